// vsamp_adamw: argument checks and launches.
#include <cmath>

#include "vsamp_adamw.cuh"
#include "vsamp_grid.h"
#include "vsamp_host.h"

namespace vsamp {

static_assert(AdamShape<true>::PerSm == AdamShape<false>::PerSm, "one grid");

static bool at_multiple(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

template <typename TP, typename TG>
static vsamp_status launch_adamw(const AdamParams& p, bool master, bool bits8, const DeviceInfo& d, cudaStream_t s) {
  const int64_t most = (int64_t)d.sm_count * AdamShape<true>::PerSm;
  const unsigned grid = (unsigned)(p.chunks < most ? p.chunks : most);
  if constexpr (sizeof(TP) == 2) {
    if (master)
      return launch_1d(bits8 ? adamw_kernel<TP, TG, true, true> : adamw_kernel<TP, TG, true, false>, grid, kAdamThreads, 0, s,
                       p);
  }
  return launch_1d(bits8 ? adamw_kernel<TP, TG, false, true> : adamw_kernel<TP, TG, false, false>, grid, kAdamThreads, 0, s,
                   p);
}

}  // namespace vsamp

using namespace vsamp;

extern "C" vsamp_status vsamp_adamw(const vsamp_adamw_tensor* tensors, int32_t count, vsamp_dtype param_dt,
                                    vsamp_dtype grad_dt, int32_t state_bits, const vsamp_adamw_rule* rule, void* stream) {
  if (!tensors || !rule || count <= 0) return VSAMP_ERR_INVALID_ARG;
  if ((param_dt != VSAMP_F32 && param_dt != VSAMP_BF16) || (grad_dt != VSAMP_F32 && grad_dt != VSAMP_BF16))
    return VSAMP_ERR_INVALID_ARG;
  if (state_bits != 32 && state_bits != 8) return VSAMP_ERR_INVALID_ARG;
  const vsamp_adamw_rule& r = *rule;
  if (!(r.beta1 >= 0 && r.beta1 < 1 && r.beta2 >= 0 && r.beta2 < 1 && r.eps >= 0 && r.weight_decay >= 0) ||
      !std::isfinite((float)r.eps) || !std::isfinite((float)r.weight_decay) || (r.eps > 0 && r.eps < 0x1p-126))
    return VSAMP_ERR_INVALID_ARG;
  if (!r.lr_dev && !(r.lr >= 0 && std::isfinite((float)r.lr))) return VSAMP_ERR_INVALID_ARG;
  if (!r.step_dev && r.step < 1) return VSAMP_ERR_INVALID_ARG;
  if (!at_multiple(r.lr_dev, 4) || !at_multiple(r.step_dev, 8) || !at_multiple(r.grad_scale, 4)) return VSAMP_ERR_INVALID_ARG;
  const bool bits8 = state_bits == 8;
  const unsigned pb = param_dt == VSAMP_F32 ? 4 : 2, gb = grad_dt == VSAMP_F32 ? 4 : 2, sb = bits8 ? 1 : 4;
  bool masters = false, first = true;
  for (int32_t k = 0; k < count; ++k) {
    const vsamp_adamw_tensor& t = tensors[k];
    if (t.n < 0) return VSAMP_ERR_INVALID_ARG;
    if (t.n > (1LL << 34)) return VSAMP_ERR_UNSUPPORTED;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || (bits8 && (!t.m_scale || !t.v_scale))) return VSAMP_ERR_INVALID_ARG;
    if (!at_multiple(t.param, pb) || !at_multiple(t.grad, gb) || !at_multiple(t.m, sb) || !at_multiple(t.v, sb) ||
        !at_multiple(t.master, 4) || !at_multiple(t.m_scale, 4) || !at_multiple(t.v_scale, 4))
      return VSAMP_ERR_INVALID_ARG;
    if (first) masters = t.master != nullptr;
    first = false;
    if (masters != (t.master != nullptr) || (masters && param_dt == VSAMP_F32)) return VSAMP_ERR_INVALID_ARG;
  }
  if (first) return VSAMP_OK;   // nothing but empty tensors
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return VSAMP_ERR_CUDA;
  }
  DeviceInfo d;
  const vsamp_status st = device_info(dev, d);
  if (st != VSAMP_OK) return st;
  AdamParams p{};
  p.lr = (float)r.lr;
  p.b1 = (float)r.beta1;
  p.b2 = (float)r.beta2;
  p.one_b1 = (float)(1.0 - r.beta1);
  p.one_b2 = (float)(1.0 - r.beta2);
  p.eps = (float)r.eps;
  p.wd = (float)r.weight_decay;
  p.ln_b1 = (float)std::log(r.beta1);
  p.ln_b2 = (float)std::log(r.beta2);
  if (!r.step_dev) {
    p.c1 = (float)(-1.0 / std::expm1((double)r.step * std::log(r.beta1)));
    p.c2 = (float)(1.0 / std::sqrt(-std::expm1((double)r.step * std::log(r.beta2))));
  }
  p.step = (uint32_t)r.step;
  for (uint32_t k = 0; k < 10; ++k) {
    p.k0[k] = (uint32_t)r.seed + k * 0x9E3779B9u;
    p.k1[k] = (uint32_t)(r.seed >> 32) + k * 0xBB67AE85u;
  }
  p.lr_dev = r.lr_dev;
  p.step_dev = r.step_dev;
  p.grad_scale = r.grad_scale;
  // With 8-bit states long chunks keep the fetches ahead of the arithmetic (67M elements: 203 us with 128 blocks, 238 with
  // 32), short ones spread few elements over the device (150 tensors of 20,000: 16.8 us with 32 blocks, 17.1 with 128; one
  // of 4M: 15.4 and 16.6). Steps with 32-bit states are the better the shorter the chunks (67M: 283 us with 32 blocks, 287
  // with 128; 150 tensors of 200,000: 128 and 136).
  int64_t total = 0;
  for (int32_t k = 0; k < count; ++k) total += tensors[k].n;
  p.chunk_blocks = bits8 && total > (int64_t)d.sm_count * AdamShape<true>::PerSm * 4 * 128 * kBlock ? 128 : 32;
  const int64_t chunk = (int64_t)p.chunk_blocks * kBlock;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t k = 0;
  while (k < count) {
    int64_t chunks = 0;
    p.count = 0;
    for (; k < count && p.count < (uint32_t)kAdamTensors; ++k) {
      const vsamp_adamw_tensor& t = tensors[k];
      if (t.n == 0) continue;
      const int64_t more = (t.n + chunk - 1) / chunk;
      if (chunks + more > 0x7FFFFFFFLL) break;
      AdamTensor& a = p.t[p.count++];
      a.param = static_cast<unsigned char*>(t.param);
      a.master = t.master;
      a.grad = static_cast<const unsigned char*>(t.grad);
      a.m = static_cast<unsigned char*>(t.m);
      a.v = static_cast<unsigned char*>(t.v);
      a.m_scale = t.m_scale;
      a.v_scale = t.v_scale;
      a.n = t.n;
      a.first_chunk = (uint32_t)chunks;
      a.index = t.index;
      a.aligned = at_multiple(t.param, 4 * pb) && at_multiple(t.master, 16) && at_multiple(t.grad, 4 * gb) &&
                  at_multiple(t.m, 4 * sb) && at_multiple(t.v, 4 * sb);
      chunks += more;
    }
    if (p.count == 0) break;
    p.chunks = (uint32_t)chunks;
    vsamp_status e;
    if (param_dt == VSAMP_F32)
      e = grad_dt == VSAMP_F32 ? launch_adamw<float, float>(p, masters, bits8, d, s)
                               : launch_adamw<float, __nv_bfloat16>(p, masters, bits8, d, s);
    else
      e = grad_dt == VSAMP_F32 ? launch_adamw<__nv_bfloat16, float>(p, masters, bits8, d, s)
                               : launch_adamw<__nv_bfloat16, __nv_bfloat16>(p, masters, bits8, d, s);
    if (e != VSAMP_OK) return e;
  }
  return VSAMP_OK;
}
