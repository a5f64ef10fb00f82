// vsamp_head_pack and vsamp_head_logits: argument checks and launches.
#include <atomic>

#include "vsamp_grid.h"
#include "vsamp_head.cuh"
#include "vsamp_host.h"

namespace vsamp {

// The shape of packed weights, or false for arguments that have none.
static bool head_shape(vsamp_dtype scale_dt, int32_t has_zeros, int64_t V, int64_t D, int32_t group, HeadShape& s) {
  if (scale_dt != VSAMP_F32 && scale_dt != VSAMP_BF16) return false;
  if (group != 32 && group != 64 && group != 128) return false;
  if (V <= 0 || D <= 0 || V > 0x7FFFFFF0LL || D > (1 << 24) || D % group != 0) return false;
  s.V = V;
  s.D = D;
  s.group = group;
  s.scale_bytes = scale_dt == VSAMP_F32 ? 4 : 2;
  s.has_zeros = has_zeros != 0;
  return true;
}

template <typename T, int NT, int RT, int GROUP, int PF>
static vsamp_status launch_head_cfg(HeadParams p, const DeviceInfo& d, int dev, cudaStream_t stream) {
  auto kern = head_kernel<T, NT, RT, GROUP, PF>;
  // Warps share a row tile when there are not enough tiles for every warp of the device.
  const int64_t sets = (p.s.tiles() + RT - 1) / RT;
  const int64_t warps = (int64_t)d.sm_count * kHeadWarps;
  p.split = 1;
  while (p.split < kHeadWarps && sets * p.split * 2 <= warps && p.split * 2 <= p.units) p.split *= 2;
  const int red = p.split > 1 ? kHeadWarps * RT * NT * 4 * 32 * 4 : 0;
  const int64_t unit_bytes = (int64_t)kHeadUnitSteps * kHeadTerms<T> * NT * 8 * 32;
  const int ring = kHeadWarps * PF * RT * p.s.record();
  const int64_t most = (d.optin - red - ring) / unit_bytes;
  if (most < 1) return VSAMP_ERR_UNSUPPORTED;
  p.chunk = p.units <= most ? p.units : (int)most;
  p.ring_off = (int)(p.chunk * unit_bytes);
  p.red_off = p.ring_off + ring;
  const int smem = p.red_off + red;
  // the kernel's limit is raised to the device's once, so concurrent callers never lower it under each other
  static std::atomic<bool> raised[64];
  if (dev >= 64 || !raised[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, d.optin) != cudaSuccess) {
      cudaGetLastError();
      return VSAMP_ERR_CUDA;
    }
    if (dev < 64) raised[dev].store(true, std::memory_order_release);
  }
  const int64_t ctas = (sets * p.split + kHeadWarps - 1) / kHeadWarps;
  return launch_1d(kern, grid_of(ctas < d.sm_count ? ctas : d.sm_count), kHeadWarps * 32, (size_t)smem, stream, false,
                   p);
}

template <typename T, int NT, int RT, int PF>
static vsamp_status launch_head_nt(const HeadParams& p, const DeviceInfo& d, int dev, cudaStream_t s) {
  if (p.s.group == 32) return launch_head_cfg<T, NT, RT, 32, PF>(p, d, dev, s);
  if (p.s.group == 64) return launch_head_cfg<T, NT, RT, 64, PF>(p, d, dev, s);
  return launch_head_cfg<T, NT, RT, 128, PF>(p, d, dev, s);
}

template <typename T>
static vsamp_status launch_head(HeadParams p, const DeviceInfo& d, int dev, cudaStream_t s) {
  p.units = p.s.units();
  p.vec = (reinterpret_cast<uintptr_t>(p.hidden) & 15u) == 0 && (p.ldh * sizeof(T)) % 16 == 0;
  for (int64_t m = 0; m < p.M; m += 64) {
    p.m0 = m;
    p.rows = (int)(p.M - m < 64 ? p.M - m : 64);
    const vsamp_status st = p.rows <= 8    ? launch_head_nt<T, 1, 1, 4>(p, d, dev, s)
                            : p.rows <= 16 ? launch_head_nt<T, 2, 2, 2>(p, d, dev, s)
                            : p.rows <= 24 ? launch_head_nt<T, 3, 2, 2>(p, d, dev, s)
                            : p.rows <= 32 ? launch_head_nt<T, 4, 2, 2>(p, d, dev, s)
                                           : launch_head_nt<T, 8, 1, 4>(p, d, dev, s);
    if (st != VSAMP_OK) return st;
  }
  return VSAMP_OK;
}

}  // namespace vsamp

using namespace vsamp;

extern "C" {

size_t vsamp_head_packed_size(vsamp_dtype scale_dt, int32_t has_zeros, int64_t V, int64_t D, int32_t group) {
  HeadShape s;
  return head_shape(scale_dt, has_zeros, V, D, group, s) ? (size_t)s.total() : 0;
}

vsamp_status vsamp_head_pack(const uint8_t* codes, const void* scales, vsamp_dtype scale_dt, const uint8_t* zeros,
                             int64_t V, int64_t D, int32_t group, void* packed, size_t packed_bytes, void* stream) {
  HeadShape s;
  if (!codes || !scales || !packed) return VSAMP_ERR_INVALID_ARG;
  if (!head_shape(scale_dt, zeros != nullptr, V, D, group, s)) return VSAMP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(scales) & (unsigned)(s.scale_bytes - 1)) != 0) return VSAMP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(packed) & 15u) != 0 || packed_bytes < (size_t)s.total()) return VSAMP_ERR_INVALID_ARG;
  HeadPackParams p{};
  p.s = s;
  p.codes = codes;
  p.scales = static_cast<const unsigned char*>(scales);
  p.zeros = zeros;
  p.packed = static_cast<unsigned char*>(packed);
  return launch_1d(head_pack_kernel, grid_of((s.tiles() * s.blocks() * 128 + 1023) / 1024), 256, 0,
                   static_cast<cudaStream_t>(stream), false, p);
}

vsamp_status vsamp_head_logits(const void* hidden, vsamp_dtype dt, int64_t M, int64_t ldh, const void* packed,
                               size_t packed_bytes, vsamp_dtype scale_dt, int32_t has_zeros, int64_t V, int64_t D,
                               int32_t group, void* logits, vsamp_dtype out_dt, int64_t ld, void* stream) {
  HeadShape s;
  if (!hidden || !packed || !logits) return VSAMP_ERR_INVALID_ARG;
  if ((dt != VSAMP_F32 && dt != VSAMP_BF16) || (out_dt != VSAMP_F32 && out_dt != VSAMP_BF16)) return VSAMP_ERR_INVALID_ARG;
  if (!head_shape(scale_dt, has_zeros, V, D, group, s)) return VSAMP_ERR_INVALID_ARG;
  if (M <= 0 || ldh < D || ld < V) return VSAMP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(hidden) & (dt == VSAMP_F32 ? 3u : 1u)) != 0 ||
      (reinterpret_cast<uintptr_t>(logits) & (out_dt == VSAMP_F32 ? 3u : 1u)) != 0 ||
      (reinterpret_cast<uintptr_t>(packed) & 15u) != 0 || packed_bytes < (size_t)s.total())
    return VSAMP_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return VSAMP_ERR_CUDA;
  }
  DeviceInfo d;
  const vsamp_status st = device_info(dev, d);
  if (st != VSAMP_OK) return st;
  HeadParams p{};
  p.s = s;
  p.packed = static_cast<const unsigned char*>(packed);
  p.hidden = static_cast<const unsigned char*>(hidden);
  p.M = M;
  p.ldh = ldh;
  p.logits = static_cast<unsigned char*>(logits);
  p.ld = ld;
  p.out_f32 = out_dt == VSAMP_F32;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return dt == VSAMP_F32 ? launch_head<float>(p, d, dev, cs) : launch_head<__nv_bfloat16>(p, d, dev, cs);
}

}  // extern "C"
