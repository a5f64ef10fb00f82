// vsamp_head_pack and vsamp_head_logits: argument checks and launches.
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

template <typename T, int NT, int SB, bool ZEROS>
static vsamp_status launch_head_cfg(HeadParams p, const DeviceInfo& d, cudaStream_t stream) {
  auto kern = head_kernel<T, NT, SB, ZEROS>;
  const int64_t steps = p.s.blocks() * (kHeadBlock / 16);
  const int64_t step_bytes = (int64_t)NT * kHeadTerms<T> * 256;
  // chunks of a multiple of eight steps (a largest group) within half of an SM's shared memory, or all of it
  int64_t most = (d.optin / 2) / step_bytes / 8 * 8;
  if (steps > most && steps <= (int64_t)d.optin / step_bytes) most = steps;
  if (most < 8) return VSAMP_ERR_UNSUPPORTED;
  p.chunk = steps < most ? steps : most;
  const int smem = (int)(p.chunk * step_bytes);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return VSAMP_ERR_CUDA;
  }
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kHeadWarps * 32, smem) != cudaSuccess || per_sm < 1) {
    cudaGetLastError();
    return VSAMP_ERR_CUDA;
  }
  const int64_t ctas = (p.s.tiles() + kHeadWarps - 1) / kHeadWarps;
  const int64_t resident = (int64_t)per_sm * d.sm_count;
  return launch_1d(kern, grid_of(ctas < resident ? ctas : resident), kHeadWarps * 32, (size_t)smem, stream, false, p);
}

template <typename T, int NT>
static vsamp_status launch_head_nt(const HeadParams& p, const DeviceInfo& d, cudaStream_t s) {
  if (p.s.scale_bytes == 4)
    return p.s.has_zeros ? launch_head_cfg<T, NT, 4, true>(p, d, s) : launch_head_cfg<T, NT, 4, false>(p, d, s);
  return p.s.has_zeros ? launch_head_cfg<T, NT, 2, true>(p, d, s) : launch_head_cfg<T, NT, 2, false>(p, d, s);
}

template <typename T>
static vsamp_status launch_head(HeadParams p, const DeviceInfo& d, cudaStream_t s) {
  for (int64_t m = 0; m < p.M; m += 64) {
    p.m0 = m;
    p.rows = (int)(p.M - m < 64 ? p.M - m : 64);
    const vsamp_status st = p.rows <= 8    ? launch_head_nt<T, 1>(p, d, s)
                            : p.rows <= 16 ? launch_head_nt<T, 2>(p, d, s)
                            : p.rows <= 32 ? launch_head_nt<T, 4>(p, d, s)
                                           : launch_head_nt<T, 8>(p, d, s);
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
  return launch_1d(head_pack_kernel, grid_of((s.code_bytes() / 4 + 1023) / 1024), 256, 0,
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
  return dt == VSAMP_F32 ? launch_head<float>(p, d, cs) : launch_head<__nv_bfloat16>(p, d, cs);
}

}  // extern "C"
