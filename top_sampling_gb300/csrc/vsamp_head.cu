// vsamp_head_pack and vsamp_head_logits: argument checks and launches.
#include "vsamp_grid.h"
#include "vsamp_head_launch.cuh"

namespace vsamp {

// One thread per 32-bit word of codes, then per scale and zero point.
__global__ void __launch_bounds__(256) head_pack_kernel(const HeadPackParams p) {
  begin_overlapped();
  const HeadShape s = p.s;
  const int64_t nb = s.blocks(), ng = s.groups(), per_unit = kHeadUnit / s.group;
  const int64_t words = s.tiles() * nb * 128, scales = s.tiles() * ng * 16;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  const int64_t first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t i = first; i < words; i += stride) {
    // word i: tile, block, lane, step
    const int step = (int)(i & 3), lane = (int)((i >> 2) & 31);
    const int64_t blk = (i >> 7) % nb, tile = (i >> 7) / nb;
    uint32_t word = 0;
    for (int n = 0; n < 8; ++n) {
      const int pair = n & 3, hi = n >> 2;
      const int64_t row = tile * 16 + (lane >> 2) + (pair & 1) * 8;
      const int64_t k = blk * kHeadBlock + step * 16 + (lane & 3) * 2 + (pair >> 1) * 8 + hi;
      uint32_t q = 0;
      if (row < s.V && k < s.D) q = (p.codes[row * (s.D / 2) + k / 2] >> ((k & 1) * 4)) & 15u;
      word |= q << (n * 4);
    }
    unsigned char* rec = p.packed + tile * s.tile_bytes() + (blk / 2) * s.record();
    reinterpret_cast<uint32_t*>(rec)[(blk & 1) * 128 + (i & 127)] = word;
  }
  for (int64_t i = first; i < scales; i += stride) {
    // scale i: tile, group, row and row + 8
    const int64_t tile = i / (ng * 16), g = (i / 16) % ng, unit = g / per_unit;
    const int64_t row = tile * 16 + ((i >> 1) & 7) + (i & 1) * 8;
    const bool in = row < s.V;
    const int64_t rec_blocks = nb - 2 * unit < 2 ? nb - 2 * unit : 2;
    const int64_t rec_groups = ng - unit * per_unit < per_unit ? ng - unit * per_unit : per_unit;
    unsigned char* at = p.packed + tile * s.tile_bytes() + unit * s.record() + rec_blocks * 512;
    const int64_t j = (g - unit * per_unit) * 16 + (i & 15);
    if (s.scale_bytes == 4)
      reinterpret_cast<uint32_t*>(at)[j] = in ? reinterpret_cast<const uint32_t*>(p.scales)[row * ng + g] : 0u;
    else
      reinterpret_cast<unsigned short*>(at)[j] =
          in ? reinterpret_cast<const unsigned short*>(p.scales)[row * ng + g] : (unsigned short)0;
    if (s.has_zeros) at[rec_groups * 16 * s.scale_bytes + j] = in ? (p.zeros[row * ng + g] & 15u) : 0;
  }
}

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

static vsamp_status launch_head(HeadParams p, const DeviceInfo& d, int dev, cudaStream_t s) {
  p.units = p.s.units();
  const int most = p.terms == 3 ? 16 : 64;   // hidden rows per launch: at most 8 column tiles (6 of fp32 terms)
  for (int64_t m = 0; m < p.M; m += most) {
    p.m0 = m;
    p.rows = (int)(p.M - m < most ? p.M - m : most);
    p.term_tiles = (p.rows + 7) / 8;
    const vsamp_status st = p.s.group == 32   ? launch_head_group<32>(p, d, dev, s)
                            : p.s.group == 64 ? launch_head_group<64>(p, d, dev, s)
                                              : launch_head_group<128>(p, d, dev, s);
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
                   static_cast<cudaStream_t>(stream), p);
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
  p.terms = dt == VSAMP_F32 ? 3 : 1;
  p.vec = (reinterpret_cast<uintptr_t>(hidden) & 15u) == 0 && (ldh * 2) % 16 == 0;
  return launch_head(p, d, dev, cs);
}

}  // extern "C"
