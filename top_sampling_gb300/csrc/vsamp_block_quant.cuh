// Quantisation into e4m3 blocks of 128, of a matrix and of its transpose in one pass over it.
//
//   scale = max(max |x| / 448, 2^-126) over a block (1 x 128 or 128 x 128), code = e4m3(x * (1 / scale)), nearest even.
//
// One CTA takes a tile of 128 x 128 elements, which holds whole blocks of both directions: it is read once, every
// maximum is formed from registers, and the transpose goes through 16 KB of shared memory so that both outputs are
// written in rows of 128 bytes.
#pragma once

#include "vsamp_device.cuh"
#include "vsamp_vec.cuh"

namespace vsamp {

constexpr int kBlock = 128;          // elements of a block along the inner dimension, rows of a 128 x 128 one
constexpr int kQuantThreads = 256;
constexpr float kE4m3Max = 448.0f;
constexpr uint32_t kInfBits = 0x7F800000u;

struct BlockQuantParams {
  const unsigned char* x;
  int64_t R, C, ldx;
  unsigned char* codes;
  int64_t ldc;
  float* scales;
  int64_t lds;
  unsigned char* codes_t;
  int64_t ldt;
  float* scales_t;
  int64_t ldst;
  int64_t col_tiles, tiles;
  int aligned;      // every row of x begins on the boundary of a thread's vector
};

// The scale of a block from the bits of its largest magnitude (those of NaN are above those of an infinity, and both
// above every finite value's); inv is what its elements are multiplied with, 0 for a block that is not finite.
__device__ __forceinline__ float block_scale(uint32_t amax_bits, float& inv) {
  const float s = fmaxf(__fdiv_rn(__uint_as_float(amax_bits), kE4m3Max), 0x1p-126f);
  const bool bad = amax_bits >= kInfBits;
  inv = bad ? 0.0f : __frcp_rn(s);
  return bad ? __uint_as_float(0x7FC00000u) : s;
}

// Two e4m3 codes, a in the low byte; magnitudes above 448 become 448.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_quad(float a, float b, float c, float d) {
  return e4m3_pair(a, b) | (e4m3_pair(c, d) << 16);
}

template <typename T>
struct QuantRow {   // eight elements of a row
  static constexpr int VE = sizeof(T) == 4 ? 4 : 8, N = 8 / VE;
  static __device__ __forceinline__ void load(const unsigned char* p, int left, bool aligned, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      ElemVec<T, VE> e;
      const int n = left - k * VE;
      if (n >= VE) e.load(p + k * VE * sizeof(T), aligned);
      else e.load_some(p + k * VE * sizeof(T), n, 0u);
#pragma unroll
      for (int j = 0; j < VE; ++j) v[k * VE + j] = e.at(j);
    }
  }
};

template <typename T, bool TILE, bool PLAIN, bool TURNED>
__global__ void __launch_bounds__(kQuantThreads) block_quant_kernel(const BlockQuantParams p) {
  begin_overlapped();
  __shared__ __align__(16) unsigned char turned[TURNED ? kBlock * kBlock : 16];
  __shared__ uint32_t maxima[8][kBlock];
  __shared__ __align__(16) float inverse[kBlock];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = (lane & 15) * 8, r0 = warp * 16 + (lane >> 4) * 8;   // this thread's 8 x 8 elements
  for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const int64_t rt = tile / p.col_tiles, ct = tile - rt * p.col_tiles;
    const int64_t row = rt * kBlock + r0, col = ct * kBlock + c0;
    const int left = (int)(p.C - col < 8 ? p.C - col : 8);
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (row + i < p.R && left > 0)
        QuantRow<T>::load(p.x + ((row + i) * p.ldx + col) * (int64_t)sizeof(T), left, p.aligned != 0, v[i]);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
    uint32_t rmax[8], cmax[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rmax[i] = cmax[i] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b = __float_as_uint(v[i][j]) & 0x7FFFFFFFu;
        rmax[i] = max(rmax[i], b);
        cmax[j] = max(cmax[j], b);
      }
    float tile_inv = 0.0f;
    bool tile_bad = false;
    if (TILE) {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, rmax[i]);
      m = warp_max_u32(m);
      if (lane == 0) maxima[warp][0] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w) m = max(m, maxima[w][0]);
      const float s = block_scale(m, tile_inv);
      tile_bad = m >= kInfBits;
      if (threadIdx.x == 0) {
        if (PLAIN) p.scales[rt * p.lds + ct] = s;
        if (TURNED) p.scales_t[ct * p.ldst + rt] = s;
      }
    }
    if (PLAIN) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float inv = tile_inv;
        bool bad = tile_bad;
        if (!TILE) {
          uint32_t m = rmax[i];
#pragma unroll
          for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(kFullMask, m, o));
          const float s = block_scale(m, inv);
          bad = m >= kInfBits;
          if ((lane & 15) == i && row + i < p.R) p.scales[ct * p.lds + row + i] = s;
        }
        if (row + i < p.R && left > 0) {
          uint2 w;
          w.x = e4m3_quad(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv);
          w.y = e4m3_quad(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv);
          if (bad) w.x = w.y = 0u;
          unsigned char* to = p.codes + (row + i) * p.ldc + col;
          if (left == 8) *reinterpret_cast<uint2*>(to) = w;
          else
            for (int j = 0; j < left; ++j) to[j] = (unsigned char)((j < 4 ? w.x : w.y) >> ((j & 3) * 8));
        }
      }
    }
    if (TURNED) {
      if (!TILE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t m = max(cmax[j], __shfl_xor_sync(kFullMask, cmax[j], 16));
          if (lane < 16) maxima[warp][c0 + j] = m;
        }
        __syncthreads();
        if (threadIdx.x < kBlock) {
          uint32_t m = 0u;
#pragma unroll
          for (int w = 0; w < 8; ++w) m = max(m, maxima[w][threadIdx.x]);
          float inv;
          const float s = block_scale(m, inv);
          inverse[threadIdx.x] = m >= kInfBits ? -1.0f : inv;   // -1 marks a block that is not finite
          const int64_t c = ct * kBlock + threadIdx.x;
          if (c < p.C) p.scales_t[rt * p.ldst + c] = s;
        }
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float inv = TILE ? tile_inv : inverse[c0 + j];
        uint2 w;
        w.x = e4m3_quad(v[0][j] * inv, v[1][j] * inv, v[2][j] * inv, v[3][j] * inv);
        w.y = e4m3_quad(v[4][j] * inv, v[5][j] * inv, v[6][j] * inv, v[7][j] * inv);
        if (TILE ? tile_bad : inv < 0.0f) w.x = w.y = 0u;
        // 16-byte pieces of a row of 128 are permuted by the column's upper bits: two-way conflicts instead of sixteen
        const int c = c0 + j, piece = (r0 >> 4) ^ ((c >> 3) & 7);
        *reinterpret_cast<uint2*>(turned + c * kBlock + piece * 16 + (r0 & 8)) = w;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kBlock * kBlock / 16 / kQuantThreads; ++k) {
        const int i = k * kQuantThreads + threadIdx.x, c = i >> 3, piece = i & 7;
        const int64_t out_row = ct * kBlock + c, out_col = rt * kBlock + piece * 16;
        if (out_row < p.C && out_col < p.R) {
          const uint4 w = *reinterpret_cast<const uint4*>(turned + c * kBlock + ((piece ^ ((c >> 3) & 7)) * 16));
          unsigned char* to = p.codes_t + out_row * p.ldt + out_col;
          if (out_col + 16 <= p.R) *reinterpret_cast<uint4*>(to) = w;
          else {
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int b = 0; b < 16; ++b)
              if (out_col + b < p.R) to[b] = (unsigned char)(ws[b >> 2] >> ((b & 3) * 8));
          }
        }
      }
    }
    if (TILE || TURNED) __syncthreads();   // shared memory is written again for the next tile
  }
}

}  // namespace vsamp
