// Quantisation into e4m3 blocks of 128, of a matrix and of its transpose in one pass over it.
//
//   scale = max(max |x| / 448, 2^-126) over a block (1 x 128 or 128 x 128), code = e4m3(x * 448 / max |x|), nearest even
//
// One CTA takes a tile of 128 x 128 elements, which holds whole blocks of both directions: it is read once, every
// maximum is formed from registers, and the transpose goes through 16 KB of shared memory so that both outputs are
// written in rows of 128 bytes. bf16 pairs stay packed (half the registers, two maxima per instruction), a lane forms the
// scale of one row and passes it on.
//
// Measured: one direction of bf16 99 % of the copy rate (32768 x 8192: 123 us); both directions 84 % (2048 x 151936: 225 us of
// 189), where the conversions' instructions fill the issue slots; 128 x 128 blocks of fp32 both ways 89 % (32000 x 2048: 66 us).
// Four CTAs per SM for bf16 (both ways 2048 x 65536: 93 us, three 102, two 128), two for fp32, whose tiles take 64 registers
// (65536 x 2048 both ways: 134 us, three 149). Rows that do not begin on 16 bytes are read by words: 2048 x 151935 bf16 both ways
// 310 us, 65536 x 2047 fp32 204, 32000 x 2047 fp32 in 128 x 128 blocks 82.
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

// What the elements of a block are multiplied with, 448 / max, in two parts. One fp32 number is off by up to half a unit,
// and of bf16 values many lie half way between two codes: which side they fell on would be that error's.
struct BlockInverse {
  float hi, lo;   // hi below 0: the block is not finite
};

// The scale of a block from the bits of its largest magnitude (those of NaN are above those of an infinity, and both
// above every finite value's).
__device__ __forceinline__ float block_scale(uint32_t amax_bits, BlockInverse& inv) {
  const float amax = __uint_as_float(amax_bits), s = fmaxf(__fdiv_rn(amax, kE4m3Max), 0x1p-126f);
  if (amax_bits >= kInfBits) {
    inv.hi = -1.0f;
    inv.lo = 0.0f;
    return __uint_as_float(0x7FC00000u);
  }
  inv.hi = 0x1p126f;
  inv.lo = 0.0f;
  if (amax >= kE4m3Max * 0x1p-126f) {
    inv.hi = __fdiv_rn(kE4m3Max, amax);
    inv.lo = fmaf(-inv.hi, amax, kE4m3Max) * inv.hi * (1.0f / kE4m3Max);
  }
  return s;
}

// x * 448 / max, rounded once, for two elements.
__device__ __forceinline__ float2 in_units(float2 x, float2 hi, float2 lo) { return __ffma2_rn(x, hi, __fmul2_rn(x, lo)); }

// Two e4m3 codes, a in the low byte; magnitudes above 448 become 448.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_quad(float a, float b, float c, float d) {
  return e4m3_pair(a, b) | (e4m3_pair(c, d) << 16);
}

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if one of them is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A thread's 8 x 8 elements as they were read, and their largest magnitudes per row and per column as fp32 values.
template <typename T>
struct QuantTile;

template <>
struct QuantTile<float> {
  float v[8][8];
  __device__ __forceinline__ void load_row(int i, const unsigned char* p, int left, bool aligned) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      ElemVec<float, 4> e;
      e.load_row(p + k * 16, left - k * 4, aligned, 0u);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][k * 4 + j] = e.at(j);
    }
  }
  __device__ __forceinline__ void clear_row(int i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
  }
  __device__ __forceinline__ float at(int i, int j) const { return v[i][j]; }
  __device__ __forceinline__ void forget() {}
  // the largest of every row over the 16 lanes of this thread's rows; the lane's own row (lane & 7) is returned
  __device__ __forceinline__ float row_max(int lane) const {
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = fabsf(v[i][0]);
#pragma unroll
      for (int j = 1; j < 8; ++j) m[i] = max_nan(m[i], fabsf(v[i][j]));
    }
    // halves of the rows are exchanged for halves of the lanes: 8 + 4 + ... values per step instead of 8 each time
#pragma unroll
    for (int o = 4; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < o) {
          const bool up = (lane & o) != 0;
          const float mine = up ? m[i + o] : m[i], other = up ? m[i] : m[i + o];
          m[i] = max_nan(mine, __shfl_xor_sync(kFullMask, other, o));
        }
    return max_nan(m[0], __shfl_xor_sync(kFullMask, m[0], 8));
  }
  // the largest of every column over this warp's rows, to the warp's 128 words of shared memory
  __device__ __forceinline__ void column_max(int lane, float* to) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float m = fabsf(v[0][j]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(v[i][j]));
      m = max_nan(m, __shfl_xor_sync(kFullMask, m, 16));
      if (lane < 16) to[(lane & 15) * 8 + j] = m;
    }
  }
  __device__ __forceinline__ float all_max() const {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[i][j]));
    return m;
  }
};

template <>
struct QuantTile<__nv_bfloat16> {   // pairs stay packed: half the registers, two maxima per instruction
  uint32_t v[8][4];
  __device__ __forceinline__ void load_row(int i, const unsigned char* p, int left, bool aligned) {
    ElemVec<__nv_bfloat16, 8> e;
    e.load_row(p, left, aligned, 0u);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i][j] = e.w[j];
  }
  __device__ __forceinline__ void clear_row(int i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i][j] = 0u;
  }
  __device__ __forceinline__ float at(int i, int j) const {
    return __uint_as_float(j & 1 ? v[i][j >> 1] & 0xFFFF0000u : v[i][j >> 1] << 16);
  }
  // Between the two outputs: the fp32 values of the first are not kept in registers for the second.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) asm volatile("" : "+r"(v[i][j]));
  }
  __device__ __forceinline__ uint32_t mag(int i, int j) const { return v[i][j] & 0x7FFF7FFFu; }
  __device__ __forceinline__ float row_max(int lane) const {
    uint32_t m[4];   // rows i and i + 4 in one word
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = max_nan_bf16x2(max_nan_bf16x2(mag(i, 0), mag(i, 1)), max_nan_bf16x2(mag(i, 2), mag(i, 3)));
      const uint32_t b = max_nan_bf16x2(max_nan_bf16x2(mag(i + 4, 0), mag(i + 4, 1)), max_nan_bf16x2(mag(i + 4, 2), mag(i + 4, 3)));
      m[i] = max_nan_bf16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    }
#pragma unroll
    for (int o = 2; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < o) {
          const bool up = (lane & o) != 0;
          const uint32_t mine = up ? m[i + o] : m[i], other = up ? m[i] : m[i + o];
          m[i] = max_nan_bf16x2(mine, __shfl_xor_sync(kFullMask, other, o));
        }
    uint32_t r = max_nan_bf16x2(m[0], __shfl_xor_sync(kFullMask, m[0], 4));
    r = max_nan_bf16x2(r, __shfl_xor_sync(kFullMask, r, 8));
    return __uint_as_float(lane & 4 ? r & 0xFFFF0000u : r << 16);
  }
  __device__ __forceinline__ void column_max(int lane, float* to) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t m = mag(0, j);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = max_nan_bf16x2(m, mag(i, j));
      m = max_nan_bf16x2(m, __shfl_xor_sync(kFullMask, m, 16));
      if (lane < 16)
        *reinterpret_cast<float2*>(to + (lane & 15) * 8 + 2 * j) =
            make_float2(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
  }
  __device__ __forceinline__ float all_max() const {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max_nan_bf16x2(m, mag(i, j));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
};

template <typename T, bool TILE, bool PLAIN, bool TURNED>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 4 ? 2 : 4) block_quant_kernel(const BlockQuantParams p) {
  begin_overlapped();
  __shared__ __align__(16) unsigned char turned[TURNED ? kBlock * kBlock : 16];
  __shared__ __align__(16) float maxima[8][kBlock];
  __shared__ __align__(16) float inverse[2][kBlock];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = (lane & 15) * 8, r0 = warp * 16 + (lane >> 4) * 8;   // this thread's 8 x 8 elements
  for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const int64_t rt = tile / p.col_tiles, ct = tile - rt * p.col_tiles;
    const int64_t row = rt * kBlock + r0, col = ct * kBlock + c0;
    const int left = (int)(p.C - col < 8 ? p.C - col : 8);
    const int rows = (int)(p.R - row < 8 ? p.R - row : 8);
    QuantTile<T> x;
    const unsigned char* from = p.x + (row * p.ldx + col) * (int64_t)sizeof(T);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < rows && left > 0) x.load_row(i, from + i * p.ldx * (int64_t)sizeof(T), left, p.aligned != 0);
      else x.clear_row(i);
    }
    BlockInverse tile_inv = {0.0f, 0.0f};
    if (TILE) {
      uint32_t m = warp_max_u32(__float_as_uint(x.all_max()));
      if (lane == 0) maxima[warp][0] = __uint_as_float(m);
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w) m = max(m, __float_as_uint(maxima[w][0]));
      const float s = block_scale(m, tile_inv);
      if (threadIdx.x == 0) {
        if (PLAIN) p.scales[rt * p.lds + ct] = s;
        if (TURNED) p.scales_t[ct * p.ldst + rt] = s;
      }
    }
    if (PLAIN) {
      BlockInverse own = tile_inv;   // of the row lane & 7
      if (!TILE) {
        const float s = block_scale(__float_as_uint(x.row_max(lane)), own);
        const int64_t r = row + (lane & 7);
        if ((lane & 8) == 0 && r < p.R) p.scales[ct * p.lds + r] = s;
      }
      unsigned char* to = p.codes + row * p.ldc + col;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float hi = TILE ? own.hi : __shfl_sync(kFullMask, own.hi, (lane & 16) + i);
        const float lo = TILE ? own.lo : __shfl_sync(kFullMask, own.lo, (lane & 16) + i);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 y = in_units(make_float2(x.at(i, 2 * j), x.at(i, 2 * j + 1)), make_float2(hi, hi), make_float2(lo, lo));
          w[j] = e4m3_pair(y.x, y.y);
        }
        uint2 c = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        if (hi < 0.0f) c.x = c.y = 0u;
        if (i < rows && left > 0) {
          if (left == 8) *reinterpret_cast<uint2*>(to) = c;
          else
            for (int j = 0; j < left; ++j) to[j] = (unsigned char)((j < 4 ? c.x : c.y) >> ((j & 3) * 8));
        }
        to += p.ldc;
      }
    }
    if (TURNED) {
      x.forget();
      if (!TILE) {
        x.column_max(lane, maxima[warp]);
        __syncthreads();
        if (threadIdx.x < kBlock) {
          float m = maxima[0][threadIdx.x];
#pragma unroll
          for (int w = 1; w < 8; ++w) m = max_nan(m, maxima[w][threadIdx.x]);
          BlockInverse inv;
          const float s = block_scale(__float_as_uint(m), inv);
          inverse[0][threadIdx.x] = inv.hi;
          inverse[1][threadIdx.x] = inv.lo;
          const int64_t c = ct * kBlock + threadIdx.x;
          if (c < p.C) p.scales_t[rt * p.ldst + c] = s;
        }
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2) {   // two columns
        const float2 hi = TILE ? make_float2(tile_inv.hi, tile_inv.hi) : *reinterpret_cast<const float2*>(&inverse[0][c0 + j]);
        const float2 lo = TILE ? make_float2(tile_inv.lo, tile_inv.lo) : *reinterpret_cast<const float2*>(&inverse[1][c0 + j]);
        uint32_t a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = in_units(make_float2(x.at(2 * i, j), x.at(2 * i, j + 1)), hi, lo);
          const float2 z = in_units(make_float2(x.at(2 * i + 1, j), x.at(2 * i + 1, j + 1)), hi, lo);
          a[i] = e4m3_pair(y.x, z.x);
          b[i] = e4m3_pair(y.y, z.y);
        }
        uint2 ca = make_uint2(a[0] | (a[1] << 16), a[2] | (a[3] << 16)), cb = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
        if (hi.x < 0.0f) ca.x = ca.y = 0u;
        if (hi.y < 0.0f) cb.x = cb.y = 0u;
        // 16-byte pieces of a row of 128 are permuted by the column's upper bits: two-way conflicts instead of sixteen
        const int c = c0 + j, piece = (r0 >> 4) ^ ((c >> 3) & 7);
        unsigned char* to = turned + c * kBlock + piece * 16 + (r0 & 8);
        *reinterpret_cast<uint2*>(to) = ca;
        *reinterpret_cast<uint2*>(to + kBlock) = cb;
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
