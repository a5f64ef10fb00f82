// The output head with 4-bit weights (vsamp_head_pack, vsamp_head_logits):
//   logits[m, v] = sum over groups g of scale[v, g] * sum over k in g of (q[v, k] - z[v, g]) * hidden[m, k].
//
// The weights are read once per call, half a byte each, and everything else is small next to them while M stays in
// the tens: a few rows of hidden states against the whole vocabulary. So the kernel is a stream over the weights
// that feeds the warp-level matrix instruction straight from registers: q - z is at most 15 in magnitude, exact in
// bf16, products with bf16 hidden states are exact, sums are fp32, and the group's scale multiplies the fp32 sum of
// its group. (Weights widened through shared or tensor memory for tcgen05 would cost four times their bytes of
// on-chip traffic for a product that has at most 64 columns.) fp32 hidden states are split into three bf16 terms,
// multiplied one after the other.
//
// Packed layout. Vocabulary rows in tiles of 16, the inner dimension in blocks of 64 (zero padded): a block is 512
// contiguous bytes, lane l of a warp owns 16 of them: one 32-bit word per 16-wide matrix step, whose nibbles are the
// lane's eight elements of the 16 x 16 operand. Nibble pairs (i, i + 4) are one operand register:
//   i = 0: row l/4,     columns 2 (l%4) + {0, 1}        i = 1: row l/4 + 8, the same columns
//   i = 2: row l/4,     columns 2 (l%4) + 8 + {0, 1}    i = 3: row l/4 + 8, the same columns
// Scales follow as [tile][group][16], then zero points as [tile][group][16] bytes.
#pragma once

#include "vsamp.h"
#include "vsamp_device.cuh"

namespace vsamp {

constexpr int kHeadWarps = 8;
constexpr int kHeadBlock = 64;      // inner elements per block of a tile

struct HeadShape {
  int64_t V, D;
  int group;
  int scale_bytes;   // 4 (fp32) or 2 (bf16)
  int has_zeros;
  __host__ __device__ int64_t tiles() const { return (V + 15) / 16; }
  __host__ __device__ int64_t blocks() const { return (D + kHeadBlock - 1) / kHeadBlock; }
  __host__ __device__ int64_t groups() const { return D / group; }
  __host__ __device__ int64_t code_bytes() const { return tiles() * blocks() * 512; }
  __host__ __device__ int64_t scale_off() const { return code_bytes(); }
  __host__ __device__ int64_t zero_off() const { return code_bytes() + tiles() * groups() * 16 * scale_bytes; }
  __host__ __device__ int64_t total() const { return zero_off() + (has_zeros ? tiles() * groups() * 16 : 0); }
};

struct HeadPackParams {
  HeadShape s;
  const unsigned char* codes;    // [V, D / 2]
  const unsigned char* scales;   // [V, groups]
  const unsigned char* zeros;    // [V, groups] or NULL
  unsigned char* packed;
};

struct HeadParams {
  HeadShape s;
  const unsigned char* packed;
  const unsigned char* hidden;
  int64_t M, ldh;
  unsigned char* logits;
  int64_t ld;
  int out_f32;
  int64_t m0;      // first hidden row of this launch
  int rows;        // hidden rows of this launch
  int64_t chunk;   // 16-wide steps of hidden states staged at once
};

// One thread per packed 32-bit word, then per scale and zero point.
__global__ void __launch_bounds__(256) head_pack_kernel(const HeadPackParams p) {
  const HeadShape s = p.s;
  const int64_t words = s.code_bytes() / 4, ng = s.groups();
  const int64_t scales = s.tiles() * ng * 16;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  const int64_t first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t i = first; i < words; i += stride) {
    // word i: tile, block, lane, step
    const int step = (int)(i & 3), lane = (int)((i >> 2) & 31);
    const int64_t blk = (i >> 7) % s.blocks(), tile = (i >> 7) / s.blocks();
    uint32_t word = 0;
    for (int n = 0; n < 8; ++n) {
      const int pair = n & 3, hi = n >> 2;
      const int64_t row = tile * 16 + (lane >> 2) + (pair & 1) * 8;
      const int64_t k = blk * kHeadBlock + step * 16 + (lane & 3) * 2 + (pair >> 1) * 8 + hi;
      uint32_t q = 0;
      if (row < s.V && k < s.D) q = (p.codes[row * (s.D / 2) + k / 2] >> ((k & 1) * 4)) & 15u;
      word |= q << (n * 4);
    }
    reinterpret_cast<uint32_t*>(p.packed)[i] = word;
  }
  for (int64_t i = first; i < scales; i += stride) {
    const int64_t row = (i / (ng * 16)) * 16 + (i & 15), g = (i / 16) % ng;
    const bool in = row < s.V;
    if (s.scale_bytes == 4)
      reinterpret_cast<uint32_t*>(p.packed + s.scale_off())[i] =
          in ? reinterpret_cast<const uint32_t*>(p.scales)[row * ng + g] : 0u;
    else
      reinterpret_cast<unsigned short*>(p.packed + s.scale_off())[i] =
          in ? reinterpret_cast<const unsigned short*>(p.scales)[row * ng + g] : (unsigned short)0;
    if (s.has_zeros) p.packed[s.zero_off() + i] = in ? (p.zeros[row * ng + g] & 15u) : 0;
  }
}

// D += A B on 16 x 16 by 16 x 8 bf16 operands, fp32 sums
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  __nv_bfloat162 x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  x = __hsub2(x, y);
  uint32_t r;
  memcpy(&r, &x, 4);
  return r;
}

// bf16 terms per hidden value: x = hi + mid + lo for fp32, each the bf16 nearest to what is left (24 bits in all).
template <typename T>
constexpr int kHeadTerms = sizeof(T) == 4 ? 3 : 1;

// Stages the hidden states of steps [k0, k1) as the instruction's second operand: for 16-wide step k and column tile
// n, lane l needs hidden row 8 n + l/4 at inner positions 2 (l%4) + {0, 1} and + 8: two registers per term, stored as
// [step][tile][term][lane]. Rows and positions beyond the data are 0.
template <typename T, int NT>
__device__ __forceinline__ void head_stage(const HeadParams& p, uint2* sh, int64_t k0, int64_t k1) {
  constexpr int TERMS = kHeadTerms<T>;
  const int n_words = (int)(k1 - k0) * NT * 32;
  for (int i = threadIdx.x; i < n_words; i += blockDim.x) {
    const int lane = i & 31, n = (i >> 5) % NT, ks = (i >> 5) / NT;
    const int r = n * 8 + (lane >> 2);
    uint32_t reg[TERMS][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int q = 0; q < TERMS; ++q) reg[q][h] = 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t k = (k0 + ks) * 16 + (lane & 3) * 2 + h * 8 + e;
        if (r < p.rows && k < p.s.D) {
          const int64_t at = (int64_t)(p.m0 + r) * p.ldh + k;
          if constexpr (TERMS == 1) {
            reg[0][h] |= (uint32_t) reinterpret_cast<const unsigned short*>(p.hidden)[at] << (16 * e);
          } else {
            float x = reinterpret_cast<const float*>(p.hidden)[at];
#pragma unroll
            for (int q = 0; q < TERMS; ++q) {
              const __nv_bfloat16 v = __float2bfloat16_rn(x);
              reg[q][h] |= (uint32_t)__bfloat16_as_ushort(v) << (16 * e);
              // an infinity has no remainder (inf - inf would turn it into NaN)
              x = isinf(__bfloat162float(v)) ? 0.f : x - __bfloat162float(v);
            }
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < TERMS; ++q)
      sh[((ks * NT + n) * TERMS + q) * 32 + lane] = make_uint2(reg[q][0], reg[q][1]);
  }
}

// One warp per tile of 16 vocabulary rows. p.chunk: steps staged at once (a multiple of 8, so no group straddles two
// chunks), all of them when they fit.
template <typename T, int NT, int SB, bool ZEROS>
__global__ void __launch_bounds__(kHeadWarps * 32) head_kernel(const HeadParams p) {
  constexpr int TERMS = kHeadTerms<T>;
  extern __shared__ __align__(16) unsigned char head_smem[];
  uint2* sh = reinterpret_cast<uint2*>(head_smem);
  const HeadShape s = p.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t nb = s.blocks(), ng = s.groups(), nt = s.tiles(), steps = nb * (kHeadBlock / 16);
  const int group_steps = s.group / 16;
  bool staged = false;
  for (int64_t tile0 = (int64_t)blockIdx.x * kHeadWarps; tile0 < nt; tile0 += (int64_t)gridDim.x * kHeadWarps) {
    const int64_t tile = tile0 + warp;
    const uint4* codes = reinterpret_cast<const uint4*>(p.packed) + tile * nb * 32 + lane;
    const unsigned char* scales = p.packed + s.scale_off() + tile * ng * 16 * SB;
    const unsigned char* zeros = p.packed + s.zero_off() + tile * ng * 16;
    float acc[NT][4], part[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[n][j] = part[n][j] = 0.f;
    for (int64_t k0 = 0; k0 < steps; k0 += p.chunk) {
      const int64_t k1 = k0 + p.chunk < steps ? k0 + p.chunk : steps;
      if (!staged || p.chunk < steps) {
        __syncthreads();   // the last chunk has been read
        head_stage<T, NT>(p, sh, k0, k1);
        __syncthreads();
        staged = true;
      }
      if (tile >= nt) continue;
      uint32_t zlo = 0x43084308u, zhi = 0x43084308u;      // 128 + 8, twice
      float slo = 0.f, shi = 0.f;
      for (int64_t b = k0 / 4; b < k1 / 4; ++b) {
        const uint4 q4 = codes[b * 32];
        const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int step = 0; step < 4; ++step) {
          const int64_t k = b * 4 + step;
          if (k % group_steps == 0 && k / group_steps < ng) {   // a group begins
            const int64_t at = k / group_steps * 16 + (lane >> 2);
            if (SB == 4) {
              slo = reinterpret_cast<const float*>(scales)[at];
              shi = reinterpret_cast<const float*>(scales)[at + 8];
            } else {
              slo = __uint_as_float((uint32_t) reinterpret_cast<const unsigned short*>(scales)[at] << 16);
              shi = __uint_as_float((uint32_t) reinterpret_cast<const unsigned short*>(scales)[at + 8] << 16);
            }
            if (ZEROS) {
              zlo = 0x43004300u + (uint32_t)zeros[at] * 0x00010001u;
              zhi = 0x43004300u + (uint32_t)zeros[at + 8] * 0x00010001u;
            }
          }
          const uint32_t w = q[step];
          const uint32_t a0 = sub_bf16x2((w & 0x000F000Fu) | 0x43004300u, zlo);
          const uint32_t a1 = sub_bf16x2(((w >> 4) & 0x000F000Fu) | 0x43004300u, zhi);
          const uint32_t a2 = sub_bf16x2(((w >> 8) & 0x000F000Fu) | 0x43004300u, zlo);
          const uint32_t a3 = sub_bf16x2(((w >> 12) & 0x000F000Fu) | 0x43004300u, zhi);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int t = 0; t < TERMS; ++t) {
              const uint2 h = sh[(((k - k0) * NT + n) * TERMS + t) * 32 + lane];
              mma_bf16(part[n], a0, a1, a2, a3, h.x, h.y);
            }
          if ((k + 1) % group_steps == 0) {   // a group ends
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              acc[n][0] = fmaf(slo, part[n][0], acc[n][0]);
              acc[n][1] = fmaf(slo, part[n][1], acc[n][1]);
              acc[n][2] = fmaf(shi, part[n][2], acc[n][2]);
              acc[n][3] = fmaf(shi, part[n][3], acc[n][3]);
              part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0.f;
            }
          }
        }
      }
    }
    // accumulator j of column tile n: vocabulary row l/4 (+ 8 for j >= 2), hidden row 8 n + 2 (l%4) + (j & 1)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t v = tile * 16 + (lane >> 2) + (j >> 1) * 8;
        const int r = n * 8 + 2 * (lane & 3) + (j & 1);
        if (r < p.rows && v < s.V) {
          const int64_t at = (int64_t)(p.m0 + r) * p.ld + v;
          if (p.out_f32) reinterpret_cast<float*>(p.logits)[at] = acc[n][j];
          else reinterpret_cast<__nv_bfloat16*>(p.logits)[at] = __float2bfloat16_rn(acc[n][j]);
        }
      }
    }
  }
}

}  // namespace vsamp
