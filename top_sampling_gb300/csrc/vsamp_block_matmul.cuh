// Product of two matrices in e4m3 blocks of 128.
//
//   out[m, n] = sum over blocks j of sa[m, j] * sb[n, j] * sum over k in j of a[m, k] * b[n, k]
#pragma once

#include "vsamp_block_quant.cuh"

namespace vsamp {

struct BlockMatmulParams {
  const unsigned char* a;
  const unsigned char* b;
  const float* sa;
  const float* sb;
  int64_t lda, ldsa, ldb, ldsb;
  int64_t M, N, K, ldo;
  unsigned char* out;
  int accumulate;
};

__device__ __forceinline__ float e4m3_value(unsigned char c) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"((uint32_t)c));
  return __half2float(__ushort_as_half((unsigned short)(r & 0xFFFFu)));
}

// 64 x 64 results per CTA, 4 x 4 per thread, fp32 multiply-adds.
template <typename TO, bool TILE>
__global__ void __launch_bounds__(256) block_matmul_kernel(const BlockMatmulParams p) {
  begin_overlapped();
  __shared__ float as[32][65], bs[32][65];
  const int64_t col_tiles = (p.N + 63) / 64;
  const int64_t m0 = blockIdx.x / col_tiles * 64, n0 = blockIdx.x % col_tiles * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float total[4][4] = {};
  for (int64_t j = 0; j * kBlock < p.K; ++j) {
    float part[4][4] = {};
    for (int k0 = 0; k0 < kBlock; k0 += 32) {
      __syncthreads();
      for (int i = threadIdx.x; i < 64 * 32; i += 256) {
        const int r = i >> 5, k = i & 31;
        const int64_t kk = j * kBlock + k0 + k;
        as[k][r] = kk < p.K && m0 + r < p.M ? e4m3_value(p.a[(m0 + r) * p.lda + kk]) : 0.0f;
        bs[k][r] = kk < p.K && n0 + r < p.N ? e4m3_value(p.b[(n0 + r) * p.ldb + kk]) : 0.0f;
      }
      __syncthreads();
      for (int k = 0; k < 32; ++k)
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int x = 0; x < 4; ++x) part[y][x] = fmaf(as[k][ty * 4 + y], bs[k][tx * 4 + x], part[y][x]);
    }
    for (int y = 0; y < 4; ++y)
      for (int x = 0; x < 4; ++x) {
        const int64_t m = m0 + ty * 4 + y, n = n0 + tx * 4 + x;
        if (m < p.M && n < p.N)
          total[y][x] = fmaf(part[y][x], p.sa[j * p.ldsa + m] * (TILE ? p.sb[n / kBlock * p.ldsb + j] : p.sb[j * p.ldsb + n]),
                             total[y][x]);
      }
  }
  for (int y = 0; y < 4; ++y)
    for (int x = 0; x < 4; ++x) {
      const int64_t m = m0 + ty * 4 + y, n = n0 + tx * 4 + x;
      if (m < p.M && n < p.N) {
        TO* o = reinterpret_cast<TO*>(p.out) + m * p.ldo + n;
        const float v = p.accumulate ? total[y][x] + (float)*o : total[y][x];
        *o = (TO)v;
      }
    }
}

}  // namespace vsamp
