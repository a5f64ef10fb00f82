// Product of two matrices in e4m3 blocks of 128 on the tensor cores.
//
//   out[m, n] = sum over blocks j of sa[m, j] * sb[n, j] * sum over k in j of a[m, k] * b[n, k]
//
// One CTA per SM walks over tiles of 128 x 256 results. A warp copies blocks of both operands into a ring in shared memory
// (tensor copies with the 128-byte swizzle the tensor cores read), another issues four products of 32 inner elements per
// block into one of two accumulators in tensor memory, and eight warps take each finished block out of tensor memory and
// add it, scaled, to fp32 sums in registers: the sum of a block's 128 products is the only one that the tensor core
// forms. A row of a is a lane, so its scale is one register; a 128 x 128 block's scale of b is the same for a warp's 128
// columns, and with one scale per row of b the column scales are read from shared memory as broadcasts.
//
// Every wait is bounded. A CTA one of whose waits gave up lets its copies and products end, frees its tensor memory and
// leaves NaN in the results that it had not finished.
#pragma once

#include "vsamp_block_quant.cuh"
#include "vsamp_tensor.cuh"

namespace vsamp {

constexpr int kMmRows = 128, kMmCols = 256, kMmStages = 4;
constexpr int kMmThreads = 320;                     // eight warps of sums, the copying warp, the issuing warp
constexpr int kMmABytes = kMmRows * kBlock, kMmBBytes = kMmCols * kBlock, kMmStageBytes = kMmABytes + kMmBBytes;
constexpr int kMmColumns = 512;                     // of tensor memory: two accumulators
constexpr int kMmOutOff = kMmStages * kMmStageBytes;            // 2 KB per warp to turn results into rows
constexpr int kMmScaleOff = kMmOutOff + 8 * 2048;               // two sets of 128 column scales per warp
constexpr int kMmBarOff = kMmScaleOff + 8 * 2 * 128 * 4;
constexpr int kMmSmem = kMmBarOff + 128 + 1024;                 // and what aligns the ring to 1024 bytes

struct BlockMatmulParams {
  const float* sa;
  const float* sb;
  int64_t ldsa, ldsb;
  int64_t M, N, ldo;
  int64_t items;             // tiles times parts of the inner dimension
  unsigned char* out;
  float* part;               // [parts, M, ldp] sums of a part each, when there are several
  int64_t ldp;
  int row_tiles, blocks, parts;
  int a_rows;                // rows of a per copy
  int accumulate, vec;       // vec: rows of the output begin on 16-byte boundaries
  int drop_loads;            // test: copies are expected and never made
  long long wait_cycles;
};

struct MmItem {
  int64_t m0, n0;
  int j0, j1;
};
__device__ __forceinline__ MmItem mm_item(const BlockMatmulParams& p, int64_t item) {
  const int64_t tile = item / p.parts;
  const int part = (int)(item - tile * p.parts);
  const int64_t nt = tile / p.row_tiles;
  MmItem w;
  w.m0 = (tile - nt * p.row_tiles) * kMmRows;
  w.n0 = nt * kMmCols;
  w.j0 = (int)((int64_t)p.blocks * part / p.parts);
  w.j1 = (int)((int64_t)p.blocks * (part + 1) / p.parts);
  return w;
}

// 32 rows of a warp's results, 128 columns from n0 on, to rows of T: written, or added to what is there in fp32.
template <typename T, bool ADD>
__device__ __forceinline__ void mm_store(const float2 (&acc)[64], unsigned char* turn, T* out, int64_t ldo, int64_t m0,
                                         int64_t M, int64_t n0, int64_t N, int lane, bool vec) {
  constexpr bool F32 = sizeof(T) == 4 || ADD;   // what is turned: fp32, or what is written
  constexpr int W = F32 ? 4 : 8;                // elements of 16 bytes
  constexpr int C = 4 * W;                      // columns per turn: 64 bytes of a row
#pragma unroll
  for (int c = 0; c < 128 / C; ++c) {
    if (n0 + c * C >= N) break;
    // 16-byte pieces of a row are permuted by the row, so that neither side meets bank conflicts
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (F32) {
          const float2 a = acc[c * 8 + q * 2 + i / 2];
          u[i] = __float_as_uint(i & 1 ? a.y : a.x);
        } else {
          const __nv_bfloat162 h = __float22bfloat162_rn(acc[c * 16 + q * 4 + i]);
          memcpy(&u[i], &h, 4);
        }
      }
      *reinterpret_cast<uint4*>(turn + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 2), q = lane & 3;
      const uint4 w = *reinterpret_cast<const uint4*>(turn + r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
      const int64_t m = m0 + r, n = n0 + c * C + q * W;
      if (m < M && n < N) {
        unsigned char* to = reinterpret_cast<unsigned char*>(out + m * ldo + n);
        const int left = (int)(N - n < W ? N - n : W);
        if constexpr (ADD) {
          ElemVec<T, 4> e;
          e.load_row(to, left, vec, 0u);
          const float f[4] = {e.at(0) + __uint_as_float(w.x), e.at(1) + __uint_as_float(w.y), e.at(2) + __uint_as_float(w.z),
                              e.at(3) + __uint_as_float(w.w)};
          e.set(f);
          e.store_row(to, left, vec);
        } else {
          ElemVec<T, W> e;
          e.w[0] = w.x;
          e.w[1] = w.y;
          e.w[2] = w.z;
          e.w[3] = w.w;
          e.store_row(to, left, vec);
        }
      }
    }
    __syncwarp();
  }
}

template <typename TO, bool TILE>
__global__ void __launch_bounds__(kMmThreads, 1) block_matmul_kernel(const BlockMatmulParams p,
                                                                     const __grid_constant__ CUtensorMap a_map,
                                                                     const __grid_constant__ CUtensorMap b_map) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((0u - smem_addr(smem_raw)) & 1023u);
  const uint32_t ring = smem_addr(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kMmBarOff);   // a stage's copies have landed
  uint64_t* empty = full + kMmStages;                               // a stage's products are done
  uint64_t* done = empty + kMmStages;                               // an accumulator holds a block
  uint64_t* taken = done + 2;                                       // an accumulator has been read
  uint64_t* drain = taken + 2;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* dead = reinterpret_cast<volatile int*>(tmem_at + 1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMmStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&done[i], 1);
      mbar_init(&taken[i], 8);
    }
    mbar_init(drain, 1);
    *dead = 0;
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(smem_addr(tmem_at), kMmColumns);
  if (threadIdx.x == 256) {
    tma_prefetch_map(&a_map);
    tma_prefetch_map(&b_map);
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = *tmem_at;
  begin_overlapped();
  uint32_t n = 0;   // blocks so far, of every warp by itself
  bool alive = true;

  if (warp == 8) {
    if (lane == 0) {
      const uint32_t bytes = (uint32_t)(p.a_rows * kBlock + kMmBBytes);
      for (int64_t item = blockIdx.x; alive && item < p.items; item += gridDim.x) {
        const MmItem w = mm_item(p, item);
        for (int j = w.j0; j < w.j1; ++j, ++n) {
          const uint32_t s = n % kMmStages, turn = n / kMmStages;
          if (!wait_alive(&empty[s], (turn & 1) ^ 1, dead, p.wait_cycles)) {
            alive = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], bytes);
          if (!p.drop_loads) {
            tma_load_2d(ring + s * kMmStageBytes, &a_map, j * kBlock, (int32_t)w.m0, smem_addr(&full[s]));
            tma_load_2d(ring + s * kMmStageBytes + kMmABytes, &b_map, j * kBlock, (int32_t)w.n0, smem_addr(&full[s]));
          }
        }
      }
    }
  } else if (warp == 9) {
    if (lane == 0) {
      constexpr uint32_t idesc = umma_e4m3(kMmRows, kMmCols);
      for (int64_t item = blockIdx.x; alive && item < p.items; item += gridDim.x) {
        const MmItem w = mm_item(p, item);
        for (int j = w.j0; j < w.j1; ++j, ++n) {
          const uint32_t s = n % kMmStages, b = n & 1;
          if (!wait_alive(&taken[b], ((n >> 1) & 1) ^ 1, dead, p.wait_cycles) ||
              !wait_alive(&full[s], (n / kMmStages) & 1, dead, p.wait_cycles)) {
            alive = false;
            break;
          }
          tcgen05_fence_after();
          const uint64_t da = umma_operand(ring + s * kMmStageBytes), db = umma_operand(ring + s * kMmStageBytes + kMmABytes);
#pragma unroll
          for (int k = 0; k < kBlock / 32; ++k) umma_f8(tmem + b * kMmCols, da + 2 * k, db + 2 * k, idesc, k > 0);
          umma_commit(smem_addr(&empty[s]));
          umma_commit(smem_addr(&done[b]));
        }
      }
    }
  } else {
    const int half = warp >> 2;                        // columns 128 half .. of the tile
    const uint32_t lanes = (uint32_t)(warp & 3) * 32;  // of tensor memory: rows of the tile
    unsigned char* turn = smem + kMmOutOff + warp * 2048;
    float* cols = reinterpret_cast<float*>(smem + kMmScaleOff) + warp * 256;
    const uint32_t from = tmem + (lanes << 16) + half * 128;
    for (int64_t item = blockIdx.x; item < p.items; item += gridDim.x) {
      const MmItem w = mm_item(p, item);
      const int64_t row0 = w.m0 + lanes, col0 = w.n0 + half * 128;
      const bool active = row0 < p.M && col0 < p.N;    // otherwise the warp has no results here
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.0f, 0.0f);
      const float* sa = p.sa + row0 + lane;
      const bool row = row0 + lane < p.M;
      // scales are fetched two blocks ahead
      auto row_scale = [&](int j) { return row && j < w.j1 ? sa[j * p.ldsa] : 0.0f; };
      auto col_scale = [&](int j) -> float4 {
        float4 c = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!active || j >= w.j1) return c;
        if (TILE) {
          c.x = p.sb[col0 / kBlock * p.ldsb + j];
        } else {
          const int64_t at = col0 + lane * 4;
          const float* q = p.sb + j * p.ldsb + at;
          if (at + 4 <= p.N) c = *reinterpret_cast<const float4*>(q);
          else {
            if (at < p.N) c.x = q[0];
            if (at + 1 < p.N) c.y = q[1];
            if (at + 2 < p.N) c.z = q[2];
          }
        }
        return c;
      };
      float r0 = row_scale(w.j0), r1 = row_scale(w.j0 + 1);
      float4 c0 = col_scale(w.j0), c1 = col_scale(w.j0 + 1);
      for (int j = w.j0; alive && j < w.j1; ++j, ++n) {
        const uint32_t b = n & 1;
        const float rs = r0;
        const float4 cs = c0;
        r0 = r1;
        c0 = c1;
        r1 = row_scale(j + 2);
        c1 = col_scale(j + 2);
        if (!TILE) *reinterpret_cast<float4*>(cols + b * 128 + lane * 4) = cs;
        const bool ok = wait_alive(&done[b], (n >> 1) & 1, dead, p.wait_cycles);
        alive = __all_sync(kFullMask, ok);   // also orders the column scales within the warp
        if (!alive) break;
        tcgen05_fence_after();
        if (active) {
          const float2 s = TILE ? make_float2(rs * cs.x, rs * cs.x) : make_float2(rs, rs);
          const float* cb = cols + b * 128;
          float t[2][16];
          tmem_load16(from + b * kMmCols, t[0]);
          tmem_wait(t[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (c < 7) tmem_load16(from + b * kMmCols + (c + 1) * 16, t[(c + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 v = make_float2(t[c & 1][2 * i], t[c & 1][2 * i + 1]);
              if (TILE) {
                acc[c * 8 + i] = __ffma2_rn(v, s, acc[c * 8 + i]);
              } else {
                const float2 q = *reinterpret_cast<const float2*>(cb + c * 16 + 2 * i);
                acc[c * 8 + i] = __ffma2_rn(__fmul2_rn(v, s), q, acc[c * 8 + i]);
              }
            }
            if (c < 7) tmem_wait(t[(c + 1) & 1]);
          }
        }
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&taken[b]));
      }
      if (!alive) {
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = make_float2(__int_as_float(0x7FC00000), __int_as_float(0x7FC00000));
      }
      if (active) {
        if (p.parts > 1) {
          float* to = p.part + (item % p.parts) * p.M * p.ldp;
          mm_store<float, false>(acc, turn, to, p.ldp, row0, p.M, col0, p.N, lane, true);
        } else if (p.accumulate) {
          mm_store<TO, true>(acc, turn, reinterpret_cast<TO*>(p.out), p.ldo, row0, p.M, col0, p.N, lane, p.vec != 0);
        } else {
          mm_store<TO, false>(acc, turn, reinterpret_cast<TO*>(p.out), p.ldo, row0, p.M, col0, p.N, lane, p.vec != 0);
        }
      }
    }
  }
  __syncwarp();
  tcgen05_fence_before();
  __syncthreads();
  if (*dead) {
    // copies and products under way end before shared and tensor memory are given up
    if (threadIdx.x == 256 && !p.drop_loads)
      for (uint32_t k = n < kMmStages ? 0 : n - kMmStages; k < n; ++k)
        (void)mbar_wait_bounded(&full[k % kMmStages], (k / kMmStages) & 1, 4000000000LL);
    if (threadIdx.x == 288) {
      umma_commit(smem_addr(drain));
      (void)mbar_wait_bounded(drain, 0, 4000000000LL);
    }
    __syncthreads();
  }
  if (warp == 9) {
    __syncwarp();
    tcgen05_fence_after();
    tmem_free(tmem, kMmColumns);
  }
}

// Sums of the parts of the inner dimension, in their order.
template <typename TO>
__global__ void __launch_bounds__(256) block_matmul_join_kernel(const BlockMatmulParams p) {
  begin_overlapped();
  const int64_t quads = p.ldp / 4, total = p.M * quads;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / quads, n = (i - m * quads) * 4;
    const float* q = p.part + m * p.ldp + n;
    float4 s = *reinterpret_cast<const float4*>(q);
    for (int k = 1; k < p.parts; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(q + k * p.M * p.ldp);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    TO* to = reinterpret_cast<TO*>(p.out) + m * p.ldo + n;
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) to[e] = (TO)(p.accumulate ? v[e] + (float)to[e] : v[e]);
  }
}

}  // namespace vsamp
