// Product of two matrices in e4m3 blocks of 128 on the tensor cores.
//
//   out[m, n] = sum over blocks j of sa[m, j] * sb[n, j] * sum over k in j of a[m, k] * b[n, k]
//
// One CTA per SM walks over tiles of 128 x 256 results, or a pair of CTAs over tiles of 256 x 256. A warp copies blocks of
// both operands into a ring in shared memory (tensor copies with the 128-byte swizzle the tensor cores read), another issues
// four products of 32 inner elements per block into one of two accumulators in tensor memory, and sixteen warps take each
// finished block out of tensor memory and add it, scaled, to fp32 sums in registers: the sum of a block's 128 products is
// the only one that the tensor core forms. With 128 x 128 blocks of b, whose scale is the same for a warp's 64 columns, a row
// of a is a lane, and its scale one register; with one scale per row of b a lane takes 4 rows and 16 columns.
//
// What bounds it with many rows is the sums, not the products (512 cycles per block at the tensor cores' rate, 4.6 PFLOP/s
// measured): 2048 x 16384 x 32768 takes 750 us (2.9 PFLOP/s), 700 without the multiply-adds, 650 without reading tensor
// memory, 474 as products alone. Each of the sixteen warps takes every block, one wait, two reads of tensor memory of about
// 100 cycles and 32 paired multiply-adds; and a product waits until its accumulator has been read, two blocks back, through
// a completion (235 cycles), that reading and a release (190). So the warp with the scales joins the products' arrival, which
// leaves one wait (850 -> 754 us), and all operands of copies and products come from uniform registers (894 -> 849). Four
// accumulators of 128 columns, two issuing warps, deeper reads in smaller steps were measured and are slower. A pair of CTAs
// holds half of b each: 32 KB per block and CTA instead of 48, which 64 bytes per cycle from the L2 would take 750 cycles for.
//
// With few rows it streams b: 64 x 151936 x 4096 takes 100 us (96 % of the copy rate).
//
// Every wait is bounded. A CTA one of whose waits gave up lets its copies and products end, frees its tensor memory and
// leaves NaN in the results that it had not finished. A pair's CTAs tell each other how many blocks they copied, since one
// may have given up before the other: rank 0, on whose barriers the copies of both are counted, waits for those of both.
#pragma once

#include "vsamp_block_quant.cuh"
#include "vsamp_tensor.cuh"

namespace vsamp {

constexpr int kMmRows = 128, kMmCols = 256;         // results of a CTA by itself; of a CTA of a pair as many
constexpr int kMmWarps = 16;                        // warps of sums: 32 rows x 64 columns each
constexpr int kMmThreads = kMmWarps * 32 + 128;     // and a warpgroup: the copying, the issuing, the scales' warp, one idle
constexpr int kMmSumRegs = 112, kMmOtherRegs = 32;  // registers per thread: 512 x 112 + 128 x 32 of the launch's 640 x 96
constexpr int kMmColumns = 512;                     // of tensor memory: two accumulators
// A block's scales, 128 of rows and 256 of columns, have a ring of their own: they are read after the block's products are
// done, when its stage may be written again. Block n is copied once the products of block n - stages are done, whose
// accumulator had held block n - stages - 2: every warp had read that one out of it, and used all scales of the block before.
// So eight sets do for up to five stages.
constexpr int kMmScaleSets = 8, kMmScaleBytes = (kMmRows + kMmCols) * 4;

template <int G>
struct MmShape {
  static constexpr int ABytes = kMmRows * kBlock, BRows = kMmCols / G, BBytes = BRows * kBlock;
  static constexpr int StageBytes = ABytes + BBytes, Stages = G == 1 ? 3 : 4;
  static constexpr int OutOff = Stages * StageBytes;            // per warp 32 rows of 128 bytes of results
  static constexpr int ScaleOff = OutOff + kMmWarps * 4096;
  static constexpr int BarOff = ScaleOff + kMmScaleSets * kMmScaleBytes;
  static constexpr int Smem = BarOff + 256 + 1024;              // and what aligns the ring to 1024 bytes
};

struct BlockMatmulParams {
  const float* sb;           // of 128 x 128 blocks: the others come by their tensor map
  int64_t ldsb, ldo;
  int M, N;
  int items;                 // tiles as a whole, then parts of the inner dimension of the others
  int whole;                 // tiles as a whole
  unsigned char* out;
  float* part;               // [tile, part, part_rows, 256] sums of the divided tiles
  int part_rows;             // rows of a tile, or of the matrix if that has fewer
  int across, inner_tiles;   // tiles follow each other along a row of results, or down a column; tiles of one
  int blocks, parts;
  int a_rows;                // rows of a per copy
  int accumulate;
  // Results leave as boxes of the output's tensor map, whose rows begin on 16-byte boundaries: 2, all of them; 1, those of 64
  // whole columns (a copy ends at a multiple of 16 bytes, so the rows' end has to be one); 0, none.
  int boxes;
  int pairs;                 // rows of results begin on the boundary of two elements
  int drop_loads;            // test: copies are expected and never made
  int stop0, stop1;          // test: blocks after which the copying warp of a CTA of rank 0, 1 ends
  long long wait_cycles;
};

// Where a tile begins.
__device__ __forceinline__ void mm_origin(const BlockMatmulParams& p, int tile, int tile_rows, int& m0, int& n0) {
  const int u = tile / p.inner_tiles, v = tile - u * p.inner_tiles;
  m0 = (p.across ? u : v) * tile_rows;
  n0 = (p.across ? v : u) * kMmCols;
}

struct MmItem {
  int m0, n0, j0, j1;
  int part;   // of all parts, -1 for a tile as a whole
};
template <int G>
__device__ __forceinline__ MmItem mm_item(const BlockMatmulParams& p, int item) {
  MmItem w;
  w.part = item - p.whole;
  int tile = item;
  w.j0 = 0;
  w.j1 = p.blocks;
  if (w.part >= 0) {
    const int t = w.part / p.parts, k = w.part - t * p.parts;
    tile = p.whole + t;
    w.j0 = (int)((int64_t)p.blocks * k / p.parts);
    w.j1 = (int)((int64_t)p.blocks * (k + 1) / p.parts);
  }
  mm_origin(p, tile, kMmRows * G, w.m0, w.n0);
  return w;
}

// Columns of a tile that are computed: whole 64 of a warp, fewer at the matrix' end (19456 x 64 x 15000: 54 us, with all 256
// columns 57). A pair's halves of b are halves of them.
__device__ __forceinline__ int mm_columns(const BlockMatmulParams& p, int n0) {
  return p.N - n0 < kMmCols ? (p.N - n0 + 63) & ~63 : kMmCols;
}

// Sums of a warp's 32 rows x 64 columns. TILE: a lane has a row, its columns 2 i and 2 i + 1 in acc[i]. Otherwise acc[4 k + 2 h
// + i] holds the columns 8 k + 2 (lane % 4) and the next of row 16 h + 8 i + lane / 4: 16 columns' scales per lane instead of
// 64, which took more of the registers and of shared memory's reads (151936 x 2048 x 2048, added: 750 us, 772 with a row per
// lane).
//
// 32 rows x 128 bytes of results, 32 fp32 or 64 bf16 columns, to the warp's box. A row's 16-byte pieces are permuted by the
// row (the 128-byte swizzle): no bank conflicts.
template <typename T, bool TILE>
__device__ __forceinline__ void mm_box(const float2 (&acc)[32], int c, unsigned char* box, int lane) {
  if constexpr (TILE) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      uint4 w;
      if constexpr (sizeof(T) == 4) {
        const float2 a = acc[c * 16 + q * 2], b = acc[c * 16 + q * 2 + 1];
        w = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
      } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 h = __float22bfloat162_rn(acc[q * 4 + i]);
          memcpy(&u[i], &h, 4);
        }
        w = make_uint4(u[0], u[1], u[2], u[3]);
      }
      *reinterpret_cast<uint4*>(box + lane * 128 + ((q ^ (lane & 7)) << 4)) = w;
    }
  } else {
    const int r = lane >> 2, e = lane & 3;
#pragma unroll
    for (int hi = 0; hi < 4; ++hi) {
      unsigned char* to = box + (8 * hi + r) * 128;
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<float2*>(to + (((2 * k + (e >> 1)) ^ r) << 4) + (e & 1) * 8) = acc[(c * 4 + k) * 4 + hi];
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<__nv_bfloat162*>(to + ((k ^ r) << 4) + e * 4) = __float22bfloat162_rn(acc[k * 4 + hi]);
      }
    }
  }
}

// A warp's 32 rows x 64 columns to boxes of the map; the copies run on while the warp goes on.
template <typename T, bool TILE>
__device__ __forceinline__ void mm_store_boxes(const float2 (&acc)[32], unsigned char* box, const CUtensorMap* map, int m0,
                                               int n0, int N, int part, int lane, bool add) {
  constexpr int C = 128 / sizeof(T);   // columns of a box
#pragma unroll
  for (int c = 0; c < 64 / C; ++c) {
    if (n0 + c * C >= N) break;
    if (lane == 0) bulk_read_done();   // of the box's last use
    __syncwarp();
    mm_box<T, TILE>(acc, c, box, lane);
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) tma_store_3d(map, n0 + c * C, m0, part, smem_addr(box), add);
  }
}

// The same to rows at any address, fp32 in the box, 16 rows of 64 columns at a time: a lane takes two neighbours (`pairs`:
// every row begins on their boundary) or two columns 32 apart: 32003 x 2050 x 1501 added to fp32 171 us and 180, 32003 x 2302 x
// 1501 added to bf16 219 and 539 (of pairs, eight rows are read at once; one after another they take 364).
template <typename T, bool TILE, bool ADD16>
__device__ __forceinline__ void mm_store_rows(const float2 (&acc)[32], unsigned char* box, T* out, int64_t ldo, int m0, int M,
                                              int n0, int N, int lane, bool add, bool pairs) {
#pragma unroll 1
  for (int h = 0; h < 32 && m0 + h < M; h += 16) {
    if (lane == 0) bulk_read_done();   // an earlier tile may have left as a box
    __syncwarp();
    if constexpr (TILE) {
      if ((lane & 16) == h) {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const float2 a = acc[q * 2], b = acc[q * 2 + 1];
          *reinterpret_cast<float4*>(box + (lane & 15) * 256 + ((q ^ (lane & 7)) << 4)) = make_float4(a.x, a.y, b.x, b.y);
        }
      }
    } else {
      const int r = lane >> 2, e = lane & 3;
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<float2*>(box + (8 * i + r) * 256 + (((2 * k + (e >> 1)) ^ r) << 4) + (e & 1) * 8) =
              h ? acc[k * 4 + 2 + i] : acc[k * 4 + i];
    }
    __syncwarp();
    const int rows = M - m0 - h < 16 ? M - m0 - h : 16, c = pairs ? 2 * lane : lane;
    T* to = out + (m0 + h) * ldo + n0 + c;
    if (pairs && n0 + c + 1 < N) {
      auto value = [&](int r) {
        return *reinterpret_cast<const float2*>(box + r * 256 + (((lane >> 1) ^ (r & 7)) << 4) + (lane & 1) * 8);
      };
      if constexpr (ADD16) {   // the sums are added before the rounding; what they are added to is read eight rows at once
        constexpr int kAhead = 8;
#pragma unroll 1
        for (int r = 0; r < rows; r += kAhead, to += kAhead * ldo) {
          __nv_bfloat162 w[kAhead];
#pragma unroll
          for (int k = 0; k < kAhead; ++k)
            if (r + k < rows) w[k] = *reinterpret_cast<const __nv_bfloat162*>(to + k * ldo);
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const float2 v = value(r + k), u = __bfloat1622float2(w[k]);
            if (r + k < rows) *reinterpret_cast<__nv_bfloat162*>(to + k * ldo) = __float22bfloat162_rn(make_float2(v.x + u.x, v.y + u.y));
          }
        }
      } else {
#pragma unroll 8
        for (int r = 0; r < rows; ++r, to += ldo) {
          const float2 v = value(r);
          if constexpr (sizeof(T) == 2)
            *reinterpret_cast<__nv_bfloat162*>(to) = __float22bfloat162_rn(v);
          else if (add)   // one addition per element and call: the same result every time; below 2^-126 this one counts zeros
            asm volatile("red.relaxed.gpu.global.add.v2.f32 [%0], {%1, %2};" ::"l"(to), "f"(v.x), "f"(v.y) : "memory");
          else
            *reinterpret_cast<float2*>(to) = v;
        }
      }
    } else {
      const int step = pairs ? 64 : 32;   // of pairs only the last column is left
#pragma unroll 1
      for (int k = 0; k < 64 && n0 + c + k < N; k += step, to += step) {
        T* at = to;
        const int piece = (c + k) >> 2;
#pragma unroll 8
        for (int r = 0; r < rows; ++r, at += ldo) {
          const float v = *reinterpret_cast<const float*>(box + r * 256 + ((piece ^ (r & 7)) << 4) + (c & 3) * 4);
          if constexpr (sizeof(T) == 4) {
            if (add) asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(at), "f"(v) : "memory");
            else *at = v;
          } else {
            *at = (T)(ADD16 ? v + (float)*at : v);
          }
        }
      }
    }
  }
}

// 32 columns of a block, times the row's scale (and the 128 x 128 block's of b), to the sums.
__device__ __forceinline__ void mm_sums(const float (&t)[32], float2 rs, float2 (&acc)[32], int at) {
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[at + i] = __ffma2_rn(make_float2(t[2 * i], t[2 * i + 1]), rs, acc[at + i]);
}

// 16 rows and 32 columns of a block, times the scales of both.
__device__ __forceinline__ void mm_sums(const float (&t)[16], const float (&rs)[4], const float2 (&cs)[4], float2 (&acc)[32],
                                        int c, int h) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float r = rs[2 * h + i];
      float2& a = acc[(c * 4 + k) * 4 + 2 * h + i];
      a = __ffma2_rn(__fmul2_rn(make_float2(t[4 * k + 2 * i], t[4 * k + 2 * i + 1]), make_float2(r, r)), cs[k], a);
    }
}

// ADD16: bf16 results are added to what is there. A kernel of its own, since those reads take registers that the others miss
// (16384 x 8192 x 2048 written as bf16: 263 us, 270 in one kernel with it).
template <typename TO, bool TILE, int G, bool ADD16>
__global__ void __launch_bounds__(kMmThreads, 1) block_matmul_kernel(const BlockMatmulParams p,
                                                                     const __grid_constant__ CUtensorMap a_map,
                                                                     const __grid_constant__ CUtensorMap b_map,
                                                                     const __grid_constant__ CUtensorMap o_map,
                                                                     const __grid_constant__ CUtensorMap sa_map,
                                                                     const __grid_constant__ CUtensorMap sb_map,
                                                                     const __grid_constant__ CUtensorMap p_map) {
  using S = MmShape<G>;
  constexpr bool kPair = G == 2;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((0u - smem_addr(smem_raw)) & 1023u);
  const uint32_t ring = smem_addr(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::BarOff);   // a stage's copies have landed (rank 0's)
  uint64_t* done = full + S::Stages;                                // a stage's products are done: an accumulator holds them
  uint64_t* taken = done + S::Stages;                               // an accumulator has been read (rank 0's)
  uint64_t* drain = taken + 2;
  uint64_t* scaled = drain + 1;                                     // a set of scales has landed
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(scaled + kMmScaleSets);
  volatile int* dead = reinterpret_cast<volatile int*>(tmem_at + 1);
  volatile uint32_t* other = tmem_at + 2;   // of the pair's other CTA, at the end: blocks copied, and whether it gave up
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = kPair ? blockIdx.x & 1 : 0;
  const int first = blockIdx.x / G, stride = gridDim.x / G;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::Stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&done[i], 2);   // the products and the scales
    }
    for (int i = 0; i < 2; ++i) mbar_init(&taken[i], kMmWarps * G);
    for (int i = 0; i < kMmScaleSets; ++i) mbar_init(&scaled[i], 1);
    mbar_init(drain, 1);
    *dead = 0;
    *other = 0;
    fence_mbar_init();
  }
  if (warp == kMmWarps + 1) tmem_alloc<G>(smem_addr(tmem_at), kMmColumns);
  if (threadIdx.x == kMmWarps * 32) {
    tma_prefetch_map(&a_map);
    tma_prefetch_map(&b_map);
    tma_prefetch_map(&sa_map);
    if (!TILE) tma_prefetch_map(&sb_map);
    if (p.boxes) tma_prefetch_map(&o_map);
  }
  tcgen05_fence_before();
  __syncthreads();
  if (kPair) cluster_barrier_shared();   // the barriers and tensor memory of both CTAs are ready
  tcgen05_fence_after();
  const uint32_t tmem = *tmem_at;
  begin_overlapped();
  uint32_t n = 0;   // blocks so far, of every warp by itself
  bool alive = true;

  if (warp >= kMmWarps) {
    fewer_registers<kMmOtherRegs>();
    uint32_t s = 0, turn = 0;   // stage of block n, and the parity of its phase
    if (warp == kMmWarps) {
      const uint32_t bytes = (uint32_t)(p.a_rows * kBlock + S::BBytes) * G;
      for (int item = first; alive && item < p.items; item += stride) {
        const MmItem w = mm_item<G>(p, item);
        const int row0 = w.m0 + (int)rank * kMmRows, col0 = w.n0 + (int)rank * (mm_columns(p, w.n0) / G);
        for (int j = w.j0; j < w.j1; ++j, ++n) {
          alive = __all_sync(kFullMask, wait_alive<G>(&done[s], turn ^ 1, dead, p.wait_cycles)) &&
                  n < (uint32_t)(rank ? p.stop1 : p.stop0);
          if (!alive) break;
          if (elect_one()) {
            const uint32_t set = n % kMmScaleSets, scales = ring + S::ScaleOff + set * kMmScaleBytes;
            const uint32_t at = ring + s * S::StageBytes;
            if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
            mbar_arrive_expect_tx(&scaled[set], TILE ? kMmRows * 4 : kMmScaleBytes);
            if (!p.drop_loads) {
              if (kPair) {
                const uint32_t bar = dsmem_map(&full[s], 0);
                tma_load_2d_pair(at, &a_map, j * kBlock, row0, bar);
                tma_load_2d_pair(at + S::ABytes, &b_map, j * kBlock, col0, bar);
              } else {
                tma_load_2d(at, &a_map, j * kBlock, row0, smem_addr(&full[s]));
                tma_load_2d(at + S::ABytes, &b_map, j * kBlock, col0, smem_addr(&full[s]));
              }
              tma_load_2d(scales, &sa_map, row0, j, smem_addr(&scaled[set]));
              if (!TILE) tma_load_2d(scales + kMmRows * 4, &sb_map, w.n0, j, smem_addr(&scaled[set]));
            }
          }
          __syncwarp();
          if (++s == S::Stages) {
            s = 0;
            turn ^= 1;
          }
        }
      }
    } else if (warp == kMmWarps + 1 && rank == 0) {
      for (int item = first; alive && item < p.items; item += stride) {
        const MmItem w = mm_item<G>(p, item);
        const uint32_t idesc = umma_e4m3(kMmRows * G, mm_columns(p, w.n0));
        for (int j = w.j0; j < w.j1; ++j, ++n) {
          const uint32_t b = n & 1;
          alive = __all_sync(kFullMask, wait_alive<G>(&full[s], turn, dead, p.wait_cycles) &&
                                            wait_alive<G>(&taken[b], ((n >> 1) & 1) ^ 1, dead, p.wait_cycles));
          if (!alive) break;
          tcgen05_fence_after();
          if (elect_one()) {
            const uint32_t at = ring + s * S::StageBytes;
            const uint64_t da = umma_operand(at), db = umma_operand(at + S::ABytes);
#pragma unroll
            for (int k = 0; k < kBlock / 32; ++k) umma_f8<G>(tmem + b * kMmCols, da + 2 * k, db + 2 * k, idesc, k > 0);
            umma_commit<G>(smem_addr(&done[s]));
          }
          __syncwarp();
          if (++s == S::Stages) {
            s = 0;
            turn ^= 1;
          }
        }
      }
    } else if (warp == kMmWarps + 2) {
      // The scales of a block's rows, times those of the 128 x 128 blocks, for the warps of sums: its arrival joins the
      // products', so that they wait once per block and read one number each.
      for (int item = first; alive && item < p.items; item += stride) {
        const MmItem w = mm_item<G>(p, item);
        const float* sb = p.sb + (TILE ? w.n0 / kBlock * p.ldsb : 0);
        const bool second = w.n0 + kBlock < p.N;
        for (int j = w.j0; j < w.j1; ++j, ++n) {
          const uint32_t set = n % kMmScaleSets;
          float t0 = 0.0f, t1 = 0.0f;
          if (TILE) {
            // plain loads: the kernel may have begun while the one that writes these scales still ran
            t0 = sb[j];
            if (second) t1 = sb[p.ldsb + j];
          }
          alive = __all_sync(kFullMask, wait_alive<G>(&scaled[set], (n / kMmScaleSets) & 1, dead, p.wait_cycles));
          if (!alive) break;
          if (TILE) {
            float* scales = reinterpret_cast<float*>(smem + S::ScaleOff + set * kMmScaleBytes);
            const float4 r = *reinterpret_cast<const float4*>(scales + lane * 4);
            float* to = scales + kMmRows + lane * 4;
            *reinterpret_cast<float4*>(to) = make_float4(r.x * t0, r.y * t0, r.z * t0, r.w * t0);
            *reinterpret_cast<float4*>(to + kMmRows) = make_float4(r.x * t1, r.y * t1, r.z * t1, r.w * t1);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&done[s]));
          if (++s == S::Stages) {
            s = 0;
            turn ^= 1;
          }
        }
      }
    }
  } else {
    more_registers<kMmSumRegs>();
    const int quarter = warp >> 2;                     // columns 64 quarter .. of the tile
    const uint32_t lanes = (uint32_t)(warp & 3) * 32;  // of tensor memory: rows of the tile
    unsigned char* box = smem + S::OutOff + warp * 4096;
    auto release = [&](uint32_t b) {   // one lane
      if (kPair) mbar_arrive_pair(dsmem_map(&taken[b], 0));
      else mbar_arrive(smem_addr(&taken[b]));
    };
    const uint32_t from = tmem + (lanes << 16) + quarter * 64;
    uint32_t s = 0, turn = 0;   // with a power of two of stages they are bits of n
    for (int item = first; item < p.items; item += stride) {
      const MmItem w = mm_item<G>(p, item);
      const int row0 = w.m0 + (int)(rank * kMmRows + lanes), col0 = w.n0 + quarter * 64;
      const bool active = row0 < p.M && col0 < p.N;    // otherwise the warp has no results here
      float2 acc[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[i] = make_float2(0.0f, 0.0f);
      for (int j = w.j0; j < w.j1; ++j, ++n) {
        const uint32_t b = n & 1, set = n % kMmScaleSets;
        const float* scales = reinterpret_cast<const float*>(smem + S::ScaleOff + set * kMmScaleBytes);
        const float* cb = scales + kMmRows + quarter * 64;                          // of columns, or
        const float* row = scales + (TILE ? kMmRows + (quarter >> 1) * kMmRows : 0) + lanes;   // of rows times the block's
        // A wait that gives up marks the CTA, and the pair's other one, which is looked at once per tile. Its warp goes on and
        // passes accumulators on that were not waited for: the next products in them reach marked CTAs alone.
        if (S::Stages == 4) {
          s = n % 4;
          turn = (n / 4) & 1;
        }
        (void)wait_alive<G>(&done[s], turn, dead, p.wait_cycles);
        if (S::Stages != 4 && ++s == S::Stages) {
          s = 0;
          turn ^= 1;
        }
        __syncwarp();
        tcgen05_fence_after();
        if (active) {
          auto read = [&] {   // all of the warp's part has been read
            tcgen05_fence_before();
            __syncwarp();
            if (lane == 0) release(b);
          };
          if constexpr (TILE) {
            const float rs = row[lane];
            const float2 r2 = make_float2(rs, rs);
            float t[32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              tmem_read(from + b * kMmCols + c * 32, t);
              if (c == 1) read();
              mm_sums(t, r2, acc, c * 16);
            }
          } else {
            float rs[4], t[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) rs[i] = row[8 * i + (lane >> 2)];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float2 cs[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) cs[k] = *reinterpret_cast<const float2*>(cb + c * 32 + 8 * k + 2 * (lane & 3));
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                tmem_read_16(from + b * kMmCols + c * 32 + (h << 20), t);
                if (c == 1 && h == 1) read();
                mm_sums(t, rs, cs, acc, c, h);
              }
            }
          }
        } else if (lane == 0) {
          release(b);
        }
      }
      if (*dead) {
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[i] = make_float2(__int_as_float(0x7FC00000), __int_as_float(0x7FC00000));
      }
      if (active) {
        const bool add = p.accumulate != 0;
        if (w.part >= 0) {
          mm_store_boxes<float, TILE>(acc, box, &p_map, row0 - w.m0, col0 - w.n0, kMmCols, w.part, lane, false);
        } else if (!ADD16 && (p.boxes == 2 || (p.boxes == 1 && col0 + 64 <= p.N))) {
          mm_store_boxes<TO, TILE>(acc, box, &o_map, row0, col0, p.N, 0, lane, add);
        } else {
          mm_store_rows<TO, TILE, ADD16>(acc, box, reinterpret_cast<TO*>(p.out), p.ldo, row0, p.M, col0, p.N, lane, add, p.pairs != 0);
        }
      }
    }
    if (lane == 0) {
      bulk_done();
      if (kPair) fence_cluster();   // its last arrivals have reached the other CTA, whose shared memory goes behind the barrier
    }
  }
  __syncwarp();
  tcgen05_fence_before();
  __syncthreads();
  bool gave_up = *dead != 0;
  uint32_t copied = n;   // by the other CTA; counts of the copying warps alone are used
  if (kPair) {
    // both CTAs have to come to the same answer: what follows, the freeing of tensor memory too, they do together
    if (threadIdx.x == kMmWarps * 32) dsmem_publish_u32(dsmem_map(const_cast<uint32_t*>(other), rank ^ 1), n * 2 + (gave_up ? 1 : 0));
    __syncwarp();
    // the other CTA's arrivals and, if neither gave up, its products have ended before this one's shared and tensor memory go
    cluster_barrier_shared();
    gave_up |= (*other & 1) != 0;
    copied = *other >> 1;
  }
  if (gave_up) {
    // copies and products under way end before shared and tensor memory are given up
    if (threadIdx.x == kMmWarps * 32 && !p.drop_loads) {
      // neither CTA is more than the stages ahead of the products; before that all copies have been waited for
      const uint32_t most = n > copied ? n : copied, half = (uint32_t)(p.a_rows * kBlock + S::BBytes);
      for (uint32_t k = most < S::Stages ? 0 : most - S::Stages; rank == 0 && k < most; ++k) {
        if (k >= n) mbar_arrive_expect_tx(&full[k % S::Stages], half);   // copied by the other CTA alone
        else if (k >= copied) mbar_complete_tx(&full[k % S::Stages], half);   // expected of it and not copied
        (void)mbar_wait_bounded(&full[k % S::Stages], (k / S::Stages) & 1, 4000000000LL);
      }
      for (uint32_t k = n < kMmScaleSets ? 0 : n - kMmScaleSets; k < n; ++k)
        (void)mbar_wait_bounded(&scaled[k % kMmScaleSets], (k / kMmScaleSets) & 1, 4000000000LL);
    }
    if (warp == kMmWarps + 1) {
      if (rank == 0 && elect_one()) umma_commit<G>(smem_addr(drain));   // by the thread that issued the products
      __syncwarp();
      (void)mbar_wait_bounded(drain, 0, 4000000000LL);
      __syncwarp();
    }
    __syncthreads();
    if (kPair) cluster_barrier_shared();
  }
  if (warp == kMmWarps + 1) {
    __syncwarp();
    tcgen05_fence_after();
    tmem_free<G>(tmem, kMmColumns);
  }
}

// Sums of the parts of the divided tiles, in their order.
template <typename TO>
__global__ void __launch_bounds__(256) block_matmul_join_kernel(const BlockMatmulParams p, int tile_rows) {
  begin_overlapped();
  constexpr int Q = kMmCols / 4;
  const int tiles = (p.items - p.whole) / p.parts;
  const int64_t total = (int64_t)tiles * p.part_rows * Q, one = (int64_t)p.part_rows * kMmCols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / Q;
    const int t = (int)(row / p.part_rows), r = (int)(row - (int64_t)t * p.part_rows), c = (int)(i - row * Q) * 4;
    int m, n;
    mm_origin(p, p.whole + t, tile_rows, m, n);
    m += r;
    n += c;
    if (m >= p.M || n >= p.N) continue;
    const float* q = p.part + t * p.parts * one + (int64_t)r * kMmCols + c;
    float4 s = *reinterpret_cast<const float4*>(q);
    for (int k = 1; k < p.parts; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(q + k * one);
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
