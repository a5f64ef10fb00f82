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
// Packed layout. Vocabulary rows in tiles of 16, the inner dimension in units of 128 (two blocks of 64): the record of
// a tile and unit is contiguous, so a warp streams its tile's records in order. A record holds, for each of its one
// or two blocks, 512 bytes of codes (lane l of a warp owns 16: one 32-bit word per 16-wide matrix step, whose nibbles
// are the lane's eight elements of the 16 x 16 operand), then the scales of its groups as [group][8][2] (rows r and
// r + 8 side by side, the two a lane needs), then their zero points the same way as bytes. Nibble pairs (i, i + 4)
// of a word are one operand register:
//   i = 0: row l/4,     columns 2 (l%4) + {0, 1}        i = 1: row l/4 + 8, the same columns
//   i = 2: row l/4,     columns 2 (l%4) + 8 + {0, 1}    i = 3: row l/4 + 8, the same columns
// The last record of a tile has only the blocks and groups that D reaches. One record of slack ends the buffer.
#pragma once

#include "vsamp.h"
#include "vsamp_device.cuh"

namespace vsamp {

constexpr int kHeadWarps = 16;
constexpr int kHeadBlock = 64;      // inner elements per block of a tile
constexpr int kHeadUnit = 128;      // inner elements a warp processes at once: two blocks, the largest group
constexpr int kHeadUnitSteps = kHeadUnit / 16;

struct HeadShape {
  int64_t V, D;
  int group;
  int scale_bytes;   // 4 (fp32) or 2 (bf16)
  int has_zeros;
  __host__ __device__ int64_t tiles() const { return (V + 15) / 16; }
  __host__ __device__ int units() const { return (int)((D + kHeadUnit - 1) / kHeadUnit); }
  __host__ __device__ int blocks() const { return (int)((D + kHeadBlock - 1) / kHeadBlock); }
  __host__ __device__ int groups() const { return (int)(D / group); }
  __host__ __device__ int group_bytes() const { return 16 * (scale_bytes + has_zeros); }
  // bytes of a whole record, and of a tile (all of its records)
  __host__ __device__ int record() const { return 1024 + kHeadUnit / group * group_bytes(); }
  __host__ __device__ int64_t tile_bytes() const { return (int64_t)blocks() * 512 + (int64_t)groups() * group_bytes(); }
  // one record of slack: a warp fetches whole records, also where a tile's last one is shorter
  __host__ __device__ int64_t total() const { return tiles() * tile_bytes() + record(); }
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
  int vec;         // hidden rows are 16-byte aligned
  int units;       // units of the inner dimension (the last one may be padded)
  int chunk;       // units of hidden states staged at once
  int ring_off;    // bytes of staged states; the warps' rings follow, then the parts of split rows
  int red_off;
  int split;       // warps that share a row tile, each with its part of the inner dimension
};

// One thread per 32-bit word of codes, then per scale and zero point.
__global__ void __launch_bounds__(256) head_pack_kernel(const HeadPackParams p) {
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

// D = A B + C on 16 x 16 by 16 x 8 bf16 operands, fp32 sums
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b,
                                         float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
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

// (w & mask) | base: one instruction when both constants are in registers
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t base) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(base));
  return r;
}

// bf16 terms per hidden value: x = hi + mid + lo for fp32, each the bf16 nearest to what is left (24 bits in all).
template <typename T>
constexpr int kHeadTerms = sizeof(T) == 4 ? 3 : 1;

// Stages the hidden states of units [u0, u1) as the instruction's second operand. In step k, lane l needs hidden row
// 8 n + l/4 at inner positions 2 (l%4) + {0, 1} and + 8; they are stored as [step][term][8 NT rows][l%4], two registers
// each, so a row's 16 positions of a step are 32 contiguous bytes and the reads have constant offsets. Positions
// beyond D are 0; the places of rows beyond p.rows are not written (their columns of the product are not used).
template <typename T, int NT>
__device__ __forceinline__ void head_stage(const HeadParams& p, uint4* sh, int u0, int u1) {
  constexpr int TERMS = kHeadTerms<T>;
  const int rows = p.rows, n = (u1 - u0) * kHeadUnitSteps * rows;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    // neighbouring threads take neighbouring steps of a row: its bytes are read in order
    const int steps = (u1 - u0) * kHeadUnitSteps;
    const int r = i / steps, ks = i - r * steps;
    const int64_t k = (int64_t)u0 * kHeadUnit + ks * 16;
    const unsigned char* src = p.hidden + ((p.m0 + r) * p.ldh + k) * (int64_t)sizeof(T);
    const bool whole = p.vec && k + 16 <= p.s.D;
    uint32_t w[TERMS][8];   // pairs of neighbouring positions
    if constexpr (TERMS == 1) {
      if (whole) {
        const uint4 a = reinterpret_cast<const uint4*>(src)[0], b = reinterpret_cast<const uint4*>(src)[1];
        w[0][0] = a.x; w[0][1] = a.y; w[0][2] = a.z; w[0][3] = a.w;
        w[0][4] = b.x; w[0][5] = b.y; w[0][6] = b.z; w[0][7] = b.w;
      } else {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(src);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[0][e] = (k + 2 * e < p.s.D ? h[2 * e] : 0u) | (uint32_t)(k + 2 * e + 1 < p.s.D ? h[2 * e + 1] : 0u) << 16;
      }
    } else {
      const float* h = reinterpret_cast<const float*>(src);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float x[2];
        if (whole) {
          const float2 v = reinterpret_cast<const float2*>(src)[e];
          x[0] = v.x;
          x[1] = v.y;
        } else {
          x[0] = k + 2 * e < p.s.D ? h[2 * e] : 0.f;
          x[1] = k + 2 * e + 1 < p.s.D ? h[2 * e + 1] : 0.f;
        }
#pragma unroll
        for (int q = 0; q < TERMS; ++q) {
          uint32_t bits = 0;
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const __nv_bfloat16 v = __float2bfloat16_rn(x[z]);
            bits |= (uint32_t)__bfloat16_as_ushort(v) << (16 * z);
            // an infinity has no remainder (inf - inf would turn it into NaN)
            x[z] = isinf(__bfloat162float(v)) ? 0.f : x[z] - __bfloat162float(v);
          }
          w[q][e] = bits;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < TERMS; ++q) {
      uint4* to = sh + ((ks * TERMS + q) * (8 * NT) + r) * 2;
      to[0] = make_uint4(w[q][0], w[q][4], w[q][1], w[q][5]);
      to[1] = make_uint4(w[q][2], w[q][6], w[q][3], w[q][7]);
    }
  }
}

// 16 bytes from global to shared memory without registers; a group of such copies is awaited by its issuer.
__device__ __forceinline__ void copy_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// RT tiles of 16 vocabulary rows per warp, NT tiles of 8 hidden rows. Every warp streams the records of its row tiles
// through a ring of PF slots in shared memory (PF records of each tile in flight, no registers held by loads), across
// the ends of tiles. p.split warps of a CTA share a set of row tiles, each with a contiguous part of its units.
template <typename T, int NT, int RT, int GROUP, int PF>
__global__ void __launch_bounds__(kHeadWarps * 32, 1) head_kernel(const HeadParams p) {
  static_assert((PF & (PF - 1)) == 0, "slots are taken in turn by masking");
  constexpr int TERMS = kHeadTerms<T>;
  constexpr int GS = GROUP / 16;          // steps per group
  constexpr int NG = kHeadUnit / GROUP;   // groups per unit
  extern __shared__ __align__(128) unsigned char head_smem[];
  const HeadShape s = p.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nb = s.blocks(), ng = s.groups(), record = s.record();
  const int64_t nt = s.tiles(), tile_bytes = s.tile_bytes();
  const int part_of = warp % p.split;                     // this warp's part of the inner dimension
  const int slots = kHeadWarps / p.split;                 // sets of row tiles per CTA and round
  const int64_t stride = (int64_t)gridDim.x * slots * RT;
  const int64_t first0 = (int64_t)blockIdx.x * slots * RT, mine = (warp / p.split) * RT;
  const int rows = p.rows;
  const int gb = s.scale_bytes * 16;                      // bytes of a group's scales

  const uint32_t slot_bytes = (uint32_t)(RT * record);
  const uint32_t ring = (uint32_t)p.ring_off + (uint32_t)warp * PF * slot_bytes;   // this warp's ring, from head_smem
  const uint32_t smem0 = smem_addr(head_smem);

  const uint32_t gsel = lane >> 2;
  // two nibbles of a word, and 128 as bf16 twice; opaque, so that both stay in registers
  uint32_t nibbles, base;
  asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(nibbles));
  asm volatile("mov.b32 %0, 0x43004300;" : "=r"(base));

  // this warp's units [lo, hi) of the chunk that begins at unit c
  auto lo_of = [&](int c) { return c + min(p.chunk, p.units - c) * part_of / p.split; };
  auto hi_of = [&](int c) { return c + min(p.chunk, p.units - c) * (part_of + 1) / p.split; };
  // the next record to fetch: its tile and chunk, its address for this lane, the records left in this run of units
  int64_t f_tile = first0;
  int f_chunk = 0, f_left = 0;
  const unsigned char* f_src[RT];
  const bool tail_lane = 1024 + lane * 16 < record;       // this lane has 16 of the record's bytes beyond the codes
  auto seek = [&]() {
    f_left = hi_of(f_chunk) - lo_of(f_chunk);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      // tiles past the last one repeat it: their rows are not written
      const int64_t tile = f_tile + mine + t < nt ? f_tile + mine + t : nt - 1;
      f_src[t] = p.packed + tile * tile_bytes + (int64_t)lo_of(f_chunk) * record + lane * 16;
    }
  };
  auto next_run = [&]() {                                 // the next chunk, or the next tile's first
    while (f_left == 0) {
      f_chunk += p.chunk;
      if (f_chunk >= p.units) {
        f_chunk = 0;
        f_tile += stride;
        if (f_tile >= nt) return;
      }
      seek();
    }
  };
  auto fetch = [&](uint32_t slot) {                       // the next record of every row tile into a slot of the ring
    if (f_left > 0) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const uint32_t dst = smem0 + slot + t * record + lane * 16;
        copy_async_16(dst, f_src[t]);
        copy_async_16(dst + 512, f_src[t] + 512);
        if (tail_lane) copy_async_16(dst + 1024, f_src[t] + 1024);
        f_src[t] += record;
      }
      if (--f_left == 0) next_run();
    }
    copy_async_commit();
  };
  seek();
  if (f_left == 0) next_run();
#pragma unroll
  for (int i = 0; i < PF; ++i) fetch(ring + i * slot_bytes);
  uint32_t turn = 0;

  for (int64_t first = first0; first < nt; first += stride) {
    const int64_t tile = first + mine;
    float acc[RT][NT][4];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][n][j] = 0.f;
    for (int c0 = 0; c0 < p.units; c0 += p.chunk) {
      if (p.chunk < p.units || first == first0) {
        __syncthreads();   // the last chunk has been read
        head_stage<T, NT>(p, reinterpret_cast<uint4*>(head_smem), c0, min(c0 + p.chunk, p.units));
        __syncthreads();
      }
      const int u1 = hi_of(c0);
      for (int u = lo_of(c0); u < u1; ++u) {
        copy_async_wait<PF - 1>();
        __syncwarp();
        const uint32_t rec = ring + (turn++ & (PF - 1)) * slot_bytes;
        const uint2* su = reinterpret_cast<const uint2*>(head_smem) + (u - c0) * (kHeadUnitSteps * TERMS * 32 * NT) + lane;
        // a group of 128 fills a record, smaller ones may leave the last record with fewer blocks and groups
        const int blocks = NG == 1 ? 2 : min(nb - 2 * u, 2), groups = min(ng - u * NG, NG);
        float part[RT][NT][4];
        uint4 q4[RT];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (NG == 1 || g < groups) {
            float slo[RT], shi[RT];
            uint32_t zlo[RT], zhi[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
              const unsigned char* sc = head_smem + rec + t * record + blocks * 512;
              if (s.scale_bytes == 4) {
                const float2 v = reinterpret_cast<const float2*>(sc + g * gb)[gsel];
                slo[t] = v.x;
                shi[t] = v.y;
              } else {
                const uint32_t v = reinterpret_cast<const uint32_t*>(sc + g * gb)[gsel];
                slo[t] = __uint_as_float(v << 16);
                shi[t] = __uint_as_float(v & 0xFFFF0000u);
              }
              // 128 + zero point as bf16, twice
              zlo[t] = zhi[t] = 0x43084308u;
              if (s.has_zeros) {
                const uint32_t z = reinterpret_cast<const unsigned short*>(sc + groups * gb + g * 16)[gsel];
                zlo[t] = 0x43004300u + (z & 0xFFu) * 0x00010001u;
                zhi[t] = 0x43004300u + (z >> 8) * 0x00010001u;
              }
            }
#pragma unroll
            for (int i = 0; i < GS; ++i) {
              const int k = g * GS + i;
              uint2 h[NT][TERMS];
#pragma unroll
              for (int q = 0; q < TERMS; ++q)
#pragma unroll
                for (int n = 0; n < NT; ++n) h[n][q] = su[((k * TERMS + q) * NT + n) * 32];
#pragma unroll
              for (int t = 0; t < RT; ++t) {
                if (k % 4 == 0) q4[t] = reinterpret_cast<const uint4*>(head_smem + rec + t * record)[(k / 4) * 32 + lane];
                const uint32_t w = k % 4 == 0 ? q4[t].x : k % 4 == 1 ? q4[t].y : k % 4 == 2 ? q4[t].z : q4[t].w;
                // 128 + q as bf16, minus 128 + zero point: exact
                const uint32_t a0 = sub_bf16x2(and_or(w, nibbles, base), zlo[t]);
                const uint32_t a1 = sub_bf16x2(and_or(w >> 4, nibbles, base), zhi[t]);
                const uint32_t a2 = sub_bf16x2(and_or(w >> 8, nibbles, base), zlo[t]);
                const uint32_t a3 = sub_bf16x2(and_or(w >> 12, nibbles, base), zhi[t]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  float (&d)[4] = part[t][n];
                  if (i == 0) mma_bf16(d, a0, a1, a2, a3, h[n][0], 0.f, 0.f, 0.f, 0.f);
                  else mma_bf16(d, a0, a1, a2, a3, h[n][0], d[0], d[1], d[2], d[3]);
#pragma unroll
                  for (int q = 1; q < TERMS; ++q) mma_bf16(d, a0, a1, a2, a3, h[n][q], d[0], d[1], d[2], d[3]);
                }
              }
            }
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                acc[t][n][0] = fmaf(slo[t], part[t][n][0], acc[t][n][0]);
                acc[t][n][1] = fmaf(slo[t], part[t][n][1], acc[t][n][1]);
                acc[t][n][2] = fmaf(shi[t], part[t][n][2], acc[t][n][2]);
                acc[t][n][3] = fmaf(shi[t], part[t][n][3], acc[t][n][3]);
              }
          }
        }
        __syncwarp();   // every lane has read the slot
        fetch(rec);
      }
    }
    if (p.split > 1) {
      // the parts are added in order by the first warp of the set
      float* red = reinterpret_cast<float*>(head_smem + p.red_off);
      constexpr int W = RT * NT * 4;
      if (part_of > 0) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) red[(warp * W + (t * NT + n) * 4 + j) * 32 + lane] = acc[t][n][j];
      }
      __syncthreads();
      if (part_of == 0) {
        for (int o = 1; o < p.split; ++o)
#pragma unroll
          for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[t][n][j] += red[((warp + o) * W + (t * NT + n) * 4 + j) * 32 + lane];
      }
      __syncthreads();
      if (part_of > 0) continue;
    }
    // accumulator j of column tile n: vocabulary row l/4 (+ 8 for j >= 2), hidden row 8 n + 2 (l%4) + (j & 1)
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t v = (tile + t) * 16 + (lane >> 2) + (j >> 1) * 8;
          const int r = n * 8 + 2 * (lane & 3) + (j & 1);
          if (r < rows && v < s.V) {
            const int64_t at = (p.m0 + r) * p.ld + v;
            if (p.out_f32) reinterpret_cast<float*>(p.logits)[at] = acc[t][n][j];
            else reinterpret_cast<__nv_bfloat16*>(p.logits)[at] = __float2bfloat16_rn(acc[t][n][j]);
          }
        }
      }
  }
  copy_async_wait<0>();
}

}  // namespace vsamp
