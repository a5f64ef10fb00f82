// The output head with 4-bit weights (vsamp_head_pack, vsamp_head_logits):
//   logits[m, v] = sum over groups g of scale[v, g] * sum over k in g of (q[v, k] - z[v, g]) * hidden[m, k].
//
// The weights are read once per call, half a byte each, and everything else is small next to them while M stays in
// the tens: a few rows of hidden states against the whole vocabulary. So the kernel is a stream over the weights
// that feeds the warp-level matrix instruction straight from registers: q - z is at most 15 in magnitude, exact in
// bf16, products with bf16 hidden states are exact, sums are fp32, and the group's scale multiplies the fp32 sum of
// its group. fp32 hidden states are split into three bf16 terms, each a column of its own.
//
// What bounds it. M = 1: the bytes (151936 x 4096, groups of 128: 55 us, 87% of the copy rate). From about eight rows on
// the issue slots and the matrix unit together: widening costs 11 instructions per eight weights and lane, a product of
// eight columns about four slots and eight cycles of its unit (measured alone: 8.1 cycles; beside 12 independent
// multiply-adds 16.4), so 24 rows take 70 us where the bytes take 37 (151936 x 2560, groups of 32). From six column tiles
// on (33 rows) a warp holds one row tile, so every matrix step reads all staged states from shared memory again for 16
// vocabulary rows (2 KB at eight tiles, 16 cycles of an SM's shared memory), and long rows are staged in parts on every
// round: 64 rows of 50000 x 4096 take 127 us where the bytes take 18, with instructions in 31% of the issue slots.
// The states are three columns each in fp32 and the weights are read once per 16 of them (50000 x 4096: 38 us for one row,
// 50 for 8, 97 for 9, 119 for 16, 475 for 64; bf16 25, 28, 32, 35, 127).
// Tried instead for many rows: tcgen05 with the scale folded into the weights as two exact bf16 terms in tensor memory,
// so that one accumulator runs over all groups. 24 rows took 117 us (one block of 64 in flight per 128 rows), 64 rows
// of 50000 x 4096 107 us against 127, and the long accumulation cost digits (3.5e-6 of the result against 1.6e-7). Both
// come from the folding; an accumulator per group, scaled in fp32 as here, was not tried.
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
  int terms;       // bf16 terms of a hidden value (1, or 3 for fp32)
  int term_tiles;  // column tiles per term: term q of hidden row r is column q * 8 * term_tiles + r
  int vec;         // hidden rows are 16-byte aligned
  int units;       // units of the inner dimension (the last one may be padded)
  int chunk;       // units of hidden states staged at once
  int ring_off;    // bytes of staged states; the warps' rings follow, then the parts of split rows
  int red_off;
  int split;       // warps that share a row tile, each with its part of the inner dimension
};

// D = A B + C on 16 x 16 by 16 x 8 bf16 operands, fp32 sums
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b,
                                         float c0, float c1, float c2, float c3) {
  asm(
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

// Stages the hidden states of units [u0, u1) as the instruction's second operand, NT column tiles of 8. In step k, lane
// l needs column 8 n + l/4 at inner positions 2 (l%4) + {0, 1} and + 8; they are stored as
// [two steps][8 NT columns][l%4], four registers each (the two of both steps), so a lane reads two steps at once and the
// reads have constant offsets. A bf16 row is a column; an fp32 row is three (x = hi + mid + lo, each the bf16 nearest to
// what is left: 24 bits in all), in column tiles of their own, so that one lane holds the sums of all three. Positions
// beyond D are 0; columns without a row are not written (their part of the product is not used).
template <int NT>
__device__ __forceinline__ void head_stage(const HeadParams& p, uint4* sh, int u0, int u1) {
  const int rows = p.rows, steps = (u1 - u0) * kHeadUnitSteps, n = steps * rows;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    // neighbouring threads take neighbouring steps of a row: its bytes are read in order
    const int r = i / steps, ks = i - r * steps;
    const int64_t k = (int64_t)u0 * kHeadUnit + ks * 16;
    const bool whole = p.vec && k + 16 <= p.s.D;
    uint2* to = reinterpret_cast<uint2*>(sh + ((ks >> 1) * (8 * NT) + r) * 4) + (ks & 1);
    if (p.terms == 1) {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p.hidden) + (p.m0 + r) * p.ldh + k;
      uint32_t w[8];   // pairs of neighbouring positions
      if (whole) {
        const uint4 a = reinterpret_cast<const uint4*>(h)[0], b = reinterpret_cast<const uint4*>(h)[1];
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = (k + 2 * e < p.s.D ? h[2 * e] : 0u) | (uint32_t)(k + 2 * e + 1 < p.s.D ? h[2 * e + 1] : 0u) << 16;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) to[2 * j] = make_uint2(w[j], w[j + 4]);
    } else {
      const float* h = reinterpret_cast<const float*>(p.hidden) + (p.m0 + r) * p.ldh + k;
      float x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = k + e < p.s.D ? h[e] : 0.f;
      for (int q = 0; q < 3; ++q) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          uint32_t bits = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x[e]));
          // a finite value beyond the largest bf16 begins with that; an infinity has no remainder (inf - inf is NaN)
          if ((bits & 0x7FFFu) == 0x7F80u && !isinf(x[e])) bits -= 1;
          if (e & 1) w[e / 2] |= bits << 16;
          else w[e / 2] = bits;
          x[e] = isinf(x[e]) ? 0.f : x[e] - __uint_as_float(bits << 16);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) to[2 * j] = make_uint2(w[j], w[j + 4]);
        to += p.term_tiles * 64;
      }
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

// RT tiles of 16 vocabulary rows per warp, NT tiles of 8 columns (hidden rows, or their terms), groups of GROUP, scales
// of SB bytes. Every warp streams the records of its row tiles through a ring of PF slots in shared memory (PF records of
// each tile in flight, no registers held by loads: with the records in registers the loop spilled), across the ends of
// tiles. Several row tiles per warp share the reads of the staged states and hide each other's latency. p.split warps
// of a CTA share a set of row tiles, each with a contiguous part of its units.
template <int NT, int RT, int GROUP, int SB, bool ZEROS, int PF, int MAXW>
__global__ void __launch_bounds__(MAXW * 32, 1) head_kernel(const HeadParams p) {
  static_assert((PF & (PF - 1)) == 0, "slots are taken in turn by masking");
  constexpr int GS = GROUP / 16;          // steps per group
  constexpr int NG = kHeadUnit / GROUP;   // groups per unit
  extern __shared__ __align__(128) unsigned char head_smem[];
  begin_overlapped();
  const HeadShape s = p.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int GB = 16 * (SB + (ZEROS ? 1 : 0));         // bytes of a group's scales and zero points
  constexpr int record = 1024 + NG * GB;
  const int nb = s.blocks(), ng = s.groups();
  const int64_t nt = s.tiles(), tile_bytes = s.tile_bytes();
  const int part_of = warp % p.split;                     // this warp's part of the inner dimension
  const int slots = (int)(blockDim.x >> 5) / p.split;               // sets of row tiles per CTA and round
  const int64_t stride = (int64_t)gridDim.x * slots * RT;
  const int64_t first0 = (int64_t)blockIdx.x * slots * RT, mine = (warp / p.split) * RT;
  const int rows = p.rows;

  constexpr uint32_t slot_bytes = RT * record;
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
    float2 acc[RT][NT][2];   // rows l/4 and l/4 + 8, two columns each
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[t][n][0] = acc[t][n][1] = make_float2(0.f, 0.f);
    for (int c0 = 0; c0 < p.units; c0 += p.chunk) {
      if (p.chunk < p.units || first == first0) {
        __syncthreads();   // the last chunk has been read
        head_stage<NT>(p, reinterpret_cast<uint4*>(head_smem), c0, min(c0 + p.chunk, p.units));
        __syncthreads();
      }
      const int u1 = hi_of(c0);
      for (int u = lo_of(c0); u < u1; ++u) {
        copy_async_wait<PF - 1>();
        __syncwarp();
        const uint32_t rec = ring + (turn++ & (PF - 1)) * slot_bytes;
        const uint4* su = reinterpret_cast<const uint4*>(head_smem) + (u - c0) * (kHeadUnitSteps / 2 * 32 * NT) + lane;
        // a group of 128 fills a record, smaller ones may leave the last record with fewer blocks and groups
        const int blocks = NG == 1 ? 2 : min(nb - 2 * u, 2), groups = min(ng - u * NG, NG);
        float part[RT][NT][4];
        uint4 q4[RT], h4[NT];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (NG == 1 || g < groups) {
            float slo[RT], shi[RT];
            uint32_t zlo[RT], zhi[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
              const unsigned char* sc = head_smem + rec + t * record + blocks * 512;
              if (SB == 4) {
                const float2 v = reinterpret_cast<const float2*>(sc + g * 64)[gsel];
                slo[t] = v.x;
                shi[t] = v.y;
              } else {
                const uint32_t v = reinterpret_cast<const uint32_t*>(sc + g * 32)[gsel];
                slo[t] = __uint_as_float(v << 16);
                shi[t] = __uint_as_float(v & 0xFFFF0000u);
              }
              // 128 + zero point as bf16, twice
              zlo[t] = zhi[t] = 0x43084308u;
              if (ZEROS) {
                const uint32_t z = reinterpret_cast<const unsigned short*>(sc + groups * (16 * SB) + g * 16)[gsel];
                zlo[t] = __byte_perm(z, 0x43u, 0x4040);
                zhi[t] = __byte_perm(z, 0x43u, 0x4141);
              }
            }
#pragma unroll
            for (int i = 0; i < GS; ++i) {
              const int k = g * GS + i;
              if (k % 2 == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n) h4[n] = su[(k / 2 * NT + n) * 32];
              }
              uint2 h[NT];
#pragma unroll
              for (int n = 0; n < NT; ++n) h[n] = k % 2 == 0 ? make_uint2(h4[n].x, h4[n].y) : make_uint2(h4[n].z, h4[n].w);
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
                  if (i == 0) mma_bf16(d, a0, a1, a2, a3, h[n], 0.f, 0.f, 0.f, 0.f);
                  else mma_bf16(d, a0, a1, a2, a3, h[n], d[0], d[1], d[2], d[3]);
                }
              }
            }
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                acc[t][n][0] = __ffma2_rn(make_float2(slo[t], slo[t]), make_float2(part[t][n][0], part[t][n][1]), acc[t][n][0]);
                acc[t][n][1] = __ffma2_rn(make_float2(shi[t], shi[t]), make_float2(part[t][n][2], part[t][n][3]), acc[t][n][1]);
              }
          }
        }
        __syncwarp();   // every lane has read the slot
        fetch(rec);
      }
    }
    if (p.split > 1) {
      // the parts are added in order by the first warp of the set
      float2* red = reinterpret_cast<float2*>(head_smem + p.red_off);
      constexpr int W = RT * NT * 2;
      if (part_of > 0) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) red[(warp * W + (t * NT + n) * 2 + j) * 32 + lane] = acc[t][n][j];
      }
      __syncthreads();
      if (part_of == 0) {
        for (int o = 1; o < p.split; ++o)
#pragma unroll
          for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                acc[t][n][j] = __fadd2_rn(acc[t][n][j], red[((warp + o) * W + (t * NT + n) * 2 + j) * 32 + lane]);
      }
      __syncthreads();
      if (part_of > 0) continue;
    }
    // accumulator j of column tile n: vocabulary row l/4 (+ 8 for j >= 2), column 8 n + 2 (l%4) + (j & 1)
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n < p.term_tiles) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t v = (tile + t) * 16 + (lane >> 2) + (j >> 1) * 8;
            const int r = n * 8 + 2 * (lane & 3) + (j & 1);
            auto sum = [&](int i) { return (j & 1) ? acc[t][i][j >> 1].y : acc[t][i][j >> 1].x; };
            float y = sum(n);
            if (NT % 3 == 0 && p.terms == 3) {   // smallest terms first
              constexpr int TT = NT / 3;
              if (n < TT) y += sum((n + TT) % NT) + sum((n + 2 * TT) % NT);
            }
            if (r < rows && v < s.V) {
              const int64_t at = (p.m0 + r) * p.ld + v;
              if (p.out_f32) reinterpret_cast<float*>(p.logits)[at] = y;
              else reinterpret_cast<__nv_bfloat16*>(p.logits)[at] = __float2bfloat16_rn(y);
            }
          }
        }
      }
  }
  copy_async_wait<0>();
}

}  // namespace vsamp
