// Scoring of given tokens (vsamp_score_tokens) and its gradient (vsamp_score_tokens_backward).
//
// Forward. With s_v = (x_v - m) / T, S = sum e^s_v and A = sum s_v e^s_v a row needs
//   log-probability of t   min(s_t - log S, 0)
//   entropy                log S - A / S
//   rank of t              #{v : x_v > x_t, or x_v = x_t and v < t}
//   the N alternatives     the first N tokens in the order (value descending, index ascending)
// Rows are cut into fixed 4 KB pieces, one warp each; a piece is read once into registers, its maximum m_p is found
// and S_p, A_p are formed relative to it, so no pass waits for the row maximum and the sums of a row depend on V
// alone. A second launch folds the pieces of every row:
//   S = sum 2^((m_p - m) c) S_p,   A = sum 2^((m_p - m) c) (A_p + (m_p - m) c S_p),   c = log2(e) / T.
// A piece with S_p < 2, in which one token outweighs the others, records S_p - 1 without that token's 1, beside which
// the others' digits would be lost.
// -inf marks a masked token (probability 0); NaN and +inf are row errors.
//
// Alternatives. A piece also records the maxima of its eight 512-byte chunks. The first N tokens of the order lie in
// the first N chunks in the order (chunk maximum descending, chunk index ascending): a token of any later chunk is
// preceded by the maxima of N chunks. So the finish re-reads N chunks, whatever the data.
#pragma once

#include "vsamp.h"
#include "vsamp_device.cuh"
#include "vsamp_vec.cuh"

namespace vsamp {

constexpr int kScorePiece = 4096;      // bytes of a row per warp
constexpr int kScoreChunks = 8;        // 512-byte chunks per piece: one 16-byte vector per lane each
constexpr int kScoreWarps = 8;
constexpr int kScoreFinishThreads = 256;
constexpr int kKeep = 4;               // chunk maxima that a thread of the finish keeps in registers
constexpr int kScoreChunkList = 2 * VSAMP_SCORE_ALT_MAX + 64;   // chunks read again per row
constexpr int kScoreList = 512;        // alternatives' candidates kept on chip; more of them take the radix path

struct ScoreParams {
  const unsigned char* x;
  int64_t B, V, ld;
  const float* temperature;
  const int32_t* token;
  int N;                 // alternatives per row
  int vec;               // rows are 16-byte aligned
  int np;                // pieces per row; B * np < 2^31
  uint32_t np_mul;       // id / np = umulhi(id, np_mul) >> np_shift for np > 1
  int np_shift;
  uint32_t inner0, inner1;   // whole pieces in [inner0, inner1) are read by aligned vectors (all but one at the very ends)
  float4* rec;           // [B, np] {m_p, S_p, or below 1 for S_p - 1, A_p, tokens before the given one}
  float* chunk_max;      // [B, np, 8] (N > 0)
  float* logprob;
  float* entropy;
  int32_t* rank;
  int32_t* alt_idx;
  float* alt_lp;
  float* row_max;
  float* row_logsum;
  int32_t* row_status;
};

struct ScoreGradParams {
  const unsigned char* x;
  int64_t B, V, ld, ldo;
  const float* temperature;
  const int32_t* token;
  const float* dlogprob;
  const float* dentropy;
  const float* row_max;
  const float* row_logsum;
  const float* entropy;
  unsigned char* dx;
  int32_t* row_status;
  int64_t spans;         // CTAs per row
};

template <typename T>
struct ScoreType;
template <>
struct ScoreType<float> {
  static constexpr int ES = 4, VE = 4;
  static constexpr uint32_t kMasked = 0xFF800000u;   // a 32-bit word of -inf
  static __device__ __forceinline__ float load(const unsigned char* p, int64_t i) {
    return reinterpret_cast<const float*>(p)[i];
  }
  // element j of a 16-byte vector
  static __device__ __forceinline__ float at(const uint32_t (&w)[4], int j) { return __uint_as_float(w[j]); }
  static __device__ __forceinline__ void put(uint32_t (&w)[4], int j, float f) { w[j] = __float_as_uint(f); }
  static __device__ __forceinline__ void store(unsigned char* p, int64_t i, float f) {
    reinterpret_cast<float*>(p)[i] = f;
  }
};
template <>
struct ScoreType<__nv_bfloat16> {
  static constexpr int ES = 2, VE = 8;
  static constexpr uint32_t kMasked = 0xFF80FF80u;
  static __device__ __forceinline__ float load(const unsigned char* p, int64_t i) {
    return __uint_as_float((uint32_t) reinterpret_cast<const unsigned short*>(p)[i] << 16);
  }
  static __device__ __forceinline__ float at(const uint32_t (&w)[4], int j) {
    return __uint_as_float((j & 1) ? (w[j >> 1] & 0xFFFF0000u) : (w[j >> 1] << 16));
  }
  // bits of a value that is exactly a bf16
  static __device__ __forceinline__ void put(uint32_t (&w)[4], int j, float f) {
    const uint32_t b = __float_as_uint(f);
    w[j >> 1] = (j & 1) ? ((w[j >> 1] & 0xFFFFu) | (b & 0xFFFF0000u)) : ((w[j >> 1] & 0xFFFF0000u) | (b >> 16));
  }
  static __device__ __forceinline__ void store(unsigned char* p, int64_t i, float f) {
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f);
  }
};

// s_v log2(e) = ((x down - m down) up) c for a temperature T > 0, where no step but the last leaves fp32's range when the
// result does not. `scale` is 1 for ordinary temperatures; below 1e-37 it is 2^60 and stands in `up` (1 / T would
// overflow), above 1e36 it is 2^-60 and stands in `down` (x - m could, and 1 / T loses digits).
struct ScoreRate {
  float T, c, scale, up, down;
  static __device__ __forceinline__ float read(const float* temperature, int64_t row) {
    return temperature && temperature[row] > 0.f ? temperature[row] : 1.f;
  }
  static __device__ __forceinline__ bool ordinary(float T) { return T >= 1e-37f && T <= 1e36f; }
  static __device__ __forceinline__ ScoreRate of(float T) {
    ScoreRate r;
    r.T = T;
    r.scale = ordinary(T) ? 1.f : T < 1.f ? 0x1p60f : 0x1p-60f;
    r.up = fmaxf(r.scale, 1.f);
    r.down = fminf(r.scale, 1.f);
    r.c = kLog2e / (T * r.scale);
    return r;
  }
  __device__ __forceinline__ float exponent(float x, float m) const { return fmaf(x, down, -m * down) * up * c; }
  __device__ __forceinline__ float s(float x, float m) const { return fmaf(x, down, -m * down) / (T * down); }
};

// max that returns NaN when either operand is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
  return v;
}
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The vector of elements [e, e + VE) of a row; elements at or beyond V read as -inf.
template <typename T>
__device__ __forceinline__ void score_load(const unsigned char* xr, int64_t e, int64_t V, int vec, uint32_t (&w)[4]) {
  using Ty = ScoreType<T>;
  ElemVec<T, Ty::VE> v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.w[i] = Ty::kMasked;
  if (e < V) v.load_row(xr + e * Ty::ES, V - e, vec, Ty::kMasked & (Ty::ES == 4 ? 0xFFFFFFFFu : 0xFFFFu));
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = v.w[i];
}

// Maximum of two registers of a vector's type; NaN if either holds one.
template <typename T>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (sizeof(T) == 4) asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The maximum that a register of partial maxima holds.
template <typename T>
__device__ __forceinline__ float max_of_word(uint32_t a) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(a);
  else return max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
}

// Elements of a lane's vectors that are larger than xt (or_equal: or equal to it).
template <typename T>
__device__ __forceinline__ uint32_t count_larger(const uint32_t (&w)[kScoreChunks][4], float xt, bool or_equal) {
  if constexpr (sizeof(T) == 4) {
    uint32_t n = 0;
    if (or_equal) {
#pragma unroll
      for (int i = 0; i < kScoreChunks; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) n += __uint_as_float(w[i][j]) >= xt ? 1u : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < kScoreChunks; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) n += __uint_as_float(w[i][j]) > xt ? 1u : 0u;
    }
    return n;
  } else {
    // pairs: 1.0 per true comparison, at most 32 per half: exact in bf16
    const __nv_bfloat162 t = __float2bfloat162_rn(xt);
    __nv_bfloat162 n = __float2bfloat162_rn(0.f);
    if (or_equal) {
#pragma unroll
      for (int i = 0; i < kScoreChunks; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          __nv_bfloat162 x;
          memcpy(&x, &w[i][j], 4);
          n = __hadd2(n, __hge2(x, t));
        }
    } else {
#pragma unroll
      for (int i = 0; i < kScoreChunks; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          __nv_bfloat162 x;
          memcpy(&x, &w[i][j], 4);
          n = __hadd2(n, __hgt2(x, t));
        }
    }
    return (uint32_t)(__low2float(n) + __high2float(n));
  }
}

// A lane's sums of 2^s2 and s2 2^s2 over its vectors. A masked token must add 0 to both, and s2 2^s2 is NaN at s2 = -inf.
// RAISE, for ordinary temperatures: s2 = (x - m) c, and elements are raised to `lowest`, whose exponential is flushed to
// 0 (2^-150), two bf16 at once. Otherwise (a temperature so large that no finite value is that low, or so small that no
// value lies between, or outside ScoreRate's ordinary ones) the exponents are raised.
// (One fused multiply-add x c - m c instead of the difference and the product is 8% fewer instructions, but then the
// maximum's own exponential is not exactly 1, and a row with one likely token loses the digits of its log-probability.)
template <typename T, bool RAISE>
__device__ __forceinline__ void score_sums(const uint32_t (&w)[kScoreChunks][4], float m, const ScoreRate& r, float lowest,
                                           float& S, float& A) {
  using Ty = ScoreType<T>;
  const float md = RAISE ? -m : -m * r.down;
  const float2 m2 = make_float2(md, md), c2 = make_float2(r.c, r.c);
  float2 S2[2] = {{0.f, 0.f}, {0.f, 0.f}}, A2[2] = {{0.f, 0.f}, {0.f, 0.f}};
  uint32_t low = __float_as_uint(lowest);
  if (sizeof(T) == 2) low = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rd(lowest)) * 0x10001u;
#pragma unroll
  for (int i = 0; i < kScoreChunks; ++i) {
    uint32_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = RAISE ? max_word<T>(w[i][j], low) : w[i][j];
#pragma unroll
    for (int j = 0; j < Ty::VE; j += 2) {
      const float2 x = make_float2(Ty::at(v, j), Ty::at(v, j + 1));
      float2 s;
      if (RAISE) {
        s = __fmul2_rn(__fadd2_rn(x, m2), c2);
      } else {
        const float2 d = __ffma2_rn(x, make_float2(r.down, r.down), m2);
        s = __fmul2_rn(__fmul2_rn(d, make_float2(r.up, r.up)), c2);
        s = make_float2(fmaxf(s.x, -150.f), fmaxf(s.y, -150.f));
      }
      const float2 e = make_float2(ex2_approx(s.x), ex2_approx(s.y));
      const int k = (j >> 1) & 1;
      S2[k] = __fadd2_rn(S2[k], e);
      A2[k] = __ffma2_rn(s, e, A2[k]);
    }
  }
  S = (S2[0].x + S2[1].x) + (S2[0].y + S2[1].y);
  A = (A2[0].x + A2[1].x) + (A2[0].y + A2[1].y);
}

// A piece that begins s bytes (4 WS + 2 odd) past a 16-byte boundary, from the aligned vectors around it: w holds the
// lane's vector of every chunk, `extra` the vector after the piece (lane 0). A lane's elements begin in its own vector and
// end in the next lane's, lane 31's in the next chunk's first. (2048 x 151935 bf16: 109 us, aligned rows 98; by 32-bit
// words 180.)
template <int WS>
__device__ __forceinline__ void realign_piece(uint32_t (&w)[kScoreChunks][4], const uint4& extra, uint32_t odd) {
  const int lane = threadIdx.x & 31;
  const uint32_t last[4] = {extra.x, extra.y, extra.z, extra.w};
#pragma unroll
  for (int i = 0; i < kScoreChunks; ++i) {
    uint32_t c[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      c[k] = w[i][k];
      c[4 + k] = 0;
      if (k <= WS) {
        const uint32_t after = i + 1 < kScoreChunks ? w[i + 1 < kScoreChunks ? i + 1 : 0][k] : last[k];
        c[4 + k] = __shfl_sync(kFullMask, lane == 0 ? after : w[i][k], (lane + 1) & 31);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) w[i][k] = __funnelshift_r(c[k + WS], c[k + WS + 1 < 8 ? k + WS + 1 : 7], odd * 8);
  }
}

// The sum of a piece in which one token outweighs all others (S < 2), without that token: beside its 1 the others' digits
// are lost, and with them those of the row's log S. One lane's sum holds the 1; that lane's 128 bytes are read again, a
// word per lane. Below 1.
template <typename T>
__device__ __forceinline__ float sum_of_others(const unsigned char* xr, int32_t e0, int32_t V, float m, const ScoreRate& r,
                                               float mine) {
  using Ty = ScoreType<T>;
  constexpr int CE = kScorePiece / Ty::ES / kScoreChunks, WE = 4 / Ty::ES;   // elements per chunk, per word
  const int lane = threadIdx.x & 31;
  const int holder = (__ffs(__ballot_sync(kFullMask, mine >= 1.f)) - 1) & 31;
  float S = lane == holder ? 0.f : mine;
  const int64_t e = (int64_t)e0 + (lane >> 2) * CE + holder * Ty::VE + (lane & 3) * WE;
#pragma unroll
  for (int j = 0; j < WE; ++j) {
    const float x = V - e > j ? Ty::load(xr, e + j) : -INFINITY;
    S += x == m ? 0.f : ex2_approx(fmaxf(r.exponent(x, m), -150.f));
  }
  return fminf(warp_sum_f(S), 0x1.fffffep-1f);
}

// One warp, one piece of a row (the id-th of all): its record, and the maxima of its chunks. The piece is held in
// registers.
template <typename T, bool ALT>
__device__ __forceinline__ void score_piece(const ScoreParams& p, uint32_t row, int piece, uint32_t id, int32_t t,
                                            float4* rec, float* chunk_max) {
  using Ty = ScoreType<T>;
  constexpr int PE = kScorePiece / Ty::ES;      // elements per piece
  constexpr int CE = PE / kScoreChunks;         // elements per chunk
  const int lane = threadIdx.x & 31;
  const int32_t e0 = piece * PE;
  const int32_t V = (int32_t)p.V;
  const unsigned char* xr = p.x + (int64_t)row * p.ld * Ty::ES;
  uint32_t w[kScoreChunks][4];
  if (PE <= V - e0 && id >= p.inner0 && id < p.inner1) {
    const unsigned char* at = xr + (int64_t)e0 * Ty::ES;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(at) & 15);   // the same for the whole row
    at += lane * 16 - (int)off;
#pragma unroll
    for (int i = 0; i < kScoreChunks; ++i) {
      const uint4 v = ldg_stream(at + i * 512);
      w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
    }
    if (off) {
      // the vectors before the first and after the last element hold elements of the piece, too
      uint4 extra = make_uint4(0, 0, 0, 0);
      if (lane == 0) extra = ldg_stream(at + kScorePiece);
      if (off < 4) realign_piece<0>(w, extra, off & 2);
      else if (off < 8) realign_piece<1>(w, extra, off & 2);
      else if (off < 12) realign_piece<2>(w, extra, off & 2);
      else realign_piece<3>(w, extra, off & 2);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kScoreChunks; ++i) score_load<T>(xr, (int64_t)e0 + i * CE + lane * Ty::VE, p.V, p.vec, w[i]);
  }
  const float T1 = ScoreRate::read(p.temperature, row), c = p.temperature ? kLog2e / T1 : kLog2e;
  const bool known = t >= 0 && t < V;
  const float xt = known ? Ty::load(xr, t) : INFINITY;

  // maximum of the lane's vectors, of the chunks and of the piece
  float m = -INFINITY;
  if (ALT) {
    float mine = 0.f;    // lane i < 8: maximum of chunk i
#pragma unroll
    for (int i = 0; i < kScoreChunks; ++i) {
      const float cm = warp_max_nan(
          max_of_word<T>(max_word<T>(max_word<T>(w[i][0], w[i][1]), max_word<T>(w[i][2], w[i][3]))));
      if (lane == i) mine = cm;
      m = max_nan(m, cm);
    }
    if (lane < kScoreChunks) chunk_max[lane] = mine;
  } else {
    uint32_t a = max_word<T>(w[0][0], w[0][1]), b = max_word<T>(w[0][2], w[0][3]);
#pragma unroll
    for (int i = 1; i < kScoreChunks; ++i) {
      a = max_word<T>(a, max_word<T>(w[i][0], w[i][1]));
      b = max_word<T>(b, max_word<T>(w[i][2], w[i][3]));
    }
    m = warp_max_nan(max_of_word<T>(max_word<T>(a, b)));
  }

  // tokens before the given one: ties count in the pieces before its own, up to its place in its own
  uint32_t before = 0;
  if (known && m >= xt) {   // a piece below the given token has none (false for NaN too)
    if (t - e0 >= PE) {
      before = count_larger<T>(w, xt, true);
    } else if (t < e0) {
      before = count_larger<T>(w, xt, false);
    } else {
      // the larger ones, and the equal ones of the vectors before its own; in its own vector one by one
      const int at = t - e0;
      before = count_larger<T>(w, xt, false);
#pragma unroll
      for (int i = 0; i < kScoreChunks; ++i) {
        const int first = i * CE + lane * Ty::VE;
        if (first < at) {
#pragma unroll
          for (int j = 0; j < Ty::VE; ++j) before += Ty::at(w[i], j) == xt && first + j < at ? 1u : 0u;
        }
      }
    }
  }
  before = warp_sum_u32(before);

  float S = 0.f, A = 0.f;
  if (m > -INFINITY && m < INFINITY) {   // false for NaN too
    // 104 log2(e) > 150; below m, too: at a temperature far below the maximum's last place it is m itself
    const float lowest = fmaf(-104.f, T1, m);
    float mine;   // this lane's sum
    if (__builtin_expect(ScoreRate::ordinary(T1) && lowest < m && lowest > -3.3e38f, 1))
      score_sums<T, true>(w, m, ScoreRate{T1, c, 1.f, 1.f, 1.f}, lowest, mine, A);
    else
      score_sums<T, false>(w, m, ScoreRate::of(T1), lowest, mine, A);
    S = warp_sum_f(mine);
    if (__builtin_expect(S < 2.f, 0)) S = sum_of_others<T>(xr, e0, V, m, ScoreRate::of(T1), mine);
    A = warp_sum_f(A);
  }
  if (lane == 0) *rec = make_float4(m, S, A, __uint_as_float(before));
}

// One warp per piece, the piece in registers: 32 warps per SM hold 128 KB of loads in flight. About six instructions per
// bf16 element beside the exponential. 2048 x 151936 bf16, a quarter of the rows ignored: 79.5 us with the finish, 88% of
// the copy rate; small batches are bound by the two launches and their first loads (256 rows: 24.6 us with 20
// alternatives where the bytes take 12). A persistent form that copies the next piece to shared
// memory meanwhile ran 15% more instructions and was slower (108 against 91 us at the time).
template <typename T, bool ALT>
__global__ void __launch_bounds__(kScoreWarps * 32, 4) score_piece_kernel(const ScoreParams p) {
  begin_overlapped();
  const uint32_t id = blockIdx.x * kScoreWarps + (threadIdx.x >> 5);
  const uint32_t row = p.np > 1 ? __umulhi(id, p.np_mul) >> p.np_shift : id;
  if (row >= (uint32_t)p.B) return;
  const int32_t t = p.token[row];
  if (t == VSAMP_TOKEN_IGNORE) return;
  score_piece<T, ALT>(p, row, (int)(id - row * (uint32_t)p.np), id, t, p.rec + id,
                      ALT ? p.chunk_max + (int64_t)id * kScoreChunks : nullptr);
}

struct ScoreRow {
  int status;
  float m, logsum, entropy;
  uint32_t before;
  ScoreRate rate;
  // the log-probability of a token from its logit: the same for the given token and for an alternative
  __device__ __forceinline__ float logprob(float x) const { return fminf(rate.s(x, m) - logsum, 0.f); }
};

// A warp folds the piece records of a row (every lane returns the same values). The first kFoldKeep records per lane are
// read at once and kept; `load` may run before the row's token is known.
constexpr int kFoldKeep = 4;
struct ScoreFold {
  const float4* all;
  float4 rec[kFoldKeep];
  // the row's records, in global or shared memory
  __device__ __forceinline__ void load(const ScoreParams& p, const float4* r) {
    all = r;
#pragma unroll
    for (int i = 0; i < kFoldKeep; ++i) {
      const int k = i * 32 + (int)(threadIdx.x & 31);
      rec[i] = k < p.np ? r[k] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(const ScoreParams& p, F f) const {
#pragma unroll
    for (int i = 0; i < kFoldKeep; ++i) f(rec[i]);
    for (int k = kFoldKeep * 32 + (int)(threadIdx.x & 31); k < p.np; k += 32) f(all[k]);
  }
  __device__ __forceinline__ ScoreRow row(const ScoreParams& p, int64_t at, int32_t t) const {
    const float temp = p.temperature ? p.temperature[at] : 1.f;
    ScoreRow r;
    r.rate = ScoreRate::of(ScoreRate::read(p.temperature, at));
    float m = -INFINITY;
    each(p, [&](float4 q) { m = max_nan(m, q.x); });
    m = warp_max_nan(m);
    float S = 0.f, A = 0.f;
    uint32_t before = 0, ones = 0;   // pieces of which S holds all but the maximum's own 1
    const bool finite = m > -INFINITY && m < INFINITY;
    if (finite) {
      each(p, [&](float4 q) {
        before += __float_as_uint(q.w);
        if (q.x > -INFINITY) {
          const float d = fmaxf(r.rate.exponent(q.x, m), -150.f);
          const float f = ex2_approx(d), sum = q.y < 1.f ? q.y + 1.f : q.y;
          const bool one = q.y < 1.f && q.x == m;
          ones += one ? 1u : 0u;
          S = fmaf(f, one ? q.y : sum, S);
          A = fmaf(f, fmaf(d, sum, q.z), A);
        }
      });
    }
    S = warp_sum_f(S);
    A = warp_sum_f(A);
    ones = warp_sum_u32(ones);
    r.before = warp_sum_u32(before);
    r.m = m;
    // log1p of the sum without one 1, which keeps the digits of the others' where one token outweighs them
    r.logsum = log1pf(S + ((float)ones - 1.f));
    r.entropy = fmaxf(r.logsum - 0.69314718056f * (A / (S + (float)ones)), 0.f);
    r.status = VSAMP_OK;
    if (!finite) r.status = VSAMP_ERR_NONFINITE;
    else if (isnan(temp) || isinf(temp) || t < 0 || (int64_t)t >= p.V) r.status = VSAMP_ERR_INVALID_ARG;
    return r;
  }
};

// The given token's logit, NaN if it is none.
template <typename T>
__device__ __forceinline__ float score_logit(const ScoreParams& p, int64_t row, int32_t t) {
  return t >= 0 && (int64_t)t < p.V ? ScoreType<T>::load(p.x + row * p.ld * ScoreType<T>::ES, t) : __int_as_float(0x7FC00000);
}

__device__ __forceinline__ void score_write(const ScoreParams& p, int64_t row, int32_t t, float xt, const ScoreRow& r) {
  const bool skip = t == VSAMP_TOKEN_IGNORE;
  const bool ok = r.status == VSAMP_OK && !skip;
  const float none = skip ? 0.f : __int_as_float(0x7FC00000);
  if (p.logprob) p.logprob[row] = ok ? r.logprob(xt) : none;
  if (p.entropy) p.entropy[row] = ok ? r.entropy : none;
  if (p.rank) p.rank[row] = ok ? (int32_t)r.before : -1;
  if (p.row_max) p.row_max[row] = ok ? r.m : none;
  if (p.row_logsum) p.row_logsum[row] = ok ? r.logsum : none;
  if (p.row_status) p.row_status[row] = r.status;
}

// No alternatives: one warp per row.
template <typename T>
__global__ void __launch_bounds__(128) score_finish_kernel(const ScoreParams p) {
  begin_overlapped();
  for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); row < p.B; row += (int64_t)gridDim.x * 4) {
    ScoreFold fold;
    fold.load(p, p.rec + row * p.np);
    const int32_t t = p.token[row];
    const float xt = score_logit<T>(p, row, t);
    ScoreRow r{};
    if (t != VSAMP_TOKEN_IGNORE) r = fold.row(p, row, t);
    if ((threadIdx.x & 31) == 0) score_write(p, row, t, xt, r);
  }
}

// Threshold of the `want` largest of the 64-bit keys that for_each visits (all different, at least `want` of them,
// want > 0): exactly `want` keys are >= the value returned. Byte-wise radix search; it stops when a whole group of
// equal leading bytes is taken. Called by all threads of the CTA.
template <typename F>
__device__ uint64_t score_radix_select(F for_each, uint32_t want, uint32_t* hist, uint32_t* bc) {
  uint64_t prefix = 0, mask = 0;
  for (int shift = 56; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    for_each([&](uint64_t k) {
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1u);
    });
    __syncthreads();
    if (threadIdx.x < 32) {
      // lane l holds bins 255 - 8 l down to 248 - 8 l
      const int top = 255 - 8 * (int)threadIdx.x;
      uint32_t n[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[i] = hist[top - i];
        sum += n[i];
      }
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kFullMask, incl, o);
        if (threadIdx.x >= o) incl += v;
      }
      uint32_t above = incl - sum;
      if (above < want && incl >= want) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < want && above + n[i] >= want) {
            bc[0] = (uint32_t)(top - i);
            bc[1] = above;
            bc[2] = n[i];
          }
          above += n[i];
        }
      }
    }
    __syncthreads();
    prefix |= (uint64_t)bc[0] << shift;
    mask |= 0xFFull << shift;
    want -= bc[1];
    const bool whole = bc[2] == want;
    __syncthreads();
    if (whole) break;
  }
  return prefix;
}

// One CTA per row. The last warp folds the records while the others look for the alternatives:
//   1. every group of threads takes the largest of its chunks; the N-th largest of these is a bound that at least N
//      chunks reach, so every alternative does;
//   2. the chunks at or above the bound are listed (their number is close to N; an arrangement that lists many more
//      is cut to the N that the lemma above needs by a radix search);
//   3. the tokens of the listed chunks at or above the bound are listed, again close to N of them (if they are more than
//      the list holds, above a bound from every thread's largest token, and failing that by a radix search for the last
//      alternative), and each one's place is the number of larger ones.
// Keys are (value, index) pairs in the order's sense, all different. Bound by latency: a chain of about eight dependent
// steps, about 5 us beside the pieces' kernel, whatever N (20 alternatives of 256 rows: 24.6 us against 18.7 without).
struct ScoreAltSmem {
  __align__(16) uint64_t list[kScoreList];
  __align__(16) uint64_t best[kScoreFinishThreads];
  uint32_t hist[256];
  uint32_t bc[3];
  int32_t chunks[kScoreChunkList];
  uint32_t n_chunks, n_list;
  uint64_t bound;
  ScoreRow row;
};

template <typename T>
__device__ __forceinline__ void score_finish_alt(const ScoreParams& p, int64_t row, int32_t t, const float4* rec,
                                                 const float* cm, ScoreAltSmem& sm) {
  using Ty = ScoreType<T>;
  constexpr int CE = kScorePiece / Ty::ES / kScoreChunks;
  constexpr int NT = kScoreFinishThreads, NW = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float qnan = __int_as_float(0x7FC00000);
  constexpr uint32_t kNone = 0x007FFFFFu;   // key of -inf
  // threads per group: as many as leave three groups with chunks for every alternative, eight at most
  const int holders = p.np * kScoreChunks < NT ? p.np * kScoreChunks : NT;
  const int gs = holders >= 24 * p.N ? 8 : holders >= 12 * p.N ? 4 : holders >= 6 * p.N ? 2 : 1;
  const int groups = (holders + gs - 1) / gs;
  // what the row needs first is read at once: the first chunk maxima of every thread, the last warp's records
  const int64_t nch = (int64_t)p.np * kScoreChunks;
  float kept[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) kept[i] = i * NT + tid < nch ? cm[i * NT + tid] : -INFINITY;
  ScoreFold fold;
  if (warp == NW - 1) fold.load(p, rec);
  const bool skip = t == VSAMP_TOKEN_IGNORE;
  int32_t* oi = p.alt_idx + row * p.N;
  float* ol = p.alt_lp + row * p.N;
  uint32_t found = 0;
  if (skip) {
    if (tid == 0) score_write(p, row, t, 0.f, ScoreRow{});
  } else {
    const unsigned char* xr = p.x + row * p.ld * Ty::ES;
    auto each_chunk = [&](auto f) {
      auto one = [&](float x, int64_t i) {
        const uint32_t k = key_f32_bits(__float_as_uint(x));
        if (k > kNone) f(((uint64_t)k << 32) | (uint32_t)~(uint32_t)i);
      };
#pragma unroll
      for (int i = 0; i < kKeep; ++i) one(kept[i], i * NT + tid);
#pragma unroll 4
      for (int64_t i = kKeep * NT + tid; i < nch; i += NT) one(cm[i], i);
    };
    uint64_t mine = 0;
    each_chunk([&](uint64_t k) { mine = k > mine ? k : mine; });
    for (int o = 1; o < gs; o <<= 1) {
      const uint64_t v = __shfl_xor_sync(kFullMask, mine, o);
      mine = v > mine ? v : mine;
    }
    if (tid % gs == 0) sm.best[tid / gs] = mine;
    if (tid == 0) {
      sm.n_chunks = sm.n_list = 0;
      sm.bound = 0;
    }
    __syncthreads();
    if (warp == NW - 1) {
      const float xt = score_logit<T>(p, row, t);
      const ScoreRow r = fold.row(p, row, t);
      if (lane == 0) {
        score_write(p, row, t, xt, r);
        sm.row = r;
      }
    }
    for (int g = tid; g < groups; g += NT - 32) {   // the first warps: the fold is the last one's
      if (warp == NW - 1) break;
      const uint64_t k = sm.best[g];
      int larger = 0;
#pragma unroll 8
      for (int i = 0; i < groups; ++i) larger += sm.best[i] > k ? 1 : 0;
      if (larger == p.N - 1 && k > 0) sm.bound = k;     // one group, if that many groups have a token
    }
    __syncthreads();
    uint64_t cut = sm.bound;
    const ScoreRow r = sm.row;
    if (r.status == VSAMP_OK) {
      auto list_chunks = [&]() {
        each_chunk([&](uint64_t k) {
          if (k >= cut) {
            const uint32_t at = atomicAdd(&sm.n_chunks, 1u);
            if (at < kScoreChunkList) sm.chunks[at] = (int32_t)~(uint32_t)k;
          }
        });
        __syncthreads();
      };
      list_chunks();
      if (sm.n_chunks > 2 * (uint32_t)p.N + 64) {   // far more than N: at least N of them, so the search finds its N-th
        cut = score_radix_select(each_chunk, (uint32_t)p.N, sm.hist, sm.bc);
        if (tid == 0) sm.n_chunks = 0;
        __syncthreads();
        list_chunks();
      }
      const uint32_t nc = sm.n_chunks;
      const uint32_t lowest = max((uint32_t)(cut >> 32), kNone + 1);
      auto each_token = [&](auto f) {
        for (uint32_t i = warp; i < nc; i += 4 * NW) {   // four sm.chunks in flight
          uint32_t w[4][4];
          int64_t e[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t at = i + u * NW;
            e[u] = at < nc ? (int64_t)sm.chunks[at] * CE + lane * Ty::VE : p.V;
            score_load<T>(xr, e[u], p.V, p.vec, w[u]);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < Ty::VE; ++j) {
              const uint32_t k = key_f32_bits(__float_as_uint(Ty::at(w[u], j)));
              if (k >= lowest) f(((uint64_t)k << 32) | (uint32_t)~(uint32_t)(e[u] + j));
            }
        }
      };
      // (once the list has run over, the rest is not counted: that many atomics on one word would take microseconds)
      auto to_list = [&](uint64_t k) {
        if (*reinterpret_cast<volatile uint32_t*>(&sm.n_list) <= kScoreList) {
          const uint32_t at = atomicAdd(&sm.n_list, 1u);
          if (at < kScoreList) sm.list[at] = k;
        }
      };
      uint32_t n = kScoreList + 1;
      if (cut != 0 || nc * CE <= kScoreList) {   // without a bound every token passes
        each_token(to_list);
        __syncthreads();
        n = sm.n_list;
      }
      if (n > kScoreList) {
        // too many (a row of few chunks, or of many equal tokens): a bound from every thread's largest token
        __syncthreads();   // every thread has read the count that is set back below, so all of them are here
        uint64_t top = 0;
        each_token([&](uint64_t k) { top = k > top ? k : top; });
        sm.best[tid] = top;
        if (tid == 0) {
          sm.bound = 0;
          sm.n_list = 0;
        }
        __syncthreads();
        int larger = 0;
#pragma unroll 8
        for (int i = 0; i < NT; ++i) larger += sm.best[i] > top ? 1 : 0;
        if (larger == p.N - 1 && top > 0) sm.bound = top;
        __syncthreads();
        const uint64_t above = sm.bound;
        each_token([&](uint64_t k) {
          if (k >= above) to_list(k);
        });
        __syncthreads();
        n = sm.n_list;
      }
      if (n > kScoreList) {
        // still more: find the last alternative by radix search, list the N exactly
        const uint64_t last = score_radix_select(each_token, (uint32_t)p.N, sm.hist, sm.bc);
        if (tid == 0) sm.n_list = 0;
        __syncthreads();
        each_token([&](uint64_t k) {
          if (k >= last) sm.list[atomicAdd(&sm.n_list, 1u)] = k;
        });
        __syncthreads();
        n = sm.n_list;
      }
      found = n < (uint32_t)p.N ? n : (uint32_t)p.N;
      for (uint32_t i = tid; i < n; i += NT) {
        const uint64_t k = sm.list[i];
        uint32_t place = 0;
#pragma unroll 4
        for (uint32_t j = 0; j < n; ++j) place += sm.list[j] > k ? 1u : 0u;
        if (place < (uint32_t)p.N) {
          oi[place] = (int32_t)~(uint32_t)k;
          ol[place] = r.logprob(value_of_key32((uint32_t)(k >> 32)));
        }
      }
    }
  }
  for (uint32_t j = found + tid; j < (uint32_t)p.N; j += NT) {
    oi[j] = -1;
    ol[j] = qnan;
  }
}

template <typename T>
__global__ void __launch_bounds__(kScoreFinishThreads) score_finish_alt_kernel(const ScoreParams p) {
  __shared__ ScoreAltSmem sm;
  begin_overlapped();
  for (int64_t row = blockIdx.x; row < p.B; row += gridDim.x) {
    score_finish_alt<T>(p, row, p.token[row], p.rec + row * p.np, p.chunk_max + row * p.np * kScoreChunks, sm);
    __syncthreads();   // the next row reuses the shared arrays
  }
}

// Both steps in one launch: a cluster of CTAs takes a row, its warps write the records of their pieces into the first
// CTA's shared memory, and that CTA finishes the row. For small batches (see the launch): 4 x 32000 fp32 with five
// alternatives 6.5 us, bound by the chain of dependent steps.
template <typename T, bool ALT>
__global__ void __launch_bounds__(kScoreWarps * 32, 4) score_row_kernel(const ScoreParams p) {
  static_assert(kScoreWarps * 32 == kScoreFinishThreads, "the first CTA's threads finish the row");
  extern __shared__ __align__(16) unsigned char score_smem[];   // first CTA: [np] records, [np, 8] chunk maxima
  __shared__ ScoreAltSmem sm;
  cluster_begun_arrive();
  begin_overlapped();
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t C = cluster.num_blocks(), rank = cluster.block_rank(), row = blockIdx.x / C;
  float4* rec = reinterpret_cast<float4*>(score_smem);
  float* cm = reinterpret_cast<float*>(rec + p.np);
  const int32_t t = p.token[row];
  cluster_begun_wait();   // the first CTA's shared memory may be written
  if (t != VSAMP_TOKEN_IGNORE) {
    float4* rec0 = cluster.map_shared_rank(rec, 0);
    float* cm0 = cluster.map_shared_rank(cm, 0);
    for (int piece = rank * kScoreWarps + (threadIdx.x >> 5); piece < p.np; piece += C * kScoreWarps)
      score_piece<T, ALT>(p, row, piece, row * (uint32_t)p.np + piece, t, rec0 + piece, cm0 + piece * kScoreChunks);
  }
  cluster.sync();   // every record is in the first CTA
  if (rank != 0) return;
  if (ALT) {
    score_finish_alt<T>(p, row, t, rec, cm, sm);
  } else if (threadIdx.x < 32) {
    ScoreFold fold;
    fold.load(p, rec);
    const float xt = score_logit<T>(p, row, t);
    ScoreRow r{};
    if (t != VSAMP_TOKEN_IGNORE) r = fold.row(p, row, t);
    if (threadIdx.x == 0) score_write(p, row, t, xt, r);
  }
}

// ------------------------------------------------------------------------------------------------
// Gradient with respect to the logits: with g, h the gradients of the log-probability and the entropy,
//   dx_v = [g (d_vt - p_v) - h p_v (log p_v + H)] / T,   p_v = e^s_v / S.
// Elementwise: one read and one write of the row.
// ------------------------------------------------------------------------------------------------
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;   // 16-byte vectors per thread

// One row's constants. With q = 2^s2, s2 = (x - m) log2(e) / T, the gradient off the given token is
//   -p (g + h (log p + H)) / T = q (k0 + k1 s2)
struct GradRow {
  float m, c, k0, k1;
  __device__ __forceinline__ float at(float x) const {
    const float s = fmaxf((x - m) * c, -150.f);   // a masked token: 2^-150 is 0 in the flushed exponential
    return ex2_approx(s) * fmaf(k1, s, k0);
  }
};

// The same where k0 + k1 s2 could pass fp32's range (extreme temperatures, largest g and h): the constants are held
// without 1 / T, which comes last, and a token without probability has the gradient 0, not 0 * inf.
struct GradRowWide {
  ScoreRate rate;
  float m, k0, k1;
  // own: g for the given token, 0 for the others
  __device__ __forceinline__ float at(float x, float own) const {
    const float s = fmaxf(rate.exponent(x, m), -150.f), q = ex2_approx(s);
    return ((q > 0.f ? fmaf(q * s, k1, q * k0) : 0.f) + own) * (1.f / (rate.T * rate.scale)) * rate.scale;
  }
};

template <typename T>
__device__ __forceinline__ void grad_vector(const GradRow& r, uint32_t (&w)[4]) {
  using Ty = ScoreType<T>;
  const float2 m2 = make_float2(-r.m, -r.m), c2 = make_float2(r.c, r.c);
  const float2 k02 = make_float2(r.k0, r.k0), k12 = make_float2(r.k1, r.k1);
  uint32_t out[4];
#pragma unroll
  for (int j = 0; j < Ty::VE; j += 2) {
    float2 s = __fmul2_rn(__fadd2_rn(make_float2(Ty::at(w, j), Ty::at(w, j + 1)), m2), c2);
    s = make_float2(fmaxf(s.x, -150.f), fmaxf(s.y, -150.f));
    const float2 d = __fmul2_rn(make_float2(ex2_approx(s.x), ex2_approx(s.y)), __ffma2_rn(k12, s, k02));
    if constexpr (Ty::ES == 4) {
      out[j] = __float_as_uint(d.x);
      out[j + 1] = __float_as_uint(d.y);
    } else {
      const __nv_bfloat162 v = __floats2bfloat162_rn(d.x, d.y);
      memcpy(&out[j / 2], &v, 4);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = out[j];
}

// One CTA per row and span of kGradThreads * kGradVecs vectors. Vectors begin at the first 16-byte boundary of the
// gradient's row, whatever the logits' row's; the elements before and after the whole vectors belong to the row's first
// CTA. Streaming loads and stores: nothing is reused. Bound by the bytes: 2048 x 151936 bf16, a quarter of the rows
// ignored, 162.5 us, the copy rate.
template <typename T>
__global__ void __launch_bounds__(kGradThreads) score_grad_kernel(const ScoreGradParams p) {
  using Ty = ScoreType<T>;
  constexpr int VE = Ty::VE;
  constexpr int64_t SPAN = (int64_t)kGradThreads * kGradVecs;   // vectors
  begin_overlapped();
  const int64_t total = p.B * p.spans;
  for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
    const int64_t row = id / p.spans, span = id - row * p.spans;
    const unsigned char* xr = p.x + row * p.ld * Ty::ES;
    unsigned char* dr = p.dx + row * p.ldo * Ty::ES;
    const int32_t t = p.token[row];
    const bool skip = t == VSAMP_TOKEN_IGNORE;
    const int xa = (int)((16 - (reinterpret_cast<uintptr_t>(xr) & 15)) & 15) / Ty::ES;
    const int da = (int)((16 - (reinterpret_cast<uintptr_t>(dr) & 15)) & 15) / Ty::ES;
    const bool same = xa == da;   // the logits' row has the same boundary
    const int64_t head = da < p.V ? da : p.V, nv = (p.V - head) / VE;
    const int64_t v0 = span * SPAN + threadIdx.x;
    uint32_t w[kGradVecs][4];
    if (!skip && same) {
#pragma unroll
      for (int i = 0; i < kGradVecs; ++i) {
        const int64_t v = v0 + i * kGradThreads;
        if (v < nv) {
          const uint4 q = ldg_stream(xr + (head + v * VE) * Ty::ES);
          w[i][0] = q.x; w[i][1] = q.y; w[i][2] = q.z; w[i][3] = q.w;
        }
      }
    } else if (!skip) {
#pragma unroll
      for (int i = 0; i < kGradVecs; ++i) {
        const int64_t v = v0 + i * kGradThreads;
        if (v < nv) {
          ElemVec<T, VE> q;
          q.load(xr + (head + v * VE) * Ty::ES, false);
#pragma unroll
          for (int k = 0; k < 4; ++k) w[i][k] = q.w[k];
        }
      }
    }
    const float temp = p.temperature ? p.temperature[row] : 1.f;
    const float m = p.row_max[row], ls = p.row_logsum[row];
    const float H = p.dentropy ? p.entropy[row] : 0.f;
    const bool args = t >= 0 && (int64_t)t < p.V && !isnan(temp) && !isinf(temp);
    const bool ok = args && isfinite(m) && isfinite(ls) && isfinite(H);
    const float T1 = temp > 0.f ? temp : 1.f, invT = 1.f / T1, e = -expf(-ls);
    const float g = !skip && p.dlogprob ? p.dlogprob[row] : 0.f;
    const float h = !skip && p.dentropy ? p.dentropy[row] : 0.f;
    GradRow r;
    r.m = m;
    r.c = kLog2e / T1;
    r.k0 = (g + h * (H - ls)) * (e * invT);
    r.k1 = h * 0.69314718056f * (e * invT);
    const bool wide = !ScoreRate::ordinary(T1) || fmaf(fabsf(r.k1), 150.f, fabsf(r.k0)) > 3.4e38f;
    const float fill = skip ? 0.f : __int_as_float(0x7FC00000);
    if (p.row_status && span == 0 && threadIdx.x == 0)
      p.row_status[row] = skip || ok ? VSAMP_OK : args ? VSAMP_ERR_NONFINITE : VSAMP_ERR_INVALID_ARG;
    if (ok && wide) {   // a rare row: element by element
      const GradRowWide rw{ScoreRate::of(T1), m, (g + h * (H - ls)) * e, h * 0.69314718056f * e};
      const int64_t first = span == 0 ? 0 : head + span * SPAN * VE, last = head + (span + 1) * SPAN * VE;
      for (int64_t v = first + threadIdx.x; v < (span + 1 == p.spans || last > p.V ? p.V : last); v += kGradThreads)
        Ty::store(dr, v, rw.at(Ty::load(xr, v), v == t ? g : 0.f));
      continue;
    }
    auto one = [&](int64_t v) {
      float d = fill;
      if (ok) d = r.at(Ty::load(xr, v)) + (v == t ? g * invT : 0.f);
      Ty::store(dr, v, d);
    };
    const int64_t tv = ok && t >= head ? (t - head) / VE : -1;   // the vector that holds the given token
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
      const int64_t v = v0 + i * kGradThreads;
      if (v < nv) {
        if (!ok) {
          const uint32_t b = skip ? 0u : Ty::ES == 4 ? 0x7FC00000u : 0x7FC07FC0u;
          w[i][0] = w[i][1] = w[i][2] = w[i][3] = b;
        } else if (v != tv) {
          grad_vector<T>(r, w[i]);
        } else {
          const int at = (int)(t - head - v * VE);
          float f[VE];
#pragma unroll
          for (int j = 0; j < VE; ++j) f[j] = r.at(Ty::at(w[i], j)) + (j == at ? g * invT : 0.f);
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            if constexpr (Ty::ES == 4) w[i][j] = __float_as_uint(f[j]);
            else Ty::put(w[i], j, __bfloat162float(__float2bfloat16_rn(f[j])));
          }
        }
        __stcs(reinterpret_cast<uint4*>(dr + (head + v * VE) * Ty::ES), make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]));
      }
    }
    if (span == 0) {
      if ((int64_t)threadIdx.x < head) one(threadIdx.x);
      const int64_t e = head + nv * VE + threadIdx.x;
      if (threadIdx.x < VE && e < p.V) one(e);
    }
  }
}

}  // namespace vsamp
