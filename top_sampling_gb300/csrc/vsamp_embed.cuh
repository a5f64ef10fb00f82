// Embedding lookup (vsamp_embed) and its gradient by sorted tokens (vsamp_embed_backward).
//
// Lookup: out[n, :] = scale * table[token[n], :], the product in fp32, rounded once.
//
// Gradient: dtable[v, :] = (dtable[v, :] +) scale * sum over n with token[n] = v of dout[n, :]. The result depends on
// the inputs alone: no atomics on floating values, every sum in a fixed order.
//   Few positions: a CTA per position and column span finds the later positions of its token (and leaves if there is
//   an earlier one) and adds their rows in order.
//   Many positions: they are sorted by (token, position) with a stable radix sort, in one CTA while the others write
//   the zeros of the untouched rows, or in several launches for long lists. The sorted list is cut into fixed tiles,
//   each summed in order. A run of equal tokens inside a tile is written at once; the first and last run of a tile,
//   which may go on in the neighbours, leave partial sums that the run's first tile joins in tile order.
#pragma once

#include "vsamp.h"
#include "vsamp_device.cuh"
#include "vsamp_vec.cuh"

namespace vsamp {

constexpr int kSortThreads = 512;
constexpr int kSortPer = 8;                              // keys per thread
constexpr int kSortTile = kSortThreads * kSortPer;       // keys per CTA
constexpr int kSortBits = 8;
constexpr int kSortBins = 1 << kSortBits;
constexpr int kEmbedTile = 16;                           // sorted positions per tile of the sums
constexpr int kJoinSpan = 1024;                          // columns per CTA of the join
constexpr uint32_t kNoToken = 0xFFFFFFFFu;               // sorts after every token

struct EmbedParams {
  const int32_t* token;
  int64_t N;
  const unsigned char* table;
  int64_t V, D, ldt;
  float scale;
  unsigned char* out;
  int64_t ldo;
  int32_t* row_status;
};

struct EmbedGradParams {
  const int32_t* token;
  int64_t N;
  const unsigned char* dout;
  int64_t D, ldd, V;
  float scale;
  unsigned char* dtable;
  int64_t ldt;
  int accumulate;
  int aligned;             // every row of dout and of the table begins on a vector's boundary
  uint2* keys[2];          // {token or kNoToken, position}
  uint32_t* hist;          // [tiles, bins]
  float* part;             // [2 * sum tiles, ldp] partial sums of the first and last run of a tile
  int64_t ldp;
  uint32_t* runs;          // [sum tiles] tiles where a run over several tiles begins, in any order
  uint32_t* n_runs;
  int64_t tiles;           // sort tiles
  int64_t sums;            // sum tiles
};

constexpr int kEmbedThreads = 256;

// WHOLE: every row of the table and of the output is whole aligned vectors.
// tx threads of a CTA along a row (a power of two), kEmbedThreads / tx rows per CTA, kEmbedUnroll vectors per thread and
// row so that their loads are in flight together (two took a sixth longer; 16384 x 4096 bf16: 32 us, 90% of the copy rate).
constexpr int kEmbedUnroll = 4;

template <typename TI, typename TO, int VE, bool WHOLE>
__global__ void __launch_bounds__(kEmbedThreads) embed_kernel(const EmbedParams p, int tx, int spans) {
  constexpr int U = kEmbedUnroll;
  begin_overlapped();
  const int col = threadIdx.x & (tx - 1), per = kEmbedThreads / tx, D = (int)p.D;
  const int64_t total = (p.N + per - 1) / per * spans;
  for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
    const int64_t group = spans == 1 ? id : id / spans;
    const int64_t n = group * per + threadIdx.x / tx;
    const int c0 = ((int)(id - group * spans) * U * tx + col) * VE;
    if (n >= p.N) continue;
    const int32_t t = p.token[n];
    const bool skip = t == VSAMP_TOKEN_IGNORE;
    const bool ok = t >= 0 && (int64_t)t < p.V;
    if (p.row_status && c0 == 0) p.row_status[n] = ok || skip ? VSAMP_OK : VSAMP_ERR_INVALID_ARG;
    const unsigned char* src = p.table + (ok ? (int64_t)t * p.ldt : 0) * (int64_t)sizeof(TI);
    unsigned char* dst = p.out + n * p.ldo * (int64_t)sizeof(TO);
    // vectors begin at the output row's first boundary of a vector; the elements before it go one by one
    constexpr int OB = VE * (int)sizeof(TO), IB = VE * (int)sizeof(TI);
    const int head = WHOLE ? 0 : (int)((OB - (reinterpret_cast<uintptr_t>(dst) & (OB - 1))) & (OB - 1)) / (int)sizeof(TO);
    const int first = head + c0;
    src += (int64_t)first * (int)sizeof(TI);
    dst += (int64_t)first * (int)sizeof(TO);
    const bool aligned = WHOLE || (reinterpret_cast<uintptr_t>(src) & (IB - 1)) == 0;
    ElemVec<TI, VE> v[U];
    if (ok) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = u * tx * VE;
        if (first + c < D) {
          if (WHOLE) v[u].load(src + c * (int)sizeof(TI), true);
          else v[u].load_row(src + c * (int)sizeof(TI), D - first - c, aligned, 0u);
        }
      }
    }
    const float fill = skip ? 0.f : __int_as_float(0x7FC00000);
    auto put = [&](const ElemVec<TI, VE>& x, ElemVec<TO, VE>& o) {
      float f[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) f[j] = ok ? x.at(j) * p.scale : fill;
      o.set(f);
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = u * tx * VE;
      if (first + c < D) {
        ElemVec<TO, VE> o;
        put(v[u], o);
        if (WHOLE) o.store(dst + c * (int)sizeof(TO), true);
        else o.store_row(dst + c * (int)sizeof(TO), D - first - c, true);
      }
    }
    if (!WHOLE && c0 == 0 && head > 0) {
      const int left = head < D ? head : D;
      ElemVec<TI, VE> x;
      ElemVec<TO, VE> o;
      if (ok) x.load_some(src - (int64_t)head * (int)sizeof(TI), left, 0u);
      put(x, o);
      o.store_some(dst - (int64_t)head * (int)sizeof(TO), left);
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Stable radix sort of (token, position), kSortBits at a time.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ uint2 embed_key(const EmbedGradParams& p, int pass, int64_t i) {
  if (pass > 0) return p.keys[(pass - 1) & 1][i];
  const int32_t t = p.token[i];
  return make_uint2(t >= 0 && (int64_t)t < p.V ? (uint32_t)t : kNoToken, (uint32_t)i);
}

__global__ void __launch_bounds__(kSortThreads) embed_hist_kernel(const EmbedGradParams p, int pass) {
  __shared__ uint32_t hist[kSortBins];
  begin_overlapped();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.n_runs = 0;
  for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    for (int i = threadIdx.x; i < kSortBins; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    for (int j = 0; j < kSortPer; ++j) {
      const int64_t i = tile * kSortTile + j * kSortThreads + threadIdx.x;
      if (i < p.N) atomicAdd(&hist[(embed_key(p, pass, i).x >> (pass * kSortBits)) & (kSortBins - 1)], 1u);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kSortBins; i += kSortThreads) p.hist[tile * kSortBins + i] = hist[i];
    __syncthreads();
  }
}

// Every CTA derives the places of its tile's keys from the histograms of all tiles: keys of smaller digits, keys of
// the same digit in earlier tiles, then the order inside the tile (warp by warp, 32 consecutive keys at a time).
__global__ void __launch_bounds__(kSortThreads) embed_scatter_kernel(const EmbedGradParams p, int pass) {
  constexpr int NW = kSortThreads / 32;
  __shared__ uint32_t base[kSortBins];
  __shared__ uint32_t count[NW][kSortBins];   // keys of each digit in every warp's part of the tile
  __shared__ uint32_t wsum[kSortBins / 32];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  begin_overlapped();
  for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    uint32_t all = 0, earlier = 0;
    if (t < kSortBins) {
      for (int64_t k = 0; k < p.tiles; ++k) {
        const uint32_t h = p.hist[k * kSortBins + t];
        all += h;
        if (k < tile) earlier += h;
      }
      uint32_t incl = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kFullMask, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) wsum[warp] = incl;
      base[t] = incl - all + earlier;
    }
    for (int i = t; i < NW * kSortBins; i += kSortThreads) (&count[0][0])[i] = 0;
    __syncthreads();
    if (t < kSortBins) {
      uint32_t add = 0;
      for (int w = 0; w < warp; ++w) add += wsum[w];
      base[t] += add;
    }
    // a warp's part: kSortPer * 32 consecutive keys
    uint2 key[kSortPer];
    uint32_t place[kSortPer];
    const int64_t w0 = tile * kSortTile + (int64_t)warp * kSortPer * 32;
#pragma unroll
    for (int j = 0; j < kSortPer; ++j) {
      const int64_t i = w0 + j * 32 + lane;
      const bool in = i < p.N;
      key[j] = in ? embed_key(p, pass, i) : make_uint2(0, 0);
      const uint32_t d = in ? (key[j].x >> (pass * kSortBits)) & (kSortBins - 1) : kSortBins;
      const uint32_t same = __match_any_sync(kFullMask, d);
      const uint32_t before = __popc(same & ((1u << lane) - 1u));
      if (in) {
        place[j] = count[warp][d] + before;
      }
      __syncwarp();
      if (in && before == 0) count[warp][d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    // exclusive sums over the warps
    if (t < kSortBins) {
      uint32_t run = base[t];
      for (int w = 0; w < NW; ++w) {
        const uint32_t c = count[w][t];
        count[w][t] = run;
        run += c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortPer; ++j) {
      const int64_t i = w0 + j * 32 + lane;
      if (i < p.N) {
        const uint32_t d = (key[j].x >> (pass * kSortBits)) & (kSortBins - 1);
        p.keys[pass & 1][count[warp][d] + place[j]] = key[j];
      }
    }
    __syncthreads();
  }
}

// Zeros over nrows byte ranges of row_bytes (the last one last_bytes) that begin row_stride apart: a warp per range.
struct ZeroParams {
  unsigned char* base;
  int64_t row_stride, row_bytes, last_bytes, nrows;
};
constexpr int64_t kZeroSpan = 16384;   // bytes per range of a contiguous table

__device__ __forceinline__ void zero_ranges(const ZeroParams& z, int64_t warp, int64_t nwarps) {
  const int lane = threadIdx.x & 31;
  for (int64_t r = warp; r < z.nrows; r += nwarps) {
    unsigned char* p = z.base + r * z.row_stride;
    const int64_t bytes = r + 1 == z.nrows ? z.last_bytes : z.row_bytes;
    // up to the first 16-byte boundary, whole vectors, the rest (elements are 2 or 4 bytes, so steps of 2)
    int64_t head = (16 - (int64_t)(reinterpret_cast<uintptr_t>(p) & 15)) & 15;
    if (head > bytes) head = bytes;
    const int64_t nv = (bytes - head) / 16, tail = head + nv * 16;
    if (lane * 2 < head) *reinterpret_cast<unsigned short*>(p + lane * 2) = 0;
    uint4* q = reinterpret_cast<uint4*>(p + head);
#pragma unroll 4
    for (int64_t i = lane; i < nv; i += 32) __stcs(q + i, make_uint4(0, 0, 0, 0));
    if (tail + lane * 2 < bytes) *reinterpret_cast<unsigned short*>(p + tail + lane * 2) = 0;
  }
}

__global__ void __launch_bounds__(kEmbedThreads) embed_zero_kernel(const ZeroParams z) {
  begin_overlapped();
  zero_ranges(z, (int64_t)blockIdx.x * (kEmbedThreads / 32) + (threadIdx.x >> 5), (int64_t)gridDim.x * (kEmbedThreads / 32));
}

// One CTA sorts up to kSortOne positions on chip, the others write zeros (no z: z.nrows = 0 and a grid of one CTA).
// A key is token << pos_bits | position: 32 bits hold both, the marker token V included. Least significant digit
// first, stable: a warp takes consecutive keys 32 at a time, equal digits keep their order. A thread's keys and their
// places among equal digits of its warp stay in registers between the count and the move, so one buffer is enough.
// 16384 positions take about 30 us in one CTA, bound by the warp matches; beside the zeros of a large table (1.2 GB, 186
// us) they cost nothing. Where the zeros end sooner, or nothing is zeroed, the sort stands alone: 16384 positions take 64
// us into 32000 x 1024 bf16 (bytes: 15), about what the sort in several launches takes for one position more (63).
constexpr int kSortOne = 16384;
constexpr int kSortOneThreads = 1024;
constexpr int kSortOnePer = kSortOne / kSortOneThreads;
constexpr int kSortOneBins = 512;   // digits of up to nine bits: two passes for vocabularies of up to 2^18
struct SortOneSmem {
  uint32_t key[kSortOne];
  uint16_t count[kSortOneThreads / 32][kSortOneBins];
  uint32_t wsum[kSortOneBins / 32];
};

__global__ void __launch_bounds__(kSortOneThreads) embed_sort_one_kernel(const EmbedGradParams p, const ZeroParams z,
                                                                         int pos_bits, int digit_bits, int passes) {
  begin_overlapped();
  if (blockIdx.x > 0) {
    zero_ranges(z, (int64_t)(blockIdx.x - 1) * (kSortOneThreads / 32) + (threadIdx.x >> 5),
                (int64_t)(gridDim.x - 1) * (kSortOneThreads / 32));
    return;
  }
  extern __shared__ __align__(16) unsigned char sort_smem[];
  SortOneSmem& S = *reinterpret_cast<SortOneSmem*>(sort_smem);
  constexpr int NW = kSortOneThreads / 32;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int n = (int)p.N, per = (n + NW * 32 - 1) / (NW * 32);   // 32-key steps per warp
  if (t == 0) *p.n_runs = 0;
#pragma unroll
  for (int j = 0; j < kSortOnePer; ++j) {   // all loads in flight
    const int i = j * kSortOneThreads + t;
    if (i < n) {
      const int32_t tok = p.token[i];
      const uint32_t v = tok >= 0 && (int64_t)tok < p.V ? (uint32_t)tok : (uint32_t)p.V;
      S.key[i] = v << pos_bits | (uint32_t)i;
    }
  }
  const int w0 = warp * per * 32 + lane;
  const uint32_t digit_mask = (1u << digit_bits) - 1u;
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pos_bits + pass * digit_bits;
    for (int i = t; i < NW * kSortOneBins; i += kSortOneThreads) (&S.count[0][0])[i] = 0;
    __syncthreads();
    uint32_t key[kSortOnePer], same[kSortOnePer];
#pragma unroll
    for (int j = 0; j < kSortOnePer; ++j) {
      if (j < per) {
        const int i = w0 + j * 32;
        key[j] = i < n ? S.key[i] : 0u;
        same[j] = __match_any_sync(kFullMask, i < n ? (key[j] >> shift) & digit_mask : kSortOneBins);
      }
    }
#pragma unroll
    for (int j = 0; j < kSortOnePer; ++j) {
      if (j < per) {
        const bool in = w0 + j * 32 < n;
        const uint32_t d = (key[j] >> shift) & digit_mask;
        const uint32_t had = in ? S.count[warp][d] : 0u, before = __popc(same[j] & ((1u << lane) - 1u));
        __syncwarp();
        if (in && before == 0) S.count[warp][d] = (uint16_t)(had + __popc(same[j]));
        __syncwarp();
        same[j] = had + before;   // the key's place among its warp's keys of the digit
      }
    }
    __syncthreads();
    uint32_t all = 0, incl = 0;
    if (t < kSortOneBins) {   // this digit's keys
#pragma unroll 8
      for (int w = 0; w < NW; ++w) all += S.count[w][t];
      incl = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kFullMask, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) S.wsum[warp] = incl;
    }
    __syncthreads();
    if (t < kSortOneBins) {   // where every warp's keys of the digit begin
      uint32_t run = incl - all;
      for (int w = 0; w < warp; ++w) run += S.wsum[w];
#pragma unroll 8
      for (int w = 0; w < NW; ++w) {
        const uint32_t c = S.count[w][t];
        S.count[w][t] = (uint16_t)run;
        run += c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortOnePer; ++j)
      if (j < per && w0 + j * 32 < n) S.key[S.count[warp][(key[j] >> shift) & digit_mask] + same[j]] = key[j];
    __syncthreads();
  }
  for (int i = t; i < n; i += kSortOneThreads) {
    const uint32_t v = S.key[i] >> pos_bits;
    p.keys[0][i] = make_uint2(v < (uint32_t)p.V ? v : kNoToken, S.key[i] & ((1u << pos_bits) - 1u));
  }
}

// Columns [c, c + VE) of a position's row of dout (0 beyond D). whole: every row is aligned whole vectors.
template <typename TI, int VE>
__device__ __forceinline__ void load_dout(const EmbedGradParams& p, bool whole, bool aligned, int64_t position, int64_t c,
                                          ElemVec<TI, VE>& v) {
  const unsigned char* at = p.dout + (position * p.ldd + c) * (int64_t)sizeof(TI);
  if (whole) v.load(at, true);
  else v.load_row(at, p.D - c, aligned, 0u);
}

// Adds `n` rows of dout in order; row i is at position pos(i). Eight rows are in flight at a time.
template <typename TI, int VE, typename F>
__device__ __forceinline__ void add_rows(const EmbedGradParams& p, int64_t c, int n, F pos, float (&sum)[VE]) {
  int i = 0;
  for (; i + 8 <= n; i += 8) {
    ElemVec<TI, VE> v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) load_dout(p, false, p.aligned, pos(i + j), c, v[j]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < VE; ++e) sum[e] += v[j].at(e);
  }
  for (; i < n; ++i) {
    ElemVec<TI, VE> v;
    load_dout(p, false, p.aligned, pos(i), c, v);
#pragma unroll
    for (int e = 0; e < VE; ++e) sum[e] += v.at(e);
  }
}

// One row's span of the table: scale * sum, added or written, one rounding.
template <typename TO, int VE>
__device__ __forceinline__ void put_row(const EmbedGradParams& p, bool whole, uint32_t tok, int64_t c,
                                        float (&sum)[VE]) {
  unsigned char* at = p.dtable + ((int64_t)tok * p.ldt + c) * (int64_t)sizeof(TO);
#pragma unroll
  for (int e = 0; e < VE; ++e) sum[e] *= p.scale;
  ElemVec<TO, VE> v;
  if (p.accumulate) {
    if (whole) v.load(at, true);
    else v.load_row(at, p.D - c, p.aligned, 0u);
#pragma unroll
    for (int e = 0; e < VE; ++e) sum[e] += v.at(e);
  }
  v.set(sum);
  if (whole) v.store(at, true);
  else v.store_row(at, p.D - c, p.aligned);
}

// Few positions (N <= kEmbedFew): a CTA per position and span of columns, no workspace. Every CTA compares its token
// with all of them (4 KB at most, from L2), which is cheaper than a sort's launches: 509 positions of 1001 fp32 columns
// take 7 us against 22 with the sort. The comparisons and the longest run's chain grow with the positions; takes_few has
// the figures of both forms.
constexpr int kEmbedFew = 1024;

template <typename TI, typename TO, int VE>
__global__ void __launch_bounds__(kEmbedThreads) embed_few_kernel(const EmbedGradParams p, int spans) {
  __shared__ uint32_t bits[kEmbedFew / 32];
  __shared__ uint16_t list[kEmbedFew];
  __shared__ int count;
  begin_overlapped();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n0 = (int)(blockIdx.x / spans), N = (int)p.N;
  const int32_t tok = p.token[n0];
  if (tok < 0 || (int64_t)tok >= p.V) return;
  for (int i = warp * 32; i < kEmbedFew; i += kEmbedThreads) {
    const uint32_t b = __ballot_sync(kFullMask, i + lane < N && p.token[i + lane] == tok);
    if (lane == 0) bits[i / 32] = b;
  }
  __syncthreads();
  if (warp == 0) {   // lane l: positions 32 l .. 32 l + 31
    uint32_t b = bits[lane];
    const uint32_t first = __ballot_sync(kFullMask, b != 0);
    const int low = __shfl_sync(kFullMask, __ffs(b) - 1, __ffs(first) - 1) + 32 * (__ffs(first) - 1);
    int incl = __popc(b);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFullMask, incl, o);
      if (lane >= o) incl += v;
    }
    int at = incl - __popc(b);
    for (; b; b &= b - 1) list[at++] = (uint16_t)(lane * 32 + __ffs(b) - 1);
    if (lane == 31) count = low == n0 ? incl : 0;   // an earlier position of the token has these rows
  }
  __syncthreads();
  const int n = count;
  const int64_t c = ((int64_t)(blockIdx.x % spans) * kEmbedThreads + threadIdx.x) * VE;
  if (n == 0 || c >= p.D) return;
  float sum[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) sum[e] = 0.f;
  add_rows<TI, VE>(p, c, n, [&](int i) { return (int)list[i]; }, sum);
  put_row<TO, VE>(p, false, (uint32_t)tok, c, sum);
}

// Sums of one tile of kEmbedTile sorted positions: a CTA per tile and span of columns. A tile is read in two halves:
// eight rows in flight per thread and three CTAs per SM (all sixteen at once held 174 registers, one CTA per SM, and
// took twice the time). 16384 x 4096 bf16: 35 us for 190 MB read and written. Writing part of the zeros from this launch
// instead, beside the sums, was slower at every split (264 us and more for the whole gradient against 235).
constexpr int kSumBatch = 8;

template <typename TI, typename TO, int VE, bool WHOLE>
__global__ void __launch_bounds__(kEmbedThreads, 3) embed_sum_kernel(const EmbedGradParams p, int last, int spans) {
  const uint2* keys = p.keys[last];
  begin_overlapped();
  for (int64_t id = blockIdx.x; id < p.sums * spans; id += gridDim.x) {
    const int64_t tile = spans == 1 ? id : id / spans;
    const int64_t span = id - tile * spans, c = (span * kEmbedThreads + threadIdx.x) * VE;
    const int64_t i0 = tile * kEmbedTile, i1 = i0 + kEmbedTile < p.N ? i0 + kEmbedTile : p.N;
    const uint32_t prev = i0 > 0 ? keys[i0 - 1].x : kNoToken;
    const uint32_t next = i1 < p.N ? keys[i1].x : kNoToken;
    const uint32_t head = keys[i0].x, tail = keys[i1 - 1].x;
    bool from_before = prev == head;   // the run at hand began in an earlier tile
    // the tile where a run begins that goes on past it puts it on the join's list
    if (span == 0 && threadIdx.x == 0 && tail == next && tail != kNoToken && !(from_before && head == tail))
      p.runs[atomicAdd(p.n_runs, 1u)] = (uint32_t)tile;
    if (c >= p.D) continue;
    float sum[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) sum[e] = 0.f;
    for (int64_t b = i0; b < i1; b += kSumBatch) {
      uint2 key[kSumBatch];
      ElemVec<TI, VE> v[kSumBatch];
#pragma unroll
      for (int i = 0; i < kSumBatch; ++i) key[i] = b + i < i1 ? keys[b + i] : make_uint2(kNoToken, 0);
#pragma unroll
      for (int i = 0; i < kSumBatch; ++i)
        if (key[i].x != kNoToken) load_dout(p, WHOLE, p.aligned, key[i].y, c, v[i]);
      const uint32_t after_batch = b + kSumBatch < i1 ? keys[b + kSumBatch].x : next;
#pragma unroll
      for (int i = 0; i < kSumBatch; ++i) {
        if (key[i].x != kNoToken) {
#pragma unroll
          for (int e = 0; e < VE; ++e) sum[e] += v[i].at(e);
          const bool end = b + i + 1 == i1;   // of the tile
          const uint32_t after = end ? next : i + 1 < kSumBatch ? key[i + 1 < kSumBatch ? i + 1 : 0].x : after_batch;
          if (after != key[i].x || end) {
            if (!from_before && after != key[i].x) {
              put_row<TO, VE>(p, WHOLE, key[i].x, c, sum);
            } else {
              // slot 0: the tile's first run, slot 1: its last (a run that fills the tile from before has slot 0)
              // (the parts' rows are padded to whole vectors)
              ElemVec<float, VE> part;
              part.set(sum);
              part.store(reinterpret_cast<unsigned char*>(p.part + (tile * 2 + (from_before ? 0 : 1)) * p.ldp + c), true);
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) sum[e] = 0.f;
            from_before = false;
          }
        }
      }
    }
  }
}

// Tiles after `tile` that begin with tok, for a run that goes on past its tile: called by a whole warp, which looks at
// 32 tiles at a time, then at 32 points of what is left.
__device__ __forceinline__ int64_t run_tiles(const uint2* keys, int64_t tile, int64_t tiles, uint32_t tok) {
  const int lane = threadIdx.x & 31;
  auto holds = [&](int64_t k) { return k < tiles && keys[k * kEmbedTile].x == tok; };
  uint32_t b = __ballot_sync(kFullMask, holds(tile + 1 + lane));
  if (b != kFullMask) return __popc(b);
  int64_t lo = tile + 32, hi = tiles;   // lo holds the token, hi does not
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 31) / 32;
    b = __ballot_sync(kFullMask, lo + step * lane < hi && holds(lo + step * lane));
    lo += step * (__popc(b) - 1);
    if (lo + step < hi) hi = lo + step;
  }
  return lo - tile;
}

// Runs over several tiles, from the list that the sums left (a fixed grid: the list's length is only known on the device):
// a CTA per run and kJoinSpan columns, four per thread, adds
// the run's parts in tile order, kJoinBatch in flight.
constexpr int kJoinBatch = 16;

template <typename TO>
__global__ void __launch_bounds__(kEmbedThreads) embed_join_kernel(const EmbedGradParams p, int last, int spans) {
  const uint2* keys = p.keys[last];
  begin_overlapped();
  const int64_t total = (int64_t)*p.n_runs * spans;
  for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
    const int64_t run = id / spans, tile = p.runs[run];
    const uint32_t tok = keys[tile * kEmbedTile + kEmbedTile - 1].x;
    const int64_t end = tile + run_tiles(keys, tile, p.sums, tok);   // the last tile of the run
    const int64_t c = (id - run * spans) * kJoinSpan + threadIdx.x * 4;
    if (c >= p.D) continue;
    // parts are padded to ldp, a multiple of 8, columns; slot 1 of the first tile, slot 0 of the others
    auto at = [&](int64_t k, int slot) { return *reinterpret_cast<const float4*>(p.part + (k * 2 + slot) * p.ldp + c); };
    float4 sum = at(tile, 1);
    auto add = [&](const float4& v) {
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    };
    int64_t k = tile + 1;
    for (; k + kJoinBatch <= end + 1; k += kJoinBatch) {
      float4 v[kJoinBatch];
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) v[i] = at(k + i, 0);
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) add(v[i]);
    }
    for (; k <= end; ++k) add(at(k, 0));
    float all[4] = {sum.x, sum.y, sum.z, sum.w};
    put_row<TO, 4>(p, false, tok, c, all);
  }
}

}  // namespace vsamp
