// Embedding lookup (vsamp_embed) and its gradient by sorted tokens (vsamp_embed_backward).
//
// Lookup: out[n, :] = scale * table[token[n], :], the product in fp32, rounded once.
//
// Gradient: dtable[v, :] = (dtable[v, :] +) scale * sum over n with token[n] = v of dout[n, :]. The positions are
// sorted by (token, position) with a stable radix sort; the sorted list is cut into fixed tiles, each summed in
// order in fp32. A run of equal tokens inside a tile is written at once, the first and last run of a tile, which may
// go on in the neighbours, leave partial sums that the run's first tile joins in tile order. So the result depends
// on the inputs alone: no atomics on floating values, whatever the launch.
#pragma once

#include "vsamp.h"
#include "vsamp_device.cuh"

namespace vsamp {

constexpr int kSortThreads = 512;
constexpr int kSortPer = 8;                              // keys per thread
constexpr int kSortTile = kSortThreads * kSortPer;       // keys per CTA
constexpr int kSortBits = 8;
constexpr int kSortBins = 1 << kSortBits;
constexpr int kEmbedTile = 16;                           // sorted positions per tile of the sums
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
  uint2* keys[2];          // {token or kNoToken, position}
  uint32_t* hist;          // [tiles, bins]
  float* part;             // [2 * sum tiles, D] partial sums of the first and last run of a tile
  int64_t tiles;           // sort tiles
  int64_t sums;            // sum tiles
};

template <typename T>
__device__ __forceinline__ float elem_load(const unsigned char* p, int64_t i) {
  if constexpr (sizeof(T) == 4) return reinterpret_cast<const float*>(p)[i];
  else return __uint_as_float((uint32_t) reinterpret_cast<const unsigned short*>(p)[i] << 16);
}
template <typename T>
__device__ __forceinline__ void elem_store(unsigned char* p, int64_t i, float f) {
  if constexpr (sizeof(T) == 4) reinterpret_cast<float*>(p)[i] = f;
  else reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f);
}

constexpr int kEmbedThreads = 256;
constexpr int kEmbedSpan = 1024;     // columns per CTA and step

template <typename TI, typename TO>
__global__ void __launch_bounds__(kEmbedThreads) embed_kernel(const EmbedParams p) {
  const int64_t spans = (p.D + kEmbedSpan - 1) / kEmbedSpan;
  const int64_t total = p.N * spans;
  for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
    const int64_t n = id / spans, c0 = (id - n * spans) * kEmbedSpan;
    const int32_t t = p.token[n];
    const bool skip = t == VSAMP_TOKEN_IGNORE;
    const bool ok = t >= 0 && (int64_t)t < p.V;
    if (p.row_status && c0 == 0 && threadIdx.x == 0) p.row_status[n] = ok || skip ? VSAMP_OK : VSAMP_ERR_INVALID_ARG;
    const unsigned char* src = p.table + (ok ? (int64_t)t * p.ldt : 0) * (int64_t)sizeof(TI);
    unsigned char* dst = p.out + n * p.ldo * (int64_t)sizeof(TO);
    const float fill = skip ? 0.f : __int_as_float(0x7FC00000);
    for (int64_t c = c0 + threadIdx.x; c < c0 + kEmbedSpan && c < p.D; c += kEmbedThreads)
      elem_store<TO>(dst, c, ok ? elem_load<TI>(src, c) * p.scale : fill);
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

template <typename TO>
__global__ void __launch_bounds__(kEmbedThreads) embed_zero_kernel(const EmbedGradParams p) {
  const int64_t total = p.V * p.D;
  for (int64_t i = (int64_t)blockIdx.x * kEmbedThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kEmbedThreads) {
    const int64_t v = i / p.D;
    elem_store<TO>(p.dtable, v * p.ldt + (i - v * p.D), 0.f);
  }
}

// Sums of one tile of kEmbedTile sorted positions: block (tile, columns).
template <typename TI, typename TO>
__global__ void __launch_bounds__(kEmbedThreads) embed_sum_kernel(const EmbedGradParams p, int last) {
  const uint2* keys = p.keys[last];
  const int64_t spans = (p.D + kEmbedThreads - 1) / kEmbedThreads;
  for (int64_t id = blockIdx.x; id < p.sums * spans; id += gridDim.x) {
    const int64_t tile = id / spans;
    const int64_t c = (id - tile * spans) * kEmbedThreads + threadIdx.x;
    const int64_t i0 = tile * kEmbedTile, i1 = i0 + kEmbedTile < p.N ? i0 + kEmbedTile : p.N;
    if (c >= p.D) continue;
    const uint32_t prev = i0 > 0 ? keys[i0 - 1].x : kNoToken;
    const uint32_t next = i1 < p.N ? keys[i1].x : kNoToken;
    float sum = 0.f;
    int64_t start = i0;
    for (int64_t i = i0; i < i1; ++i) {
      const uint2 k = keys[i];
      if (k.x == kNoToken) break;
      sum += elem_load<TI>(p.dout, (int64_t)k.y * p.ldd + c);
      const uint32_t after = i + 1 < i1 ? keys[i + 1].x : next;
      if (after == k.x && i + 1 < i1) continue;
      // the run ends here, or goes on in the next tile
      const bool from_before = start == i0 && prev == k.x;
      const bool goes_on = i + 1 == i1 && after == k.x;
      if (!from_before && !goes_on) {
        const int64_t at = (int64_t)k.x * p.ldt + c;
        float r = sum * p.scale;
        if (p.accumulate) r += elem_load<TO>(p.dtable, at);
        elem_store<TO>(p.dtable, at, r);
      } else {
        // slot 0: the tile's first run, slot 1: its last (a run that fills the tile has slot 0)
        p.part[(tile * 2 + (from_before ? 0 : 1)) * p.D + c] = sum;
      }
      sum = 0.f;
      start = i + 1;
    }
  }
}

// Runs over several tiles: the tile where a run begins adds up its parts in order.
template <typename TO>
__global__ void __launch_bounds__(kEmbedThreads) embed_join_kernel(const EmbedGradParams p, int last) {
  const uint2* keys = p.keys[last];
  const int64_t spans = (p.D + kEmbedThreads - 1) / kEmbedThreads;
  for (int64_t id = blockIdx.x; id < p.sums * spans; id += gridDim.x) {
    const int64_t tile = id / spans;
    const int64_t c = (id - tile * spans) * kEmbedThreads + threadIdx.x;
    const int64_t i0 = tile * kEmbedTile, i1 = i0 + kEmbedTile;
    if (c >= p.D || i1 >= p.N) continue;
    const uint32_t tok = keys[i1 - 1].x;
    if (tok == kNoToken || keys[i1].x != tok) continue;               // no run goes on from this tile
    if (i0 > 0 && keys[i0].x == tok && keys[i0 - 1].x == tok) continue;   // it began earlier
    float sum = p.part[(tile * 2 + 1) * p.D + c];
    for (int64_t k = tile + 1; k < p.sums && keys[k * kEmbedTile].x == tok; ++k) sum += p.part[(k * 2) * p.D + c];
    const int64_t at = (int64_t)tok * p.ldt + c;
    float r = sum * p.scale;
    if (p.accumulate) r += elem_load<TO>(p.dtable, at);
    elem_store<TO>(p.dtable, at, r);
  }
}

}  // namespace vsamp
