// vsamp_embed and vsamp_embed_backward: argument checks and launches.
#include "vsamp_embed.cuh"
#include "vsamp_grid.h"

namespace vsamp {

static bool type_ok(vsamp_dtype dt) { return dt == VSAMP_F32 || dt == VSAMP_BF16; }
static bool elem_aligned(const void* p, vsamp_dtype dt) {
  return (reinterpret_cast<uintptr_t>(p) & (dt == VSAMP_F32 ? 3u : 1u)) == 0;
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Radix passes for tokens below V and the marker of positions without a token, which sorts last in each digit
static int sort_passes(int64_t V) {
  int bits = 1;
  while (bits < 32 && (V >> bits) != 0) ++bits;   // V itself fits: the marker's low bits are larger than any token's
  return ceil_div(bits, kSortBits);
}

template <typename TI, typename TO>
static vsamp_status launch_embed(const EmbedParams& p, cudaStream_t s) {
  const int64_t spans = ceil_div(p.D, kEmbedSpan);
  return launch_1d(embed_kernel<TI, TO>, grid_of(p.N * spans), kEmbedThreads, 0, s, false, p);
}

template <typename TI, typename TO>
static vsamp_status launch_embed_grad(const EmbedGradParams& p, cudaStream_t s) {
  vsamp_status st = VSAMP_OK;
  if (!p.accumulate) {
    st = launch_1d(embed_zero_kernel<TO>, grid_of(ceil_div(p.V * p.D, kEmbedThreads * 8)), kEmbedThreads, 0, s, false, p);
    if (st != VSAMP_OK) return st;
  }
  const int passes = sort_passes(p.V);
  for (int k = 0; k < passes; ++k) {
    st = launch_1d(embed_hist_kernel, grid_of(p.tiles), kSortThreads, 0, s, false, p, k);
    if (st != VSAMP_OK) return st;
    st = launch_1d(embed_scatter_kernel, grid_of(p.tiles), kSortThreads, 0, s, false, p, k);
    if (st != VSAMP_OK) return st;
  }
  const int last = (passes - 1) & 1;
  const unsigned grid = grid_of(p.sums * ceil_div(p.D, kEmbedThreads));
  st = launch_1d(embed_sum_kernel<TI, TO>, grid, kEmbedThreads, 0, s, false, p, last);
  if (st != VSAMP_OK) return st;
  return launch_1d(embed_join_kernel<TO>, grid, kEmbedThreads, 0, s, false, p, last);
}

struct EmbedPlan {
  int64_t tiles, sums;
  size_t keys, hist, part, total;
};
static EmbedPlan embed_plan(int64_t N, int64_t D) {
  EmbedPlan e;
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  e.tiles = ceil_div(N, kSortTile);
  e.sums = ceil_div(N, kEmbedTile);
  e.keys = up((size_t)N * sizeof(uint2));
  e.hist = up((size_t)e.tiles * kSortBins * 4);
  e.part = up((size_t)e.sums * 2 * (size_t)D * 4);
  e.total = 2 * e.keys + e.hist + e.part;
  return e;
}

}  // namespace vsamp

using namespace vsamp;

extern "C" {

vsamp_status vsamp_embed(const int32_t* token, int64_t N, const void* table, vsamp_dtype dt, int64_t V, int64_t D,
                         int64_t ldt, float scale, void* out, vsamp_dtype out_dt, int64_t ldo, int32_t* row_status,
                         void* stream) {
  if (!token || !table || !out || !type_ok(dt) || !type_ok(out_dt)) return VSAMP_ERR_INVALID_ARG;
  if (N <= 0 || V <= 0 || D <= 0 || ldt < D || ldo < D) return VSAMP_ERR_INVALID_ARG;
  if (!elem_aligned(table, dt) || !elem_aligned(out, out_dt)) return VSAMP_ERR_INVALID_ARG;
  if (V > 0x7FFFFFF0LL || N > 0x7FFFFFFFLL || D > 0x7FFFFFFFLL) return VSAMP_ERR_UNSUPPORTED;
  EmbedParams p{};
  p.token = token;
  p.N = N;
  p.table = static_cast<const unsigned char*>(table);
  p.V = V;
  p.D = D;
  p.ldt = ldt;
  p.scale = scale;
  p.out = static_cast<unsigned char*>(out);
  p.ldo = ldo;
  p.row_status = row_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dt == VSAMP_F32)
    return out_dt == VSAMP_F32 ? launch_embed<float, float>(p, s) : launch_embed<float, __nv_bfloat16>(p, s);
  return out_dt == VSAMP_F32 ? launch_embed<__nv_bfloat16, float>(p, s)
                             : launch_embed<__nv_bfloat16, __nv_bfloat16>(p, s);
}

size_t vsamp_embed_workspace_size(int64_t N, int64_t D) {
  if (N <= 0 || D <= 0 || N > 0x7FFFFFFFLL || D > 0x7FFFFFFFLL) return 0;
  return embed_plan(N, D).total;
}

vsamp_status vsamp_embed_backward(const int32_t* token, int64_t N, const void* dout, vsamp_dtype dt, int64_t D,
                                  int64_t ldd, float scale, int64_t V, void* dtable, vsamp_dtype table_dt,
                                  int64_t ldt, int32_t accumulate, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  if (!token || !dout || !dtable || !type_ok(dt) || !type_ok(table_dt)) return VSAMP_ERR_INVALID_ARG;
  if (N <= 0 || V <= 0 || D <= 0 || ldt < D || ldd < D) return VSAMP_ERR_INVALID_ARG;
  if (!elem_aligned(dout, dt) || !elem_aligned(dtable, table_dt)) return VSAMP_ERR_INVALID_ARG;
  if (V > 0x7FFFFFF0LL || N > 0x7FFFFFFFLL || D > 0x7FFFFFFFLL) return VSAMP_ERR_UNSUPPORTED;
  const EmbedPlan e = embed_plan(N, D);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0 || workspace_bytes < e.total)
    return VSAMP_ERR_INVALID_ARG;
  EmbedGradParams p{};
  p.token = token;
  p.N = N;
  p.dout = static_cast<const unsigned char*>(dout);
  p.D = D;
  p.ldd = ldd;
  p.V = V;
  p.scale = scale;
  p.dtable = static_cast<unsigned char*>(dtable);
  p.ldt = ldt;
  p.accumulate = accumulate != 0;
  unsigned char* w = static_cast<unsigned char*>(workspace);
  p.keys[0] = reinterpret_cast<uint2*>(w);
  p.keys[1] = reinterpret_cast<uint2*>(w + e.keys);
  p.hist = reinterpret_cast<uint32_t*>(w + 2 * e.keys);
  p.part = reinterpret_cast<float*>(w + 2 * e.keys + e.hist);
  p.tiles = e.tiles;
  p.sums = e.sums;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dt == VSAMP_F32)
    return table_dt == VSAMP_F32 ? launch_embed_grad<float, float>(p, s) : launch_embed_grad<float, __nv_bfloat16>(p, s);
  return table_dt == VSAMP_F32 ? launch_embed_grad<__nv_bfloat16, float>(p, s)
                               : launch_embed_grad<__nv_bfloat16, __nv_bfloat16>(p, s);
}

}  // extern "C"
