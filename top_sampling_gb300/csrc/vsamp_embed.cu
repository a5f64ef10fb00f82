// vsamp_embed and vsamp_embed_backward: argument checks and launches.
#include <atomic>

#include "vsamp_embed.cuh"
#include "vsamp_grid.h"
#include "vsamp_host.h"

namespace vsamp {

static bool type_ok(vsamp_dtype dt) { return dt == VSAMP_F32 || dt == VSAMP_BF16; }
static bool elem_aligned(const void* p, vsamp_dtype dt) {
  return (reinterpret_cast<uintptr_t>(p) & (dt == VSAMP_F32 ? 3u : 1u)) == 0;
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

static int bits_of(int64_t n) {   // values 0 .. n fit
  int bits = 1;
  while (bits < 62 && (n >> bits) != 0) ++bits;
  return bits;
}

// Whether every row begins on the boundary of a vector of ve elements.
static bool rows_aligned(const void* p, int64_t ld, int es, int ve) {
  return (reinterpret_cast<uintptr_t>(p) % (unsigned)(ve * es)) == 0 && ld % ve == 0;
}

template <typename TI, typename TO, int VE>
static vsamp_status launch_embed_ve(const EmbedParams& p, bool whole, cudaStream_t s) {
  const int64_t nv = ceil_div(p.D, VE);
  int tx = 1;   // threads along a row
  while (tx < kEmbedThreads && tx * kEmbedUnroll < nv) tx *= 2;
  const int64_t spans = ceil_div(nv, (int64_t)tx * kEmbedUnroll), rows = ceil_div(p.N, kEmbedThreads / tx);
  return launch_1d(whole ? embed_kernel<TI, TO, VE, true> : embed_kernel<TI, TO, VE, false>,
                   grid_of(rows * spans), kEmbedThreads, 0, s, p, tx, (int)spans);
}

template <typename TI, typename TO>
static vsamp_status launch_embed(const EmbedParams& p, cudaStream_t s) {
  constexpr int VE = sizeof(TI) == 2 && sizeof(TO) == 2 ? 8 : 4;   // 16 bytes of the wider type
  const bool whole = p.D % VE == 0 && rows_aligned(p.table, p.ldt, sizeof(TI), VE) &&
                     rows_aligned(p.out, p.ldo, sizeof(TO), VE);
  return launch_embed_ve<TI, TO, VE>(p, whole, s);
}

template <typename TO>
static ZeroParams zero_params(const EmbedGradParams& p) {
  ZeroParams z{};
  z.base = p.dtable;
  const int64_t es = sizeof(TO);
  if (p.ldt == p.D || p.V == 1) {   // one contiguous range in equal pieces
    const int64_t bytes = p.V * p.D * es;
    z.row_stride = z.row_bytes = kZeroSpan;
    z.nrows = ceil_div(bytes, kZeroSpan);
    z.last_bytes = bytes - (z.nrows - 1) * kZeroSpan;
  } else {
    z.row_stride = p.ldt * es;
    z.row_bytes = z.last_bytes = p.D * es;
    z.nrows = p.V;
  }
  return z;
}

template <typename TI, typename TO, int VE>
static vsamp_status launch_embed_sums(const EmbedGradParams& p, int last, const DeviceInfo& d, cudaStream_t s) {
  const int64_t spans = ceil_div(ceil_div(p.D, VE), kEmbedThreads);
  const vsamp_status st = launch_1d(p.aligned && p.D % VE == 0 ? embed_sum_kernel<TI, TO, VE, true>
                                                               : embed_sum_kernel<TI, TO, VE, false>,
                                    grid_of(p.sums * spans), kEmbedThreads, 0, s, p, last, (int)spans);
  if (st != VSAMP_OK) return st;
  const int64_t jspans = ceil_div(p.D, kJoinSpan);
  const int64_t most = p.sums * jspans, resident = (int64_t)d.sm_count * 8;   // the list's length is not known here
  return launch_1d(embed_join_kernel<TO>, grid_of(most < resident ? most : resident), kEmbedThreads, 0, s, p,
                   last, (int)jspans);
}

template <typename TI, typename TO, int VE>
static vsamp_status launch_embed_few(const EmbedGradParams& p, cudaStream_t s) {
  const int64_t spans = ceil_div(ceil_div(p.D, VE), kEmbedThreads);
  return launch_1d(embed_few_kernel<TI, TO, VE>, grid_of(p.N * spans), kEmbedThreads, 0, s, p, (int)spans);
}

// Whether a call takes the form of few positions (embed_few_kernel) instead of the sort. Added to the table it wins as far
// as it goes (1,024 positions: 1,001 fp32 columns 10.4 against 22.0 us, 8,192 columns 18.6 against 27.5, 64 columns 6.5
// against 16.8). Written whole it waits for the zeros, which the sort runs beside: it wins up to about 300 positions
// (256: 15.1 against 17.1 us for a table of 65 MB, 17.1 against 18.7 for 77 MB; 384: 24.0 against 17.2 and 23.7 against
// 19.2; 1,024: 25.3 against 17.9), and with small tables, whose zeros are short (2 MB, 1,024 positions: 11.5 against 14.9
// us; 26 MB, 700: 11.7 against 15.9). A table of 1.2 GB takes 192 against 190 us at 256 positions.
// The tokens are not known here: 1,024 positions of one token, added in one chain, take 84 us against 20.
constexpr int64_t kFewWhole = 256, kFewSmallTable = 32 << 20;
static bool takes_few(int64_t N, bool accumulate, int64_t table_bytes) {
  return N <= (accumulate || table_bytes <= kFewSmallTable ? (int64_t)kEmbedFew : kFewWhole);
}

template <typename TI, typename TO>
static vsamp_status launch_embed_grad(EmbedGradParams p, const DeviceInfo& d, int dev, cudaStream_t s) {
  constexpr int VE = sizeof(TI) == 2 && sizeof(TO) == 2 ? 8 : 4;
  p.aligned = rows_aligned(p.dout, p.ldd, sizeof(TI), VE) && rows_aligned(p.dtable, p.ldt, sizeof(TO), VE);
  vsamp_status st = VSAMP_OK;
  ZeroParams z{};
  if (!p.accumulate) z = zero_params<TO>(p);
  const int64_t zero_warps = z.nrows < (int64_t)d.sm_count * 64 ? z.nrows : (int64_t)d.sm_count * 64;
  if (takes_few(p.N, p.accumulate, p.V * p.D * (int64_t)sizeof(TO))) {
    if (z.nrows > 0) {
      st = launch_1d(embed_zero_kernel, grid_of(ceil_div(zero_warps, kEmbedThreads / 32)), kEmbedThreads, 0, s, z);
      if (st != VSAMP_OK) return st;
    }
    return launch_embed_few<TI, TO, VE>(p, s);
  }
  int last = 0;
  const int pos_bits = bits_of(p.N - 1), token_bits = bits_of(p.V);
  if (p.N <= kSortOne && pos_bits + token_bits <= 32) {
    static std::atomic<bool> raised[64];
    const int smem = (int)sizeof(SortOneSmem);
    if (dev >= 64 || !raised[dev].load(std::memory_order_acquire)) {
      if (cudaFuncSetAttribute(embed_sort_one_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return VSAMP_ERR_CUDA;
      }
      if (dev < 64) raised[dev].store(true, std::memory_order_release);
    }
    const int64_t zero_ctas = ceil_div(zero_warps, kSortOneThreads / 32);
    const int64_t most = 2 * (int64_t)d.sm_count - 1;   // two CTAs fit an SM
    const int passes = (int)ceil_div(token_bits, 9), digit_bits = (int)ceil_div(token_bits, passes);
    st = launch_1d(embed_sort_one_kernel, grid_of(1 + (zero_ctas < most ? zero_ctas : most)), kSortOneThreads,
                   (size_t)smem, s, p, z, pos_bits, digit_bits, passes);
    if (st != VSAMP_OK) return st;
  } else {
    if (z.nrows > 0) {
      st = launch_1d(embed_zero_kernel, grid_of(ceil_div(zero_warps, kEmbedThreads / 32)), kEmbedThreads, 0, s, z);
      if (st != VSAMP_OK) return st;
    }
    // the marker's low bits are larger than any token's: V itself fits token_bits
    const int passes = (int)ceil_div(token_bits, kSortBits);
    for (int k = 0; k < passes; ++k) {
      st = launch_1d(embed_hist_kernel, grid_of(p.tiles), kSortThreads, 0, s, p, k);
      if (st != VSAMP_OK) return st;
      st = launch_1d(embed_scatter_kernel, grid_of(p.tiles), kSortThreads, 0, s, p, k);
      if (st != VSAMP_OK) return st;
    }
    last = (passes - 1) & 1;
  }
  return launch_embed_sums<TI, TO, VE>(p, last, d, s);
}

struct EmbedPlan {
  int64_t tiles, sums, ldp;
  size_t keys, hist, part, runs, total;
};
static EmbedPlan embed_plan(int64_t N, int64_t D) {
  EmbedPlan e;
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  e.tiles = ceil_div(N, kSortTile);
  e.sums = ceil_div(N, kEmbedTile);
  e.ldp = ceil_div(D, 8) * 8;
  e.keys = up((size_t)N * sizeof(uint2));
  e.hist = up((size_t)e.tiles * kSortBins * 4);
  e.part = up((size_t)e.sums * 2 * (size_t)e.ldp * 4);
  e.runs = up((size_t)e.sums * 4) + 256;
  e.total = 2 * e.keys + e.hist + e.part + e.runs;
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
  if (V > 0x7FFFFFF0LL || N > 0x7FFFFFFFLL || D > 0x3FFFFFFFLL) return VSAMP_ERR_UNSUPPORTED;
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
  if (N <= 0 || D <= 0 || N > 0x7FFFFFFFLL || D > 0x3FFFFFFFLL) return 0;
  return N <= kFewWhole ? 16 : embed_plan(N, D).total;   // few positions need none
}

vsamp_status vsamp_embed_backward(const int32_t* token, int64_t N, const void* dout, vsamp_dtype dt, int64_t D,
                                  int64_t ldd, float scale, int64_t V, void* dtable, vsamp_dtype table_dt,
                                  int64_t ldt, int32_t accumulate, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  if (!token || !dout || !dtable || !type_ok(dt) || !type_ok(table_dt)) return VSAMP_ERR_INVALID_ARG;
  if (N <= 0 || V <= 0 || D <= 0 || ldt < D || ldd < D) return VSAMP_ERR_INVALID_ARG;
  if (!elem_aligned(dout, dt) || !elem_aligned(dtable, table_dt)) return VSAMP_ERR_INVALID_ARG;
  if (V > 0x7FFFFFF0LL || N > 0x7FFFFFFFLL || D > 0x3FFFFFFFLL) return VSAMP_ERR_UNSUPPORTED;
  const EmbedPlan e = embed_plan(N, D);
  const size_t need = takes_few(N, accumulate != 0, V * D * (table_dt == VSAMP_F32 ? 4 : 2)) ? 16 : e.total;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0 || workspace_bytes < need)
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
  p.runs = reinterpret_cast<uint32_t*>(w + 2 * e.keys + e.hist + e.part);
  p.n_runs = p.runs + (e.runs - 256) / 4;
  p.tiles = e.tiles;
  p.sums = e.sums;
  p.ldp = e.ldp;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return VSAMP_ERR_CUDA;
  }
  DeviceInfo d;
  const vsamp_status st = device_info(dev, d);
  if (st != VSAMP_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dt == VSAMP_F32)
    return table_dt == VSAMP_F32 ? launch_embed_grad<float, float>(p, d, dev, s)
                                 : launch_embed_grad<float, __nv_bfloat16>(p, d, dev, s);
  return table_dt == VSAMP_F32 ? launch_embed_grad<__nv_bfloat16, float>(p, d, dev, s)
                               : launch_embed_grad<__nv_bfloat16, __nv_bfloat16>(p, d, dev, s);
}

}  // extern "C"
