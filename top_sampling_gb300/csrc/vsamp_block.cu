// vsamp_block_quantize and vsamp_block_matmul: argument checks and launches.
#include <atomic>
#include <climits>

#include "vsamp_block_matmul.cuh"
#include "vsamp_block_quant.cuh"
#include "vsamp_grid.h"
#include "vsamp_host.h"

namespace vsamp {

static bool at_multiple(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
static int64_t ceil_blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }
static bool kind_ok(vsamp_block_kind k) { return k == VSAMP_BLOCK_ROW || k == VSAMP_BLOCK_TILE; }

// Whether (codes, ld, scales, lds) can hold a matrix of rows x cols in blocks of `kind`.
static bool matrix_ok(const void* codes, int64_t ld, const float* scales, int64_t lds, vsamp_block_kind kind, int64_t rows,
                      int64_t cols) {
  if (!codes || !scales || !at_multiple(codes, 16) || ld < cols || ld % 16 != 0) return false;
  if (kind == VSAMP_BLOCK_TILE) return at_multiple(scales, 4) && lds >= ceil_blocks(cols);
  return at_multiple(scales, 16) && lds >= rows && lds % 4 == 0;
}

// Rows of `width` bytes, `stride` apart.
struct Region {
  __int128 at, stride, width, rows;
  Region(const void* p, int64_t n, int64_t ld, int64_t cols, int elem)
      : at(reinterpret_cast<uintptr_t>(p)), stride((__int128)ld * elem), width(p ? (__int128)cols * elem : 0), rows(n) {}
  __int128 end() const { return at + (rows - 1) * stride + width; }
};
static Region codes_region(const void* p, int64_t ld, int64_t rows, int64_t cols) { return Region(p, rows, ld, cols, 1); }
static Region scales_region(const void* p, int64_t ld, vsamp_block_kind kind, int64_t rows, int64_t cols) {
  if (kind == VSAMP_BLOCK_TILE) return Region(p, ceil_blocks(rows), ld, ceil_blocks(cols), 4);
  return Region(p, ceil_blocks(cols), ld, rows, 4);
}
// Whether two regions have memory in common. Ranges of columns of one array, whose rows are equally far apart, do not; other
// regions are taken from their first byte to their last.
static bool share(const Region& a, const Region& b) {
  if (!a.width || !b.width || a.end() <= b.at || b.end() <= a.at) return false;
  const __int128 stride = a.rows > 1 ? a.stride : b.stride;   // that of a single row says nothing
  if (stride <= 0 || (a.rows > 1 && b.rows > 1 && a.stride != b.stride)) return true;
  const __int128 off = ((b.at - a.at) % stride + stride) % stride;   // of b's rows behind those of a
  return off < a.width || off + b.width > stride;
}

template <typename T, bool TILE>
static vsamp_status launch_quant(const BlockQuantParams& p, cudaStream_t s) {
  const unsigned grid = grid_of(p.tiles);
  if (p.codes && p.codes_t) return launch_1d(block_quant_kernel<T, TILE, true, true>, grid, kQuantThreads, 0, s, p);
  if (p.codes) return launch_1d(block_quant_kernel<T, TILE, true, false>, grid, kQuantThreads, 0, s, p);
  return launch_1d(block_quant_kernel<T, TILE, false, true>, grid, kQuantThreads, 0, s, p);
}

// cuTensorMapEncodeTiled of the installed driver, or null.
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiled encode_tiled() {
  static std::atomic<void*> found{nullptr};
  void* fn = found.load(std::memory_order_acquire);
  if (!fn) {
    cudaDriverEntryPointQueryResult how;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &how) != cudaSuccess ||
        how != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    found.store(fn, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(fn);
}

// A map of a code matrix for copies of box_rows rows of one block.
static bool codes_map(CUtensorMap& map, const uint8_t* codes, int64_t ld, int64_t rows, int64_t cols, int box_rows) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t size[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {(cuuint32_t)kBlock, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), size, stride, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map of the scales of 1 x 128 blocks, [blocks, rows], for copies of box_rows rows' scales of one block.
static bool scales_map(CUtensorMap& map, const float* scales, int64_t ld, int64_t rows, int64_t cols, int box_rows) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t size[2] = {(cuuint64_t)rows, (cuuint64_t)ceil_blocks(cols)}, stride[1] = {(cuuint64_t)ld * 4};
  const cuuint32_t box[2] = {(cuuint32_t)box_rows, 1}, step[2] = {1, 1};
  return encode(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(scales), size, stride, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map of [planes, rows, cols] results for boxes of 32 rows of 128 bytes.
static bool results_map(CUtensorMap& map, void* out, bool f32, int64_t ld, int64_t rows, int64_t cols, int planes) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t es = f32 ? 4 : 2;
  const cuuint64_t size[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t stride[2] = {(cuuint64_t)ld * es, (cuuint64_t)(rows * ld) * es};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / es), 32, 1}, step[3] = {1, 1, 1};
  return encode(&map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, out, size, stride, box,
                step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int64_t kMmSms = 152;   // the division of the inner dimension goes by sizes alone

// Whether the numbers of rows, columns, blocks and tiles keep within the kernel's 32-bit arithmetic.
static bool mm_fits(int64_t M, int64_t N, int64_t K) {
  return M <= 0x7FFFFE00LL && N <= 0x7FFFFE00LL && K <= 0x7FFFFE00LL && (double)M * N < 3e13;
}

// Whether pairs of CTAs take tiles of 256 rows: they need less of the L2 (2048 x 16384 x 4096: 103 us, single CTAs 111;
// 256 x 151936 x 4096: 136 and 147; 512 x 2048 x 32000: 37 and 40), and lose a little where there are few tiles (400 x 4096 x
// 4096: 17.3 and 16.6; 129 x 20000 x 2048: 19.2 and 18.8). A tile of 128 rows has nothing to pair.
static bool mm_pair(int64_t M) { return M > kMmRows; }

// How the tiles are divided. Whole rounds of tiles over the CTAs (or pairs) go as they are; the tiles that are left over, or
// all if there are fewer than CTAs, may be cut into parts of the inner dimension. Time goes by the blocks that the longest
// CTA walks over, and about six blocks' worth for each tile's start and end; parts are written and read again. Divided and
// whole (M x K x N, us): 64 x 151936 x 4096 108 (9 parts) and 574; 512 x 32000 x 2048 38 (4) and 102; 16 x 32000 x 2048 15 (16)
// and 97; 300 x 100000 x 300 30 (16) and 304. 1000 x 4000 x 4000 stays whole: 19, and 28 with two parts. Of 2048 x 151936 x
// 4096 only the rest of 52 tiles is divided: 866, and 914 whole, in bursts of ten; in long runs, at the power limit, 1,010 and
// 1,000, the same within what the clock varies.
struct MmPlan {
  int64_t tiles, whole;   // whole: tiles that are not divided
  int parts, part_rows;
  size_t bytes() const { return whole < tiles ? (size_t)((tiles - whole) * parts) * (size_t)part_rows * kMmCols * 4 : 0; }
};
static MmPlan mm_plan(int64_t M, int64_t N, int64_t K) {
  const int64_t g = mm_pair(M) ? 2 : 1, rows = kMmRows * g, at_once = kMmSms / g, blocks = ceil_blocks(K);
  MmPlan p;
  p.tiles = ((M + rows - 1) / rows) * ((N + kMmCols - 1) / kMmCols);
  p.whole = p.tiles;
  p.parts = 1;
  p.part_rows = (int)(M < rows ? M : rows);
  const int64_t rest = p.tiles % at_once;
  const double rounds = (double)((p.tiles - rest) / at_once) * (double)(blocks + 6);
  double least = rounds + (rest ? (double)(blocks + 6) : 0.0);
  for (int s = 2; rest && s <= 64 && blocks / s >= 4; ++s) {
    const double t = rounds + (double)((rest * s + at_once - 1) / at_once) * ((double)((blocks + s - 1) / s) + 6) + 8 +
                     (double)rest * p.part_rows * kMmCols * s * 8 / 1.5e6;
    if (t < least * 0.95) {
      p.whole = p.tiles - rest;
      p.parts = s;
      least = t;
    }
  }
  return p;
}

struct MatmulMaps {
  CUtensorMap a, b, o, sa, sb, p;
};

template <typename TO, bool TILE, int G, bool ADD16>
static vsamp_status launch_matmul_g(const BlockMatmulParams& p, const MatmulMaps& m, const DeviceInfo& d, int dev,
                                    cudaStream_t s) {
  auto kern = block_matmul_kernel<TO, TILE, G, ADD16>;
  constexpr int smem = MmShape<G>::Smem;
  static std::atomic<bool> raised[64];
  if (dev >= 64 || !raised[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
      cudaGetLastError();
      return VSAMP_ERR_CUDA;
    }
    if (dev < 64) raised[dev].store(true, std::memory_order_release);
  }
  const int64_t most = d.sm_count / G;
  const unsigned grid = (unsigned)(p.items < most ? p.items : most) * G;
  if (G == 1) return launch_1d(kern, grid, kMmThreads, smem, s, p, m.a, m.b, m.o, m.sa, m.sb, m.p);
  return launch_clusters(kern, grid, G, kMmThreads, smem, s, p, m.a, m.b, m.o, m.sa, m.sb, m.p);
}

template <typename TO, bool TILE, bool ADD16 = false>
static vsamp_status launch_matmul(const BlockMatmulParams& p, const MatmulMaps& m, bool pair, const DeviceInfo& d, int dev,
                                  cudaStream_t s) {
  const vsamp_status st = pair ? launch_matmul_g<TO, TILE, 2, ADD16>(p, m, d, dev, s)
                               : launch_matmul_g<TO, TILE, 1, ADD16>(p, m, d, dev, s);
  if (st != VSAMP_OK || p.whole == p.items) return st;
  const int64_t tiles = (p.items - p.whole) / p.parts;
  const int64_t ctas = (tiles * p.part_rows * (kMmCols / 4) + 255) / 256, most = (int64_t)d.sm_count * 8;
  return launch_1d(block_matmul_join_kernel<TO>, grid_of(ctas < most ? ctas : most), 256, 0, s, p, pair ? 2 * kMmRows : kMmRows);
}

}  // namespace vsamp

using namespace vsamp;

extern "C" {

vsamp_status vsamp_block_quantize(const void* x, vsamp_dtype dt, int64_t R, int64_t C, int64_t ldx,
                                  vsamp_block_kind kind, uint8_t* codes, int64_t ldc, float* scales, int64_t lds,
                                  uint8_t* codes_t, int64_t ldt, float* scales_t, int64_t ldst, void* stream) {
  if (!x || (dt != VSAMP_F32 && dt != VSAMP_BF16) || !kind_ok(kind)) return VSAMP_ERR_INVALID_ARG;
  if (R <= 0 || C <= 0 || ldx < C || !at_multiple(x, dt == VSAMP_F32 ? 4 : 2)) return VSAMP_ERR_INVALID_ARG;
  if (!codes != !scales || !codes_t != !scales_t || (!codes && !codes_t)) return VSAMP_ERR_INVALID_ARG;
  if (codes && !matrix_ok(codes, ldc, scales, lds, kind, R, C)) return VSAMP_ERR_INVALID_ARG;
  if (codes_t && !matrix_ok(codes_t, ldt, scales_t, ldst, kind, C, R)) return VSAMP_ERR_INVALID_ARG;
  if (R > 0x7FFFFF00LL || C > 0x7FFFFF00LL) return VSAMP_ERR_UNSUPPORTED;
  const Region all[5] = {Region(x, R, ldx, C, dt == VSAMP_F32 ? 4 : 2), codes_region(codes, ldc, R, C),
                         scales_region(scales, lds, kind, R, C), codes_region(codes_t, ldt, C, R),
                         scales_region(scales_t, ldst, kind, C, R)};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (share(all[i], all[j])) return VSAMP_ERR_INVALID_ARG;
  BlockQuantParams p{};
  p.x = static_cast<const unsigned char*>(x);
  p.R = R;
  p.C = C;
  p.ldx = ldx;
  p.codes = codes;
  p.ldc = ldc;
  p.scales = scales;
  p.lds = lds;
  p.codes_t = codes_t;
  p.ldt = ldt;
  p.scales_t = scales_t;
  p.ldst = ldst;
  p.col_tiles = ceil_blocks(C);
  p.tiles = ceil_blocks(R) * p.col_tiles;
  p.aligned = at_multiple(x, 16) && ldx * (dt == VSAMP_F32 ? 4 : 2) % 16 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dt == VSAMP_F32)
    return kind == VSAMP_BLOCK_TILE ? launch_quant<float, true>(p, s) : launch_quant<float, false>(p, s);
  return kind == VSAMP_BLOCK_TILE ? launch_quant<__nv_bfloat16, true>(p, s) : launch_quant<__nv_bfloat16, false>(p, s);
}

size_t vsamp_block_matmul_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || !mm_fits(M, N, K)) return 0;
  return mm_plan(M, N, K).bytes();
}

vsamp_status vsamp_block_matmul(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, const uint8_t* b,
                                int64_t ldb, const float* sb, int64_t ldsb, vsamp_block_kind b_kind, int64_t M,
                                int64_t N, int64_t K, void* out, vsamp_dtype out_dt, int64_t ldo, int32_t accumulate,
                                void* workspace, size_t workspace_bytes, void* stream) {
  if (!kind_ok(b_kind) || (out_dt != VSAMP_F32 && out_dt != VSAMP_BF16) || !out) return VSAMP_ERR_INVALID_ARG;
  if (M <= 0 || N <= 0 || K <= 0 || ldo < N || !at_multiple(out, out_dt == VSAMP_F32 ? 4 : 2)) return VSAMP_ERR_INVALID_ARG;
  if (!matrix_ok(a, lda, sa, ldsa, VSAMP_BLOCK_ROW, M, K) || !matrix_ok(b, ldb, sb, ldsb, b_kind, N, K))
    return VSAMP_ERR_INVALID_ARG;
  if (!mm_fits(M, N, K)) return VSAMP_ERR_UNSUPPORTED;
  const MmPlan plan = mm_plan(M, N, K);
  const size_t need = plan.bytes();
  if (need && (!workspace || !at_multiple(workspace, 16) || workspace_bytes < need)) return VSAMP_ERR_INVALID_ARG;
  // what is written shares no memory with what is read
  const Region read[4] = {codes_region(a, lda, M, K), scales_region(sa, ldsa, VSAMP_BLOCK_ROW, M, K), codes_region(b, ldb, N, K),
                          scales_region(sb, ldsb, b_kind, N, K)};
  const Region result(out, M, ldo, N, out_dt == VSAMP_F32 ? 4 : 2), room(need ? workspace : nullptr, 1, 0, (int64_t)need, 1);
  for (const Region& r : read)
    if (share(r, result) || share(r, room)) return VSAMP_ERR_INVALID_ARG;
  if (share(result, room)) return VSAMP_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return VSAMP_ERR_CUDA;
  }
  DeviceInfo d;
  const vsamp_status st = device_info(dev, d);
  if (st != VSAMP_OK) return st;
  if (d.optin < MmShape<1>::Smem || d.optin < MmShape<2>::Smem) return VSAMP_ERR_UNSUPPORTED;
  const bool pair = mm_pair(M);
  const int64_t tile_rows = pair ? 2 * kMmRows : kMmRows;
  BlockMatmulParams p{};
  p.sb = sb;
  p.ldsb = ldsb;
  p.M = (int)M;
  p.N = (int)N;
  p.ldo = ldo;
  p.out = static_cast<unsigned char*>(out);
  p.blocks = (int)ceil_blocks(K);
  // The matrix with fewer rows stays in the L2 while the other one is walked through once. With more rows of a, along rows of
  // results and down columns: 32003 x 2050 x 1501 167 and 175 us, 151936 x 2048 x 2048 772 and 799; with more rows of b,
  // 2048 x 151936 x 4096, 1,028 and 876.
  p.across = M > N;
  p.inner_tiles = (int)(p.across ? (N + kMmCols - 1) / kMmCols : (M + tile_rows - 1) / tile_rows);
  p.parts = plan.parts;
  p.whole = (int)plan.whole;
  p.items = (int)(plan.whole + (plan.tiles - plan.whole) * plan.parts);
  p.part = static_cast<float*>(workspace);
  p.part_rows = plan.part_rows;
  p.a_rows = (int)(M < kMmRows ? M : kMmRows);
  p.accumulate = accumulate != 0;
  const int es = out_dt == VSAMP_F32 ? 4 : 2;
  // bf16 sums are added and rounded once, by the warps themselves; a stride of a tensor map has 40 bits
  if (at_multiple(out, 16) && ldo * es % 16 == 0 && !(p.accumulate && es == 2) && (double)M * ldo * es < 1e12)
    p.boxes = N * es % 16 == 0 ? 2 : 1;
  p.pairs = at_multiple(out, 2 * es) && ldo % 2 == 0;
  const long long wc = env_ll("VSAMP_WAIT_CYCLES", 0);
  p.wait_cycles = wc > 0 ? wc : 4000000000LL;   // ~2 s at the maximum SM clock
  p.drop_loads = env_int("VSAMP_TEST_DROP_LOADS", 0) != 0 ? 1 : 0;
  const int stop0 = env_int("VSAMP_TEST_STOP_LOADS_0", 0), stop1 = env_int("VSAMP_TEST_STOP_LOADS_1", 0);
  p.stop0 = stop0 > 0 ? stop0 : INT_MAX;
  p.stop1 = stop1 > 0 ? stop1 : INT_MAX;
  const bool tile = b_kind == VSAMP_BLOCK_TILE;
  MatmulMaps m{};
  if (!codes_map(m.a, a, lda, M, K, p.a_rows) || !codes_map(m.b, b, ldb, N, K, pair ? kMmCols / 2 : kMmCols) ||
      !scales_map(m.sa, sa, ldsa, M, K, kMmRows) || (!tile && !scales_map(m.sb, sb, ldsb, N, K, kMmCols)))
    return VSAMP_ERR_CUDA;
  if (p.boxes && !results_map(m.o, out, es == 4, ldo, M, N, 1)) return VSAMP_ERR_CUDA;
  if (need && !results_map(m.p, p.part, true, kMmCols, p.part_rows, kMmCols, p.items - p.whole)) return VSAMP_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (out_dt == VSAMP_F32)
    return tile ? launch_matmul<float, true>(p, m, pair, d, dev, s) : launch_matmul<float, false>(p, m, pair, d, dev, s);
  using B = __nv_bfloat16;
  if (accumulate)
    return tile ? launch_matmul<B, true, true>(p, m, pair, d, dev, s) : launch_matmul<B, false, true>(p, m, pair, d, dev, s);
  return tile ? launch_matmul<B, true>(p, m, pair, d, dev, s) : launch_matmul<B, false>(p, m, pair, d, dev, s);
}

}  // extern "C"
