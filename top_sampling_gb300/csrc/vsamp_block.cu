// vsamp_block_quantize and vsamp_block_matmul: argument checks and launches.
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

template <typename T, bool TILE>
static vsamp_status launch_quant(const BlockQuantParams& p, cudaStream_t s) {
  const unsigned grid = grid_of(p.tiles);
  if (p.codes && p.codes_t) return launch_1d(block_quant_kernel<T, TILE, true, true>, grid, kQuantThreads, 0, s, p);
  if (p.codes) return launch_1d(block_quant_kernel<T, TILE, true, false>, grid, kQuantThreads, 0, s, p);
  return launch_1d(block_quant_kernel<T, TILE, false, true>, grid, kQuantThreads, 0, s, p);
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
  (void)M;
  (void)N;
  (void)K;
  return 0;
}

vsamp_status vsamp_block_matmul(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, const uint8_t* b,
                                int64_t ldb, const float* sb, int64_t ldsb, vsamp_block_kind b_kind, int64_t M,
                                int64_t N, int64_t K, void* out, vsamp_dtype out_dt, int64_t ldo, int32_t accumulate,
                                void* workspace, size_t workspace_bytes, void* stream) {
  if (!kind_ok(b_kind) || (out_dt != VSAMP_F32 && out_dt != VSAMP_BF16) || !out) return VSAMP_ERR_INVALID_ARG;
  if (M <= 0 || N <= 0 || K <= 0 || ldo < N || !at_multiple(out, out_dt == VSAMP_F32 ? 4 : 2)) return VSAMP_ERR_INVALID_ARG;
  if (!matrix_ok(a, lda, sa, ldsa, VSAMP_BLOCK_ROW, M, K) || !matrix_ok(b, ldb, sb, ldsb, b_kind, N, K))
    return VSAMP_ERR_INVALID_ARG;
  const size_t need = vsamp_block_matmul_workspace_size(M, N, K);
  if (need && (!workspace || !at_multiple(workspace, 16) || workspace_bytes < need)) return VSAMP_ERR_INVALID_ARG;
  if (M > 0x7FFFFF00LL || N > 0x7FFFFF00LL || K > 0x7FFFFF00LL) return VSAMP_ERR_UNSUPPORTED;
  BlockMatmulParams p{};
  p.a = a;
  p.b = b;
  p.sa = sa;
  p.sb = sb;
  p.lda = lda;
  p.ldsa = ldsa;
  p.ldb = ldb;
  p.ldsb = ldsb;
  p.M = M;
  p.N = N;
  p.K = K;
  p.ldo = ldo;
  p.out = static_cast<unsigned char*>(out);
  p.accumulate = accumulate != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = grid_of(((M + 63) / 64) * ((N + 63) / 64));
  if (out_dt == VSAMP_F32)
    return launch_1d(b_kind == VSAMP_BLOCK_TILE ? block_matmul_kernel<float, true> : block_matmul_kernel<float, false>, grid,
                     256, 0, s, p);
  return launch_1d(b_kind == VSAMP_BLOCK_TILE ? block_matmul_kernel<__nv_bfloat16, true>
                                              : block_matmul_kernel<__nv_bfloat16, false>, grid, 256, 0, s, p);
}

}  // extern "C"
