// vsamp_score_tokens and vsamp_score_tokens_backward: argument checks and launches.
#include "vsamp_grid.h"
#include "vsamp_host.h"
#include "vsamp_score.cuh"

namespace vsamp {

static int64_t score_pieces(vsamp_dtype dt, int64_t V) {
  const int64_t pe = kScorePiece / (dt == VSAMP_F32 ? 4 : 2);
  return (V + pe - 1) / pe;
}

template <typename T>
static vsamp_status launch_score(const ScoreParams& p, const DeviceInfo& d, cudaStream_t s) {
  // One launch where a cluster's warps take a piece each and the pieces fill the device once at most: it saves a launch
  // (64 rows of 32000 fp32 with 20 alternatives: 7.4 against 8.2 us, and less host time); beyond, the finish of a row
  // holds up its cluster's place (256 rows: 15.9 against 12.4 us; 256 of 151936 bf16, two pieces a warp: 30 against 26).
  if (p.np <= 8 * kScoreWarps && p.B * p.np <= 16 * (int64_t)d.sm_count) {
    const int C = (p.np + kScoreWarps - 1) / kScoreWarps;
    return launch_clusters(p.N > 0 ? score_row_kernel<T, true> : score_row_kernel<T, false>, (unsigned)(p.B * C),
                           (unsigned)C, kScoreWarps * 32, (size_t)p.np * (p.N > 0 ? 48 : 16), s, p);
  }
  const unsigned grid = grid_of((p.B * p.np + kScoreWarps - 1) / kScoreWarps);
  const vsamp_status st =
      launch_1d(p.N > 0 ? score_piece_kernel<T, true> : score_piece_kernel<T, false>, grid, kScoreWarps * 32, 0, s,
                p);
  if (st != VSAMP_OK) return st;
  if (p.N > 0) return launch_1d(score_finish_alt_kernel<T>, grid_of(p.B), kScoreFinishThreads, 0, s, p);
  return launch_1d(score_finish_kernel<T>, grid_of((p.B + 3) / 4), 128, 0, s, p);
}

template <typename T>
static vsamp_status launch_score_grad(ScoreGradParams p, cudaStream_t s) {
  constexpr int64_t SPAN = (int64_t)kGradThreads * kGradVecs * ScoreType<T>::VE;
  p.spans = (p.V + SPAN - 1) / SPAN;   // covers the whole vectors wherever they begin
  return launch_1d(score_grad_kernel<T>, grid_of(p.B * p.spans), kGradThreads, 0, s, p);
}

static vsamp_status score_check(const void* logits, vsamp_dtype dt, int64_t B, int64_t V, int64_t ld) {
  if (!logits) return VSAMP_ERR_INVALID_ARG;
  if (dt != VSAMP_F32 && dt != VSAMP_BF16) return VSAMP_ERR_INVALID_ARG;
  if (B <= 0 || V <= 0 || ld < V) return VSAMP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) & (dt == VSAMP_F32 ? 3u : 1u)) != 0) return VSAMP_ERR_INVALID_ARG;
  if (V > 0x7FFFFFF0LL || B > 0x7FFFFFFFLL) return VSAMP_ERR_UNSUPPORTED;
  return VSAMP_OK;
}

}  // namespace vsamp

using namespace vsamp;

extern "C" {

size_t vsamp_score_workspace_size(vsamp_dtype dt, int64_t B, int64_t V, int32_t N) {
  if ((dt != VSAMP_F32 && dt != VSAMP_BF16) || B <= 0 || V <= 0 || V > 0x7FFFFFF0LL || B > 0x7FFFFFFFLL || N < 0 ||
      N > VSAMP_SCORE_ALT_MAX)
    return 0;
  const size_t pieces = (size_t)B * (size_t)score_pieces(dt, V);
  return pieces * (N > 0 ? 48 : 16);
}

vsamp_status vsamp_score_tokens(const void* logits, vsamp_dtype dt, int64_t B, int64_t V, int64_t ld,
                                const float* temperature, const int32_t* token, int32_t N, float* logprob,
                                float* entropy, int32_t* rank, int32_t* alt_idx, float* alt_lp, float* row_max,
                                float* row_logsum, int32_t* row_status, void* workspace, size_t workspace_bytes,
                                void* stream) {
  vsamp_status st = score_check(logits, dt, B, V, ld);
  if (st != VSAMP_OK) return st;
  if (!token || N < 0 || N > VSAMP_SCORE_ALT_MAX) return VSAMP_ERR_INVALID_ARG;
  if (N > 0 && (!alt_idx || !alt_lp)) return VSAMP_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0 ||
      workspace_bytes < vsamp_score_workspace_size(dt, B, V, N))
    return VSAMP_ERR_INVALID_ARG;
  ScoreParams p{};
  p.x = static_cast<const unsigned char*>(logits);
  p.B = B;
  p.V = V;
  p.ld = ld;
  p.temperature = temperature;
  p.token = token;
  p.N = N;
  const int64_t es = dt == VSAMP_F32 ? 4 : 2;
  p.vec = (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 && (B == 1 || (ld * es) % 16 == 0);
  const int64_t np = score_pieces(dt, V);
  if (np * B > 0x7FFFFFFFLL) return VSAMP_ERR_UNSUPPORTED;
  p.np = (int)np;
  // id / np for id < 2^31: with l = ceil(log2 np), ceil(2^(31 + l) / np) is exact to 31 bits
  int l = 0;
  while ((1LL << l) < np) ++l;
  p.np_mul = (uint32_t)(((1ULL << (31 + l)) + (uint64_t)np - 1) / (uint64_t)np);
  p.np_shift = l - 1;
  // the aligned vectors around the first or the last whole piece may reach out of the logits: these take loads of elements
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(logits), xl = x0 + (uintptr_t)((B - 1) * ld * es);
  const uintptr_t x1 = xl + (uintptr_t)(V * es);
  const int64_t whole = V * es / kScorePiece;
  p.inner0 = vectors_inside(x0, kScorePiece, x0, x1) ? 0u : 1u;
  p.inner1 = (uint32_t)(B * np);
  if (whole > 0 && !vectors_inside(xl + (uintptr_t)((whole - 1) * kScorePiece), kScorePiece, x0, x1))
    p.inner1 = (uint32_t)((B - 1) * np + whole - 1);
  p.rec = static_cast<float4*>(workspace);
  p.chunk_max = N > 0 ? reinterpret_cast<float*>(p.rec + B * np) : nullptr;
  p.logprob = logprob;
  p.entropy = entropy;
  p.rank = rank;
  p.alt_idx = alt_idx;
  p.alt_lp = alt_lp;
  p.row_max = row_max;
  p.row_logsum = row_logsum;
  p.row_status = row_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return VSAMP_ERR_CUDA;
  }
  DeviceInfo d;
  st = device_info(dev, d);
  if (st != VSAMP_OK) return st;
  return dt == VSAMP_F32 ? launch_score<float>(p, d, s) : launch_score<__nv_bfloat16>(p, d, s);
}

vsamp_status vsamp_score_tokens_backward(const void* logits, vsamp_dtype dt, int64_t B, int64_t V, int64_t ld,
                                         const float* temperature, const int32_t* token, const float* dlogprob,
                                         const float* dentropy, const float* row_max, const float* row_logsum,
                                         const float* entropy, void* dlogits, int64_t ldd, int32_t* row_status,
                                         void* stream) {
  vsamp_status st = score_check(logits, dt, B, V, ld);
  if (st != VSAMP_OK) return st;
  if (!token || !row_max || !row_logsum || (!dlogprob && !dentropy) || (dentropy && !entropy))
    return VSAMP_ERR_INVALID_ARG;
  st = score_check(dlogits, dt, B, V, ldd);
  if (st != VSAMP_OK) return st;
  ScoreGradParams p{};
  p.x = static_cast<const unsigned char*>(logits);
  p.B = B;
  p.V = V;
  p.ld = ld;
  p.ldo = ldd;
  p.temperature = temperature;
  p.token = token;
  p.dlogprob = dlogprob;
  p.dentropy = dentropy;
  p.row_max = row_max;
  p.row_logsum = row_logsum;
  p.entropy = entropy;
  p.dx = static_cast<unsigned char*>(dlogits);
  p.row_status = row_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dt == VSAMP_F32 ? launch_score_grad<float>(p, s) : launch_score_grad<__nv_bfloat16>(p, s);
}

}  // extern "C"
