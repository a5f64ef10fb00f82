// The AdamW step of many tensors in one launch.
//
//   g = grad * scale, m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2
//   p = p - lr (wd p + (m / (1 - b1^t)) / (sqrt(v) / sqrt(1 - b2^t) + eps))
//
// A stream over memory: each element is read and written once. A warp takes 128 consecutive elements of a tensor, four
// per lane, which is also a block of the 8-bit states: their new scale is one maximum over the warp's registers, and one
// Philox call gives a lane's four elements their random bits. The next blocks are on their way while a warp computes. The
// tensors' addresses travel in the kernel's parameters (up to 384 per launch), so a step needs no table in device memory
// and can be captured as it is.
//
// Measured: 32-bit states 95 % of the copy rate (65.5M elements: fp32 283 us, bf16 with masters 281); 8-bit states 71 % (311M
// fp32 parameters with bf16 gradients 925 us of 657): 85 instructions per element issue in 72 % of the slots, 16 warps per SM
// wait for each other's results; bf16 parameters without masters draw a second set of words (65.5M: 249 us, of 32 bits 230).
// More warps with fewer blocks each, copies through shared memory and paired arithmetic were measured and are slower. 150 tensors
// of 13,700 elements: 10 us.
#pragma once

#include "vsamp_block_quant.cuh"

namespace vsamp {

constexpr int kAdamThreads = 256;
constexpr int kAdamTensors = 384;    // of 80 bytes: 30,720 of a launch's 32,764 parameter bytes
// Blocks of 128 elements that a warp fetches at a time, and CTAs per SM. 67M parameters: 8-bit states (fp32 parameters, bf16
// gradients) 4 blocks and 2 CTAs 203 us, 2 and 3 221, 2 and 2 243, 1 and 4 258; 32-bit ones move with none of it (2 and 2
// 289 us, 4 and 2 303, their floor is 281).
template <bool BITS8>
struct AdamShape {
  static constexpr int Unroll = BITS8 ? 4 : 2, PerSm = 2;
};

struct AdamTensor {
  unsigned char* param;
  float* master;
  const unsigned char* grad;
  unsigned char* m;
  unsigned char* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  uint32_t first_chunk;   // chunks of the tensors before it
  uint32_t index;
  uint32_t aligned;       // every array begins on the boundary of a lane's vector
  uint32_t pad;
};

struct AdamParams {
  AdamTensor t[kAdamTensors];
  uint32_t count, chunks, chunk_blocks;   // a CTA takes a chunk of blocks of a tensor at a time
  float lr, b1, b2, one_b1, one_b2, eps, wd;
  float ln_b1, ln_b2, c1, c2;      // logarithms of the betas; 1 / (1 - b1^t), 1 / sqrt(1 - b2^t) of the host's step
  uint32_t step, k0[10], k1[10];   // Philox round keys
  const float* lr_dev;
  const int64_t* step_dev;
  const float* grad_scale;
};
static_assert(sizeof(AdamTensor) == 80 && sizeof(AdamParams) <= 32764, "kernel parameters");

// Philox4x32-10 with the round keys in the kernel's parameters: operands of the exclusive ors, no registers.
__device__ __forceinline__ uint4 adam_words(const AdamParams& p, uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3) {
  uint4 c = make_uint4(c0, c1, c2, c3);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    unsigned long long p0, p1;
    asm("mul.wide.u32 %0, %1, %2;" : "=l"(p0) : "r"(c.x), "r"(0xD2511F53u));
    asm("mul.wide.u32 %0, %1, %2;" : "=l"(p1) : "r"(c.z), "r"(0xCD9E8D57u));
    c = make_uint4((uint32_t)(p1 >> 32) ^ c.y ^ p.k0[r], (uint32_t)p1, (uint32_t)(p0 >> 32) ^ c.w ^ p.k1[r], (uint32_t)p0);
  }
  return c;
}

// A magnitude in units of the scale to one of the two e4m3 values next to it, up with the probability of its place
// between them: u is 16 random bits, times 16, and 8. e4m3 keeps three fraction bits, so 20 bits of an fp32 magnitude are
// dropped: the random bits are added below the kept ones and carry into them. Below 2^-6 the values are 2^-9 apart: those
// of [2^-6, 2^-5), minus 2^-6.
__device__ __forceinline__ float e4m3_stochastic(float y, uint32_t u) {
  const float base = y < 0x1p-6f ? 0x1p-6f : 0.0f;
  const float q = __uint_as_float((__float_as_uint(y + base) + u) & 0xFFF00000u) - base;
  return q;   // 480 for a block's largest at most, which the conversion takes for 448
}

// Two e4m3 codes (the lower 16 bits) as fp32.
__device__ __forceinline__ float2 e4m3_values(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(codes));
  __half2 h;
  memcpy(&h, &r, 4);
  return __half22float2(h);
}

// A reciprocal of one unit's error: far below what the step, lr times the quotient, has of the parameter. Its divisor is 0 or
// at least 2^-126, since an eps between them is refused and 2^-75 is the least root.
__device__ __forceinline__ float rcp_near(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The scale of a block of moments: the largest magnitude times fp32 1/448 (a division, as the quantisation's, would differ in the
// last bit half of the time and cost more). inv is what they are multiplied with, 0 for a block that is not finite. It is the
// scale's reciprocal after a Newton step: that of a division for all 2^23 significands on GB300 (compared at ten exponents from
// 2^-126 to 2^119; the approximation before the step differs for 1,108,522 of them), a division itself is slower (67M elements
// 219 us, 203). Moments and roots are formed in separately rounded operations. So the codes are those of elementary fp32
// operations, which a random rounding else leaves by a whole code where the last bit decides (one element of 10^6), and the
// next steps' scales with them.
__device__ __forceinline__ float moment_scale(uint32_t amax_bits, float& inv) {
  const float s = fmaxf(__uint_as_float(amax_bits) * (1.0f / kE4m3Max), 0x1p-126f);
  const bool bad = amax_bits >= kInfBits;
  const float near = rcp_near(s);
  inv = bad ? 0.0f : fmaf(near, fmaf(-s, near, 1.0f), near);
  return bad ? __uint_as_float(0x7FC00000u) : s;
}

template <typename T, bool FULL>
__device__ __forceinline__ void adam_load(ElemVec<T, 4>& e, const unsigned char* base, int64_t i, int left, bool aligned) {
  const unsigned char* p = base + i * (int64_t)sizeof(T);
  if (FULL) e.load(p, true);
  else e.load_row(p, left, aligned, 0u);
}
template <typename T, bool FULL>
__device__ __forceinline__ void adam_store(unsigned char* base, int64_t i, int left, bool aligned, const float (&f)[4]) {
  ElemVec<T, 4> e;
  e.set(f);
  unsigned char* p = base + i * (int64_t)sizeof(T);
  if (FULL) e.store(p, true);
  else e.store_row(p, left, aligned);
}
template <bool FULL>
__device__ __forceinline__ uint32_t codes_load(const unsigned char* base, int64_t i, int left, bool aligned) {
  if (FULL || (left >= 4 && aligned)) return *reinterpret_cast<const uint32_t*>(base + i);
  uint32_t w = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < left) w |= (uint32_t)base[i + j] << (8 * j);
  return w;
}
template <bool FULL>
__device__ __forceinline__ void codes_store(unsigned char* base, int64_t i, int left, bool aligned, uint32_t w) {
  if (FULL || (left >= 4 && aligned)) *reinterpret_cast<uint32_t*>(base + i) = w;
  else
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) base[i + j] = (unsigned char)(w >> (8 * j));
}

struct AdamNow {   // the step's numbers, whether they came from the host or the device
  float gs, lr, c1, c2;
  uint32_t step;
};

constexpr int kAdamWarps = kAdamThreads / 32;

// A lane's four elements of blocks b, b + kAdamWarps, ... (U of them) as they were read.
template <typename TP, typename TG, bool MASTER, bool BITS8, int U>
struct AdamRaw {
  ElemVec<float, 4> value[MASTER || sizeof(TP) == 4 ? U : 1];
  ElemVec<__nv_bfloat16, 4> value16[MASTER || sizeof(TP) == 4 ? 1 : U];
  ElemVec<TG, 4> g[U];
  ElemVec<float, 4> m[BITS8 ? 1 : U], v[BITS8 ? 1 : U];
  uint32_t mw[U], vw[U];
  float ms[U], vs[U];

  template <bool FULL>
  __device__ __forceinline__ void load(const AdamTensor& t, int64_t b0, int lane) {
    const bool aligned = t.aligned != 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t b = b0 + u * kAdamWarps, i = b * kBlock + lane * 4;
      const int left = FULL ? 4 : (int)(t.n - i < 4 ? (t.n - i > 0 ? t.n - i : 0) : 4);
      if constexpr (MASTER)
        adam_load<float, FULL>(value[u], reinterpret_cast<const unsigned char*>(t.master), i, left, aligned);
      else if constexpr (sizeof(TP) == 4)
        adam_load<float, FULL>(value[u], t.param, i, left, aligned);
      else
        adam_load<__nv_bfloat16, FULL>(value16[u], t.param, i, left, aligned);
      adam_load<TG, FULL>(g[u], t.grad, i, left, aligned);
      if constexpr (BITS8) {
        mw[u] = codes_load<FULL>(t.m, i, left, aligned);
        vw[u] = codes_load<FULL>(t.v, i, left, aligned);
        ms[u] = t.m_scale[b];
        vs[u] = t.v_scale[b];
      } else {
        adam_load<float, FULL>(m[u], t.m, i, left, aligned);
        adam_load<float, FULL>(v[u], t.v, i, left, aligned);
      }
    }
  }
};

// The step of those elements. FULL: whole blocks on aligned addresses.
template <typename TP, typename TG, bool MASTER, bool BITS8, int U, bool FULL>
__device__ __forceinline__ void adam_step(const AdamParams& p, const AdamTensor& t, const AdamNow& now,
                                          const AdamRaw<TP, TG, MASTER, BITS8, U>& raw, int64_t b0, int lane) {
  constexpr bool kDrawParam = sizeof(TP) == 2 && !MASTER;   // a bf16 parameter without master is rounded at random
  const bool aligned = t.aligned != 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t b = b0 + u * kAdamWarps, i = b * kBlock + lane * 4;
    const int left = FULL ? 4 : (int)(t.n - i < 4 ? (t.n - i > 0 ? t.n - i : 0) : 4);
    float value[4], m[4], v[4], root[4];
    if constexpr (BITS8) {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float2 a = e4m3_values(raw.mw[u] >> (8 * j)), r = e4m3_values(raw.vw[u] >> (8 * j));
        m[j] = a.x * raw.ms[u];
        m[j + 1] = a.y * raw.ms[u];
        v[j] = r.x * raw.vs[u];
        v[j + 1] = r.y * raw.vs[u];
        v[j] *= v[j];
        v[j + 1] *= v[j + 1];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[j] = raw.m[u].at(j);
        v[j] = raw.v[u].at(j);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (MASTER || sizeof(TP) == 4) value[j] = raw.value[u].at(j);
      else value[j] = raw.value16[u].at(j);
      const float g = raw.g[u].at(j) * now.gs;
      m[j] = __fadd_rn(__fmul_rn(p.b1, m[j]), __fmul_rn(p.one_b1, g));
      v[j] = __fadd_rn(__fmul_rn(p.b2, v[j]), __fmul_rn(__fmul_rn(p.one_b2, g), g));
      root[j] = __fsqrt_rn(v[j]);
      const float change = m[j] * now.c1 * rcp_near(fmaf(root[j], now.c2, p.eps));
      value[j] = fmaf(-now.lr, fmaf(p.wd, value[j], change), value[j]);
    }
    if (MASTER) adam_store<float, FULL>(reinterpret_cast<unsigned char*>(t.master), i, left, aligned, value);
    if (kDrawParam) {
      const uint4 w = adam_words(p, (uint32_t)(i >> 2), 0x80000000u, now.step, t.index);
      const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((__float_as_uint(value[j]) & kInfBits) != kInfBits)
          value[j] = __uint_as_float((__float_as_uint(value[j]) + (h[j] & 0xFFFFu)) & 0xFFFF0000u);
    }
    adam_store<TP, FULL>(t.param, i, left, aligned, value);
    if constexpr (BITS8) {
      // what lies behind the tensor's end was read as zeros and is one still
      const uint32_t ma = warp_max_u32(__float_as_uint(
          max_nan(max_nan(fabsf(m[0]), fabsf(m[1])), max_nan(fabsf(m[2]), fabsf(m[3])))));
      const uint32_t va = warp_max_u32(__float_as_uint(max_nan(max_nan(root[0], root[1]), max_nan(root[2], root[3]))));
      float mi, vi;
      const float m_new = moment_scale(ma, mi), v_new = moment_scale(va, vi);
      const uint4 w = adam_words(p, (uint32_t)(i >> 2), 0u, now.step, t.index);
      const uint32_t h[4] = {w.x, w.y, w.z, w.w};
      float y[4], r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = copysignf(e4m3_stochastic(fabsf(m[j]) * mi, ((h[j] >> 12) & 0xFFFF0u) | 8u), m[j]);
        r[j] = e4m3_stochastic(root[j] * vi, ((h[j] << 4) & 0xFFFF0u) | 8u);
        if (root[j] > 0.0f) r[j] = fmaxf(r[j], 0x1p-9f);
      }
      uint32_t mc = e4m3_quad(y[0], y[1], y[2], y[3]), vc = e4m3_quad(r[0], r[1], r[2], r[3]);
      if (ma >= kInfBits) mc = 0u;
      if (va >= kInfBits) vc = 0u;
      codes_store<FULL>(t.m, i, left, aligned, mc);
      codes_store<FULL>(t.v, i, left, aligned, vc);
      if (lane == 0) {
        t.m_scale[b] = m_new;
        t.v_scale[b] = v_new;
      }
    } else {
      adam_store<float, FULL>(t.m, i, left, aligned, m);
      adam_store<float, FULL>(t.v, i, left, aligned, v);
    }
  }
}

template <typename TP, typename TG, bool MASTER, bool BITS8>
__global__ void __launch_bounds__(kAdamThreads, AdamShape<BITS8>::PerSm) adamw_kernel(const __grid_constant__ AdamParams p) {
  begin_overlapped();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  AdamNow now;
  now.gs = p.grad_scale ? *p.grad_scale : 1.0f;
  now.lr = p.lr_dev ? *p.lr_dev : p.lr;
  now.c1 = p.c1;
  now.c2 = p.c2;
  now.step = p.step;
  if (p.step_dev) {
    const int64_t t = *p.step_dev;
    if (t < 1) return;
    now.step = (uint32_t)t;
    now.c1 = 1.0f / -expm1f((float)t * p.ln_b1);
    now.c2 = rsqrtf(-expm1f((float)t * p.ln_b2));
  }
  constexpr int W = kAdamWarps, U = AdamShape<BITS8>::Unroll;
  for (uint32_t chunk = blockIdx.x; chunk < p.chunks; chunk += gridDim.x) {
    uint32_t lo = 0, hi = p.count;   // the last tensor whose first chunk is not behind this one
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) >> 1;
      if (p.t[mid].first_chunk <= chunk) lo = mid;
      else hi = mid;
    }
    const AdamTensor& t = p.t[lo];
    const int64_t blocks = (t.n + kBlock - 1) / kBlock, begin = (int64_t)(chunk - t.first_chunk) * p.chunk_blocks;
    const int64_t end = begin + p.chunk_blocks < blocks ? begin + p.chunk_blocks : blocks;
    const int64_t whole = t.aligned ? (end < t.n / kBlock ? end : t.n / kBlock) : begin;   // up to here in whole vectors
    int64_t b = begin + warp;
    if (b + (U - 1) * W < whole) {
      AdamRaw<TP, TG, MASTER, BITS8, U> now_raw, next_raw;
      now_raw.template load<true>(t, b, lane);
      for (;;) {
        const int64_t next = b + U * W;
        const bool more = next + (U - 1) * W < whole;
        if (more) next_raw.template load<true>(t, next, lane);
        adam_step<TP, TG, MASTER, BITS8, U, true>(p, t, now, now_raw, b, lane);
        b = next;
        if (!more) break;
        now_raw = next_raw;
      }
    }
    for (; b < whole; b += W) {
      AdamRaw<TP, TG, MASTER, BITS8, 1> raw;
      raw.template load<true>(t, b, lane);
      adam_step<TP, TG, MASTER, BITS8, 1, true>(p, t, now, raw, b, lane);
    }
    for (; b < end; b += W) {
      AdamRaw<TP, TG, MASTER, BITS8, 1> raw;
      raw.template load<false>(t, b, lane);
      adam_step<TP, TG, MASTER, BITS8, 1, false>(p, t, now, raw, b, lane);
    }
  }
}

}  // namespace vsamp
