// The AdamW step of many tensors in one launch.
//
//   g = grad * scale, m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2
//   p = p - lr (wd p + (m / (1 - b1^t)) / (sqrt(v) / sqrt(1 - b2^t) + eps))
//
// A stream over memory: each element is read and written once. A warp takes 128 consecutive elements of a tensor, four
// per lane, which is also a block of the 8-bit states: their new scale is one maximum over the warp's registers, and one
// Philox call gives a lane's four elements their random bits. The tensors' addresses travel in the kernel's parameters
// (up to 384 per launch), so a step needs no table in device memory and can be captured as it is.
#pragma once

#include "vsamp_block_quant.cuh"

namespace vsamp {

constexpr int kAdamThreads = 256;
constexpr int kAdamTensors = 384;    // of 80 bytes: 30,720 of a launch's 32,764 parameter bytes
constexpr int kAdamChunk = 32;       // blocks of 128 elements that a CTA takes at a time

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
  uint32_t count, chunks;
  float lr, b1, b2, one_b1, one_b2, eps, wd;
  float ln_b1, ln_b2, c1, c2;      // logarithms of the betas; 1 / (1 - b1^t), 1 / sqrt(1 - b2^t) of the host's step
  uint32_t step, k0, k1;
  const float* lr_dev;
  const int64_t* step_dev;
  const float* grad_scale;
};
static_assert(sizeof(AdamTensor) == 80 && sizeof(AdamParams) <= 32764, "kernel parameters");

// A magnitude in units of the scale to one of the two e4m3 values next to it, up with the probability of its place
// between them: h is 16 random bits. Below 2^-6 the values are 2^-9 apart, above it 2^-3 of the power of two below.
__device__ __forceinline__ float e4m3_stochastic(float y, uint32_t h) {
  const int e = max((int)(__float_as_uint(y) >> 23) - 127, -6) - 3;
  const float up = __uint_as_float((uint32_t)(127 - e) << 23), down = __uint_as_float((uint32_t)(127 + e) << 23);
  return fminf(floorf(fmaf(y, up, ((float)h + 0.5f) * 0x1p-16f)) * down, kE4m3Max);
}

__device__ __forceinline__ float e4m3_to_float(uint32_t code) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(code & 0xFFu));
  return __half2float(__ushort_as_half((unsigned short)(r & 0xFFFFu)));
}

template <typename T>
__device__ __forceinline__ void adam_load(const unsigned char* base, int64_t i, int left, bool aligned, float (&f)[4]) {
  ElemVec<T, 4> e;
  const unsigned char* p = base + i * (int64_t)sizeof(T);
  if (left >= 4) e.load(p, aligned);
  else e.load_some(p, left, 0u);
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = e.at(j);
}
template <typename T>
__device__ __forceinline__ void adam_store(unsigned char* base, int64_t i, int left, bool aligned, const float (&f)[4]) {
  ElemVec<T, 4> e;
  e.set(f);
  unsigned char* p = base + i * (int64_t)sizeof(T);
  if (left >= 4) e.store(p, aligned);
  else e.store_some(p, left);
}
__device__ __forceinline__ uint32_t codes_load(const unsigned char* base, int64_t i, int left, bool aligned) {
  if (left >= 4 && aligned) return *reinterpret_cast<const uint32_t*>(base + i);
  uint32_t w = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < left) w |= (uint32_t)base[i + j] << (8 * j);
  return w;
}
__device__ __forceinline__ void codes_store(unsigned char* base, int64_t i, int left, bool aligned, uint32_t w) {
  if (left >= 4 && aligned) *reinterpret_cast<uint32_t*>(base + i) = w;
  else
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) base[i + j] = (unsigned char)(w >> (8 * j));
}

template <typename TP, typename TG, bool MASTER, bool BITS8>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamParams p) {
  begin_overlapped();
  constexpr bool kDrawParam = sizeof(TP) == 2 && !MASTER;   // a bf16 parameter without master is rounded at random
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float gs = p.grad_scale ? *p.grad_scale : 1.0f;
  const float lr = p.lr_dev ? *p.lr_dev : p.lr;
  float c1 = p.c1, c2 = p.c2;
  uint32_t step = p.step;
  if (p.step_dev) {
    const int64_t t = *p.step_dev;
    if (t < 1) return;
    step = (uint32_t)t;
    c1 = 1.0f / -expm1f((float)t * p.ln_b1);
    c2 = rsqrtf(-expm1f((float)t * p.ln_b2));
  }
  for (uint32_t chunk = blockIdx.x; chunk < p.chunks; chunk += gridDim.x) {
    uint32_t lo = 0, hi = p.count;   // the last tensor whose first chunk is not behind this one
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) >> 1;
      if (p.t[mid].first_chunk <= chunk) lo = mid;
      else hi = mid;
    }
    const AdamTensor& t = p.t[lo];
    const int64_t blocks = (t.n + kBlock - 1) / kBlock, begin = (int64_t)(chunk - t.first_chunk) * kAdamChunk;
    const int64_t end = begin + kAdamChunk < blocks ? begin + kAdamChunk : blocks;
    const bool aligned = t.aligned != 0;
    for (int64_t b = begin + warp; b < end; b += kAdamThreads / 32) {
      const int64_t i = b * kBlock + lane * 4;
      const int left = (int)(t.n - i < 4 ? (t.n - i > 0 ? t.n - i : 0) : 4);
      float value[4], g[4], m[4], v[4], root[4];
      if (MASTER) adam_load<float>(reinterpret_cast<const unsigned char*>(t.master), i, left, aligned, value);
      else adam_load<TP>(t.param, i, left, aligned, value);
      adam_load<TG>(t.grad, i, left, aligned, g);
      if (BITS8) {
        const uint32_t mw = codes_load(t.m, i, left, aligned), vw = codes_load(t.v, i, left, aligned);
        const float ms = t.m_scale[b], vs = t.v_scale[b];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          m[j] = e4m3_to_float(mw >> (8 * j)) * ms;
          v[j] = e4m3_to_float(vw >> (8 * j)) * vs;
          v[j] *= v[j];
        }
      } else {
        adam_load<float>(t.m, i, left, aligned, m);
        adam_load<float>(t.v, i, left, aligned, v);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        g[j] *= gs;
        m[j] = fmaf(p.b1, m[j], p.one_b1 * g[j]);
        v[j] = fmaf(p.b2, v[j], p.one_b2 * g[j] * g[j]);
        root[j] = sqrtf(v[j]);
        const float change = m[j] * c1 / fmaf(root[j], c2, p.eps);
        value[j] = fmaf(-lr, fmaf(p.wd, value[j], change), value[j]);
      }
      if (MASTER) adam_store<float>(reinterpret_cast<unsigned char*>(t.master), i, left, aligned, value);
      if (kDrawParam) {
        const uint4 w = philox4x32_10(make_uint4((uint32_t)(i >> 2), 0x80000000u, step, t.index), {p.k0, p.k1});
        const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if ((__float_as_uint(value[j]) & kInfBits) != kInfBits)
            value[j] = __uint_as_float((__float_as_uint(value[j]) + (h[j] & 0xFFFFu)) & 0xFFFF0000u);
      }
      adam_store<TP>(t.param, i, left, aligned, value);
      if (BITS8) {
        uint32_t ma = 0u, va = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < left) {
            ma = max(ma, __float_as_uint(m[j]) & 0x7FFFFFFFu);
            va = max(va, __float_as_uint(root[j]) & 0x7FFFFFFFu);
          }
        ma = warp_max_u32(ma);
        va = warp_max_u32(va);
        float mi, vi;
        const float ms = block_scale(ma, mi), vs = block_scale(va, vi);
        const uint4 w = philox4x32_10(make_uint4((uint32_t)(i >> 2), 0u, step, t.index), {p.k0, p.k1});
        const uint32_t h[4] = {w.x, w.y, w.z, w.w};
        float y[4], r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[j] = copysignf(e4m3_stochastic(fabsf(m[j]) * mi, h[j] >> 16), m[j]);
          r[j] = e4m3_stochastic(root[j] * vi, h[j] & 0xFFFFu);
          if (root[j] > 0.0f) r[j] = fmaxf(r[j], 0x1p-9f);
        }
        uint32_t mw = e4m3_quad(y[0], y[1], y[2], y[3]), vw = e4m3_quad(r[0], r[1], r[2], r[3]);
        if (ma >= kInfBits) mw = 0u;
        if (va >= kInfBits) vw = 0u;
        codes_store(t.m, i, left, aligned, mw);
        codes_store(t.v, i, left, aligned, vw);
        if (lane == 0) {
          t.m_scale[b] = ms;
          t.v_scale[b] = vs;
        }
      } else {
        adam_store<float>(t.m, i, left, aligned, m);
        adam_store<float>(t.v, i, left, aligned, v);
      }
    }
  }
}

}  // namespace vsamp
