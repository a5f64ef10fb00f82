// Vectors of up to 16 bytes of fp32 or bf16 elements at any element's address: whole vectors where the address allows it,
// otherwise 32-bit words (a bf16 row that begins in the middle of a word is shifted together from neighbouring words).
// Rows of an odd length, or at an odd stride, then cost about as much as aligned ones.
#pragma once

#include <cstdint>
#include <cstring>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace vsamp {

// Whether the whole aligned 16-byte vectors that hold the `bytes` bytes at `at` lie in [begin, end).
inline bool vectors_inside(uintptr_t at, uintptr_t bytes, uintptr_t begin, uintptr_t end) {
  return at - (at & 15) >= begin && at + bytes + ((0 - (at + bytes)) & 15) <= end;
}

template <typename T, int VE>
struct ElemVec {
  static constexpr int ES = (int)sizeof(T), W = VE * ES / 4;   // 32-bit words
  uint32_t w[W];

  // The VE elements at p. aligned: p is a multiple of the vector's size.
  __device__ __forceinline__ void load(const unsigned char* p, bool aligned) {
    if (aligned) {
      if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x; w[1] = v.y;
      }
    } else if (ES == 4 || (reinterpret_cast<uintptr_t>(p) & 2) == 0) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    } else {
      // the whole words between the first and the last element, and these two alone: nothing but the elements is read
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p + 2);
      uint32_t a = (uint32_t)h[0] << 16;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint32_t b = i + 1 < W ? q[i] : (uint32_t)h[VE - 1];
        w[i] = __funnelshift_r(a, b, 16);
        a = b;
      }
    }
  }
  // The first n elements at p, `fill` (an element's bits) for the others.
  __device__ __forceinline__ void load_some(const unsigned char* p, int n, uint32_t fill) {
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      uint32_t b = fill;
      if (j < n) {
        if constexpr (ES == 4) b = reinterpret_cast<const uint32_t*>(p)[j];
        else b = reinterpret_cast<const unsigned short*>(p)[j];
      }
      if constexpr (ES == 4) w[j] = b;
      else if (j & 1) w[j / 2] |= b << 16;
      else w[j / 2] = b;
    }
  }
  __device__ __forceinline__ void load_row(const unsigned char* p, int64_t left, bool aligned, uint32_t fill) {
    if (left >= VE) load(p, aligned);
    else load_some(p, (int)left, fill);
  }

  __device__ __forceinline__ float at(int j) const {
    if constexpr (ES == 4) return __uint_as_float(w[j]);
    else return __uint_as_float((j & 1) ? (w[j >> 1] & 0xFFFF0000u) : (w[j >> 1] << 16));
  }
  // fp32 values, each rounded once
  __device__ __forceinline__ void set(const float (&f)[VE]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (ES == 4) {
        w[i] = __float_as_uint(f[i]);
      } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        memcpy(&w[i], &b, 4);
      }
    }
  }

  __device__ __forceinline__ void store(unsigned char* p, bool aligned) const {
    if (aligned) {
      if constexpr (W == 8) {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
      } else if constexpr (W == 4) {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      }
    } else if (ES == 4 || (reinterpret_cast<uintptr_t>(p) & 2) == 0) {
#pragma unroll
      for (int i = 0; i < W; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
    } else {
      *reinterpret_cast<unsigned short*>(p) = (unsigned short)w[0];
#pragma unroll
      for (int i = 0; i + 1 < W; ++i) reinterpret_cast<uint32_t*>(p + 2)[i] = __funnelshift_r(w[i], w[i + 1], 16);
      *reinterpret_cast<unsigned short*>(p + W * 4 - 2) = (unsigned short)(w[W - 1] >> 16);
    }
  }
  __device__ __forceinline__ void store_some(unsigned char* p, int n) const {
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      if (j < n) {
        if constexpr (ES == 4) reinterpret_cast<uint32_t*>(p)[j] = w[j];
        else reinterpret_cast<unsigned short*>(p)[j] = (unsigned short)(w[j / 2] >> (16 * (j & 1)));
      }
    }
  }
  __device__ __forceinline__ void store_row(unsigned char* p, int64_t left, bool aligned) const {
    if (left >= VE) store(p, aligned);
    else store_some(p, (int)left);
  }
};

}  // namespace vsamp
