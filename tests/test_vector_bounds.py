"""The vectors of csrc/vsamp_vec.cuh at every alignment, compiled for the host with the address sanitizer: they read and
write the elements that they are given and nothing beyond."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")

SOURCE = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <cuda_runtime.h>
static inline uint32_t __funnelshift_r(uint32_t lo, uint32_t hi, uint32_t n) {
  return (uint32_t)((((uint64_t)hi << 32) | lo) >> (n & 31));
}
#include "vsamp_vec.cuh"

template <typename T, int VE>
static int check() {
  constexpr int ES = (int)sizeof(T), BYTES = VE * ES;
  for (int off = 0; off < 16; off += ES)
    for (int n = 1; n <= VE; ++n) {
      // the allocation ends with the last element; malloc's blocks begin on 16-byte boundaries
      const int len = off + n * ES;
      unsigned char* in = (unsigned char*)malloc(len);
      unsigned char* out = (unsigned char*)malloc(len);
      for (int i = 0; i < len; ++i) { in[i] = (unsigned char)(i * 37 + 11); out[i] = 0xEE; }
      vsamp::ElemVec<T, VE> v;
      v.load_row(in + off, n, ((uintptr_t)(in + off) % BYTES) == 0, 0u);
      v.store_row(out + off, n, ((uintptr_t)(out + off) % BYTES) == 0);
      if (memcmp(in + off, out + off, n * ES) != 0) return printf("%d bytes at offset %d, %d elements\n", ES, off, n), 1;
      for (int i = 0; i < off; ++i)
        if (out[i] != 0xEE) return printf("offset %d: byte %d written\n", off, i), 1;
      unsigned char w[VE * ES];
      memcpy(w, v.w, BYTES);
      for (int i = n * ES; i < BYTES; ++i)
        if (w[i] != 0) return printf("offset %d: element past the end not filled\n", off), 1;
      free(in);
      free(out);
    }
  return 0;
}

// every address and length around a buffer of 100 bytes at an odd place, against the vectors one by one
static int check_inside() {
  const uintptr_t begin = 1000 + 6, end = begin + 100;
  for (uintptr_t at = begin; at < end; at += 2)
    for (uintptr_t n = 2; at + n <= end; n += 2) {
      bool in = true;
      for (uintptr_t v = at / 16; v <= (at + n - 1) / 16; ++v) in = in && v * 16 >= begin && v * 16 + 16 <= end;
      if (vsamp::vectors_inside(at, n, begin, end) != in) return printf("%d bytes at %d\n", (int)n, (int)at), 1;
    }
  return 0;
}

int main() {
  return check_inside() || check<float, 4>() || check<__nv_bfloat16, 4>() || check<__nv_bfloat16, 8>();
}
"""


def test_vectors_stay_on_their_elements(tmp_path):
    if shutil.which("g++") is None or not os.path.isdir(os.path.join(CUDA, "include")):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "vec.cpp", tmp_path / "vec"
    src.write_text(SOURCE)
    flags = ["-std=c++17", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
             "-I" + os.path.join(CUDA, "include"), "-I" + os.path.join(ROOT, "top_sampling_gb300", "csrc")]
    subprocess.run(["g++", *flags, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout + run.stderr[:2000]
