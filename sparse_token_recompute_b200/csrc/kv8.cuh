// Shared by the kernels of the 8-bit K/V cache: the rows of a call, e4m3
// conversions and the power-of-two block scales.
//
// The cache holds e4m3 codes [B, N, Hkv, hd] and one fp32 scale per sequence,
// kv head and block of `block` tokens [B, Hkv, ceil(N / block)]; a code c
// stands for c * scale.  Scales are powers of two: a decoded value has the
// code's 4 significant bits, so it is exact in bf16, and a row that is
// re-encoded because its block's scale grew keeps every bit except those that
// fall below e4m3's smallest step.  e4m3 is a floating format (normal from 2^-6
// to 448): under the tight scale the values down to 2^-14 of the block's
// largest keep their 4 bits, under one 2^k too large those down to 2^(k-14),
// and from k = 19 on every value rounds to zero.  A scale falls only where
// the whole block is written.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace dllm {

constexpr float kE4m3Max = 448.0f;
// smallest scale a written block gets: its codes still decode to normal floats
constexpr float kKv8MinScale = 7.888609052210118e-31f;  // 2^-100

// The rows of a call, packed by sequence.  Either idx/count as the C entry
// points take them (idx null: positions 0 .. count[b]-1; count null: k_cap
// rows each), or the row maps a step has already built (row_off non-null).
struct Kv8Rows {
  const int32_t* idx;
  const int32_t* count;
  const int* row_off;
  const int* row_pos;
  int B, k_cap, N;
  int* status;
};

// first compact row and row count of sequence b, computed by the calling warp
// (every lane gets both; k_cap bounds a count that is out of range)
__device__ __forceinline__ void kv8_seq_rows(const Kv8Rows& R, int b, int& off, int& n) {
  if (R.row_off) {
    off = R.row_off[b];
    n = R.row_off[b + 1] - off;
    return;
  }
  if (!R.count) {
    off = b * R.k_cap;
    n = R.k_cap;
    return;
  }
  int sum = 0;
  for (int i = threadIdx.x & 31; i < b; i += 32) sum += min(max(R.count[i], 0), R.k_cap);
  const int c = R.count[b];
  off = (int)__reduce_add_sync(0xffffffffu, (unsigned)sum);
  n = min(max(c, 0), R.k_cap);
  if (c != n && R.status && (threadIdx.x & 31) == 0) raise_status(R.status, DEV_CAPACITY);
}

// four e4m3 codes (low byte first) as packed f16 (exact; NaN stays NaN)
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
// four codes times a factor 2^-k (0 for k > 24), rounded once: a product that f16 does not
// hold exactly is below 2^-21, and e4m3 has nothing between 0 and 2^-9
__device__ __forceinline__ uint32_t e4m3x4_scaled(uint32_t four, __half2 f) {
  uint32_t h[2];
  e4m3x4_to_f16x4(four, h[0], h[1]);
  uint16_t d[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), f);
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d[i]) : "r"(*reinterpret_cast<const uint32_t*>(&p)));
  }
  return d[0] | (uint32_t)d[1] << 16;
}
// two floats (|x| <= 448, or NaN) to e4m3 codes, round to nearest even, a in the low byte
__device__ __forceinline__ uint32_t floats_to_e4m3x2(float a, float b) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
  return d;
}

// smallest power of two s >= 2^-100 with a <= 448 s (a >= 0 finite): with
// a = m 2^e, 1 <= m < 2, a / 448 = (m / 1.75) 2^(e-8)
__device__ __forceinline__ float kv8_scale_for(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e <= -100 ? kKv8MinScale : __uint_as_float((uint32_t)(e + 127) << 23);
}
// 1 / s of a power of two 2^-100 .. 2^121
__device__ __forceinline__ float kv8_inverse(float s) {
  return __uint_as_float((254u << 23) - __float_as_uint(s));
}

}  // namespace dllm
