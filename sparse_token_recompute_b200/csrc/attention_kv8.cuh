// Shared by the two attention kernels over the 8-bit K/V cache: their arguments
// and the arithmetic that attention_kv8.cu's head comment describes.
#pragma once

#include "internal.h"
#include "kv8.cuh"

namespace dllm {

constexpr float kKv8Log2e = 1.4426950408889634f;
// Where the largest weight of a tile lies in f16: a reference puts it at 2^5, and stays while
// it is 2^-6 .. 2^15 (a move makes O wait and be rescaled: over random scales of four octaves
// 0.3 moves per warp and 24 tiles; 3.3, and 4 % of the time, for 2^0 .. 2^15 around 2^8).
// References fall at most 2^64 below the highest one so far, so that sums which grow with
// every fall stay floats; a tile is left where it is if even there its weights were below
// 2^-24.
constexpr float kKv8Aim = 5.0f, kKv8Low = -6.0f, kKv8High = 15.0f, kKv8Fall = 64.0f, kKv8Lost = 24.0f;
// V scales and references whose exponents (their differences) are larger than this are far:
// the weights' way into the sum, p_j 2^-e_j 2^(r - r'), could leave the range of floats
constexpr int kKv8Far = 30;
// what a reference starts with: below any score, and finite, so that a score of -infinity
// has the weight 0 from the start
constexpr float kKv8NoRef = -3.0e38f;

constexpr int kKv8MaxShares = 64;

struct Kv8Args {
  const __nv_bfloat16* q;
  const uint8_t* k8;
  const uint8_t* v8;
  const float* ks;
  const float* vs;
  __nv_bfloat16* o;
  const int* kv_len;  // null: N keys each
  Kv8Rows rows;
  int Hq, Hkv, G;
  int nblk, blk_log2;
  float scale_log2;  // log2(e) / sqrt(hd)
  int tiles;         // CTAs' worth of packed rows per (sequence, kv head)
  int S;             // key shares
  int part_rows;
  float* part_o;     // [S, part_rows, Hq, hd]
  float* part_ml;    // [S, part_rows, Hq, 2]: reference maximum (log2 units), sum
  float* st_m;       // softmax statistics (natural units), or null
  float* st_l;
};

// 2^x, relative error about 2^-22; results below 2^-126 flush to zero
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 t = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
// 2^e, e clamped to normal floats
__device__ __forceinline__ float pow2i(int e) {
  return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23);
}
// log2 of a block's V scale; -infinity for a block that holds no rows (its values are zeros)
__device__ __forceinline__ float v_exponent(float s) {
  return s >= kKv8MinScale ? (float)((int)(__float_as_uint(s) >> 23) - 127) : -INFINITY;
}
// the inverse of a power of two, 0 if it is far from 1
__device__ __forceinline__ float near_inverse(float s) {
  constexpr float lo = 1.0f / (1 << kKv8Far), hi = 1 << kKv8Far;
  return s >= lo && s <= hi ? kv8_inverse(s) : 0.f;
}
// whether a tile whose largest x_j lies d above the reference wants another one; mixed: a
// tile of several V scales far apart, whose largest weight is to be 2^8 .. 2^15
__device__ __forceinline__ bool wants_ref(float d, bool mixed = false) {
  const float lo = mixed ? 8.f : kKv8Low;
  return fabsf(d - 0.5f * (kKv8High + lo)) > 0.5f * (kKv8High - lo);
}
// moves the reference m to the tile's largest x_j, mx, but not below `low`; false: it stays
__device__ __forceinline__ bool new_ref(float mx, float& m, float& low, bool mixed = false) {
  if (!wants_ref(mx - m, mixed) || !(mx > low - kKv8Lost) || (mx < m && m <= low)) return false;
  m = fmaxf(mx - (mixed ? 12.f : kKv8Aim), low);
  low = fmaxf(low, m - kKv8Fall);
  return true;
}
// A rise after a fall may pass 2^126, where O's factor would flush to zero: O is multiplied
// twice then (not at the first reference, where O is zero)
__device__ __forceinline__ bool rises_far(float before, float after) {
  return before - after < -120.f && before > kKv8NoRef;
}
// 2^(weights' reference - sum's reference), 0 if that is far above 1
__device__ __forceinline__ float ref_factor(float d) { return d <= (float)kKv8Far ? exp2_approx(d) : 0.f; }
// (m, l) with the same l 2^m and 1 <= l < 2; l = 0 stays, with m = -inf
__device__ __forceinline__ void normal_stats(float& m, float& l) {
  if (l == 0.f) m = -INFINITY;
  if (!(l > 0.f) || l == INFINITY) return;
  const uint32_t b = __float_as_uint(l);
  m += (float)((int)(b >> 23) - 127);
  l = __uint_as_float((b & 0x7fffffu) | 0x3f800000u);
}
// exponent that brings amax into [2^14, 2^15) (0 for a row of zeros)
__device__ __forceinline__ int query_shift(float amax) {
  const int e = (int)(__float_as_uint(amax) >> 23);
  return e == 0 ? 0 : 14 + 127 - e;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void lds128(uint32_t* v, uint32_t at) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void lds64(uint32_t* v, uint32_t at) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(at) : "memory");
}

// many packed rows: tiles of 128 on tcgen05 (attention_kv8_tc.cu)
cudaError_t launch_attention_kv8_tc(const Kv8Args& A, long long ctas, int hd, cudaStream_t s);

template <auto Kernel, typename... Args>
cudaError_t launch_kv8(unsigned grid, unsigned threads, int smem, cudaStream_t s, const Args&... args) {
  if (smem > 48 * 1024) {
    const cudaError_t e = ensure_smem_attr<Kernel>(smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = la;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, Kernel, args...);
}

}  // namespace dllm
