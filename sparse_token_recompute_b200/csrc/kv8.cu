// Kernels around the 8-bit K/V cache: the q/k norm with the position rotation,
// writing selected rows into the cache, and reading rows back.  All three are
// bound by HBM (or, for a handful of rows, by the latency of a launch).
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "kv8.cuh"

namespace dllm {

namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------- q/k norm + rotation

struct NormArgs {
  Kv8Rows rows;
  const int* row_seq;  // with row maps: sequence of each compact row
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  size_t ldq, ldk, ldqo, ldko;  // elements between compact rows
  const void* q_gain;
  const void* k_gain;
  const float2* rope;  // [N, hd/2] (cos, sin), null: no rotation
  int Hq, Hkv;
  float eps;
  int k_in_cache, k_out_cache;  // keys at [B, N, Hkv, hd] rows instead of compact ones
};

struct NormRow {
  int r, seq, pos;  // compact row (-1: none), sequence, position
};

// The rows of a call one after the other from row x on: compact row x (row maps), or
// row x % k_cap of sequence x / k_cap (idx/count).
struct NormRows {
  int x, b, j, seq = -1, off = 0, n = 0;
  __device__ __forceinline__ NormRows(const NormArgs& A, int x0) : x(x0), b(0), j(0) {
    if (!A.rows.row_off) b = x0 / A.rows.k_cap, j = x0 - b * A.rows.k_cap;
  }
  __device__ __forceinline__ NormRow next(const NormArgs& A) {
    const Kv8Rows& R = A.rows;
    if (R.row_off) {
      const int i = x++;
      if (i >= R.row_off[R.B]) return NormRow{-1, 0, 0};
      return NormRow{i, A.row_seq[i], R.row_pos[i]};
    }
    if (j >= R.k_cap) j = 0, ++b;
    if (b >= R.B) return NormRow{-1, 0, 0};
    if (b != seq) {
      seq = b;
      kv8_seq_rows(R, b, off, n);
    }
    const int i = j++;
    if (i >= n) return NormRow{-1, 0, 0};
    int pos = i;
    bool bad;
    if (R.idx) {
      const int32_t* l = R.idx + (size_t)b * R.k_cap;
      pos = l[i];
      bad = i > 0 && l[i - 1] >= pos;
    } else {
      bad = false;
    }
    const bool out = (unsigned)pos >= (unsigned)R.N;
    if ((bad || out) && (threadIdx.x & 31) == 0) raise_status(R.status, DEV_BAD_INDEX);
    return NormRow{out ? -1 : off + i, b, pos};
  }
};

// Head vectors of HD bf16: HD/16 lanes per head, each with 8 elements j.. of the
// first half and their partners j + HD/2.., so that the rotation is in one lane
// and a head's sum of squares is 2 or 3 shuffles.  A row's heads (queries, then
// keys) are spread over `lanes` threads, each with PASSES of them; a thread takes
// `rows` rows one after the other, the next one's vectors on their way while it
// works on the current.  The sums, the norm and the rotation are fp32, rounded once
// when stored.  Bound by HBM, closely followed by instruction issue (66 % active): hence
// addresses that are set up once per thread, and gains in shared memory as bf16 (fp32
// there, with twice the reads: 66 us; in registers, at the cost of a CTA per SM: 75).  32
// sequences x up to 308 rows of 32 + 32 heads of 128 (279 MB): 62.6 us, 4.5 TB/s.
template <int HD, int PASSES>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_rope_kernel(const NormArgs A, int lanes, int rows) {
  griddep_launch_dependents();
  griddep_wait();
  using bf = __nv_bfloat16;
  constexpr int LPH = HD / 16;
  __shared__ uint4 s_gain[2][HD / 8];  // bf16
  if (threadIdx.x < HD / 4)
    s_gain[threadIdx.x / (HD / 8)][threadIdx.x % (HD / 8)] =
        static_cast<const uint4*>(threadIdx.x < HD / 8 ? A.q_gain : A.k_gain)[threadIdx.x % (HD / 8)];
  __syncthreads();
  const int l = threadIdx.x % lanes;
  const int e = (l % LPH) * 8;  // first element of this lane in each half
  const int heads = A.Hq + A.Hkv, per_pass = lanes / LPH;
  const int h0 = blockIdx.y * PASSES * per_pass + l / LPH;  // this lane's first head
  // the lanes of one head: in each pass all of them have a head or none has
  const unsigned group = ((1u << LPH) - 1u) << ((threadIdx.x & 31) / LPH * LPH);
  // per pass: where this lane's elements of row 0 lie and go, and the rows' strides (of
  // compact rows, or of cache rows where the stride is a whole key row)
  const char* src[PASSES];
  char* dst[PASSES];
  uint32_t ld_in[PASSES], ld_out[PASSES];  // bytes
  const uint4* gain[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int h = h0 + p * per_pass;
    const bool is_q = h < A.Hq;
    const size_t at = (size_t)(is_q ? h : h - A.Hq) * HD + e;
    src[p] = static_cast<const char*>(is_q ? A.q : A.k) + at * 2;
    dst[p] = static_cast<char*>(is_q ? A.q_out : A.k_out) + at * 2;
    ld_in[p] = 2 * (uint32_t)(is_q ? A.ldq : A.k_in_cache ? A.Hkv * HD : A.ldk);
    ld_out[p] = 2 * (uint32_t)(is_q ? A.ldqo : A.k_out_cache ? A.Hkv * HD : A.ldko);
    gain[p] = s_gain[is_q ? 0 : 1] + e / 8;
  }
  NormRows list(A, (blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes) * rows);
  NormRow w = list.next(A);
  uint4 v[PASSES][2];
  auto load = [&](const NormRow& t, int p) {
    const int h = h0 + p * per_pass;
    if (t.r < 0 || h >= heads) return;
    // (rows of at least 128 bytes: their numbers fit 32 bits)
    const uint32_t row = h >= A.Hq && A.k_in_cache ? (uint32_t)t.seq * A.rows.N + t.pos : t.r;
    const char* at = src[p] + (uint64_t)row * ld_in[p];
    v[p][0] = *reinterpret_cast<const uint4*>(at);
    v[p][1] = *reinterpret_cast<const uint4*>(at + HD);
  };
#pragma unroll
  for (int p = 0; p < PASSES; ++p) load(w, p);
  for (int i = 0; i < rows; ++i) {
    const NormRow next = i + 1 < rows ? list.next(A) : NormRow{-1, 0, 0};
    float cs[8], sn[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float4 c = make_float4(1.f, 0.f, 1.f, 0.f);
      if (A.rope && w.r >= 0)
        c = __ldg(reinterpret_cast<const float4*>(A.rope + (size_t)w.pos * (HD / 2) + e) + k);
      cs[2 * k] = c.x, sn[2 * k] = c.y, cs[2 * k + 1] = c.z, sn[2 * k + 1] = c.w;
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int h = h0 + p * per_pass;
      const uint32_t xa[4] = {v[p][0].x, v[p][0].y, v[p][0].z, v[p][0].w};
      const uint32_t xb[4] = {v[p][1].x, v[p][1].y, v[p][1].z, v[p][1].w};
      float a[8], b[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[2 * k] = __uint_as_float(xa[k] << 16), a[2 * k + 1] = __uint_as_float(xa[k] & 0xffff0000u);
        b[2 * k] = __uint_as_float(xb[k] << 16), b[2 * k + 1] = __uint_as_float(xb[k] & 0xffff0000u);
      }
      load(next, p);
      if (w.r < 0 || h >= heads) continue;
      float ss = 0.f, s1 = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(a[k], a[k], ss), s1 = fmaf(b[k], b[k], s1);
      ss += s1;
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
      const float r = rsqrtf(ss * (1.0f / HD) + A.eps);
      uint32_t ya[4], yb[4];
      float ga[8], gb[8];
      unpack8(gain[p][0], ga);
      unpack8(gain[p][HD / 16], gb);
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        const float *fa = ga + k, *fb = gb + k;
        float y[4], z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = a[k + i] * r * fa[i], t = b[k + i] * r * fb[i];
          y[i] = x * cs[k + i] - t * sn[k + i];
          z[i] = t * cs[k + i] + x * sn[k + i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const __nv_bfloat162 u0 = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
          const __nv_bfloat162 u1 = __floats2bfloat162_rn(z[2 * i], z[2 * i + 1]);
          ya[k / 2 + i] = *reinterpret_cast<const uint32_t*>(&u0);
          yb[k / 2 + i] = *reinterpret_cast<const uint32_t*>(&u1);
        }
      }
      const uint32_t row = h >= A.Hq && A.k_out_cache ? (uint32_t)w.seq * A.rows.N + w.pos : w.r;
      char* to = dst[p] + (uint64_t)row * ld_out[p];
      *reinterpret_cast<uint4*>(to) = make_uint4(ya[0], ya[1], ya[2], ya[3]);
      *reinterpret_cast<uint4*>(to + HD) = make_uint4(yb[0], yb[1], yb[2], yb[3]);
    }
    w = next;
  }
}

// fp32 rows (small models, any even head_dim up to 256): one warp per row and head
__global__ void __launch_bounds__(kThreads) qk_norm_rope_f32_kernel(const NormArgs A, int HD) {
  const int heads = A.Hq + A.Hkv;
  const size_t u = (size_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int x = (int)(u / heads), h = (int)(u % heads);
  const NormRow w = NormRows(A, x).next(A);
  if (w.r < 0) return;
  const int r = w.r, seq = w.seq, pos = w.pos;
  const int lane = threadIdx.x & 31, half = HD / 2;
  const bool is_q = h < A.Hq;
  const size_t cache_row = ((size_t)seq * A.rows.N + pos) * A.Hkv * HD;
  const float* src = static_cast<const float*>(is_q ? A.q : A.k) +
                     (is_q ? r * A.ldq + (size_t)h * HD
                           : (A.k_in_cache ? cache_row : r * A.ldk) + (size_t)(h - A.Hq) * HD);
  float* dst = static_cast<float*>(is_q ? A.q_out : A.k_out) +
               (is_q ? r * A.ldqo + (size_t)h * HD
                     : (A.k_out_cache ? cache_row : r * A.ldko) + (size_t)(h - A.Hq) * HD);
  const float* g = static_cast<const float*>(is_q ? A.q_gain : A.k_gain);
  float a[4], b[4], ss = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = lane + 32 * i;
    a[i] = j < half ? src[j] : 0.f;
    b[i] = j < half ? src[j + half] : 0.f;
    ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
  }
  const float rs = rsqrtf(warp_sum(ss) / (float)HD + A.eps);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = lane + 32 * i;
    if (j >= half) break;
    const float2 t = A.rope ? A.rope[(size_t)pos * half + j] : make_float2(1.f, 0.f);
    const float y = a[i] * rs * g[j], z = b[i] * rs * g[j + half];
    dst[j] = y * t.x - z * t.y;
    dst[j + half] = z * t.x + y * t.y;
  }
}

// ---------------------------------------------------------------- write

struct WriteArgs {
  Kv8Rows rows;
  const __nv_bfloat16* x[2];  // K and V rows
  size_t ld[2];
  uint8_t* c8[2];
  float* scale[2];
  int Hkv, blk_log2, nblk;
  int hpc;     // heads per CTA
  int groups;  // ceil(Hkv / hpc)
};

// the first place of a strictly ascending list whose value is not below v, found by
// the whole warp: 32 probes per round
__device__ __forceinline__ int warp_lower_bound(const int* __restrict__ l, int n, int v) {
  int lo = 0, len = n;  // the place is in [lo, lo + len]
  const int lane = threadIdx.x & 31;
  while (len > 0) {
    const int step = (len + 31) / 32;
    const int at = lane * step + step - 1;  // last of this lane's piece
    const bool below = at < len && l[lo + at] < v;
    const int k = __popc(__ballot_sync(0xffffffffu, below));  // whole pieces below v
    lo += k * step;
    len = min(step - 1, len - k * step);
    if (len < 0) len = 0;
  }
  return lo;
}

// One CTA = one block of tokens of one sequence and `hpc` kv heads.  It finds the
// rows that fall in its block; then 1, 2, 4 or 8 warps take one (head, K or V) at a
// time, as many as hold its new rows in registers: largest magnitude, the block's
// scale, encode and store.  Tokens that are kept are read only where the scale grew.
// Few rows are bound by the way list -> rows -> scale -> kept codes, each a trip to
// memory, and by instruction issue (78 % active); many by HBM.  32 sequences, 32 heads of
// 128, blocks of 64: up to 308 of 1536 rows (206 MB) 47 us, 4.4 TB/s; all rows (1.2 GB)
// 202 us, 6.0 TB/s (before, one warp with a second look at the rows: 234).  Four CTAs per
// SM 50 and 201 us, six 52 and 222.
template <int HD>
__global__ void __launch_bounds__(kThreads, 5) kv8_write_kernel(const WriteArgs A) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int LPR = HD / 8;       // lanes per bf16 row (16 bytes each)
  constexpr int RPL = 32 / LPR;     // rows per load of a warp
  constexpr int NL = 8;             // loads of a lane at a time: RPL * NL rows of a warp
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps * RPL * NL >= 128, "a block's rows fit the registers");
  constexpr int LPO = HD / 16;      // lanes per row of codes
  constexpr int RPO = 32 / LPO;
  const Kv8Rows& R = A.rows;
  const int block = 1 << A.blk_log2;
  const int grp = blockIdx.x % A.groups;
  const int bb = blockIdx.x / A.groups;
  const int blk = bb % A.nblk, b = bb / A.nblk;
  const int p0 = blk << A.blk_log2;
  const int tokens = min(block, R.N - p0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  __shared__ int s_row[128];        // by token of the block: its compact row, or -1
  __shared__ int s_new_row[128];    // the new rows, compacted in token order
  __shared__ uint8_t s_tok[128];    // their tokens, then the tokens that are kept
  __shared__ int s_cnt[4];
  __shared__ uint32_t s_top[2][kWarps];
  // A list of up to SCAN * 256 rows is read whole, all entries at once (those of idx while
  // the count is on its way); in a longer one the block's first row is searched for (at 308
  // rows 55.1 us against 54.9, with twice the CTAs 62.5 against 59.9).
  constexpr int SCAN = 4;
  const int* list = R.row_off || !R.idx ? nullptr : R.idx + (size_t)b * R.k_cap;
  int pos[SCAN];
  auto read_list = [&](int rows) {
#pragma unroll
    for (int i = 0; i < SCAN; ++i) {
      const int j = threadIdx.x + i * kThreads;
      pos[i] = j < rows ? list[j] : -1;
    }
  };
  if (list && R.k_cap <= SCAN * kThreads) read_list(R.k_cap);
  if (threadIdx.x < 128) s_row[threadIdx.x] = -1;
  int off, n;
  kv8_seq_rows(R, b, off, n);
  if (R.row_off) list = R.row_pos + off;
  const bool scan = (R.row_off ? n : R.k_cap) <= SCAN * kThreads;
  if (R.row_off && scan) read_list(n);
  __syncthreads();
  // (a repeated position: the later row)
  auto put = [&](int j, int p) {
    const unsigned t = (unsigned)p - (unsigned)p0;
    if (j < n && t < (unsigned)tokens) atomicMax(&s_row[t], off + j);
  };
  if (!list) {
    if (threadIdx.x < tokens) put(p0 + threadIdx.x, p0 + threadIdx.x);
  } else if (scan) {
#pragma unroll
    for (int i = 0; i < SCAN; ++i) put(threadIdx.x + i * kThreads, pos[i]);
  } else {
    const int j = warp_lower_bound(list, n, p0) + threadIdx.x;
    if (threadIdx.x < tokens && j < n) put(j, list[j]);
  }
  if (!R.row_off && R.status && blk == 0 && grp == 0) {  // one CTA per sequence looks the list over
    for (int j = threadIdx.x; j < n; j += kThreads) {
      const int p = list ? list[j] : j;
      if (p < 0 || p >= R.N || (list && j > 0 && list[j - 1] >= p))
        raise_status(R.status, DEV_BAD_INDEX);
    }
  }
  __syncthreads();
  const int mine = threadIdx.x < 128 ? s_row[threadIdx.x] : -1;
  const unsigned has = __ballot_sync(0xffffffffu, mine >= 0);
  if (lane == 0 && warp < 4) s_cnt[warp] = __popc(has);
  __syncthreads();
  const int n_new = s_cnt[0] + s_cnt[1] + s_cnt[2] + s_cnt[3];
  if (n_new == 0) return;
  if (threadIdx.x < tokens) {
    int at = __popc(has & ((1u << lane) - 1u));  // new rows before this token
    for (int w = 0; w < warp; ++w) at += s_cnt[w];
    if (mine >= 0) s_new_row[at] = mine;
    s_tok[mine >= 0 ? at : n_new + (int)threadIdx.x - at] = (uint8_t)threadIdx.x;
  }
  __syncthreads();

  const int h0 = grp * A.hpc, h1 = min(A.Hkv, h0 + A.hpc);
  const int units = 2 * (h1 - h0);
  int wpu = 1;  // warps per (head, K or V)
  while (wpu * NL * RPL < n_new) wpu *= 2;
  const int part = warp & (wpu - 1);
  const int sub = lane / LPR, e = (lane % LPR) * 8;
  const int k0 = part * RPL + sub, k_step = wpu * RPL;  // this lane's new rows
  for (int u0 = 0, turn = 0; u0 < units; u0 += kWarps / wpu, turn ^= 1) {
    const int u = u0 + warp / wpu;
    const bool active = u < units;
    const int kv = u & 1, h = h0 + (u >> 1);
    const char* src = reinterpret_cast<const char*>(A.x[kv] + (size_t)h * HD + e);
    const uint32_t ld = 2 * (uint32_t)A.ld[kv];  // bytes
    uint8_t* dst = A.c8[kv] + (((size_t)b * R.N + p0) * A.Hkv + h) * HD;
    float* sp = A.scale[kv] + ((size_t)b * A.Hkv + h) * A.nblk + blk;
    const float s_old = active ? *sp : 0.f;
    uint4 v[NL];
    uint32_t mx = 0;  // two running maxima of |x| as bf16 bits
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int k = k0 + i * k_step;
      v[i] = make_uint4(0, 0, 0, 0);
      if (active && k < n_new) v[i] = *reinterpret_cast<const uint4*>(src + (uint64_t)(uint32_t)s_new_row[k] * ld);
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      mx = __vmaxu2(mx, v[i].x & 0x7fff7fffu);
      mx = __vmaxu2(mx, v[i].y & 0x7fff7fffu);
      mx = __vmaxu2(mx, v[i].z & 0x7fff7fffu);
      mx = __vmaxu2(mx, v[i].w & 0x7fff7fffu);
    }
    uint32_t top = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
    if (top >= 0x7f80u) {  // infinities or NaN among this warp's: they do not count, and become NaN
      top = 0;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        uint32_t* q = reinterpret_cast<uint32_t*>(&v[i]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t lo = q[t] & 0x7fffu, hi = (q[t] >> 16) & 0x7fffu;
          if (lo < 0x7f80u) top = max(top, lo);
          else q[t] |= 0x7fu;
          if (hi < 0x7f80u) top = max(top, hi);
          else q[t] |= 0x7f0000u;
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
    }
    if (wpu > 1) {  // (a buffer is written again two turns on, past the next turn's barrier)
      if (lane == 0) s_top[turn][warp] = top;
      __syncthreads();
      for (int w = 0; w < wpu; ++w) top = max(top, s_top[turn][warp - part + w]);
    }
    if (!active) continue;
    const float amax = __uint_as_float(top << 16);
    const bool had = s_old >= kKv8MinScale;  // (false for NaN) the block holds rows already
    const bool same = n_new < tokens && had && amax <= kE4m3Max * s_old;
    const float s = same ? s_old : kv8_scale_for(amax);
    const float inv = kv8_inverse(s);
    // (powers of two of bf16's range: products that bf16 does not hold exactly are below
    // 2^-126, and those round to zero codes)
    const __nv_bfloat162 inv2 = __float2bfloat162_rn(inv);
    const uint32_t token_bytes = A.Hkv * HD;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int k = k0 + i * k_step;
      if (k >= n_new) continue;
      uint32_t q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t c[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&q[t]), inv2);
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&y);
        c[t] = floats_to_e4m3x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
      }
      *reinterpret_cast<uint2*>(dst + s_tok[k] * token_bytes + e) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    }
    if (same) continue;
    if (lane == 0 && part == 0) *sp = s;
    // the kept tokens at the new scale (a block without rows yet: zeros)
    const __half2 f = __float2half2_rn(had ? s_old * inv : 0.f);
    const int t_step = wpu * RPO;
    for (int t0 = n_new + part * RPO + lane / LPO; t0 < tokens; t0 += NL * t_step) {
      uint4 w[NL];
      uint32_t at[NL];
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        w[i] = make_uint4(0, 0, 0, 0);
        at[i] = 0;
        if (t0 + i * t_step >= tokens) continue;
        at[i] = s_tok[t0 + i * t_step] * token_bytes + (lane % LPO) * 16;
        if (had) w[i] = *reinterpret_cast<const uint4*>(dst + at[i]);
      }
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        if (t0 + i * t_step >= tokens) continue;
        *reinterpret_cast<uint4*>(dst + at[i]) =
            make_uint4(e4m3x4_scaled(w[i].x, f), e4m3x4_scaled(w[i].y, f), e4m3x4_scaled(w[i].z, f),
                       e4m3x4_scaled(w[i].w, f));
      }
    }
  }
}

// ---------------------------------------------------------------- read

struct ReadArgs {
  Kv8Rows rows;
  const int* row_seq;
  const uint8_t* c8[2];
  const float* scale[2];
  __nv_bfloat16* out[2];
  size_t ld[2];
  int Hkv, hd_log2, blk_log2, nblk;
};

// `lanes` threads per row, 16 codes of K and of V per thread and turn; several rows one
// after the other, so that the addresses of a row cost little: what is fixed for a
// thread is its place in the row.  Bound by HBM (a third read, two thirds written): 32 x
// 1536 rows of 32 heads of 128 (1.2 GB) 202 us, 6.0 TB/s.
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const ReadArgs A, int lanes, int rows) {
  griddep_launch_dependents();
  griddep_wait();
  const Kv8Rows& R = A.rows;
  const int x0 = (blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes) * rows;
  const int vecs = (A.Hkv << A.hd_log2) >> 4;
  int seq = -1, off = 0, n = 0;
  for (int i = 0; i < rows; ++i) {
    const int x = x0 + i;
    int r, pos;
    if (R.row_off) {
      if (x >= R.row_off[R.B]) return;
      r = x, seq = A.row_seq[x], pos = R.row_pos[x];
    } else {
      if (x >= R.B * R.k_cap) return;
      const int b = x / R.k_cap, j = x - b * R.k_cap;
      if (b != seq) {
        seq = b;
        kv8_seq_rows(R, b, off, n);
      }
      if (j >= n) continue;
      r = off + j, pos = j;
      if (R.idx) {
        const int32_t* l = R.idx + (size_t)b * R.k_cap;
        pos = l[j];
        if ((pos < 0 || pos >= R.N || (j > 0 && l[j - 1] >= pos)) && (threadIdx.x & 31) == 0)
          raise_status(R.status, DEV_BAD_INDEX);
      } else if (j >= R.N && (threadIdx.x & 31) == 0) {
        raise_status(R.status, DEV_BAD_INDEX);
      }
      if (pos < 0 || pos >= R.N) continue;
    }
    const size_t in = ((size_t)seq * R.N + pos) * vecs;
    const size_t sc = (size_t)seq * A.Hkv * A.nblk + (pos >> A.blk_log2);
    for (int c = threadIdx.x % lanes; c < vecs; c += lanes) {
      const int at = ((c << 4) >> A.hd_log2) * A.nblk;
      uint4 w[2];
      float s[2];
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        w[kv] = __ldg(reinterpret_cast<const uint4*>(A.c8[kv]) + in + c);
        s[kv] = __ldg(A.scale[kv] + sc + at);
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t q[4] = {w[kv].x, w[kv].y, w[kv].z, w[kv].w};
        uint32_t y[8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          uint32_t h[2];
          e4m3x4_to_f16x4(q[t], h[0], h[1]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
            const __nv_bfloat162 u = __floats2bfloat162_rn(f.x * s[kv], f.y * s[kv]);
            y[2 * t + k] = *reinterpret_cast<const uint32_t*>(&u);
          }
        }
        uint4* dst = reinterpret_cast<uint4*>(A.out[kv] + (size_t)r * A.ld[kv]) + 2 * c;
        dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
        dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
      }
    }
  }
}

int log2_of(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

template <typename K, typename... Args>
cudaError_t launch(K kernel, dim3 grid, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = la;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// threads that share a row of `units` equal pieces: a power of two of whole warps
int lanes_for(int units) { return std::min(kThreads, 32 * (1 << log2_of((units + 31) / 32))); }

Kv8Rows rows_of(const Kv8RowMap& m) {
  return Kv8Rows{m.idx, m.count, m.row_off, m.row_pos, m.B, m.k_cap, m.N, m.status};
}

}  // namespace

cudaError_t launch_qk_norm_rope(const Kv8RowMap& m, const void* q, size_t ldq, const void* k,
                                size_t ldk, void* q_out, size_t ldqo, void* k_out, size_t ldko,
                                const void* q_gain, const void* k_gain, const float2* rope, int Hq,
                                int Hkv, int hd, float eps, bool bf16, bool k_in_cache,
                                bool k_out_cache, cudaStream_t s) {
  const int cap = m.M_cap;
  if (cap <= 0) return cudaSuccess;
  NormArgs A{rows_of(m), m.row_seq, q,    k,  q_out, k_out, ldq, ldk,        ldqo,       ldko, q_gain,
             k_gain,     rope,      Hq,   Hkv, eps,  k_in_cache, k_out_cache};
  ProfScope prof("qk_norm_rope", s);
  if (!bf16) {
    const size_t units = (size_t)cap * (Hq + Hkv);
    qk_norm_rope_f32_kernel<<<(unsigned)((units + 7) / 8), kThreads, 0, s>>>(A, hd);
    return cudaGetLastError();
  }
  // at most 256 threads per row and 4 heads per thread; more heads: more CTAs
  const int lph = hd / 16, lanes = lanes_for((Hq + Hkv) * lph);
  const int need = ((Hq + Hkv) * lph + lanes - 1) / lanes;
  const int passes = need <= 2 ? need : 4;
  const int per = kThreads / lanes, chunk = passes * lanes / lph;  // rows and heads per CTA
  // several rows per thread once the GPU is full (3 CTAs per SM): above one took 86 us, up
  // to four 66, up to eight 70
  const int rows = std::max(1, std::min(4, cap / (per * 3 * num_sms())));
  const dim3 grid((unsigned)((cap + per * rows - 1) / (per * rows)), (unsigned)((Hq + Hkv + chunk - 1) / chunk));
  auto go = [&](auto hd_c) {
    constexpr int HD = decltype(hd_c)::value;
    if (passes == 1) return launch(qk_norm_rope_kernel<HD, 1>, grid, s, A, lanes, rows);
    if (passes == 2) return launch(qk_norm_rope_kernel<HD, 2>, grid, s, A, lanes, rows);
    return launch(qk_norm_rope_kernel<HD, 4>, grid, s, A, lanes, rows);
  };
  return hd == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
}

cudaError_t launch_kv8_write(const Kv8RowMap& m, const __nv_bfloat16* k, size_t ldk,
                             const __nv_bfloat16* v, size_t ldv, uint8_t* k8, float* ks,
                             uint8_t* v8, float* vs, int Hkv, int hd, int block, cudaStream_t s) {
  if (m.M_cap <= 0) return cudaSuccess;
  const int nblk = (m.N + block - 1) / block;
  // heads per CTA: fewer repeat the list's way, more leave a longer tail (308 of 1536 rows:
  // 4 heads 60 us, 8 55, 16 57; all rows: 213, 214, 225)
  const int hpc = std::min(Hkv, 8);
  const int groups = (Hkv + hpc - 1) / hpc;
  WriteArgs A{rows_of(m), {k, v}, {ldk, ldv}, {k8, v8}, {ks, vs}, Hkv, log2_of(block), nblk, hpc, groups};
  ProfScope prof("kv8_write", s);
  const unsigned grid = (unsigned)((size_t)m.B * nblk * groups);
  return hd == 128 ? launch(kv8_write_kernel<128>, grid, s, A) : launch(kv8_write_kernel<64>, grid, s, A);
}

cudaError_t launch_kv8_read(const Kv8RowMap& m, const uint8_t* k8, const float* ks,
                            const uint8_t* v8, const float* vs, __nv_bfloat16* k, size_t ldk,
                            __nv_bfloat16* v, size_t ldv, int Hkv, int hd, int block,
                            cudaStream_t s) {
  if (m.M_cap <= 0) return cudaSuccess;
  const int nblk = (m.N + block - 1) / block;
  ReadArgs A{rows_of(m), m.row_seq, {k8, v8}, {ks, vs}, {k, v}, {ldk, ldv}, Hkv, log2_of(hd),
             log2_of(block), nblk};
  ProfScope prof("kv8_read", s);
  const int lanes = lanes_for(Hkv * hd / 16);
  const int per = kThreads / lanes;
  // several rows per CTA once the GPU is full (8 CTAs per SM): at 32 x 1536 rows up to four
  // take 200 us, one 204, up to eight 206
  const int rows = std::max(1, std::min(4, m.M_cap / (per * 8 * num_sms())));
  return launch(kv8_read_kernel, (unsigned)((m.M_cap + per * rows - 1) / (per * rows)), s, A, lanes, rows);
}

}  // namespace dllm
