// Kernels around the 8-bit K/V cache: the q/k norm with the position rotation,
// writing selected rows into the cache, and reading rows back.  All three are
// bound by HBM (or, for a handful of rows, by the latency of a launch).
#include <algorithm>

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

// compact row, sequence and position of row `j` of sequence `b` (idx/count) or of
// compact row `x` (row maps); false: no such row, or a position outside the sequence
__device__ __forceinline__ bool norm_row(const NormArgs& A, int x, int& r, int& seq, int& pos) {
  const Kv8Rows& R = A.rows;
  if (R.row_off) {
    r = x;
    if (x >= R.row_off[R.B]) return false;
    seq = A.row_seq[x];
    pos = R.row_pos[x];
    return true;
  }
  seq = x / R.k_cap;
  const int j = x - seq * R.k_cap;
  int off, n;
  kv8_seq_rows(R, seq, off, n);
  if (j >= n) return false;
  r = off + j;
  pos = j;
  if (R.idx) {
    const int32_t* l = R.idx + (size_t)seq * R.k_cap;
    pos = l[j];
    if ((pos < 0 || pos >= R.N || (j > 0 && l[j - 1] >= pos)) && (threadIdx.x & 31) == 0)
      raise_status(R.status, DEV_BAD_INDEX);
  } else if (j >= R.N && (threadIdx.x & 31) == 0) {
    raise_status(R.status, DEV_BAD_INDEX);
  }
  return pos >= 0 && pos < R.N;
}

// Head vectors of HD bf16: HD/16 lanes per head, each with 8 elements j.. of the
// first half and their partners j + HD/2.., so that the rotation is in one lane
// and a head's sum of squares is 2 or 3 shuffles.  A row's heads (queries, then
// keys) are spread over `lanes` threads; the sums, the norm and the rotation are
// fp32, rounded once when stored.
template <int HD>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const NormArgs A, int lanes) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int LPH = HD / 16;
  const int per_cta = kThreads / lanes;
  const int x = blockIdx.x * per_cta + threadIdx.x / lanes;
  const int total = A.rows.row_off ? 0x7fffffff : A.rows.B * A.rows.k_cap;
  int r, seq, pos;
  if (x >= total || !norm_row(A, x, r, seq, pos)) return;
  const int l = threadIdx.x % lanes;
  const int e = (l % LPH) * 8;  // first element of this lane in each half
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  if (A.rope) {
    const float4* t = reinterpret_cast<const float4*>(A.rope + (size_t)pos * (HD / 2) + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldg(t + i);
      cs[2 * i] = v.x, sn[2 * i] = v.y, cs[2 * i + 1] = v.z, sn[2 * i + 1] = v.w;
    }
  }
  const size_t cache_row = (size_t)seq * A.rows.N + pos;
  using bf = __nv_bfloat16;
  const bf* qi = static_cast<const bf*>(A.q) + (size_t)r * A.ldq;
  const bf* ki = static_cast<const bf*>(A.k) + (A.k_in_cache ? cache_row * A.Hkv * HD : (size_t)r * A.ldk);
  bf* qo = static_cast<bf*>(A.q_out) + (size_t)r * A.ldqo;
  bf* ko = static_cast<bf*>(A.k_out) + (A.k_out_cache ? cache_row * A.Hkv * HD : (size_t)r * A.ldko);
  const int heads = A.Hq + A.Hkv;
  for (int h = l / LPH; h < heads; h += lanes / LPH) {
    const bool is_q = h < A.Hq;
    const size_t at = (size_t)(is_q ? h : h - A.Hq) * HD + e;
    const bf* src = (is_q ? qi : ki) + at;
    bf* dst = (is_q ? qo : ko) + at;
    const bf* gain = static_cast<const bf*>(is_q ? A.q_gain : A.k_gain) + e;
    float a[8], b[8], g[8];
    unpack8(*reinterpret_cast<const uint4*>(src), a);
    unpack8(*reinterpret_cast<const uint4*>(src + HD / 2), b);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
    // the lanes of one head: every head of a warp's pass exists or none of its lanes does
    const unsigned group = ((1u << LPH) - 1u) << ((threadIdx.x & 31) / LPH * LPH);
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
    const float rs = rsqrtf(ss * (1.0f / HD) + A.eps);
    unpack8(__ldg(reinterpret_cast<const uint4*>(gain)), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = a[i] * rs * g[i];
    unpack8(__ldg(reinterpret_cast<const uint4*>(gain + HD / 2)), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = b[i] * rs * g[i];
    float y[8], z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = a[i] * cs[i] - b[i] * sn[i];
      z[i] = b[i] * cs[i] + a[i] * sn[i];
    }
    *reinterpret_cast<uint4*>(dst) = pack8(y);
    *reinterpret_cast<uint4*>(dst + HD / 2) = pack8(z);
  }
}

// fp32 rows (small models, any even head_dim up to 256): one warp per row and head
__global__ void __launch_bounds__(kThreads) qk_norm_rope_f32_kernel(const NormArgs A, int HD) {
  const int heads = A.Hq + A.Hkv;
  const size_t u = (size_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int x = (int)(u / heads), h = (int)(u % heads);
  int r, seq, pos;
  if (!A.rows.row_off && x >= A.rows.B * A.rows.k_cap) return;
  if (!norm_row(A, x, r, seq, pos)) return;
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
// rows that fall in its block; then each warp takes one (head, K or V) at a time:
// largest magnitude of the new rows, the block's scale, encode and store.  Tokens
// that are kept are read only where the scale grew.
template <int HD>
__global__ void __launch_bounds__(kThreads) kv8_write_kernel(const WriteArgs A) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int LPR = HD / 8;       // lanes per bf16 row (16 bytes each)
  constexpr int RPL = 32 / LPR;     // rows per load of a warp
  constexpr int NL = 8;             // loads that stay in registers: RPL * NL rows
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
  __shared__ uint8_t s_new_tok[128];
  __shared__ int s_first, s_off, s_n, s_cnt[4];
  if (threadIdx.x < 128) s_row[threadIdx.x] = -1;
  if (warp == 0) {
    int off, n;
    kv8_seq_rows(R, b, off, n);
    const int* list = R.row_off ? R.row_pos + off : (R.idx ? R.idx + (size_t)b * R.k_cap : nullptr);
    const int first = list ? warp_lower_bound(list, n, p0) : min(p0, n);
    if (lane == 0) s_first = first, s_off = off, s_n = n;
  }
  __syncthreads();
  const int off = s_off, n = s_n, first = s_first;
  const int* list = R.row_off ? R.row_pos + off : (R.idx ? R.idx + (size_t)b * R.k_cap : nullptr);
  if (!R.row_off && R.status && blk == 0 && grp == 0) {  // one CTA per sequence looks the list over
    for (int j = threadIdx.x; j < n; j += kThreads) {
      const int p = list ? list[j] : j;
      if (p < 0 || p >= R.N || (list && j > 0 && list[j - 1] >= p))
        raise_status(R.status, DEV_BAD_INDEX);
    }
  }
  if (threadIdx.x < block) {
    const int j = first + threadIdx.x;
    if (j < n) {
      const int t = (list ? list[j] : j) - p0;
      if (t >= 0 && t < tokens) atomicMax(&s_row[t], off + j);  // a repeated position: the later row
    }
  }
  __syncthreads();
  const int mine = threadIdx.x < 128 ? s_row[threadIdx.x] : -1;
  const unsigned has = __ballot_sync(0xffffffffu, mine >= 0);
  if (lane == 0 && warp < 4) s_cnt[warp] = __popc(has);
  __syncthreads();
  const int n_new = s_cnt[0] + s_cnt[1] + s_cnt[2] + s_cnt[3];
  if (n_new == 0) return;
  if (mine >= 0) {
    int at = __popc(has & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) at += s_cnt[w];
    s_new_row[at] = mine;
    s_new_tok[at] = (uint8_t)threadIdx.x;
  }
  __syncthreads();

  const int h0 = grp * A.hpc, h1 = min(A.Hkv, h0 + A.hpc);
  const int sub = lane / LPR, e = (lane % LPR) * 8;
  for (int u = warp; u < 2 * (h1 - h0); u += kThreads / 32) {
    const int kv = u & 1, h = h0 + (u >> 1);
    const __nv_bfloat16* src = A.x[kv] + (size_t)h * HD + e;
    uint8_t* dst = A.c8[kv] + (((size_t)b * R.N + p0) * A.Hkv + h) * HD;
    float* sp = A.scale[kv] + ((size_t)b * A.Hkv + h) * A.nblk + blk;
    const float s_old = *sp;
    uint4 v[NL];
    uint32_t mx = 0;  // two running maxima of |x| as bf16 bits
    auto load = [&](int base) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int k = base + i * RPL + sub;
        v[i] = make_uint4(0, 0, 0, 0);
        if (k < n_new)
          v[i] = *reinterpret_cast<const uint4*>(src + (size_t)s_new_row[k] * A.ld[kv]);
      }
    };
    auto magnitude = [&]() {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        mx = __vmaxu2(mx, v[i].x & 0x7fff7fffu);
        mx = __vmaxu2(mx, v[i].y & 0x7fff7fffu);
        mx = __vmaxu2(mx, v[i].z & 0x7fff7fffu);
        mx = __vmaxu2(mx, v[i].w & 0x7fff7fffu);
      }
    };
    const bool once = n_new <= NL * RPL;
    for (int base = 0; base < n_new; base += NL * RPL) {
      load(base);
      magnitude();
    }
    uint32_t top = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
    const bool odd = top >= 0x7f80u;  // an infinity or NaN among them: they do not count
    if (odd) {
      top = 0;
      for (int k = sub; k < n_new; k += RPL) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + (size_t)s_new_row[k] * A.ld[kv]);
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo = q[i] & 0x7fffu, hi = (q[i] >> 16) & 0x7fffu;
          if (lo < 0x7f80u) top = max(top, lo);
          if (hi < 0x7f80u) top = max(top, hi);
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
    }
    const float amax = __uint_as_float(top << 16);
    const bool had = s_old >= kKv8MinScale;  // (false for NaN) the block holds rows already
    const bool same = n_new < tokens && had && amax <= kE4m3Max * s_old;
    const float s = same ? s_old : kv8_scale_for(amax);
    const float inv = kv8_inverse(s);
    auto store = [&](int base) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int k = base + i * RPL + sub;
        if (k >= n_new) continue;
        float f[8];
        unpack8(v[i], f);
#pragma unroll
        for (int t = 0; t < 8; ++t) f[t] *= inv;
        if (odd) {
#pragma unroll
          for (int t = 0; t < 8; ++t)
            if (isinf(f[t])) f[t] = __uint_as_float(0x7fffffffu);
        }
        uint2 c;
        c.x = floats_to_e4m3x2(f[0], f[1]) | floats_to_e4m3x2(f[2], f[3]) << 16;
        c.y = floats_to_e4m3x2(f[4], f[5]) | floats_to_e4m3x2(f[6], f[7]) << 16;
        *reinterpret_cast<uint2*>(dst + (size_t)s_new_tok[k] * A.Hkv * HD + e) = c;
      }
    };
    if (once) {
      store(0);
    } else {  // more rows than the registers hold: a second look, from the caches
      for (int base = 0; base < n_new; base += NL * RPL) {
        load(base);
        store(base);
      }
    }
    if (!same) {
      if (lane == 0) *sp = s;
      // the kept tokens at the new scale (a block without rows yet: zeros)
      const float f = had ? s_old * inv : 0.f;
      for (int t = lane / LPO; t < tokens; t += RPO) {
        if (s_row[t] >= 0) continue;
        uint4* at = reinterpret_cast<uint4*>(dst + (size_t)t * A.Hkv * HD + (lane % LPO) * 16);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (had) {
          w = *at;
          uint32_t* q = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 lo = e4m3x2_to_float2(q[i]), hi = e4m3x2_to_float2(q[i] >> 16);
            q[i] = floats_to_e4m3x2(lo.x * f, lo.y * f) | floats_to_e4m3x2(hi.x * f, hi.y * f) << 16;
          }
        }
        *at = w;
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

// `lanes` threads per row, 16 codes of K and of V each per turn
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const ReadArgs A, int lanes) {
  griddep_launch_dependents();
  griddep_wait();
  const Kv8Rows& R = A.rows;
  const int x = blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
  int r, seq, pos;
  if (R.row_off) {
    if (x >= R.row_off[R.B]) return;
    r = x, seq = A.row_seq[x], pos = R.row_pos[x];
  } else {
    if (x >= R.B * R.k_cap) return;
    seq = x / R.k_cap;
    const int j = x - seq * R.k_cap;
    int off, n;
    kv8_seq_rows(R, seq, off, n);
    if (j >= n) return;
    r = off + j;
    const int32_t* l = R.idx ? R.idx + (size_t)seq * R.k_cap : nullptr;
    pos = l ? l[j] : j;
    if ((pos < 0 || pos >= R.N || (l && j > 0 && l[j - 1] >= pos)) && (threadIdx.x & 31) == 0)
      raise_status(R.status, DEV_BAD_INDEX);
    if (pos < 0 || pos >= R.N) return;
  }
  const int vecs = (A.Hkv << A.hd_log2) >> 4;
  const size_t in = ((size_t)seq * R.N + pos) * vecs;
  for (int i = threadIdx.x % lanes; i < vecs; i += lanes) {
    const size_t sc = ((size_t)seq * A.Hkv + ((i << 4) >> A.hd_log2)) * A.nblk + (pos >> A.blk_log2);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(A.c8[kv]) + in + i);
      const float s = __ldg(A.scale[kv] + sc);
      const uint32_t q[4] = {w.x, w.y, w.z, w.w};
      float f[16];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float2 lo = e4m3x2_to_float2(q[t]), hi = e4m3x2_to_float2(q[t] >> 16);
        f[4 * t] = lo.x * s, f[4 * t + 1] = lo.y * s, f[4 * t + 2] = hi.x * s, f[4 * t + 3] = hi.y * s;
      }
      uint4* dst = reinterpret_cast<uint4*>(A.out[kv] + (size_t)r * A.ld[kv] + i * 16);
      dst[0] = pack8(f);
      dst[1] = pack8(f + 8);
    }
  }
}

int log2_of(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

template <typename K, typename... Args>
cudaError_t launch(K kernel, unsigned grid, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
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
  const int lanes = lanes_for((Hq + Hkv) * (hd / 16));
  const unsigned grid = (unsigned)((cap + kThreads / lanes - 1) / (kThreads / lanes));
  return hd == 128 ? launch(qk_norm_rope_kernel<128>, grid, s, A, lanes)
                   : launch(qk_norm_rope_kernel<64>, grid, s, A, lanes);
}

cudaError_t launch_kv8_write(const Kv8RowMap& m, const __nv_bfloat16* k, size_t ldk,
                             const __nv_bfloat16* v, size_t ldv, uint8_t* k8, float* ks,
                             uint8_t* v8, float* vs, int Hkv, int hd, int block, cudaStream_t s) {
  if (m.M_cap <= 0) return cudaSuccess;
  const int nblk = (m.N + block - 1) / block;
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
  return launch(kv8_read_kernel, (unsigned)((m.M_cap + per - 1) / per), s, A, lanes);
}

}  // namespace dllm
