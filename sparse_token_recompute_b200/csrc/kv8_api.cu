// C entry points of the 8-bit K/V cache operators: argument checks, then one
// launch (two for an attention whose keys are shared among CTAs).
#include <math.h>

#include <algorithm>

#include "../../include/dllm.h"
#include "internal.h"

using namespace dllm;

namespace {

constexpr size_t kHeader = 256;                 // device status word at offset 0
constexpr long long kMaxRows = 1LL << 30;       // B * k_cap
constexpr int kMaxN = 1 << 30;                  // positions of a sequence
constexpr long long kMaxGrid = 0x7fffffffLL;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline dllm_status status_of(cudaError_t e) {
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? DLLM_OK : DLLM_ERR_CUDA;
}
inline bool block_ok(int block) { return block == 16 || block == 32 || block == 64 || block == 128; }
inline long long blocks_of(int N, int block) { return ((long long)N + block - 1) / block; }

// what the calls share: sizes of the rows and heads, and the optional workspace
dllm_status check_rows(const int32_t* idx, const int32_t* count, int k_cap, int B, int N, int Hkv,
                       int hd, const void* ws, size_t ws_bytes) {
  if (B < 0 || N < 0 || k_cap < 1 || Hkv <= 0 || hd <= 0) return DLLM_ERR_INVALID_ARG;
  if ((long long)B * k_cap > kMaxRows || (long long)Hkv * hd > (1 << 24) || N > kMaxN)
    return DLLM_ERR_UNSUPPORTED_SHAPE;
  if (!idx && !count && k_cap > N) return DLLM_ERR_CAPACITY;  // more rows than positions
  if (!aligned(idx, 4) || !aligned(count, 4)) return DLLM_ERR_INVALID_ARG;
  if (ws && (ws_bytes < kHeader || !aligned(ws, 256))) return DLLM_ERR_WORKSPACE;
  return DLLM_OK;
}

Kv8RowMap row_map(const int32_t* idx, const int32_t* count, int k_cap, int B, int N, void* ws) {
  Kv8RowMap m{};
  m.idx = idx;
  m.count = count;
  m.B = B;
  m.k_cap = k_cap;
  m.N = N;
  m.M_cap = B * k_cap;
  m.status = static_cast<int*>(ws);
  return m;
}

dllm_status check_cache(const void* k8, const float* ks, const void* v8, const float* vs) {
  if (!k8 || !ks || !v8 || !vs) return DLLM_ERR_INVALID_ARG;
  if (!aligned(k8, 16) || !aligned(v8, 16) || !aligned(ks, 4) || !aligned(vs, 4))
    return DLLM_ERR_INVALID_ARG;
  return DLLM_OK;
}

inline bool ld_ok(int ld, int width, int step) { return ld >= width && ld % step == 0; }

}  // namespace

extern "C" dllm_status dllm_rope_table(float* table, int N, int head_dim, float theta,
                                       dllm_stream_t stream) {
  if (N < 0 || head_dim <= 0 || head_dim % 2 || !(theta > 0.f) || theta == INFINITY)
    return DLLM_ERR_INVALID_ARG;
  if (N == 0) return DLLM_OK;
  if (!table || !aligned(table, 16)) return DLLM_ERR_INVALID_ARG;
  launch_rope_table(reinterpret_cast<float2*>(table), N, head_dim, theta,
                    reinterpret_cast<cudaStream_t>(stream));
  return status_of(cudaSuccess);
}

extern "C" dllm_status dllm_qk_norm_rope(const void* q, int ldq, const void* k, int ldk,
                                         int k_in_is_cache, const void* q_gain,
                                         const void* k_gain, const float* rope, void* q_out,
                                         int ldqo, void* k_out, int ldko, int k_out_is_cache,
                                         const int32_t* idx, const int32_t* count, int k_cap,
                                         int B, int N, int n_heads, int n_kv_heads, int head_dim,
                                         float eps, int dtype, void* ws, size_t ws_bytes,
                                         dllm_stream_t stream) {
  if (dtype != DLLM_F32 && dtype != DLLM_BF16) return DLLM_ERR_INVALID_ARG;
  if (n_heads <= 0 || !(eps >= 0.f) || eps == INFINITY) return DLLM_ERR_INVALID_ARG;
  const dllm_status st = check_rows(idx, count, k_cap, B, N, n_kv_heads, head_dim, ws, ws_bytes);
  if (st != DLLM_OK) return st;
  if (n_heads % n_kv_heads || (long long)n_heads * head_dim > (1 << 24)) return DLLM_ERR_UNSUPPORTED_SHAPE;
  const bool bf = dtype == DLLM_BF16;
  if (bf ? (head_dim != 64 && head_dim != 128) : (head_dim % 2 || head_dim > 256))
    return DLLM_ERR_UNSUPPORTED_SHAPE;
  if (!bf && ((long long)B * k_cap * (n_heads + n_kv_heads) + 7) / 8 > kMaxGrid)
    return DLLM_ERR_UNSUPPORTED_SHAPE;
  if (B == 0 || N == 0) return DLLM_OK;
  if (!q || !k || !q_gain || !k_gain || !q_out || !k_out) return DLLM_ERR_INVALID_ARG;
  for (const void* p : {q, k, q_gain, k_gain, static_cast<const void*>(q_out),
                        static_cast<const void*>(k_out)})
    if (!aligned(p, bf ? 16 : 4)) return DLLM_ERR_INVALID_ARG;
  if (!aligned(rope, 16)) return DLLM_ERR_INVALID_ARG;
  const int step = bf ? 8 : 1, wq = n_heads * head_dim, wk = n_kv_heads * head_dim;
  if (!ld_ok(ldq, wq, step) || !ld_ok(ldqo, wq, step) || (!k_in_is_cache && !ld_ok(ldk, wk, step)) ||
      (!k_out_is_cache && !ld_ok(ldko, wk, step)))
    return DLLM_ERR_INVALID_ARG;
  return status_of(launch_qk_norm_rope(row_map(idx, count, k_cap, B, N, ws), q, ldq, k, ldk, q_out,
                                       ldqo, k_out, ldko, q_gain, k_gain,
                                       reinterpret_cast<const float2*>(rope), n_heads, n_kv_heads,
                                       head_dim, eps, bf, k_in_is_cache != 0, k_out_is_cache != 0,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" size_t dllm_kv8_scale_count(int B, int N, int n_kv_heads, int block) {
  if (B < 0 || N < 0 || n_kv_heads <= 0 || !block_ok(block)) return 0;
  return (size_t)B * n_kv_heads * blocks_of(N, block);
}

extern "C" dllm_status dllm_kv8_write(const void* k, int ldk, const void* v, int ldv,
                                      const int32_t* idx, const int32_t* count, int k_cap, int B,
                                      int N, int n_kv_heads, int head_dim, int block, void* k8,
                                      float* k_scale, void* v8, float* v_scale, void* ws,
                                      size_t ws_bytes, dllm_stream_t stream) {
  dllm_status st = check_rows(idx, count, k_cap, B, N, n_kv_heads, head_dim, ws, ws_bytes);
  if (st != DLLM_OK) return st;
  if ((head_dim != 64 && head_dim != 128) || !block_ok(block)) return DLLM_ERR_UNSUPPORTED_SHAPE;
  if ((long long)B * n_kv_heads > kMaxGrid / std::max(1LL, blocks_of(N, block)))
    return DLLM_ERR_UNSUPPORTED_SHAPE;
  if (B == 0 || N == 0) return DLLM_OK;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return DLLM_ERR_INVALID_ARG;
  if ((st = check_cache(k8, k_scale, v8, v_scale)) != DLLM_OK) return st;
  if (!ld_ok(ldk, n_kv_heads * head_dim, 8) || !ld_ok(ldv, n_kv_heads * head_dim, 8))
    return DLLM_ERR_INVALID_ARG;
  using bf = __nv_bfloat16;
  return status_of(launch_kv8_write(row_map(idx, count, k_cap, B, N, ws), static_cast<const bf*>(k),
                                    ldk, static_cast<const bf*>(v), ldv, static_cast<uint8_t*>(k8),
                                    k_scale, static_cast<uint8_t*>(v8), v_scale, n_kv_heads,
                                    head_dim, block, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" dllm_status dllm_kv8_read(const void* k8, const float* k_scale, const void* v8,
                                     const float* v_scale, const int32_t* idx,
                                     const int32_t* count, int k_cap, int B, int N,
                                     int n_kv_heads, int head_dim, int block, void* k_out,
                                     int ldk, void* v_out, int ldv, void* ws, size_t ws_bytes,
                                     dllm_stream_t stream) {
  dllm_status st = check_rows(idx, count, k_cap, B, N, n_kv_heads, head_dim, ws, ws_bytes);
  if (st != DLLM_OK) return st;
  if ((head_dim != 64 && head_dim != 128) || !block_ok(block)) return DLLM_ERR_UNSUPPORTED_SHAPE;
  if (B == 0 || N == 0) return DLLM_OK;
  if (!k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16)) return DLLM_ERR_INVALID_ARG;
  if ((st = check_cache(k8, k_scale, v8, v_scale)) != DLLM_OK) return st;
  if (!ld_ok(ldk, n_kv_heads * head_dim, 8) || !ld_ok(ldv, n_kv_heads * head_dim, 8))
    return DLLM_ERR_INVALID_ARG;
  using bf = __nv_bfloat16;
  return status_of(launch_kv8_read(row_map(idx, count, k_cap, B, N, ws),
                                   static_cast<const uint8_t*>(k8), k_scale,
                                   static_cast<const uint8_t*>(v8), v_scale,
                                   static_cast<bf*>(k_out), ldk, static_cast<bf*>(v_out), ldv,
                                   n_kv_heads, head_dim, block,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" size_t dllm_attention_kv8_workspace_size(int B, int k_cap, int N, int n_heads,
                                                    int n_kv_heads, int head_dim) {
  if (B <= 0 || k_cap < 1 || N < 0 || N > kMaxN || n_heads <= 0 || n_kv_heads <= 0 ||
      n_heads % n_kv_heads || head_dim <= 0 || (long long)B * k_cap > kMaxRows ||
      (long long)B * k_cap * n_heads >= kMaxGrid)
    return kHeader;
  return kHeader + attention_kv8_part_bytes(B, k_cap, N, n_heads, n_kv_heads, head_dim);
}

extern "C" dllm_status dllm_attention_kv8(const void* q, const void* k8, const float* k_scale,
                                          const void* v8, const float* v_scale, void* o, float* m,
                                          float* l, const int32_t* count, const int32_t* kv_len,
                                          int B, int k_cap, int N, int n_heads, int n_kv_heads,
                                          int head_dim, int block, void* ws, size_t ws_bytes,
                                          dllm_stream_t stream) {
  if (B < 0 || k_cap < 1 || N < 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0)
    return DLLM_ERR_INVALID_ARG;
  if (n_heads % n_kv_heads || (head_dim != 64 && head_dim != 128) || !block_ok(block) ||
      (long long)B * k_cap > kMaxRows || (long long)n_heads * head_dim > (1 << 24) || N > kMaxN ||
      (long long)B * k_cap * n_heads >= kMaxGrid)
    return DLLM_ERR_UNSUPPORTED_SHAPE;
  if (B == 0) return DLLM_OK;
  if (!q || !o || (m == nullptr) != (l == nullptr)) return DLLM_ERR_INVALID_ARG;
  for (const void* p : {q, static_cast<const void*>(o)})
    if (!aligned(p, 16)) return DLLM_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(count), static_cast<const void*>(kv_len),
                        static_cast<const void*>(m), static_cast<const void*>(l)})
    if (!aligned(p, 4)) return DLLM_ERR_INVALID_ARG;
  if (N > 0) {
    const dllm_status st = check_cache(k8, k_scale, v8, v_scale);
    if (st != DLLM_OK) return st;
  }
  const size_t need = dllm_attention_kv8_workspace_size(B, k_cap, N, n_heads, n_kv_heads, head_dim);
  if (!ws || !aligned(ws, 256) || ws_bytes < need) return DLLM_ERR_WORKSPACE;
  const Kv8AttnPlan pl = attention_kv8_plan(B, k_cap, N, n_heads, n_kv_heads, head_dim,
                                            (size_t)B * k_cap, need - kHeader);
  if (pl.ctas > kMaxGrid) return DLLM_ERR_UNSUPPORTED_SHAPE;
  using bf = __nv_bfloat16;
  return status_of(launch_attention_kv8(
      row_map(nullptr, count, k_cap, B, N, ws), static_cast<const bf*>(q),
      static_cast<const uint8_t*>(k8), k_scale, static_cast<const uint8_t*>(v8), v_scale,
      static_cast<bf*>(o), kv_len, n_heads, n_kv_heads, head_dim, block,
      reinterpret_cast<float*>(static_cast<char*>(ws) + kHeader), need - kHeader, m, l,
      reinterpret_cast<cudaStream_t>(stream)));
}
