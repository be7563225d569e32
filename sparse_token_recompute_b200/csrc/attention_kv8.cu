// Attention of compact query rows over the 8-bit K/V cache.
//
// Sequence b's query rows attend to its first kv_len[b] cached keys, no mask:
// O = softmax(Q K^T / sqrt(hd)) V with K = k8 * ks, V = v8 * vs, one scale per
// (sequence, kv head, block of tokens).  A sequence without keys gives zeros.
//
// The query rows of one sequence and kv head are packed: packed row r is
// (compact row r / G, query head g * G + r % G), G query heads per kv head, so
// one pass over the keys serves all G heads.
//
// Products run on f16 operands, which hold exactly what they stand for:
//   codes   an e4m3 code is exact in f16 (3 mantissa bits, 2^-9 .. 448);
//   queries a bf16 row times the power of two that brings its largest element
//           to [2^14, 2^15): 8 bits fit f16's 11, and elements down to 2^-28
//           of the largest stay normal numbers;
//   P       exp2(score - reference), rounded to f16's 11 bits (bf16 would keep 8).
// The K scale multiplies the fp32 score.  The V scale 2^e of a key's block is an
// addend of its exponent: with x_j = score_j + e_j (log2 units) and a reference
// r at most 8 below the largest x_j,
//   O = sum_j 2^(x_j - r) v8_j,   l = sum_j 2^(x_j - r) 2^-e_j,   out = O / l,
// so that the keys with the largest weight * scale have the weights near 1, and
// f16's range is kept however far apart the blocks' scales are.
#include <algorithm>

#include "attention_kv8.cuh"

namespace dllm {

namespace {

// D(16x8) += A(16x16) B(16x8), f16 in, fp32 accumulate
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- few query rows

// packed query rows per (sequence, kv head) that still run here
constexpr int kKv8TcRows = 16;
constexpr int RW = 4;        // warps per CTA
constexpr int RM = 16;       // packed query rows per CTA
constexpr int RK = 16;       // keys per warp and turn

template <int HD>
struct RowsSmem {
  static constexpr int VB = HD / 8;                     // V bytes per lane and key
  static constexpr int V_OFF = 32 * (HD / 2);           // K codes of 16 keys, then V's,
  static constexpr int SC_OFF = V_OFF + 32 * 4 * VB;    // then the two scales
  static constexpr int STAGE = SC_OFF + 16;
  static constexpr int STAGES = HD == 128 ? 5 : 8;
  static constexpr int WARP = STAGE * STAGES;
  static constexpr int RED = RW * RM * HD * 4;          // outputs of the warps
  static constexpr int ML_OFF = RW * WARP > RED ? RW * WARP : RED;
  static constexpr int TOTAL = ML_OFF + RW * RM * 2 * 4;
};

// One CTA = up to 16 packed query rows of one (sequence, kv head) and one share of
// the keys; its warps take 16 keys each in turn.  A warp's codes go through a ring
// of cp.async copies in shared memory in which every lane reads back what it
// copied itself, laid out so that a lane's 16 bytes are its mma fragments: K along
// the head (any order of the inner index serves a product as long as Q has the
// same), V by gathering one byte of two neighbouring keys.  The codes are thus
// read once, converted in registers (one cvt per two codes), and never written
// back.
template <int HD>
__global__ void __launch_bounds__(RW * 32) attn_kv8_rows_kernel(const Kv8Args A) {
  griddep_launch_dependents();
  griddep_wait();
  using L = RowsSmem<HD>;
  constexpr int KS = HD / 16;    // k-steps of Q K^T
  constexpr int NT = HD / 8;     // n-tiles of P V
  constexpr int KV16 = HD / 64;  // 16-byte pieces of a key row per lane
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  int u = blockIdx.x;
  const int share = u % A.S;
  u /= A.S;
  const int tile = u % A.tiles;
  u /= A.tiles;
  const int kvh = u % A.Hkv, b = u / A.Hkv;
  int off, cnt;
  kv8_seq_rows(A.rows, b, off, cnt);
  const int R = cnt * A.G - tile * RM;  // packed rows left
  if (R <= 0) return;
  const int N = A.rows.N;
  int len = N;
  if (A.kv_len) {
    const int want = A.kv_len[b];
    len = min(max(want, 0), N);
    if (len != want && threadIdx.x == 0) raise_status(A.rows.status, DEV_BAD_SHAPE);
  }
  const int chunks = (len + RK - 1) / RK;
  const int per = (chunks + A.S - 1) / A.S;
  const int c_lo = min(chunks, share * per), c_hi = min(chunks, c_lo + per);

  const uint32_t ring = smem_u32(smem) + warp * L::WARP;
  const uint8_t* kbase = A.k8 + ((size_t)b * N * A.Hkv + kvh) * HD;
  const uint8_t* vbase = A.v8 + ((size_t)b * N * A.Hkv + kvh) * HD;
  const size_t row_bytes = (size_t)A.Hkv * HD;
  const size_t sc0 = ((size_t)b * A.Hkv + kvh) * A.nblk;
  // keys past the last one arrive as zeros (copies of 0 bytes from a valid row)
  auto issue = [&](int c, int slot) {
    if (c < c_hi) {
      const uint32_t st = ring + slot * L::STAGE;
      const int k0 = c * RK;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int key = k0 + n * 8 + g;
        const uint8_t* src = kbase + (size_t)min(key, len - 1) * row_bytes + t * 16;
#pragma unroll
        for (int i = 0; i < KV16; ++i)
          cp_async16(st + ((n * KV16 + i) * 32 + lane) * 16, src + i * 64, key < len);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = k0 + 2 * t + (i & 1) + (i >> 1) * 8;
        const uint8_t* src = vbase + (size_t)min(key, len - 1) * row_bytes + g * L::VB;
        if constexpr (HD == 128)
          cp_async16(st + L::V_OFF + (i * 32 + lane) * 16, src, key < len);
        else
          cp_async8(st + L::V_OFF + (i * 32 + lane) * 8, src, key < len);
      }
      if (lane < 2)
        cp_async4(st + L::SC_OFF + lane * 4, (lane == 0 ? A.ks : A.vs) + sc0 + (k0 >> A.blk_log2));
    }
    cp_commit();
  };
  // the ring's first copies are on their way before the queries are read
#pragma unroll
  for (int i = 0; i < L::STAGES - 1; ++i) issue(c_lo + warp + i * RW, i);

  // Q fragments of packed rows g and g + 8: in k-step i of a half of 64 elements, lane
  // t holds elements 16 t + 4 i .. + 3
  uint32_t qf[KS][4];
  float rs[2];  // log2 units per raw score of rows g, g + 8
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = tile * RM + g + 8 * i;
    const bool there = g + 8 * i < R;
    const size_t row = (size_t)(off + r / A.G) * A.Hq + kvh * A.G + r % A.G;
    uint4 raw[KV16][2];
    uint32_t mx = 0;
#pragma unroll
    for (int p = 0; p < KV16; ++p) {
      const uint4* src = reinterpret_cast<const uint4*>(A.q + row * HD + p * 64 + t * 16);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        raw[p][w] = there ? src[w] : make_uint4(0, 0, 0, 0);
        mx = __vmaxu2(mx, raw[p][w].x & 0x7fff7fffu);
        mx = __vmaxu2(mx, raw[p][w].y & 0x7fff7fffu);
        mx = __vmaxu2(mx, raw[p][w].z & 0x7fff7fffu);
        mx = __vmaxu2(mx, raw[p][w].w & 0x7fff7fffu);
      }
    }
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int sh = query_shift(__uint_as_float(mx << 16));
    // in two factors: the shift itself may lie outside the normal floats' exponents
    const float f0 = pow2i(sh / 2), f1 = pow2i(sh - sh / 2);
    rs[i] = A.scale_log2 * pow2i(-(sh / 2)) * pow2i(-(sh - sh / 2));
#pragma unroll
    for (int p = 0; p < KV16; ++p) {
      float f[16];
      unpack8(raw[p][0], f);
      unpack8(raw[p][1], f + 8);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        qf[p * 4 + e][i] = pack_h2(f[4 * e] * f0 * f1, f[4 * e + 1] * f0 * f1);
        qf[p * 4 + e][2 + i] = pack_h2(f[4 * e + 2] * f0 * f1, f[4 * e + 3] * f0 * f1);
      }
    }
  }

  float o[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  int slot = 0;
  for (int c = c_lo + warp; c < c_hi; c += RW) {
    cp_wait<L::STAGES - 2>();
    __syncwarp();
    issue(c + (L::STAGES - 1) * RW, slot == 0 ? L::STAGES - 1 : slot - 1);
    const uint8_t* st = smem + warp * L::WARP + slot * L::STAGE;
    if (++slot == L::STAGES) slot = 0;
    const float2 sc = *reinterpret_cast<const float2*>(st + L::SC_OFF);
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int p = 0; p < KV16; ++p) {
        const uint4 w = *reinterpret_cast<const uint4*>(st + ((n * KV16 + p) * 32 + lane) * 16);
        const uint32_t q4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma_f16(s[n], qf[p * 4 + e], e4m3x2_to_f16x2(q4[e] & 0xffffu), e4m3x2_to_f16x2(q4[e] >> 16));
      }
    }
    float ev, inv_v;
    v_scale_parts(sc.y, ev, inv_v);
    const float k0 = rs[0] * sc.x, k1 = rs[1] * sc.x;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      s[n][0] = fmaf(s[n][0], k0, ev), s[n][1] = fmaf(s[n][1], k0, ev);
      s[n][2] = fmaf(s[n][2], k1, ev), s[n][3] = fmaf(s[n][3], k1, ev);
    }
    if ((c + 1) * RK > len) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c * RK + n * 8 + 2 * t + (i & 1) >= len) s[n][i] = -INFINITY;
    }
    float alpha[2] = {1.f, 1.f};
    bool grew = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (mx > m[i] + kKv8Lazy) {
        alpha[i] = exp2_approx(m[i] - mx);
        m[i] = mx;
        grew = true;
      }
    }
    if (__any_sync(0xffffffffu, grew)) {
      l[0] *= alpha[0], l[1] *= alpha[1];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        o[n][0] *= alpha[0], o[n][1] *= alpha[0], o[n][2] *= alpha[1], o[n][3] *= alpha[1];
    }
    float p[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) p[n][i] = exp2_approx(s[n][i] - m[i >> 1]);
    l[0] = fmaf((p[0][0] + p[0][1]) + (p[1][0] + p[1][1]), inv_v, l[0]);
    l[1] = fmaf((p[0][2] + p[0][3]) + (p[1][2] + p[1][3]), inv_v, l[1]);
    const uint32_t pa[4] = {pack_h2(p[0][0], p[0][1]), pack_h2(p[0][2], p[0][3]),
                            pack_h2(p[1][0], p[1][1]), pack_h2(p[1][2], p[1][3])};
    uint32_t w[4][L::VB / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* src = st + L::V_OFF + (i * 32 + lane) * L::VB;
      if constexpr (HD == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(src);
        w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(src);
        w[i][0] = x.x, w[i][1] = x.y;
      }
    }
#pragma unroll
    for (int q = 0; q < L::VB / 4; ++q) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {  // columns 4 q + 2 j, + 1: (key, next key) byte pairs
        const uint32_t a = __byte_perm(w[0][q], w[1][q], j ? 0x7362 : 0x5140);
        const uint32_t d = __byte_perm(w[2][q], w[3][q], j ? 0x7362 : 0x5140);
        const uint32_t v[4] = {e4m3x2_to_f16x2(a & 0xffffu), e4m3x2_to_f16x2(d & 0xffffu),
                         e4m3x2_to_f16x2(a >> 16), e4m3x2_to_f16x2(d >> 16)};
        mma_f16(o[q * 4 + 2 * j], pa, v[0], v[1]);
        mma_f16(o[q * 4 + 2 * j + 1], pa, v[2], v[3]);
      }
    }
  }
  cp_wait<0>();
  __syncthreads();  // every ring is done with: the warps' outputs take its place

  float* red = reinterpret_cast<float*>(smem);
  float* ml = reinterpret_cast<float*>(smem + L::ML_OFF);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float sum = l[i];
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (t == 0) {
      float* x = ml + (warp * RM + g + 8 * i) * 2;
      x[0] = m[i], x[1] = sum;
    }
    // n-tile j of lane t: columns 2t * VB + j and (2t + 1) * VB + j
    float* dst = red + (warp * RM + g + 8 * i) * HD + 2 * t * L::VB;
#pragma unroll
    for (int j = 0; j < NT; j += 4) {
      *reinterpret_cast<float4*>(dst + j) =
          make_float4(o[j][2 * i], o[j + 1][2 * i], o[j + 2][2 * i], o[j + 3][2 * i]);
      *reinterpret_cast<float4*>(dst + L::VB + j) = make_float4(
          o[j][2 * i + 1], o[j + 1][2 * i + 1], o[j + 2][2 * i + 1], o[j + 3][2 * i + 1]);
    }
  }
  __syncthreads();
  // 8 outputs per thread and turn: the warps' results in warp order
  for (int i = threadIdx.x; i < RM * (HD / 8); i += RW * 32) {
    const int row = i / (HD / 8), e = (i % (HD / 8)) * 8;
    if (row >= R) break;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < RW; ++w) mx = fmaxf(mx, ml[(w * RM + row) * 2]);
    float sum = 0.f, acc[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] = 0.f;
#pragma unroll
    for (int w = 0; w < RW; ++w) {
      const float* x = ml + (w * RM + row) * 2;
      if (x[1] == 0.f) continue;  // no keys
      const float f = exp2_approx(x[0] - mx);
      sum += x[1] * f;
      const float* src = red + (w * RM + row) * HD + e;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(src[k], f, acc[k]);
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;  // a row without keys: zeros
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] *= inv;
    const int r = tile * RM + row;
    const size_t at = (size_t)(off + r / A.G) * A.Hq + kvh * A.G + r % A.G;
    if (A.S == 1) {
      *reinterpret_cast<uint4*>(A.o + at * HD + e) = pack8(acc);
      if (A.st_m && e == 0) {
        normal_stats(mx, sum);
        A.st_m[at] = mx / kKv8Log2e;
        A.st_l[at] = sum;
      }
    } else {
      const size_t pa = (size_t)share * A.part_rows * A.Hq + at;
      float4* dst = reinterpret_cast<float4*>(A.part_o + pa * HD + e);
      dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (e == 0) {
        normal_stats(mx, sum);
        A.part_ml[pa * 2] = mx;
        A.part_ml[pa * 2 + 1] = sum;
      }
    }
  }
}

// The shares of one output row, in share order: M = max m_s, w_s = l_s 2^(m_s - M),
// O = sum w_s o_s / sum w_s.  One warp per (row, head); an empty share has l = 0.
template <int HD>
__global__ void __launch_bounds__(256) attn_kv8_merge_kernel(const Kv8Args A) {
  constexpr int PER = HD / 32;
  griddep_launch_dependents();
  griddep_wait();
  const size_t u = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  int off, cnt;
  kv8_seq_rows(A.rows, A.rows.B - 1, off, cnt);
  if (u >= (size_t)(off + cnt) * A.Hq) return;
  const size_t stride = (size_t)A.part_rows * A.Hq;
  float mx = -INFINITY;
  for (int s = lane; s < A.S; s += 32) {
    const float2 x = *reinterpret_cast<const float2*>(A.part_ml + (s * stride + u) * 2);
    if (x.y != 0.f) mx = fmaxf(mx, x.x);
  }
  mx = warp_max(mx);
  float acc[PER], sum = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  for (int s = 0; s < A.S; ++s) {
    const float2 x = *reinterpret_cast<const float2*>(A.part_ml + (s * stride + u) * 2);
    if (x.y == 0.f) continue;
    const float w = x.y * exp2_approx(x.x - mx);
    sum += w;
    const float* src = A.part_o + (s * stride + u) * HD + lane * PER;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = fmaf(w, src[i], acc[i]);
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  __nv_bfloat16* dst = A.o + u * HD + lane * PER;
#pragma unroll
  for (int i = 0; i < PER; i += 2)
    *reinterpret_cast<__nv_bfloat162*>(dst + i) = __floats2bfloat162_rn(acc[i] * inv, acc[i + 1] * inv);
  if (A.st_m && lane == 0) {
    normal_stats(mx, sum);
    A.st_m[u] = mx / kKv8Log2e;
    A.st_l[u] = sum;
  }
}

size_t part_floats(int S, size_t rows, int Hq, int hd) {
  return S > 1 ? (size_t)S * rows * Hq * (hd + 2) : 0;
}

}  // namespace

Kv8AttnPlan attention_kv8_plan(int B, int k_cap, int N, int Hq, int Hkv, int hd, size_t M_cap,
                               size_t part_bytes) {
  Kv8AttnPlan pl{};
  const long long packed = (long long)k_cap * (Hq / Hkv);
  const int keys = std::max(N, 1);
  pl.tc = packed > kKv8TcRows;
  const int rows = pl.tc ? 128 : RM;
  const int least = pl.tc ? 128 : 256;  // keys that a share holds at least
  pl.tiles = (int)((packed + rows - 1) / rows);
  const long long units = (long long)B * Hkv * pl.tiles;
  const long long want = std::max(1LL, 2LL * num_sms() / std::max(1LL, units));  // two CTAs per SM
  pl.shares = (int)std::max(1LL, std::min({want, (long long)(keys + least - 1) / least, 64LL}));
  while (pl.shares > 1 && part_floats(pl.shares, M_cap, Hq, hd) * sizeof(float) > part_bytes) --pl.shares;
  pl.ctas = units * pl.shares;
  return pl;
}

size_t attention_kv8_part_bytes(int B, int k_cap, int N, int Hq, int Hkv, int hd) {
  const size_t M = (size_t)B * k_cap;
  const Kv8AttnPlan pl = attention_kv8_plan(B, k_cap, N, Hq, Hkv, hd, M, ~size_t(0));
  return part_floats(pl.shares, M, Hq, hd) * sizeof(float);
}

cudaError_t launch_attention_kv8(const Kv8RowMap& m, const __nv_bfloat16* q, const uint8_t* k8,
                                 const float* ks, const uint8_t* v8, const float* vs,
                                 __nv_bfloat16* o, const int* kv_len, int Hq, int Hkv, int hd,
                                 int block, float* part, size_t part_bytes, float* st_m,
                                 float* st_l, cudaStream_t s) {
  if (m.M_cap <= 0) return cudaSuccess;
  const Kv8AttnPlan pl =
      attention_kv8_plan(m.B, m.k_cap, m.N, Hq, Hkv, hd, m.M_cap, part ? part_bytes : 0);
  Kv8Args A{};
  A.q = q, A.k8 = k8, A.v8 = v8, A.ks = ks, A.vs = vs, A.o = o, A.kv_len = kv_len;
  A.rows = Kv8Rows{nullptr, m.count, m.row_off, m.row_pos, m.B, m.k_cap, m.N, m.status};
  A.Hq = Hq, A.Hkv = Hkv, A.G = Hq / Hkv;
  A.nblk = (m.N + block - 1) / block;
  while ((1 << A.blk_log2) < block) ++A.blk_log2;
  A.scale_log2 = kKv8Log2e / sqrtf((float)hd);
  A.tiles = pl.tiles;
  A.S = pl.shares;
  A.part_rows = m.M_cap;
  A.part_o = part;
  A.part_ml = pl.shares > 1 ? part + (size_t)pl.shares * m.M_cap * Hq * hd : nullptr;
  A.st_m = st_m, A.st_l = st_l;
  cudaError_t e;
  {
    ProfScope prof("attention_kv8", s);
    if (pl.tc)
      e = launch_attention_kv8_tc(A, pl.ctas, hd, s);
    else
      e = hd == 128 ? launch_kv8<attn_kv8_rows_kernel<128>>((unsigned)pl.ctas, RW * 32, RowsSmem<128>::TOTAL, s, A)
                  : launch_kv8<attn_kv8_rows_kernel<64>>((unsigned)pl.ctas, RW * 32, RowsSmem<64>::TOTAL, s, A);
  }
  if (e != cudaSuccess || pl.shares == 1) return e;
  ProfScope prof("attention_kv8_merge", s);
  const unsigned grid = (unsigned)(((size_t)m.M_cap * Hq + 7) / 8);
  return hd == 128 ? launch_kv8<attn_kv8_merge_kernel<128>>(grid, 256, 0, s, A)
                   : launch_kv8<attn_kv8_merge_kernel<64>>(grid, 256, 0, s, A);
}

}  // namespace dllm
