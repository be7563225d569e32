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
//   P       2^(x_j - r), see below, rounded to f16's 11 bits (bf16 would keep 8).
// The K scale multiplies the fp32 score.  The V scale 2^e of a key's block is an
// addend of its exponent: with x_j = score_j + e_j (log2 units) and a reference r,
//   O = sum_j 2^(x_j - r) v8_j,   l = sum_j 2^(score_j - r'),   out = O / l * 2^(r - r').
//
// f16 keeps 11 bits of a weight down to 2^-14 and has none below 2^-25, and a tile of keys
// may matter although another one's weights are far larger: that one's codes may be small
// (a scale left behind by an outlier) or zero in a channel.  So r follows the keys, up and
// down, such that each tile's largest weight is 2^-6 .. 2^15 in f16; O, in fp32, is rescaled
// where r moves.  A weight is then off by at most 2^-11 of itself, or 2^-19 of the largest
// weight * scale of its own tile: 16 keys here, 64 of the tcgen05 kernel, which also brings
// the codes of a tile of several blocks towards one scale if theirs lie far apart.  r falls by 2^64 at most; tiles
// below that lose bits from 2^-83 of the largest weight * scale on.
//
// The sum has a reference r' of its own, near the largest score, and takes a weight as
// 2^(x_j - r) * 2^-e_j * 2^(r - r').  Where 2^e_j or 2^(r - r') is far from 1
// (kKv8Far) the first factor may flush to zero though the weight counts (a block of
// zero V rows has the scale 2^-100): there the score is exponentiated anew.
#include <algorithm>
#include <type_traits>

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

// Packed query rows per (sequence, kv head) that still run here: one tile of RM.  At 1 row
// and 32 x 1536 keys, 32 heads over 32, 75 us against the tcgen05 kernel's 122; at 16 rows
// of 1 x 1536 keys over 8 heads 7.8 against 10.3.  At 20 rows over 8 heads 11.5 against 10.6
// (1 x 1536 keys) and 25 against 23 (1 x 16384); at 64 rows 39 against 30.5 (16 x 1536) and
// 317 against 180 (64 x 4096).
constexpr int kKv8TcRows = 16;
constexpr int RW = 4;        // warps per CTA
constexpr int RM = 16;       // packed query rows per CTA
constexpr int RK = 16;       // keys per warp and tile

template <int HD>
struct RowsSmem {
  static constexpr int VB = HD / 8;                     // V bytes per lane and key
  static constexpr int TILE = RW * RK * HD;             // codes of 64 keys
  static constexpr int STAGES = HD == 128 ? 3 : 5;      // of a K and a V tile each
  static constexpr int RED = RW * RM * HD * 4;          // outputs of the warps, over the ring
  static constexpr int RING = STAGES * 2 * TILE > RED ? STAGES * 2 * TILE : RED;
  static constexpr int Q_OFF = RING;                    // Q fragments, then the rows' units
  static constexpr int U_OFF = Q_OFF + HD / 16 * 512;
  static constexpr int ML_OFF = U_OFF + RM * 4;
  static constexpr int BAR_OFF = ML_OFF + RW * RM * 2 * 4;
  static constexpr int TOTAL = BAR_OFF + (2 * STAGES + 1) * 8;
  static_assert(4 * (TOTAL + 1024) <= 228 * 1024, "four CTAs per SM");
};

// One CTA = up to 16 packed query rows of one (sequence, kv head) and one share of
// the keys.  Tiles of 64 keys of K and V come by TMA (swizzled, so that the reads
// below are free of bank conflicts at head_dim 128); each warp takes 16 keys of
// every tile.  The codes are read straight into mma.sync fragments and converted in
// registers (one cvt per two codes): K along the head, 16 codes of a lane in an
// order of the inner index that Q's fragments share; V by gathering one byte of two
// keys.  With so few rows the tensor cores' rate does not matter and the kernel is
// bound by the codes' way: 2 bytes per key and head_dim element.  32 sequences x 1 row x
// 1536 keys, 32 heads of 128 over 32 (403 MB): 76 us, 5.3 TB/s; 1 x 1 x 16384 keys (134
// MB) 33 us, start-up and merge included.
template <int HD>
__global__ void __launch_bounds__(RW * 32, 4)
    attn_kv8_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const Kv8Args A) {
  griddep_launch_dependents();
  griddep_wait();
  using L = RowsSmem<HD>;
  constexpr int NT = HD / 8;     // n-tiles of P V
  constexpr int KV16 = HD / 64;  // 16-byte pieces of a key row per lane
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  int u = blockIdx.x;
  const int share = u % A.S;
  u /= A.S;
  const int tile = u % A.tiles;
  u /= A.tiles;
  const int kvh = u % A.Hkv, b = u / A.Hkv;
  const int N = A.rows.N;
  const int want = A.kv_len ? A.kv_len[b] : N;
  int off, cnt;
  kv8_seq_rows(A.rows, b, off, cnt);
  const int R = cnt * A.G - tile * RM;  // packed rows left
  if (R <= 0) return;
  const int len = min(max(want, 0), N);
  if (len != want && threadIdx.x == 0) raise_status(A.rows.status, DEV_BAD_SHAPE);
  const int all = (len + RW * RK - 1) / (RW * RK);
  const int per = (all + A.S - 1) / A.S;
  const int t_lo = min(all, share * per);
  const int T = min(all, t_lo + per) - t_lo;  // this CTA's tiles

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&bars[2 * L::STAGES]);
  auto full = [&](int st) { return smem_u32(&bars[st]); };
  auto empty = [&](int st) { return smem_u32(&bars[L::STAGES + st]); };
  const uint32_t ring = smem_u32(smem);
  int* const status = A.rows.status;
  // warps 0 and 1 read the packed rows g and g + 8 before the codes' copies fill the memory
  // system's queues (behind every CTA's first copies they took 3 us)
  uint4 raw[KV16][2];
  if (warp < 2) {
    const int r = tile * RM + g + 8 * warp;
    const size_t row = (size_t)(off + r / A.G) * A.Hq + kvh * A.G + r % A.G;
#pragma unroll
    for (int p = 0; p < KV16; ++p)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        raw[p][w] = make_uint4(0, 0, 0, 0);
        if (g + 8 * warp < R)
          raw[p][w] = *(reinterpret_cast<const uint4*>(A.q + row * HD + p * 64 + t * 16) + w);
      }
  }
  if (ring & 1023u) {  // the swizzle counts from multiples of 1024
    if (threadIdx.x == 0) raise_status(status, DEV_BAD_SHAPE);
    return;
  }
  if (threadIdx.x == 0) {
    if (T > 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    for (int i = 0; i < L::STAGES; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), RW);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  // tile i (from one thread): K, then V, into stage i % STAGES
  int issued = 0;
  auto issue = [&](int i) {
    const int st = i % L::STAGES;
    if (i >= L::STAGES && !mbar_wait(empty(st), (i / L::STAGES - 1) & 1, abort_flag, status)) return;
    mbar_arrive_expect_tx(full(st), 2 * L::TILE);
    const uint32_t dst = ring + st * 2 * L::TILE;
    const int key = (t_lo + i) * RW * RK;
    tma_load_3d(dst, &tmK, full(st), kvh * HD, key, b);
    tma_load_3d(dst + L::TILE, &tmV, full(st), kvh * HD, key, b);
    issued = i + 1;
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < min(T, L::STAGES); ++i) issue(i);

  // the scales of this warp's keys, read a tile ahead
  const size_t sc0 = ((size_t)b * A.Hkv + kvh) * A.nblk;
  auto scales_of = [&](int i) {
    const int key = ((t_lo + i) * RW + warp) * RK;
    float2 f = make_float2(0.f, 0.f);
    if (i < T && key < len) {
      f.x = __ldg(A.ks + sc0 + (key >> A.blk_log2));
      f.y = __ldg(A.vs + sc0 + (key >> A.blk_log2));
    }
    return f;
  };
  float2 next = scales_of(0);

  // Q fragments of packed rows g (by warp 0) and g + 8 (by warp 1), kept in shared memory
  // for all warps: in k-step i of a half of 64 elements, lane t has elements 16 t + 4 i .. + 3
  float* unit = reinterpret_cast<float*>(smem + L::U_OFF);  // log2 units per raw score of a row
  if (warp < 2) {
    const int i = warp;
    uint32_t mx = 0;
#pragma unroll
    for (int p = 0; p < KV16; ++p)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        mx = __vmaxu2(mx, raw[p][w].x & 0x7fff7fffu);
        mx = __vmaxu2(mx, raw[p][w].y & 0x7fff7fffu);
        mx = __vmaxu2(mx, raw[p][w].z & 0x7fff7fffu);
        mx = __vmaxu2(mx, raw[p][w].w & 0x7fff7fffu);
      }
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int sh = query_shift(__uint_as_float(mx << 16));
    // in two factors: the shift itself may lie outside the normal floats' exponents
    const float f0 = pow2i(sh / 2), f1 = pow2i(sh - sh / 2);
    if (t == 0) unit[g + 8 * i] = A.scale_log2 * pow2i(-(sh / 2)) * pow2i(-(sh - sh / 2));
#pragma unroll
    for (int p = 0; p < KV16; ++p) {
      float f[16];
      unpack8(raw[p][0], f);
      unpack8(raw[p][1], f + 8);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(smem + L::Q_OFF + (p * 4 + e) * 512 + lane * 16) + i;
        dst[0] = pack_h2(f[4 * e] * f0 * f1, f[4 * e + 1] * f0 * f1);
        dst[2] = pack_h2(f[4 * e + 2] * f0 * f1, f[4 * e + 3] * f0 * f1);
      }
    }
  }
  __syncthreads();
  const float rs[2] = {unit[g], unit[g + 8]};
  const uint32_t q_at = ring + L::Q_OFF + lane * 16;

  float o[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m[2] = {kKv8NoRef, kKv8NoRef}, low[2] = {-INFINITY, -INFINITY};  // the weights' reference
  float lm[2] = {kKv8NoRef, kKv8NoRef}, l[2] = {0.f, 0.f};               // the sum and its own
  float fc[2] = {1.f, 1.f};                                              // and what lies between them

  // Column n of an 8-key score tile is key key8(n): at head_dim 128 rows 4 apart in
  // neighbouring lanes, whose swizzled 16-byte pieces lie on different banks; V's 16-byte
  // pieces are dealt out the same way.  (At head_dim 64 a row is half a line: in order.)
  auto key8 = [](int n) { return HD == 128 ? (n & 1) * 4 + (n >> 1) : n; };
  auto piece8 = [](int n) { return HD == 128 ? (n & 1) * 4 + (n >> 1) : n; };
  // address of piece p (16 bytes) of key row r of a tile, as TMA's swizzle leaves it
  auto at = [](int r, int p) {
    return HD == 128 ? r * 128 + ((p ^ (r & 7)) << 4) : r * 64 + ((p ^ ((r >> 1) & 3)) << 4);
  };
  uint32_t k_at[2][KV16], v_at[4];
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int p = 0; p < KV16; ++p) k_at[n][p] = at(warp * RK + 8 * n + key8(g), 4 * p + t);
  int v_key[4];  // of this lane's V fragments, within the warp's 16
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v_key[i] = 8 * (i >> 1) + key8(2 * t + (i & 1));
    const int r = warp * RK + v_key[i];
    v_at[i] = L::TILE + (HD == 128 ? at(r, piece8(g)) : at(r, g >> 1) + (g & 1) * 8);
  }

  bool ok = true;
  for (int i = 0; i < T; ++i) {
    const int st = i % L::STAGES;
    const float2 sc = next;
    next = scales_of(i + 1);
    // the stage that the tile before last freed
    if (threadIdx.x == 0 && i >= 2 && i + L::STAGES - 2 < T) issue(i + L::STAGES - 2);
    __syncwarp();
    ok = __all_sync(0xffffffffu, mbar_wait(full(st), (i / L::STAGES) & 1, abort_flag, status));
    if (!ok) break;
    const uint32_t base = ring + st * 2 * L::TILE;
    const int left = len - ((t_lo + i) * RW + warp) * RK;  // of this warp's keys that exist
    if (left > 0) {
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int p = 0; p < KV16; ++p) {
        uint32_t q4[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) lds128(q4[n], base + k_at[n][p]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t qf[4];
          lds128(qf, q_at + (p * 4 + e) * 512);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            uint32_t lo, hi;
            e4m3x4_to_f16x4(q4[n][e], lo, hi);
            mma_f16(s[n], qf, lo, hi);
          }
        }
      }
      uint32_t w[4][L::VB / 4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if constexpr (HD == 128)
          lds128(w[x], base + v_at[x]);
        else
          lds64(w[x], base + v_at[x]);
      }
      const float ev = v_exponent(sc.y), inv_v = near_inverse(sc.y);
      const float k[2] = {rs[0] * sc.x, rs[1] * sc.x};  // log2 units per raw score
      if (left < RK) {  // what lies past the last key plays no part, whatever it holds
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (8 * n + key8(2 * t + (x & 1)) >= left) s[n][x] = -INFINITY;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int y = 0; y < L::VB / 4; ++y)
            if (v_key[x] >= left) w[x][y] = 0;
      }
      float top[2], f[2];
      bool move[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        top[x] = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        move[x] = wants_ref(fmaf(top[x], k[x], ev - m[x]));
        f[x] = fc[x] * inv_v;  // 0: far
      }
      if (__any_sync(0xffffffffu, move[0] || move[1] || f[0] == 0.f || f[1] == 0.f)) {
        float rise[2];
        bool twice = false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          top[x] *= k[x];
          const float before = m[x];
          move[x] = new_ref(top[x] + ev, m[x], low[x]);
          rise[x] = before - m[x];
          twice |= rises_far(before, m[x]);
          if (top[x] > lm[x] && (move[x] || f[x] == 0.f)) {
            l[x] *= exp2_approx(lm[x] - top[x]);
            lm[x] = top[x];
          }
          fc[x] = ref_factor(m[x] - lm[x]);
          f[x] = fc[x] * inv_v;
          if (f[x] == 0.f) {  // the weights anew
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int n = y >> 1, i = y & 1;
              if (8 * n + key8(2 * t + i) < left) l[x] += exp2_approx(fmaf(s[n][2 * x + i], k[x], -lm[x]));
            }
          }
        }
        twice = __any_sync(0xffffffffu, twice);
        const float a0 = exp2_approx(twice ? 0.5f * rise[0] : rise[0]), a1 = exp2_approx(twice ? 0.5f * rise[1] : rise[1]);
#pragma unroll 1
        for (int i = twice ? 0 : 1; i < 2; ++i) {
#pragma unroll
          for (int n = 0; n < NT; ++n) o[n][0] *= a0, o[n][1] *= a0, o[n][2] *= a1, o[n][3] *= a1;
        }
      }
      float p[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) p[n][x] = exp2_approx(fmaf(s[n][x], k[x >> 1], ev - m[x >> 1]));
      if (left < RK) {  // (-infinity times a zero scale is NaN)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (8 * n + key8(2 * t + (x & 1)) >= left) p[n][x] = 0.f;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        l[x] = fmaf((p[0][2 * x] + p[0][2 * x + 1]) + (p[1][2 * x] + p[1][2 * x + 1]), f[x], l[x]);
      const uint32_t pa[4] = {pack_h2(p[0][0], p[0][1]), pack_h2(p[0][2], p[0][3]),
                              pack_h2(p[1][0], p[1][1]), pack_h2(p[1][2], p[1][3])};
#pragma unroll
      for (int q = 0; q < L::VB / 4; ++q) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // bytes 4 q + 2 j, + 1 of the pieces: (key, key) pairs
          const uint32_t a = __byte_perm(w[0][q], w[1][q], j ? 0x7362 : 0x5140);
          const uint32_t d = __byte_perm(w[2][q], w[3][q], j ? 0x7362 : 0x5140);
          uint32_t v[4];
          e4m3x4_to_f16x4(a, v[0], v[2]);
          e4m3x4_to_f16x4(d, v[1], v[3]);
          mma_f16(o[q * 4 + 2 * j], pa, v[0], v[1]);
          mma_f16(o[q * 4 + 2 * j + 1], pa, v[2], v[3]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty(st));
  }
  if (!ok && threadIdx.x == 0)  // a wait ran out: the copies on their way land before the exit
    for (int i = max(0, issued - L::STAGES); i < issued; ++i)
      mbar_wait_drain(full(i % L::STAGES), (i / L::STAGES) & 1, status);
  __syncthreads();  // every tile has been read: the warps' outputs take the ring's place
  if (*abort_flag) return;

  float* red = reinterpret_cast<float*>(smem);
  float* ml = reinterpret_cast<float*>(smem + L::ML_OFF);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float sum = l[i];
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    // the warp's output: its sums over its own softmax sum, and the references' difference
    // in two factors, either of which alone stays a normal float
    const float inv = sum == 0.f ? 0.f : 1.0f / sum, f = exp2_approx(0.5f * (m[i] - lm[i]));
    normal_stats(lm[i], sum);
    if (t == 0) {
      float* x = ml + (warp * RM + g + 8 * i) * 2;
      x[0] = lm[i], x[1] = sum;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
      o[j][2 * i] = o[j][2 * i] * inv * f * f, o[j][2 * i + 1] = o[j][2 * i + 1] * inv * f * f;
    // n-tile j of lane t: byte j of V's pieces piece8(2t) and piece8(2t + 1)
    float* dst = red + (warp * RM + g + 8 * i) * HD;
#pragma unroll
    for (int j = 0; j < NT; j += 4) {
      *reinterpret_cast<float4*>(dst + piece8(2 * t) * L::VB + j) =
          make_float4(o[j][2 * i], o[j + 1][2 * i], o[j + 2][2 * i], o[j + 3][2 * i]);
      *reinterpret_cast<float4*>(dst + piece8(2 * t + 1) * L::VB + j) = make_float4(
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
    float sum = 0.f, part[RW], acc[8];
#pragma unroll
    for (int w = 0; w < RW; ++w) {
      const float* x = ml + (w * RM + row) * 2;
      part[w] = x[1] == 0.f ? 0.f : x[1] * exp2_approx(x[0] - mx);  // (0: no keys)
      sum += part[w];
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;  // a row without keys: zeros
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] = 0.f;
#pragma unroll
    for (int w = 0; w < RW; ++w) {
      const float* src = red + (w * RM + row) * HD + e;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(src[k], part[w] * inv, acc[k]);
    }
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
// W = sum w_s, O = sum (w_s / W) o_s (no partial sum above the largest o_s).  WPR warps per (row, head), each with up to 8 shares whose
// slices are on their way at once: bound by the latency of one such trip (one warp for 64
// shares took 16 us of a call; eight warps for 12 shares and 1024 rows 3 us more than two).
// An empty share has l = 0, and what its slice holds is dropped.
template <int HD, int WPR>
__global__ void __launch_bounds__(256) attn_kv8_merge_kernel(const Kv8Args A) {
  constexpr int PER = HD / 32;
  __shared__ float s_acc[WPR][HD];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t u = WPR > 1 ? blockIdx.x : (size_t)blockIdx.x * 8 + warp;
  const int s0 = WPR > 1 ? warp * 8 : 0;
  int off, cnt;
  kv8_seq_rows(A.rows, A.rows.B - 1, off, cnt);
  if (u >= (size_t)(off + cnt) * A.Hq) return;  // (a row's warps together)
  const size_t stride = (size_t)A.part_rows * A.Hq;
  auto ml_of = [&](int s) {
    return s < A.S ? *reinterpret_cast<const float2*>(A.part_ml + (s * stride + u) * 2) : make_float2(0.f, 0.f);
  };
  const float2 a = ml_of(lane), b = WPR > 4 ? ml_of(lane + 32) : make_float2(0.f, 0.f);
  float o[8][PER];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float* src = A.part_o + (min(s0 + k, A.S - 1) * stride + u) * HD + lane * PER;
    if constexpr (PER == 4)
      *reinterpret_cast<float4*>(o[k]) = *reinterpret_cast<const float4*>(src);
    else
      *reinterpret_cast<float2*>(o[k]) = *reinterpret_cast<const float2*>(src);
  }
  const float mx = warp_max(fmaxf(a.y != 0.f ? a.x : -INFINITY, b.y != 0.f ? b.x : -INFINITY));
  const float wa = a.y != 0.f ? a.y * exp2_approx(a.x - mx) : 0.f;
  const float wb = b.y != 0.f ? b.y * exp2_approx(b.x - mx) : 0.f;
  float sum = warp_sum(wa + wb), acc[PER];
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float w = __shfl_sync(0xffffffffu, s0 < 32 ? wa : wb, (s0 + k) & 31) * inv;  // 0 past the last share
#pragma unroll
    for (int x = 0; x < PER; ++x) acc[x] = fmaf(w, w != 0.f ? o[k][x] : 0.f, acc[x]);
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int x = 0; x < PER; ++x) s_acc[warp][lane * PER + x] = acc[x];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < WPR; ++w) {  // in share order
#pragma unroll
      for (int x = 0; x < PER; ++x) acc[x] += s_acc[w][lane * PER + x];
    }
  }
  __nv_bfloat16* dst = A.o + u * HD + lane * PER;
#pragma unroll
  for (int i = 0; i < PER; i += 2)
    *reinterpret_cast<__nv_bfloat162*>(dst + i) = __floats2bfloat162_rn(acc[i], acc[i + 1]);
  if (A.st_m && lane == 0) {
    float m = mx;
    normal_stats(m, sum);
    A.st_m[u] = m / kKv8Log2e;
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
  pl.tiles = (int)((packed + rows - 1) / rows);
  const long long units = (long long)B * Hkv * pl.tiles;
  // Shares hold 128 keys or more (64: 16.3 us against 11.9 for 16 rows of 1 x 1536 keys, 32
  // heads over 8; 256: 13.1).  Of the CTAs with few rows four share an SM (1 row of 8 x 16384
  // keys, 28 heads over 4: 30.8 us; three 34.9, six 35.2); of those with many, one (20 rows
  // of 4 x 1536 keys: 17.7 us against 20.8 with two), unless that leaves more than 1024 keys
  // to each (20 rows of 6 x 16384 keys: two 70 us, one 91).
  auto split = [&](int per_sm) {
    const long long fill = std::max(1LL, (long long)per_sm * num_sms() / std::max(1LL, units));
    return std::min({fill, (long long)(keys + 127) / 128, (long long)kKv8MaxShares});
  };
  long long shares = split(pl.tc ? 1 : 4);
  if (pl.tc && keys > shares * 1024) shares = split(2);
  pl.shares = (int)std::max(1LL, shares);
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
  // (no position cached: nothing is copied, and the maps point nowhere)
  CUtensorMap tk{}, tv{};
  if (!pl.tc && m.N > 0 &&
      (!tmap_codes(&tk, k8, m.B, m.N, Hkv * hd, hd, 64) || !tmap_codes(&tv, v8, m.B, m.N, Hkv * hd, hd, 64)))
    return cudaErrorInvalidValue;
  cudaError_t e;
  {
    ProfScope prof("attention_kv8", s);
    if (pl.tc)
      e = launch_attention_kv8_tc(A, pl.ctas, hd, s);
    else
      e = hd == 128 ? launch_kv8<attn_kv8_rows_kernel<128>>((unsigned)pl.ctas, RW * 32, RowsSmem<128>::TOTAL, s, tk, tv, A)
                  : launch_kv8<attn_kv8_rows_kernel<64>>((unsigned)pl.ctas, RW * 32, RowsSmem<64>::TOTAL, s, tk, tv, A);
  }
  if (e != cudaSuccess || pl.shares == 1) return e;
  ProfScope prof("attention_kv8_merge", s);
  auto merge = [&](auto hd_c) {
    constexpr int HD = decltype(hd_c)::value;
    const size_t rows = (size_t)m.M_cap * Hq;
    auto wide = [&](auto wpr_c) {
      constexpr int WPR = decltype(wpr_c)::value;
      return launch_kv8<attn_kv8_merge_kernel<HD, WPR>>((unsigned)rows, WPR * 32, 0, s, A);
    };
    if (pl.shares <= 8)
      return launch_kv8<attn_kv8_merge_kernel<HD, 1>>((unsigned)((rows + 7) / 8), 256, 0, s, A);
    if (pl.shares <= 16) return wide(std::integral_constant<int, 2>{});
    if (pl.shares <= 32) return wide(std::integral_constant<int, 4>{});
    return wide(std::integral_constant<int, 8>{});
  };
  return hd == 128 ? merge(std::integral_constant<int, 128>{}) : merge(std::integral_constant<int, 64>{});
}

}  // namespace dllm
