// Attention over the 8-bit K/V cache on the 5th-generation tensor cores: tiles of
// 128 packed query rows (see attention_kv8.cu for the arithmetic).
//
// One CTA = one (sequence, kv head), one tile of 128 packed rows and one share of
// the keys, 64 keys at a time; two CTAs share an SM, so that one's softmax overlaps
// the other's products.  Warp roles (288 threads):
//   warps 0 .. 3  converters, two for the K tiles and two for the V tiles: the codes
//                 by cp.async into a small ring (each thread reads back what it
//                 copied itself), one cvt per two codes, and f16 to slots in the
//                 128-byte-swizzled layout that TMA would have written;
//   warp 4        TMEM owner and tcgen05.mma issuer;
//   warps 5 .. 8  softmax, one packed row per thread (its TMEM lane): the thread
//                 first brings its query row to f16 in shared memory.
// TMEM holds two score tiles of 64 columns, and O.  The scores of tile j + 1 are
// computed while tile j is exponentiated; P (f16 pairs) goes over the first 32
// columns of its scores and is read from TMEM by P V.  Issue order: QK(0) QK(1)
// PV(0) QK(2) PV(1) ...  Operations of one thread complete in order, so QK(j+2)
// cannot overwrite P(j) before PV(j) has read it.  64 keys rather than 128, so that
// a thread reads its scores once and holds them in registers.
//
// Bound by shared memory: per 64 keys a CTA moves 128 KB through it (codes in and
// out 32, f16 tiles 32, Q and K for Q K^T 48, V 16) = 1024 cycles at 128 bytes a
// cycle.  32 sequences x 308 rows x 1536 keys, 32 heads of 128: over 8 kv heads 347 us
// (714 TFLOP/s; the kernel over a bf16 cache 347), over 32, where the third of each
// sequence's tiles holds 52 of 128 rows, 402 (358); under the power cap, at 1.78 GHz, 446.
// Dropped on the way, at the latter: scores read twice and 128 keys 696 us; codes through
// registers and L1 540; K and V converted in turn by the same warps 445.  Two row tiles per
// CTA over the same keys, one CTA per SM, 378 us at 256 rows against 350; codes by TMA 468
// against 441.
// Every mbarrier wait is bounded; a timeout sets DLLM_DEV_TIMEOUT, drains the MMAs,
// frees TMEM and returns.
#include <type_traits>

#include "attention_kv8.cuh"
#include "tmem.cuh"

namespace dllm {

namespace {

constexpr int BT = 128;   // packed rows per tile (= TMEM lanes)
constexpr int BK = 64;    // keys per tile
constexpr int NSC = 8;    // tiles whose scales are kept: more than the converters run ahead
constexpr int NC = 4;     // converter warps
constexpr int kThreads = (NC + 1 + 4) * 32;
constexpr uint32_t kTmemCols = 256;

template <int HD>
struct Smem {
  static constexpr int Q_TILE = BT * HD * 2;
  static constexpr int SLOT = BK * HD * 2;
  static constexpr int RAW = BK * HD;                      // codes of a tile
  static constexpr int RAWS = 2;                           // of K, and of V
  static constexpr int BUDGET = 113 * 1024;                // half of 228 KB, 1 KB reserved
  // K runs a tile ahead of V: with one V slot less both are released a tile before they
  // are needed again
  static constexpr int KS = 2, VS = HD == 128 ? 1 : 2;
  static constexpr int K_OFF = Q_TILE;
  static constexpr int V_OFF = K_OFF + KS * SLOT;
  static constexpr int RAW_OFF = V_OFF + VS * SLOT;        // [K, V][RAWS]
  static constexpr int SC_OFF = RAW_OFF + 2 * RAWS * RAW;  // [NSC][4] float4
  static constexpr int BAR_OFF = SC_OFF + NSC * 4 * 16;
  static constexpr int TOTAL = BAR_OFF + 48 * 8;
  static_assert(TOTAL <= BUDGET, "shared memory");
};

// f16 x f16 -> fp32, both operands K-major, M x N tile
constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// MIX: blocks shorter than a tile of keys, whose V scales may differ within it (413 us where
// blocks of 64 take 402)
template <int HD, bool MIX>
__global__ void __launch_bounds__(kThreads, 2) attn_kv8_tc_kernel(const Kv8Args A) {
  using L = Smem<HD>;
  griddep_launch_dependents();
  griddep_wait();
  int u = blockIdx.x;
  const int share = u % A.S;
  u /= A.S;
  const int tile = u % A.tiles;
  u /= A.tiles;
  const int kvh = u % A.Hkv, b = u / A.Hkv;
  int off, cnt;
  kv8_seq_rows(A.rows, b, off, cnt);
  const int r0 = tile * BT;
  const int R = cnt * A.G - r0;  // packed rows from this CTA's first on
  if (R <= 0) return;
  const int N = A.rows.N;
  int len = N;
  if (A.kv_len) {
    const int want = A.kv_len[b];
    len = min(max(want, 0), N);
    if (len != want && threadIdx.x == 0) raise_status(A.rows.status, DEV_BAD_SHAPE);
  }
  const int all = (len + BK - 1) / BK;
  const int per = (all + A.S - 1) / A.S;
  const int k_lo = min(all, share * per);
  const int T = min(all, k_lo + per) - k_lo;  // this CTA's K/V tiles

  extern __shared__ __align__(1024) uint8_t sm[];
  if (smem_u32(sm) & 1023u) {  // the swizzled tiles start at multiples of 1024
    if (threadIdx.x == 0) raise_status(A.rows.status, DEV_BAD_SHAPE);
    return;
  }
  float4* scales = reinterpret_cast<float4*>(sm + L::SC_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
  const uint32_t q_full = smem_u32(&bars[0]), drain_bar = smem_u32(&bars[1]);
  // per score buffer: tile j uses buffer j & 1 for the (j / 2)-th time
  auto s_full = [&](int j) { return smem_u32(&bars[2 + (j & 1)]); };
  auto p_full = [&](int j) { return smem_u32(&bars[4 + (j & 1)]); };
  auto pv_done = [&](int j) { return smem_u32(&bars[6 + (j & 1)]); };
  auto par = [](int j) { return (uint32_t)((j >> 1) & 1); };
  auto sc_full = [&](int j) { return smem_u32(&bars[8 + j % NSC]); };
  // of the slots K0 K1 V0 (V1)
  auto full_at = [&](int i) { return smem_u32(&bars[8 + NSC + i]); };
  auto empty_at = [&](int i) { return smem_u32(&bars[8 + NSC + 4 + i]); };
  static_assert(8 + NSC + 2 * 4 + 1 <= 48, "barrier area holds 48 words");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&bars[8 + NSC + 2 * 4]);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* const status = A.rows.status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sQ = smem_u32(sm);
  const int live_warps = (min(BT, R) + 31) / 32;  // softmax warps that hold a row

  // the converters' copies and scales: the first ones are on their way while the CTA is set up
  constexpr int HB = HD / 64;   // 64-element boxes of a row
  constexpr int NV = 4 * HB;    // 16-byte vectors per thread and tile
  const size_t row_bytes = (size_t)A.Hkv * HD;
  const int key0 = k_lo * BK;
  const bool is_v = warp >= NC / 2;
  // A thread's vectors of a tile: keys row, row + 8, .. + 24 of this warp's 32, HB boxes
  // each, 16 codes at 16 (lane & 3).  A warp's copy covers 8 rows of 64 bytes, and the 8
  // lanes of a store phase fall on 8 different bank groups.
  const int row = (warp & 1) * 32 + (lane >> 2);
  const uint8_t* next = (is_v ? A.v8 : A.k8) +
                        (((size_t)b * N + key0 + row) * A.Hkv + kvh) * HD + (size_t)(lane & 3) * 16;
  const size_t eight = 8 * row_bytes, step = BK * row_bytes;
  const uint32_t raw = smem_u32(sm + L::RAW_OFF) + (is_v ? L::RAWS * L::RAW : 0) + (threadIdx.x & 63) * 16;
  const uint32_t st0 = smem_u32(sm + (is_v ? L::V_OFF : L::K_OFF)) + row * 128 +
                       (((lane & 3) * 2) ^ (lane >> 2)) * 16;
  auto fetch = [&](int j) {
    if (j < T) {
      const uint32_t dst = raw + (j & 1) * L::RAW;
      const int left = len - key0 - j * BK - row;  // keys from this thread's first row on
      if (left > 24) {
#pragma unroll
        for (int i = 0; i < NV; ++i) cp_async16(dst + i * 1024, next + (i / HB) * eight + i % HB * 64);
      } else {  // keys past the last one arrive as zeros (copies of 0 bytes from a valid row)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const bool there = left > i / HB * 8;
          cp_async16(dst + i * 1024, there ? next + (i / HB) * eight + i % HB * 64 : A.k8, there);
        }
      }
      next += step;
    }
    cp_commit();
  };
  // the scales of a K/V tile, per 16 keys: by the first lanes of K's warp j & 1, read when
  // its previous turn is done
  const size_t sc0 = ((size_t)b * A.Hkv + kvh) * A.nblk;
  auto fetch_scales = [&](int j) {
    const int key = key0 + j * BK + lane * 16;
    float2 f = make_float2(0.f, 0.f);
    if (lane < 4 && j < T && key < len) {
      f.x = __ldg(A.ks + sc0 + (key >> A.blk_log2));
      f.y = __ldg(A.vs + sc0 + (key >> A.blk_log2));
    }
    return f;
  };
  float2 sc = make_float2(0.f, 0.f);
  if (warp < NC) {
    fetch(0);
    if (!is_v) sc = fetch_scales(warp);
  }
  // and a softmax thread's query row
  const int r = (warp & 3) * 32 + lane;  // packed row in the tile (= TMEM lane)
  const bool there = r < R;
  const int pr = r0 + r;
  const size_t at = (size_t)(off + (there ? pr / A.G : 0)) * A.Hq + kvh * A.G + pr % A.G;
  uint4 q_row[HD / 8];
  if (warp > NC && T > 0) {
#pragma unroll
    for (int i = 0; i < HD / 8; ++i)
      q_row[i] = there ? *(reinterpret_cast<const uint4*>(A.q + at * HD) + i) : make_uint4(0, 0, 0, 0);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(full_at(i), NC / 2);
      mbar_init(empty_at(i), 1);
    }
    for (int i = 0; i < NSC; ++i) mbar_init(sc_full(i), 1);
    for (int j = 0; j < 2; ++j) {
      mbar_init(s_full(j), 1);
      mbar_init(p_full(j), live_warps);
      mbar_init(pv_done(j), 1);
    }
    mbar_init(q_full, 128);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == NC) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto tS = [&](int j) { return tmem + (uint32_t)((j & 1) * 64); };
  const uint32_t tO = tmem + 128;

  if (warp < NC) {
    // ---------------------------------------------------------------- converters
    // Blocks shorter than a tile: where the V scales of a tile span more than six octaves, the
    // codes themselves are brought towards a common scale, by 2^-7 .. 2^1 (f16 would hold them
    // from 2^-15 to 2^7, but keys of a small block may weigh more, and then it is the scales'
    // difference that keeps their weights and the others' in range), and the largest weight
    // to 2^8 or more.  Exponent of the factor of lane's (0 .. 3) group of 16 keys.
    auto v_shift = [&](float e, bool& mixed) {
      float hi = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, 1));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 2));
      float lo = e == -INFINITY ? INFINITY : e;
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, 2));
      mixed |= hi - lo > 6.f;
      return hi - lo > 6.f ? fminf(fmaxf(e - hi + 1.f, -7.f), 1.f) : 0.f;
    };
    auto tiles = [&](auto scaled) {
      constexpr bool SCALED = decltype(scaled)::value;
      for (int j = 0; j < T; ++j) {
        fetch(j + 1);
        float by[2];  // the factors of this warp's two groups
        if constexpr (SCALED) {
          if (!mbar_wait(sc_full(j), (j / NSC) & 1, abort_flag, status)) return;
          by[0] = fabsf(scales[j % NSC * 4 + (warp & 1) * 2].w);
          by[1] = fabsf(scales[j % NSC * 4 + (warp & 1) * 2 + 1].w);
        } else if (!is_v && warp == (j & 1)) {
          bool mixed = false;
          const float e = v_exponent(sc.y), c = MIX ? v_shift(e, mixed) : 0.f;
          const float inv = near_inverse(sc.y) * (MIX ? pow2i((int)c) : 1.f);
          // (the sum takes the whole tile one way: a far scale makes it far)
          const bool near = __all_sync(0xffffffffu, lane >= 4 || key0 + j * BK + lane * 16 >= len || inv != 0.f);
          if (lane < 4)
            scales[j % NSC * 4 + lane] = make_float4(sc.x, e - c, near ? inv : 0.f, mixed ? -pow2i((int)c) : 1.f);
          __syncwarp();
          if (lane == 0) mbar_arrive(sc_full(j));
          sc = fetch_scales(j + 2);
        }
        cp_wait<1>();
        const int slot = is_v ? j % L::VS : j % L::KS;
        const int turn = is_v ? j / L::VS : j / L::KS;
        const int bar = is_v ? L::KS + slot : slot;
        if (!mbar_wait(empty_at(bar), (turn & 1) ^ 1, abort_flag, status)) return;
        const uint32_t dst = st0 + slot * L::SLOT;
        const uint32_t from = raw + (j & 1) * L::RAW;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          uint32_t q[4], h[8];
          lds128(q, from + i * 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k) e4m3x4_to_f16x4(q[k], h[2 * k], h[2 * k + 1]);
          if constexpr (SCALED) {
            const __half2 f = __float2half2_rn(by[i / HB / 2]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&h[k]), f);
              h[k] = *reinterpret_cast<const uint32_t*>(&y);
            }
          }
          const uint32_t to = dst + i % HB * (BK * 128) + i / HB * 1024;
#pragma unroll
          for (int c = 0; c < 2; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(c ? to ^ 16 : to), "r"(h[4 * c]),
                         "r"(h[4 * c + 1]), "r"(h[4 * c + 2]), "r"(h[4 * c + 3])
                         : "memory");
        }
        // generic stores before the tensor core's reads
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(full_at(bar));
      }
    };
    // V's warps: whether any tile of this CTA needs it, found before the first tile (looked at
    // in every tile it took 437 us where this takes 410, at 32 heads and blocks of 16)
    bool scaled = false;
    if (MIX && is_v) {
      for (int g = 0; g < 4 * T; g += 32) {
        const int key = key0 + (g + lane) * 16;
        const float s = key < len && g + lane < 4 * T ? __ldg(A.vs + sc0 + (key >> A.blk_log2)) : 0.f;
        v_shift(v_exponent(s), scaled);
      }
      scaled = __any_sync(0xffffffffu, scaled);
    }
    if (MIX && scaled)
      tiles(std::true_type{});
    else
      tiles(std::false_type{});
    cp_wait<0>();
  } else if (warp == NC) {
    if (lane == 0 && T > 0) {
      // ---------------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = idesc_f16(BT, BK);
      constexpr uint32_t idesc_pv = idesc_f16(BT, HD) | (1u << 16);  // V read MN-major
      bool ok = true, any = false;
      auto take = [&](int i, int turn) -> bool {
        if (!mbar_wait(full_at(i), turn & 1, abort_flag, status)) return false;
        tc_fence_after();
        return true;
      };
      auto give = [&](int i) { tc_commit(empty_at(i)); };
      // operand descriptors: the high words are constant, the low ones count 16 bytes
      const uint64_t dq = umma_desc_k_sw128(sQ), dk = umma_desc_k_sw128(smem_u32(sm + L::K_OFF)),
                     dv = umma_desc_mn_sw128(smem_u32(sm + L::V_OFF), BK * 128);
      auto qk = [&](int j) -> bool {
        const int i = j % L::KS;
        if (!take(i, j / L::KS)) return false;
        const uint64_t b0 = dk + (uint64_t)(i * (L::SLOT / 16));
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          tc_mma_bf16(tS(j), dq + ((kk >> 2) * (BT * 128) + (kk & 3) * 32) / 16,
                      b0 + ((kk >> 2) * (BK * 128) + (kk & 3) * 32) / 16, idesc_qk, kk > 0 ? 1u : 0u);
        tc_commit(s_full(j));
        give(i);
        return any = true;
      };
      auto pv = [&](int j) -> bool {
        const int i = j % L::VS;
        if (!take(L::KS + i, j / L::VS)) return false;
        if (!mbar_wait(p_full(j), par(j), abort_flag, status)) return false;
        tc_fence_after();
        const uint64_t b0 = dv + (uint64_t)(i * (L::SLOT / 16));
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          tc_mma_ts(tO, tS(j) + (uint32_t)(kk * 8), b0 + kk * 2048 / 16, idesc_pv,
                    (j > 0 || kk > 0) ? 1u : 0u);
        tc_commit(pv_done(j));
        give(L::KS + i);
        return true;
      };
      ok = mbar_wait(q_full, 0, abort_flag, status);
      tc_fence_after();
      for (int j = 0; j < 2 && j < T && ok; ++j) ok = qk(j);
      for (int j = 0; j < T && ok; ++j) ok = pv(j) && (j + 2 >= T || qk(j + 2));
      if (!ok && any) {
        tc_commit(drain_bar);
        mbar_wait_drain(drain_bar, 0, status);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    const int quad = warp & 3;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    float rs = 0.f;  // log2 units per raw score
    if (T > 0) {
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        mx = __vmaxu2(mx, q_row[i].x & 0x7fff7fffu);
        mx = __vmaxu2(mx, q_row[i].y & 0x7fff7fffu);
        mx = __vmaxu2(mx, q_row[i].z & 0x7fff7fffu);
        mx = __vmaxu2(mx, q_row[i].w & 0x7fff7fffu);
      }
      const int sh = query_shift(__uint_as_float(max(mx & 0xffffu, mx >> 16) << 16));
      const float f0 = pow2i(sh / 2), f1 = pow2i(sh - sh / 2);
      rs = A.scale_log2 * pow2i(-(sh / 2)) * pow2i(-(sh - sh / 2));
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        float f[8];
        unpack8(q_row[i], f);
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = pack_h2(f[2 * k] * f0 * f1, f[2 * k + 1] * f0 * f1);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         sQ + (i >> 3) * (BT * 128) + r * 128 + ((i & 7) ^ (r & 7)) * 16),
                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                     : "memory");
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(q_full);
    }
    float m = kKv8NoRef, low = -INFINITY;  // the weights' reference
    float lm = kKv8NoRef, l = 0.f;         // the sum and its own
    float fc = 1.f;                        // and what lies between them
    bool ok = true;
    // the sum's reference moves up to r
    auto raise_sum = [&](float r) {
      if (r > lm) {
        l *= exp2_approx(lm - r);
        lm = r;
      }
      fc = ref_factor(m - lm);
    };
    // Adds the weights of tile j to the sum where its scales or references are far, from the
    // scores anew.  (Seldom: not unrolled.)
    auto far_sum = [&](bool far, const float4* sc, int j, int nkeys) {
      float top = kKv8NoRef;
#pragma unroll 1
      for (int turn = 0; turn < 2; ++turn) {
#pragma unroll 1
        for (int g = 0; g < 4 && 16 * g < nkeys; ++g) {
          float t[16];
          __syncwarp();
          tmem_ld16(tS(j) + lane_off + 16 * g, t);
          const float k = rs * sc[g].x;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (16 * g + i >= nkeys) continue;
            if (turn == 0) top = fmaxf(top, t[i] * k);
            else if (far) l += exp2_approx(fmaf(t[i], k, -lm));
          }
        }
        if (turn == 0 && far) raise_sum(top);
      }
    };
    // a warp whose 32 rows are all past the sequence's rows takes no further part
    if (quad < live_warps) {
      for (int j = 0; j < T; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(sc_full(j), (j / NSC) & 1, abort_flag, status) &&
                                         mbar_wait(s_full(j), par(j), abort_flag, status));
        if (!ok) break;
        tc_fence_after();
        const float4* sc = scales + j % NSC * 4;
        const int nkeys = len - (k_lo + j) * BK;
        const bool far = fc == 0.f || sc[0].z == 0.f;
        if (__any_sync(0xffffffffu, far)) far_sum(far, sc, j, nkeys);
        float s[BK];
        tmem_ld32_nowait(tS(j) + lane_off, s);
        tmem_ld32_nowait(tS(j) + lane_off + 32, s + 32);
        tmem_wait_ld();
        auto tile_softmax = [&](auto last) {
          constexpr bool LAST = decltype(last)::value;  // some of the keys do not exist
          float mx = -INFINITY;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float* t = s + 16 * g;
            if (LAST) {
#pragma unroll
              for (int i = 0; i < 16; ++i) t[i] = 16 * g + i < nkeys ? t[i] : -INFINITY;
            }
            float a = fmaxf(t[0], t[1]), c = fmaxf(t[2], t[3]);
#pragma unroll
            for (int i = 4; i < 16; i += 4) {
              a = fmax3(a, t[i], t[i + 1]);
              c = fmax3(c, t[i + 2], t[i + 3]);
            }
            // (a group past the keys: -inf times a zero scale would be NaN)
            const float2 f = *reinterpret_cast<const float2*>(sc + g);
            if (!LAST || 16 * g < nkeys) mx = fmaxf(mx, fmaf(fmaxf(a, c), rs * f.x, f.y));
          }
          const bool mixed = MIX && sc[0].w < 0.f;
          if (__any_sync(0xffffffffu, wants_ref(mx - m, mixed))) {
            const float before = m;
            const bool move = new_ref(mx, m, low, mixed);
            if (move) raise_sum(sc[0].z != 0.f ? m - sc[0].y : lm);
            if (j > 0 && __any_sync(0xffffffffu, move)) {
              // O may be rescaled once PV(j-1) is complete, until P(j) is handed over
              if (!__all_sync(0xffffffffu, mbar_wait(pv_done(j - 1), par(j - 1), abort_flag, status)))
                return false;
              tc_fence_after();
              const bool twice = __any_sync(0xffffffffu, rises_far(before, m));
              const float alpha = exp2_approx(twice ? 0.5f * (before - m) : before - m);
#pragma unroll 1
              for (int c = twice ? 0 : HD; c < 2 * HD; c += HD == 128 ? 64 : 16) {
                const uint32_t at = tO + lane_off + c % HD;
                if (c == HD && twice) tmem_wait_st();  // (the second turn reads the first's)
                if constexpr (HD == 128) {  // in the scores' registers, which are read again
                  tmem_ld32_nowait(at, s);
                  tmem_ld32_nowait(at + 32, s + 32);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 64; ++i) s[i] *= alpha;
                  tmem_st32(at, reinterpret_cast<const uint32_t*>(s));
                  tmem_st32(at + 32, reinterpret_cast<const uint32_t*>(s) + 32);
                } else {
                  float o[16];
                  tmem_ld16(at, o);
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] *= alpha;
                  tmem_st16(at, reinterpret_cast<const uint32_t*>(o));
                }
              }
              if constexpr (HD == 128) {
                tmem_ld32_nowait(tS(j) + lane_off, s);
                tmem_ld32_nowait(tS(j) + lane_off + 32, s + 32);
                tmem_wait_ld();
              }
            }
          }
          float add = 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int g = 2 * h; g < 2 * h + 2; ++g) {
              const float4 f = sc[g];
              const float k = rs * f.x, e = f.y - m;
              const float2 kk = make_float2(k, k), ee = make_float2(e, e);
              float2 sum = make_float2(0.f, 0.f);
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const int c = 16 * g + i;
                float2 p = fma_f32x2(make_float2(s[c], s[c + 1]), kk, ee);
                p.x = exp2_approx(p.x);
                p.y = exp2_approx(p.y);
                if (LAST) {
                  if (c >= nkeys) p.x = 0.f;
                  if (c + 1 >= nkeys) p.y = 0.f;
                }
                sum = add_f32x2(sum, p);
                pk[c / 2 - 16 * h] = pack_h2(p.x, p.y);
              }
              add = fmaf(sum.x + sum.y, f.z, add);
            }
            // P over scores that have been read
            tmem_st16(tS(j) + lane_off + 16 * h, pk);
          }
          l = fmaf(add, far ? 0.f : fc, l);
          return true;
        };
        ok = nkeys < BK ? tile_softmax(std::true_type{}) : tile_softmax(std::false_type{});
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(j));
      }
      if (ok && T > 0) ok = __all_sync(0xffffffffu, mbar_wait(pv_done(T - 1), par(T - 1), abort_flag, status));
      tc_fence_after();
      if (ok) {
        const float inv = l == 0.f ? 0.f : 1.0f / l;  // a row without keys: zeros
        // the references' difference, in two factors that stay normal floats
        const float ref = exp2_approx(0.5f * (m - lm));
        const size_t pa = (size_t)share * A.part_rows * A.Hq + at;
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          float o[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
          if (T > 0) {
            tmem_ld32_nowait(tO + lane_off + c, o);
            tmem_wait_ld();
          }
          if (!there) continue;
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = o[i] * inv * ref * ref;
          if (A.S > 1) {
            if (T > 0) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(A.part_o + pa * HD + c + i) =
                    make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 8) *reinterpret_cast<uint4*>(A.o + at * HD + c + i) = pack8(o + i);
          }
        }
        if (there && (A.S > 1 || A.st_m)) {
          normal_stats(lm, l);
          if (A.S > 1) {
            A.part_ml[pa * 2] = lm;
            A.part_ml[pa * 2 + 1] = l;
          } else {
            A.st_m[at] = lm / kKv8Log2e;
            A.st_l[at] = l;
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == NC) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_attention_kv8_tc(const Kv8Args& A, long long ctas, int hd, cudaStream_t s) {
  auto go = [&](auto hd_c, auto mix) {
    constexpr int HD = decltype(hd_c)::value;
    return launch_kv8<attn_kv8_tc_kernel<HD, decltype(mix)::value>>((unsigned)ctas, kThreads, Smem<HD>::TOTAL, s, A);
  };
  auto of_hd = [&](auto mix) {
    return hd == 128 ? go(std::integral_constant<int, 128>{}, mix) : go(std::integral_constant<int, 64>{}, mix);
  };
  return (1 << A.blk_log2) < BK ? of_hd(std::true_type{}) : of_hd(std::false_type{});
}

}  // namespace dllm
