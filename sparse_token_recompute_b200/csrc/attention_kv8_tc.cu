// Attention over the 8-bit K/V cache on the 5th-generation tensor cores: tiles of
// 128 packed query rows (see attention_kv8.cu for the arithmetic).
//
// One CTA = one (sequence, kv head), NT tiles of 128 packed rows (A and B) and one
// share of the keys, 64 keys at a time.  Warp roles:
//   warps 0 .. 3         converters: the codes of a K or V tile by cp.async into a
//                        small ring (each thread reads back what it copied itself),
//                        one cvt per two codes, and f16 to a ring of slots in the
//                        128-byte-swizzled layout that TMA would have written;
//   warp 4               TMEM owner and tcgen05.mma issuer;
//   the others           softmax, one packed row per thread (its TMEM lane): the
//                        thread first brings its query row to f16 in shared memory.
// TMEM holds two score tiles of 64 columns per row tile, and O.  The scores of tile
// j + 1 are computed while tile j is exponentiated; P (f16 pairs) goes over the
// first 32 columns of its scores and is read from TMEM by P V.  Issue order: QK(0)
// QK(1) PV(0) QK(2) PV(1) ...  Operations of one thread complete in order, so
// QK(j+2) cannot overwrite P(j) before PV(j) has read it.  64 keys rather than 128:
// a thread holds its 64 scores in registers, and with NT = 1 two CTAs of 8 warps
// share an SM at 128 registers a thread.
// Every mbarrier wait is bounded; a timeout sets DLLM_DEV_TIMEOUT, drains the MMAs,
// frees TMEM and returns.
#include <type_traits>

#include "attention_kv8.cuh"
#include "tmem.cuh"

namespace dllm {

namespace {

constexpr int BT = 128;   // packed rows per tile (= TMEM lanes)
constexpr int BK = 64;    // keys per tile
constexpr int NSC = 8;    // tiles whose scales are kept: more than the ring runs ahead
constexpr int NC = 4;     // converter warps

template <int NT>
constexpr int nthreads() { return (NC + 1 + NT * 4) * 32; }
template <int NT>
constexpr uint32_t tmem_cols() { return NT * 256u; }

template <int HD, int NT>
struct Smem {
  static constexpr int Q_TILE = BT * HD * 2;
  static constexpr int SLOT = BK * HD * 2;
  static constexpr int RAW = BK * HD;                      // codes of a tile
  static constexpr int RAWS = NT == 1 && HD == 128 ? 2 : 4;
  // two one-tile CTAs share an SM's 228 KB (1 KB of it reserved per CTA)
  static constexpr int BUDGET = NT == 2 ? 227 * 1024 : 113 * 1024;
  static constexpr int FIT = (BUDGET - 1024 - NT * Q_TILE - RAWS * RAW) / SLOT;
  static constexpr int SLOTS = FIT < 8 ? FIT : 8;
  static constexpr int RING_OFF = NT * Q_TILE;
  static constexpr int RAW_OFF = RING_OFF + SLOTS * SLOT;
  static constexpr int SC_OFF = RAW_OFF + RAWS * RAW;      // [NSC][4] float4
  static constexpr int BAR_OFF = SC_OFF + NSC * 4 * 16;
  static constexpr int NEED = BAR_OFF + 48 * 8;
  // a pair CTA holds all 512 TMEM columns: one per SM
  static constexpr int TOTAL = (NT == 1 || NEED > 116 * 1024) ? NEED : 116 * 1024;
  static_assert(TOTAL <= BUDGET, "shared memory");
  static_assert(SLOTS >= 4 && SLOTS / 2 + 4 <= NSC, "the scales' ring outruns the tiles'");
};

// f16 x f16 -> fp32, both operands K-major, M x N tile
constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <int HD, int NT>
__global__ void __launch_bounds__(nthreads<NT>(), NT == 1 ? 2 : 1)
    attn_kv8_tc_kernel(const Kv8Args A) {
  using L = Smem<HD, NT>;
  constexpr int NS = L::SLOTS, NR = L::RAWS;
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
  const int r0 = tile * NT * BT;
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
  const int nq = NT == 2 && R > BT ? 2 : 1;

  extern __shared__ __align__(1024) uint8_t sm[];
  if (smem_u32(sm) & 1023u) {  // the swizzled tiles start at multiples of 1024
    if (threadIdx.x == 0) raise_status(A.rows.status, DEV_BAD_SHAPE);
    return;
  }
  float4* scales = reinterpret_cast<float4*>(sm + L::SC_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
  auto q_full = [&](int x) { return smem_u32(&bars[0 + x]); };
  // per row tile and score buffer (tile j uses buffer j & 1 for the (j / 2)-th time)
  auto s_full = [&](int x, int j) { return smem_u32(&bars[2 + 2 * x + (j & 1)]); };
  auto p_full = [&](int x, int j) { return smem_u32(&bars[6 + 2 * x + (j & 1)]); };
  auto pv_done = [&](int x, int j) { return smem_u32(&bars[10 + 2 * x + (j & 1)]); };
  auto par = [](int j) { return (uint32_t)((j >> 1) & 1); };
  const uint32_t drain_bar = smem_u32(&bars[14]);
  auto sc_full = [&](int j) { return smem_u32(&bars[15 + j % NSC]); };
  auto full = [&](int n) { return smem_u32(&bars[15 + NSC + n % NS]); };
  auto empty = [&](int n) { return smem_u32(&bars[15 + NSC + NS + n % NS]); };
  static_assert(15 + NSC + 2 * 8 + 1 <= 48, "barrier area holds 48 words");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&bars[15 + NSC + 2 * NS]);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* const status = A.rows.status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sQ = smem_u32(sm);
  const uint32_t sRing = smem_u32(sm + L::RING_OFF);
  // The ring's order is the issuer's: K0 K1 V0 K2 V1 ... K(T-1) V(T-2) V(T-1); the n-th
  // entry is its slot's (n / NS)-th use.
  auto use_par = [&](int n) { return (uint32_t)((n / NS) & 1); };
  auto live_warps = [&](int x) {
    const int rows = min(BT, R - x * BT);
    return rows > 0 ? (rows + 31) / 32 : 1;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full(i), 32 * NC);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < NSC; ++i) mbar_init(sc_full(i), 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(q_full(x), 128);
      for (int j = 0; j < 2; ++j) {
        mbar_init(s_full(x, j), 1);
        mbar_init(p_full(x, j), 32 * live_warps(x));
        mbar_init(pv_done(x, j), 1);
      }
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == NC) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols<NT>());
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto tS = [&](int x, int j) { return tmem + (uint32_t)(x * 128 + (j & 1) * 64); };
  auto tO = [&](int x) { return tmem + (uint32_t)(NT * 128 + x * 128); };

  if (warp < NC) {
    // ---------------------------------------------------------------- converters
    constexpr int HB = HD / 64;   // 64-element boxes of a row
    constexpr int NV = 2 * HB;    // 16-byte vectors per thread and tile
    const size_t row_bytes = (size_t)A.Hkv * HD;
    const size_t base = ((size_t)b * N * A.Hkv + kvh) * HD + (size_t)(lane & 3) * 16;
    const int key0 = k_lo * BK;
    const int ring = 2 * T;
    auto is_v = [&](int n) { return n == ring - 1 || (n > 0 && !(n & 1)); };
    auto tile_of = [&](int n) { return n == ring - 1 ? T - 1 : (n & 1) ? (n + 1) / 2 : n > 0 ? n / 2 - 1 : 0; };
    // vector i of a tile: box i % HB of keys 8 (i / HB) + lane / 4 of this warp's 16.  A
    // warp's copy covers 8 rows of 64 bytes, and the 8 lanes of a store phase fall on 8
    // different bank groups.
    auto row_of = [&](int i) { return warp * 16 + i / HB * 8 + (lane >> 2); };
    const uint32_t raw = smem_u32(sm + L::RAW_OFF) + threadIdx.x * 16;
    const size_t sc0 = ((size_t)b * A.Hkv + kvh) * A.nblk;
    const bool scaler = warp == 0 && lane < 4;  // the scales of 16 of a K/V tile's keys
    float2 sc[2];                               // of the K tiles whose copies are on their way
    auto fetch = [&](int n) {
      if (n < ring) {
        const uint8_t* src = (is_v(n) ? A.v8 : A.k8) + base;
        const int t0 = key0 + tile_of(n) * BK;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int key = t0 + row_of(i);  // keys past the last one arrive as zeros
          cp_async16(raw + (n % NR) * L::RAW + i * (NC * 32 * 16),
                     src + (size_t)min(key, len - 1) * row_bytes + i % HB * 64, key < len);
        }
      }
      cp_commit();
    };
    auto fetch_scales = [&](int j) {
      const int key = key0 + j * BK + lane * 16;
      float2 f = make_float2(0.f, 0.f);
      if (scaler && j < T && key < len) {
        f.x = __ldg(A.ks + sc0 + (key >> A.blk_log2));
        f.y = __ldg(A.vs + sc0 + (key >> A.blk_log2));
      }
      return f;
    };
#pragma unroll
    for (int n = 0; n < NR - 1; ++n) fetch(n);
    sc[0] = fetch_scales(0);
    for (int n = 0; n < ring; ++n) {
      fetch(n + NR - 1);
      if (!is_v(n) && warp == 0) {
        const int j = tile_of(n);
        sc[1] = fetch_scales(j + 1);
        if (lane < 4) {
          float4 f = make_float4(sc[0].x, 0.f, 0.f, 0.f);
          if (key0 + j * BK + lane * 16 < len) v_scale_parts(sc[0].y, f.y, f.z);
          scales[j % NSC * 4 + lane] = f;
        }
        sc[0] = sc[1];
        __syncwarp();
        if (lane == 0) mbar_arrive(sc_full(j));
      }
      cp_wait<NR - 1>();
      if (!mbar_wait(empty(n), use_par(n) ^ 1u, abort_flag, status)) break;
      const uint32_t slot = sRing + (n % NS) * L::SLOT;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int row = row_of(i);
        uint32_t q[4], h[8];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3])
                     : "r"(raw + (n % NR) * L::RAW + i * (NC * 32 * 16))
                     : "memory");
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          h[2 * k] = e4m3x2_to_f16x2(q[k] & 0xffffu);
          h[2 * k + 1] = e4m3x2_to_f16x2(q[k] >> 16);
        }
        const uint32_t at = slot + i % HB * (BK * 128) + row * 128;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           at + (((lane & 3) * 2 + c) ^ (row & 7)) * 16),
                       "r"(h[4 * c]), "r"(h[4 * c + 1]), "r"(h[4 * c + 2]), "r"(h[4 * c + 3])
                       : "memory");
      }
      // generic stores before the tensor core's reads
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(full(n));
    }
    cp_wait<0>();
  } else if (warp == NC) {
    if (lane == 0 && T > 0) {
      // ---------------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = idesc_f16(BT, BK);
      constexpr uint32_t idesc_pv = idesc_f16(BT, HD) | (1u << 16);  // V read MN-major
      bool ok = true, any = false;
      int n = 0;  // ring entries consumed
      auto take = [&]() -> int {
        if (!mbar_wait(full(n), use_par(n), abort_flag, status)) return -1;
        tc_fence_after();
        return n++;
      };
      auto give = [&](int i) { tc_commit(empty(i)); };
      auto qk = [&](int x, int j, int i) {
        const uint32_t kb = sRing + (i % NS) * L::SLOT;
        const uint32_t qb = sQ + x * L::Q_TILE;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          tc_mma_bf16(tS(x, j), umma_desc_k_sw128(qb + (kk >> 2) * (BT * 128) + (kk & 3) * 32),
                      umma_desc_k_sw128(kb + (kk >> 2) * (BK * 128) + (kk & 3) * 32), idesc_qk,
                      kk > 0 ? 1u : 0u);
        tc_commit(s_full(x, j));
        any = true;
      };
      auto pv = [&](int x, int j, int i) -> bool {
        if (!mbar_wait(p_full(x, j), par(j), abort_flag, status)) return false;
        tc_fence_after();
        const uint32_t vb = sRing + (i % NS) * L::SLOT;
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          tc_mma_ts(tO(x), tS(x, j) + (uint32_t)(kk * 8), umma_desc_mn_sw128(vb + kk * 2048, BK * 128),
                    idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
        tc_commit(pv_done(x, j));
        return true;
      };
      for (int j = 0; j < 2 && j < T && ok; ++j) {
        const int k = take();
        if (!(ok = k >= 0)) break;
        for (int x = 0; x < nq && ok; ++x) {
          if (j == 0 && !(ok = mbar_wait(q_full(x), 0, abort_flag, status))) break;
          tc_fence_after();
          qk(x, j, k);
        }
        if (ok) give(k);
      }
      for (int j = 0; j < T && ok; ++j) {
        const int v = take();
        if (!(ok = v >= 0 && pv(0, j, v))) break;
        int k = -1;
        if (j + 2 < T) {
          if (!(ok = (k = take()) >= 0)) break;
          qk(0, j + 2, k);
        }
        if (nq == 2) {
          if (!(ok = pv(1, j, v))) break;
          if (k >= 0) qk(1, j + 2, k);
        }
        give(v);
        if (k >= 0) give(k);
      }
      if (!ok && any) {
        tc_commit(drain_bar);
        mbar_wait_drain(drain_bar, 0, status);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    const int x = (warp - NC - 1) >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;  // packed row in the tile (= TMEM lane)
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const bool there = x * BT + r < R;
    const int pr = r0 + x * BT + r;
    const size_t at = (size_t)(off + (there ? pr / A.G : 0)) * A.Hq + kvh * A.G + pr % A.G;
    float rs = 0.f;  // log2 units per raw score
    if (x < nq && T > 0) {
      uint4 raw[HD / 8];
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        raw[i] = there ? *(reinterpret_cast<const uint4*>(A.q + at * HD) + i) : make_uint4(0, 0, 0, 0);
        mx = __vmaxu2(mx, raw[i].x & 0x7fff7fffu);
        mx = __vmaxu2(mx, raw[i].y & 0x7fff7fffu);
        mx = __vmaxu2(mx, raw[i].z & 0x7fff7fffu);
        mx = __vmaxu2(mx, raw[i].w & 0x7fff7fffu);
      }
      const int sh = query_shift(__uint_as_float(max(mx & 0xffffu, mx >> 16) << 16));
      const float f0 = pow2i(sh / 2), f1 = pow2i(sh - sh / 2);
      rs = A.scale_log2 * pow2i(-(sh / 2)) * pow2i(-(sh - sh / 2));
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        float f[8];
        unpack8(raw[i], f);
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = pack_h2(f[2 * k] * f0 * f1, f[2 * k + 1] * f0 * f1);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         sQ + x * L::Q_TILE + (i >> 3) * (BT * 128) + r * 128 + ((i & 7) ^ (r & 7)) * 16),
                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                     : "memory");
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(q_full(x));
    }
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    // a warp whose 32 rows are all past the sequence's rows takes no further part
    const bool live = x < nq && quad < live_warps(x);
    if (live) {
      for (int j = 0; j < T; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(sc_full(j), (j / NSC) & 1, abort_flag, status) &&
                                         mbar_wait(s_full(x, j), par(j), abort_flag, status));
        if (!ok) break;
        tc_fence_after();
        float s[BK];
        tmem_ld32_nowait(tS(x, j) + lane_off, s);
        tmem_ld32_nowait(tS(x, j) + lane_off + 32, s + 32);
        const float4* sc = scales + j % NSC * 4;
        float k[4], e[4], w[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float4 f = sc[g];
          k[g] = rs * f.x, e[g] = f.y, w[g] = f.z;
        }
        const int nkeys = len - (k_lo + j) * BK;
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
            if (!LAST || 16 * g < nkeys) mx = fmaxf(mx, fmaf(fmaxf(a, c), k[g], e[g]));
          }
          const bool need = mx > m + kKv8Lazy;
          if (__any_sync(0xffffffffu, need)) {
            const float alpha = need ? exp2_approx(m - mx) : 1.f;  // the first time: 0
            if (need) m = mx;
            l *= alpha;
            if (j > 0) {
              // O may be rescaled once PV(j-1) is complete, until P(j) is handed over
              if (!__all_sync(0xffffffffu, mbar_wait(pv_done(x, j - 1), par(j - 1), abort_flag, status)))
                return false;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < HD; c += 16) {
                float o[16];
                tmem_ld16(tO(x) + lane_off + c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= alpha;
                tmem_st16(tO(x) + lane_off + c, reinterpret_cast<const uint32_t*>(o));
              }
            }
          }
          uint32_t pk[32];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float2 kk = make_float2(k[g], k[g]), ee = make_float2(e[g] - m, e[g] - m);
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
              pk[c / 2] = pack_h2(p.x, p.y);
            }
            l = fmaf(sum.x + sum.y, w[g], l);
          }
          tmem_st32(tS(x, j) + lane_off, pk);  // P over scores that have been read
          return true;
        };
        ok = nkeys < BK ? tile_softmax(std::true_type{}) : tile_softmax(std::false_type{});
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full(x, j));
      }
      if (ok && T > 0) ok = __all_sync(0xffffffffu, mbar_wait(pv_done(x, T - 1), par(T - 1), abort_flag, status));
      tc_fence_after();
      if (ok) {
        const float inv = l == 0.f ? 0.f : 1.0f / l;  // a row without keys: zeros
        const size_t pa = (size_t)share * A.part_rows * A.Hq + at;
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          float o[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
          if (T > 0) {
            tmem_ld32_nowait(tO(x) + lane_off + c, o);
            tmem_wait_ld();
          }
          if (!there) continue;
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= inv;
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
          normal_stats(m, l);
          if (A.S > 1) {
            A.part_ml[pa * 2] = m;
            A.part_ml[pa * 2 + 1] = l;
          } else {
            A.st_m[at] = m / kKv8Log2e;
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
    tmem_dealloc(tmem, tmem_cols<NT>());
  }
}

template <int HD, int NT>
cudaError_t go(const Kv8Args& A, long long ctas, cudaStream_t s) {
  return launch_kv8<attn_kv8_tc_kernel<HD, NT>>((unsigned)ctas, nthreads<NT>(), Smem<HD, NT>::TOTAL, s, A);
}

}  // namespace

cudaError_t launch_attention_kv8_tc(const Kv8Args& A, int nt, long long ctas, int hd, cudaStream_t s) {
  if (nt == 1) return hd == 128 ? go<128, 1>(A, ctas, s) : go<64, 1>(A, ctas, s);
  return hd == 128 ? go<128, 2>(A, ctas, s) : go<64, 2>(A, ctas, s);
}

}  // namespace dllm
