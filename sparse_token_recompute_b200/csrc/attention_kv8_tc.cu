// Attention over the 8-bit K/V cache on the 5th-generation tensor cores: tiles of
// 128 packed query rows (see attention_kv8.cu for the arithmetic).
//
// One CTA = one (sequence, kv head), NT tiles of 128 packed rows (A and B) and one
// share of the keys.  Warp roles (32 + 128 + NT * 128 threads):
//   warps 0-3            converters: codes of a K or V tile of 128 keys from global
//                        memory to registers (the next tile's on their way while
//                        this one is converted), one cvt per two codes, and f16 to
//                        a ring of shared-memory slots in the 128-byte-swizzled
//                        layout that TMA would have written;
//   warp 4               TMEM owner and tcgen05.mma issuer;
//   the others           softmax, one packed row per thread (its TMEM lane): the
//                        thread first brings its query row to f16 in shared memory.
// TMEM holds S_A, S_B (fp32, 128 columns each) and O_A, O_B; P (f16 pairs) goes
// over the first 64 columns of S and is read from TMEM by P V.  The issuer
// alternates the groups, PV_A(j) QK_A(j+1) PV_B(j) QK_B(j+1), so that one group's
// softmax overlaps the other's products; operations of one thread complete in
// order, so S(j+1) cannot overwrite P(j) before PV(j) has read it.
// A row reads its scores twice, 64 columns at a time (for the maximum, then for
// the weights), so that a thread stays under 112 registers and, with NT = 1, two
// CTAs share an SM.
// Every mbarrier wait is bounded; a timeout sets DLLM_DEV_TIMEOUT, drains the MMAs,
// frees TMEM and returns.
#include "attention_kv8.cuh"
#include "tmem.cuh"

namespace dllm {

namespace {

constexpr int BT = 128;   // packed rows per tile (= TMEM lanes)
constexpr int BKV = 128;  // keys per tile
constexpr int NSC = 8;    // tiles whose scales are kept: more than the ring runs ahead

template <int NT>
constexpr int nthreads() { return 160 + NT * 128; }
template <int NT>
constexpr uint32_t tmem_cols() { return NT * 256u; }

template <int HD, int NT>
struct Smem {
  static constexpr int Q_TILE = BT * HD * 2;
  static constexpr int SLOT = BKV * HD * 2;
  static constexpr int BUDGET = NT == 2 ? 227 * 1024 : 112 * 1024;
  static constexpr int FIT = (BUDGET - 4096 - NT * Q_TILE) / SLOT;
  static constexpr int SLOTS = FIT < 8 ? FIT : 8;
  static constexpr int RING_OFF = NT * Q_TILE;
  static constexpr int SC_OFF = RING_OFF + SLOTS * SLOT;   // [NSC][8] float4
  static constexpr int BAR_OFF = SC_OFF + NSC * 8 * 16;
  static constexpr int NEED = BAR_OFF + 512 + 1024;        // + alignment slack
  // a pair CTA holds all 512 TMEM columns: one per SM
  static constexpr int TOTAL = (NT == 1 || NEED > 116 * 1024) ? NEED : 116 * 1024;
  static_assert(NT == 2 || 2 * (TOTAL + 1024) <= 228 * 1024, "two one-tile CTAs per SM");
  static_assert(SLOTS >= 2 && SLOTS / 2 < NSC, "the scales' ring outruns the tiles'");
};

// f16 x f16 -> fp32, both operands K-major, M x N tile
constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <int HD, int NT>
__global__ void __launch_bounds__(nthreads<NT>(), NT == 1 ? 2 : 1)
    attn_kv8_tc_kernel(const Kv8Args A) {
  using L = Smem<HD, NT>;
  constexpr int NS = L::SLOTS;
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
  const int all = (len + BKV - 1) / BKV;
  const int per = (all + A.S - 1) / A.S;
  const int k_lo = min(all, share * per);
  const int T = min(all, k_lo + per) - k_lo;  // this CTA's K/V tiles
  const int nq = NT == 2 && R > BT ? 2 : 1;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  float4* scales = reinterpret_cast<float4*>(sm + L::SC_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
  auto q_full = [&](int x) { return smem_u32(&bars[0 + x]); };
  auto s_full = [&](int x) { return smem_u32(&bars[2 + x]); };
  auto p_full = [&](int x) { return smem_u32(&bars[4 + x]); };
  auto pv_done = [&](int x) { return smem_u32(&bars[6 + x]); };
  const uint32_t drain_bar = smem_u32(&bars[8]);
  auto sc_full = [&](int j) { return smem_u32(&bars[9 + j % NSC]); };
  auto full = [&](int n) { return smem_u32(&bars[9 + NSC + n % NS]); };
  auto empty = [&](int n) { return smem_u32(&bars[9 + NSC + NS + n % NS]); };
  static_assert(9 + NSC + 2 * 8 + 1 <= 64, "barrier area holds 64 words");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&bars[9 + NSC + 2 * NS]);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* const status = A.rows.status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sQ = smem_u32(sm);
  const uint32_t sRing = smem_u32(sm + L::RING_OFF);
  // the n-th tile through the ring (K0 V0 K1 V1 ...) is its slot's (n / NS)-th use
  auto use_par = [&](int n) { return (uint32_t)((n / NS) & 1); };
  auto live_warps = [&](int x) {
    const int rows = min(BT, R - x * BT);
    return rows > 0 ? (rows + 31) / 32 : 1;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full(i), 128);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < NSC; ++i) mbar_init(sc_full(i), 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(q_full(x), 128);
      mbar_init(s_full(x), 1);
      mbar_init(p_full(x), 32 * live_warps(x));
      mbar_init(pv_done(x), 1);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 4) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols<NT>());
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto tS = [&](int x) { return tmem + (uint32_t)(x * 128); };
  auto tO = [&](int x) { return tmem + (uint32_t)(NT * 128 + x * 128); };

  if (warp < 4) {
    // ---------------------------------------------------------------- converters
    constexpr int NV = HD / 16;  // 16-byte vectors per thread and tile
    const size_t row_bytes = (size_t)A.Hkv * HD;
    const size_t base = ((size_t)b * N * A.Hkv + kvh) * HD + (size_t)(lane & 3) * 16;
    const int key0 = k_lo * BKV;
    // vector i of a tile: 64-element half i % (HD/64), keys 8 (i / (HD/64)) + lane / 4 of
    // this warp's 32: a warp's load covers 8 rows of 64 bytes, and the 8 lanes of a
    // store phase fall on 8 different bank groups
    auto row_of = [&](int i) { return warp * 32 + i / (HD / 64) * 8 + (lane >> 2); };
    auto fetch = [&](int n, uint4* v) {
      const uint8_t* src = ((n & 1) ? A.v8 : A.k8) + base;
      const int t0 = key0 + (n >> 1) * BKV;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int key = t0 + row_of(i);
        v[i] = make_uint4(0, 0, 0, 0);
        if (key < len)
          v[i] = __ldg(reinterpret_cast<const uint4*>(src + (size_t)key * row_bytes + i % (HD / 64) * 64));
      }
    };
    const size_t sc0 = ((size_t)b * A.Hkv + kvh) * A.nblk;
    uint4 cur[NV], nxt[NV];
    if (T > 0) fetch(0, cur);
    for (int n = 0; n < 2 * T; ++n) {
      if (n + 1 < 2 * T) fetch(n + 1, nxt);
      if (!(n & 1) && warp == 0) {  // the scales of K/V tile n / 2, per 16 keys
        if (lane < 8) {
          const int key = key0 + (n >> 1) * BKV + lane * 16;
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
          if (key < len) {
            s.x = __ldg(A.ks + sc0 + (key >> A.blk_log2));
            v_scale_parts(__ldg(A.vs + sc0 + (key >> A.blk_log2)), s.y, s.z);
          }
          scales[(n >> 1) % NSC * 8 + lane] = s;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sc_full(n >> 1));
      }
      if (!mbar_wait(empty(n), use_par(n) ^ 1u, abort_flag, status)) break;
      const uint32_t slot = sRing + (n % NS) * L::SLOT;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int row = row_of(i);
        const uint32_t q[4] = {cur[i].x, cur[i].y, cur[i].z, cur[i].w};
        uint32_t h[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          h[2 * k] = e4m3x2_to_f16x2(q[k] & 0xffffu);
          h[2 * k + 1] = e4m3x2_to_f16x2(q[k] >> 16);
        }
        const uint32_t at = slot + i % (HD / 64) * (BKV * 128) + row * 128;
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
#pragma unroll
      for (int i = 0; i < NV; ++i) cur[i] = nxt[i];
    }
  } else if (warp == 4) {
    if (lane == 0 && T > 0) {
      // ---------------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = idesc_f16(BT, BKV);
      constexpr uint32_t idesc_pv = idesc_f16(BT, HD) | (1u << 16);  // V read MN-major
      bool ok = true, any = false;
      int n = 0;  // ring tiles consumed
      auto take = [&]() -> int {
        if (!mbar_wait(full(n), use_par(n), abort_flag, status)) return -1;
        tc_fence_after();
        return n++;
      };
      auto give = [&](int i) { tc_commit(empty(i)); };
      auto qk = [&](int x, int i) {
        const uint32_t kb = sRing + (i % NS) * L::SLOT;
        const uint32_t qb = sQ + x * L::Q_TILE;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          tc_mma_bf16(tS(x), umma_desc_k_sw128(qb + (kk >> 2) * (BT * 128) + (kk & 3) * 32),
                      umma_desc_k_sw128(kb + (kk >> 2) * (BKV * 128) + (kk & 3) * 32), idesc_qk,
                      kk > 0 ? 1u : 0u);
        tc_commit(s_full(x));
        any = true;
      };
      auto pv = [&](int x, int j, int i) -> bool {
        if (!mbar_wait(p_full(x), j & 1, abort_flag, status)) return false;
        tc_fence_after();
        const uint32_t vb = sRing + (i % NS) * L::SLOT;
#pragma unroll
        for (int kk = 0; kk < BKV / 16; ++kk)
          tc_mma_ts(tO(x), tS(x) + (uint32_t)(kk * 8), umma_desc_mn_sw128(vb + kk * 2048, BKV * 128),
                    idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
        if (j == T - 1) tc_commit(pv_done(x));
        return true;
      };
      const int k0 = take();
      ok = k0 >= 0;
      for (int x = 0; x < nq && ok; ++x) {
        if (!(ok = mbar_wait(q_full(x), 0, abort_flag, status))) break;
        tc_fence_after();
        qk(x, k0);
      }
      if (ok) give(k0);
      for (int j = 0; j < T && ok; ++j) {
        const int v = take();
        if (!(ok = v >= 0 && pv(0, j, v))) break;
        int k = -1;
        if (j + 1 < T) {
          if (!(ok = (k = take()) >= 0)) break;
          qk(0, k);
        }
        if (nq == 2) {
          if (!(ok = pv(1, j, v))) break;
          if (k >= 0) qk(1, k);
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
    const int x = (warp - 5) >> 2;
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
                                         mbar_wait(s_full(x), j & 1, abort_flag, status));
        if (!ok) break;
        tc_fence_after();
        const float4* sc = scales + j % NSC * 8;
        const int nkeys = min(BKV, len - (k_lo + j) * BKV);
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < BKV; c += 64) {
          float s[64];
          tmem_ld32_nowait(tS(x) + lane_off + c, s);
          tmem_ld32_nowait(tS(x) + lane_off + c + 32, s + 32);
          tmem_wait_ld();
          if (nkeys < c + 64) {
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = c + i < nkeys ? s[i] : -INFINITY;
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float4 f = sc[c / 16 + g];
            float a = fmaxf(s[16 * g], s[16 * g + 1]);
#pragma unroll
            for (int i = 2; i < 16; i += 2) a = fmaxf(a, fmaxf(s[16 * g + i], s[16 * g + i + 1]));
            // (a group past the keys: -inf times a zero scale would be NaN)
            if (c + 16 * g < nkeys) mx = fmaxf(mx, fmaf(a, rs * f.x, f.y));
          }
        }
        const bool need = mx > m + kKv8Lazy;
        const bool rescale = __any_sync(0xffffffffu, need) && j > 0;
        float alpha = 1.f;
        if (need) {
          alpha = exp2_approx(m - mx);  // the first time: 0
          m = mx;
        }
        l *= alpha;
#pragma unroll 1
        for (int c = 0; c < BKV; c += 64) {
          float s[64];
          tmem_ld32_nowait(tS(x) + lane_off + c, s);
          tmem_ld32_nowait(tS(x) + lane_off + c + 32, s + 32);
          tmem_wait_ld();
          uint32_t pk[32];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float4 f = sc[c / 16 + g];
            const float k = rs * f.x, e = f.y - m;
            float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float p0 = exp2_approx(fmaf(s[16 * g + i], k, e));
              float p1 = exp2_approx(fmaf(s[16 * g + i + 1], k, e));
              if (nkeys < c + 64) {
                if (c + 16 * g + i >= nkeys) p0 = 0.f;
                if (c + 16 * g + i + 1 >= nkeys) p1 = 0.f;
              }
              sum0 += p0;
              sum1 += p1;
              pk[8 * g + i / 2] = pack_h2(p0, p1);
            }
            l = fmaf(sum0 + sum1, f.z, l);
          }
          // P of these 64 keys over columns of S that have been read
          tmem_st32(tS(x) + lane_off + c / 2, pk);
        }
        if (rescale) {
          // S(j) complete implies PV(j-1) complete: O is stable until P(j) is ready
#pragma unroll 1
          for (int c = 0; c < HD; c += 32) {
            float o[32];
            tmem_ld32_nowait(tO(x) + lane_off + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= alpha;
            tmem_st32(tO(x) + lane_off + c, reinterpret_cast<const uint32_t*>(o));
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full(x));
      }
      if (ok && T > 0) ok = __all_sync(0xffffffffu, mbar_wait(pv_done(x), 0, abort_flag, status));
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
  if (warp == 4) {
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
