"""GPU parity of the 8-bit K/V cache operators against the oracle in 64 bits.

The write and the read are exact (powers of two and one rounding each): codes and
scales are compared for equality.  The norm's bound counts its fp32 roundings and
the one of the store; the attention's counts the roundings of the weights to f16
(half a step is 2^-11 of a weight), of the fp32 scores, and of the store to bf16
(half a step is 2^-8)."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from _util import f64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rows_of(B, N, counts, seed):
    """idx [B, k_cap] (-7 past each count), count, and per row (sequence, position)."""
    rng = np.random.default_rng(seed)
    k = max(max(counts), 1)
    idx = np.full((B, k), -7, dtype=np.int32)
    for b, c in enumerate(counts):
        idx[b, :c] = np.sort(rng.choice(N, size=c, replace=False))
    b_of = np.concatenate([np.full(c, b) for b, c in enumerate(counts)]).astype(int)
    pos = np.concatenate([idx[b, :c] for b, c in enumerate(counts)]).astype(int)
    return (torch.from_numpy(idx).cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda"),
            b_of, pos, k)


def normal(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale


def decoded(c8, sc, block):
    N = c8.shape[1]
    s = f64(sc).repeat(block, axis=2)[:, :, :N].transpose(0, 2, 1)[..., None]
    return f64(c8.view(torch.float8_e4m3fn).float()) * s


def filled(lib, B, N, H, hd, block, seed, spread=3):
    """A cache of random codes whose scales differ by up to 2^spread from block to block."""
    c = lib.kv8_cache(B, N, H, hd, block)
    for i, t in enumerate(c):
        if i % 2 == 0:
            t.copy_((normal(t.shape, seed + i) * 100).clamp(-448, 448).to(torch.float8_e4m3fn))
        else:
            g = torch.Generator(device="cuda").manual_seed(seed + i)
            t.copy_(torch.exp2(torch.randint(-7, -6 + spread, t.shape, generator=g, device="cuda").float()))
    return c


# ------------------------------------------------------------------ norm and rotation

def norm_ref(x, g, pos, theta, eps, H):
    y = O.rms_norm(f64(x).reshape(len(pos), H, -1), f64(g), eps)
    half = y.shape[-1] // 2
    mag = np.abs(y[..., :half]) + np.abs(y[..., half:])   # |a cos| + |b sin| at most
    return O.rope(y, pos, theta).reshape(len(pos), -1), np.concatenate([mag, mag], -1).reshape(len(pos), -1)


@pytest.mark.parametrize("dtype,Hq,Hkv,hd", [("bf16", 28, 4, 128), ("bf16", 32, 32, 128), ("bf16", 6, 2, 64),
                                             ("bf16", 2, 2, 64), ("bf16", 144, 8, 128), ("bf16", 64, 32, 128),
                                             ("f32", 4, 4, 64), ("f32", 3, 1, 10),
                                             ("f32", 2, 1, 256)])
@pytest.mark.parametrize("counts,N", [([1, 0, 3], 17), ([70, 33], 200), ([1], 1)])
@pytest.mark.parametrize("cache", [False, True])
def test_norm_matches_oracle(lib, dtype, Hq, Hkv, hd, counts, N, cache):
    dt = BF if dtype == "bf16" else torch.float32
    B, eps, theta = len(counts), 1e-5, 5e5
    idx, cnt, b_of, pos, k = rows_of(B, N, counts, 1)
    M, R = len(pos), B * k
    # rows with a stride of their own: slices of a wider tensor
    wide = normal((R, (Hq + Hkv) * hd + 16), 2, 3.0).to(dt)
    q, kk = wide[:, :Hq * hd], wide[:, Hq * hd:(Hq + Hkv) * hd]
    qg, kg = (1 + 0.3 * normal((hd,), 3)).to(dt), (1 + 0.3 * normal((hd,), 4)).to(dt)
    rope = torch.zeros(N, hd // 2, 2, device="cuda")
    lib.dllm_rope_table(rope, theta)
    qo = torch.full((R, Hq * hd), 7.0, dtype=dt, device="cuda")
    ko = torch.full((B, N, Hkv, hd) if cache else (R, Hkv * hd), 7.0, dtype=dt, device="cuda")
    ws = lib.Workspace(256)
    lib.dllm_qk_norm_rope(q, kk, qg, kg, rope, qo, ko, idx, cnt, eps, ws=ws)
    assert ws.device_status() == 0
    rq, mq = norm_ref(q[:M], qg, pos, theta, eps, Hq)
    rk, mk = norm_ref(kk[:M], kg, pos, theta, eps, Hkv)
    gk = ko[torch.from_numpy(b_of), torch.from_numpy(pos)].reshape(M, -1) if cache else ko[:M]
    # fp32: hd/8 + 3 additions of one sign, the root (2 steps), three products and the
    # rotation's two, on |a| + |b|; the table's sine and cosine are half a step off
    fp32 = (hd / 8 + 3 + 2 + 3 + 3 + 2) * 2.0 ** -24
    for got, ref, mag in ((qo[:M], rq, mq), (gk, rk, mk)):
        tol = fp32 * mag + (2.0 ** -8 * (np.abs(ref) + fp32 * mag) if dtype == "bf16" else 0.0)
        assert np.all(np.abs(f64(got) - ref) <= tol)
    assert torch.all(qo[M:] == 7.0)
    if cache:
        other = torch.ones(B, N, dtype=torch.bool)
        other[torch.from_numpy(b_of), torch.from_numpy(pos)] = False
        assert torch.all(ko[other.cuda()] == 7.0)
    else:
        assert torch.all(ko[M:] == 7.0)


def test_norm_in_place_zero_rows_far_positions_and_no_rotation(lib):
    B, N, H, hd = 1, 120000, 2, 128
    idx = torch.tensor([[0, 7, 119999]], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([3], dtype=torch.int32, device="cuda")
    pos = np.array([0, 7, 119999])
    g = torch.ones(hd, dtype=BF, device="cuda")
    rope = torch.zeros(N, hd // 2, 2, device="cuda")
    lib.dllm_rope_table(rope, 1e4)
    x = normal((3, H * hd), 5).to(BF)
    x[1] = 0                                    # 0 / sqrt(0 + eps)
    rq, _ = norm_ref(x, g, pos, 1e4, 1e-6, H)
    r0, _ = norm_ref(x, g, pos, 0.0, 1e-6, H)
    q, k = x.clone(), x.clone()
    lib.dllm_qk_norm_rope(q, k, g, g, rope, q, k, idx, cnt, 1e-6)
    assert torch.equal(q, k) and torch.all(q[1] == 0)
    assert np.all(np.abs(f64(q) - rq) <= 2.0 ** -8 * np.abs(rq) + 2.0 ** -18 * 8)
    lib.dllm_qk_norm_rope(x, k, g, g, None, q, k, idx, cnt, 1e-6, N=N)
    assert np.all(np.abs(f64(q) - r0) <= 2.0 ** -8 * np.abs(r0) + 2.0 ** -18 * 8)


# ------------------------------------------------------------------ write and read

def write_ref(cache, k, v, b_of, pos, block):
    k8, ks, v8, vs = cache
    out = []
    for c8, sc, x in ((k8, ks, k), (v8, vs, v)):
        val, s = decoded(c8, sc, block), f64(sc).copy()
        O.kv8_write(val, s, f64(x[:len(pos)]).reshape(len(pos), val.shape[2], -1), b_of, pos, block)
        out += [val, s]
    return out


def assert_cache(cache, ref, block):
    for i in (0, 2):
        assert np.array_equal(f64(cache[i + 1]), ref[i + 1])
        assert np.array_equal(decoded(cache[i], cache[i + 1], block), ref[i], equal_nan=True)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("B,N,H,hd,counts", [
    (1, 1, 2, 64, [1]), (2, 100, 1, 128, [100, 37]), (3, 333, 5, 128, [40, 0, 333]), (2, 257, 9, 64, [1, 200])])
def test_write_and_read_match_oracle(lib, block, B, N, H, hd, counts):
    idx, cnt, b_of, pos, k = rows_of(B, N, counts, block)
    M, R = len(pos), B * k
    wide = normal((R, 2 * H * hd + 8), 7, 2.0).to(BF)
    kk, vv = wide[:, :H * hd], wide[:, H * hd + 8:]
    for cache in (lib.kv8_cache(B, N, H, hd, block), filled(lib, B, N, H, hd, block, 9)):
        ref = write_ref(cache, kk, vv, b_of, pos, block)
        ws = lib.Workspace(256)
        lib.dllm_kv8_write(kk, vv, idx, cnt, *cache, block, ws=ws)
        assert ws.device_status() == 0
        assert_cache(cache, ref, block)
        before = [t.clone() for t in cache]
        lib.dllm_kv8_write(kk, vv, idx, cnt, *cache, block)    # the same rows again: no change
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache, before))
        ko = torch.full((R, H * hd + 8), 7.0, dtype=BF, device="cuda")
        vo = torch.full((R, H * hd), 7.0, dtype=BF, device="cuda")
        lib.dllm_kv8_read(*cache, idx, cnt, ko[:, :H * hd], vo, block, ws=ws)
        assert ws.device_status() == 0
        for got, val in ((ko[:, :H * hd], ref[0]), (vo, ref[2])):
            assert np.array_equal(f64(got[:M]), val[b_of, pos].reshape(M, -1))
            assert torch.all(got[M:] == 7.0)
        assert torch.all(ko[:, H * hd:] == 7.0)


def test_write_of_whole_sequences_without_a_list(lib):
    B, N, H, hd, block = 2, 90, 3, 64, 32
    kk, vv = normal((B * N, H * hd), 1).to(BF), normal((B * N, H * hd), 2).to(BF)
    cache = filled(lib, B, N, H, hd, block, 3)
    b_of, pos = np.repeat(np.arange(B), N), np.tile(np.arange(N), B)
    ref = write_ref(cache, kk, vv, b_of, pos, block)
    lib.dllm_kv8_write(kk, vv, None, None, *cache, block)
    assert_cache(cache, ref, block)
    ko, vo = torch.zeros_like(kk), torch.zeros_like(vv)
    lib.dllm_kv8_read(*cache, None, None, ko, vo, block)
    assert np.array_equal(f64(ko), ref[0].reshape(B * N, -1))
    # a prefix of each sequence: count without positions
    cnt = torch.tensor([5, 40], dtype=torch.int32, device="cuda")
    b_of = np.repeat([0, 1], [5, 40])
    pos = np.concatenate([np.arange(5), np.arange(40)])
    ref = write_ref(cache, 9 * kk, vv, b_of, pos, block)
    lib.dllm_kv8_write(9 * kk, vv, None, cnt, *cache, block)
    assert_cache(cache, ref, block)


def test_write_of_extreme_values(lib):
    """Zeros, the smallest and largest bf16 values, infinities and NaN, alone and among others."""
    B, N, H, hd, block = 1, 64, 8, 64, 16
    x = normal((64, H, hd), 4)
    x[:16, 0] = 0
    x[:16, 1] = 2.0 ** -133
    x[:16, 2] *= 1e38
    x[:16, 3, 5] = math.inf
    x[:16, 4, 6] = math.nan
    x[:16, 5] = math.nan
    x[:16, 6] = -math.inf
    x[:16, 7] *= 2.0 ** -60
    x[16:32] *= 2.0 ** torch.randint(-30, 30, (16, 1, 1), generator=torch.Generator().manual_seed(1)).cuda()
    kk = x.to(BF).reshape(64, -1)
    for rows in (np.arange(64), np.arange(0, 64, 3)):
        cache = lib.kv8_cache(B, N, H, hd, block)
        idx = torch.from_numpy(rows.astype(np.int32))[None].cuda()
        ref = write_ref(cache, kk, kk, np.zeros(len(rows), int), rows, block)
        lib.dllm_kv8_write(kk, kk, idx, None, *cache, block)
        assert_cache(cache, ref, block)


def test_bad_lists_are_flagged_and_stay_inside(lib):
    B, N, H, hd, block = 3, 40, 2, 64, 16
    idx = torch.tensor([[3, 3, 39], [-1, 5, 40], [9, 4, 2147483647]], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([3, 3, 9], dtype=torch.int32, device="cuda")
    kk = torch.ones(9, H * hd, dtype=BF, device="cuda")
    guard = torch.zeros(3 * B * N, H, hd, dtype=torch.uint8, device="cuda")   # the cache between two guards
    k8 = guard[B * N:2 * B * N].view(B, N, H, hd)
    _, ks, v8, vs = lib.kv8_cache(B, N, H, hd, block)
    ws = lib.Workspace(256)
    lib.dllm_kv8_write(kk, kk, idx, cnt, k8, ks, v8, vs, block, ws=ws)
    assert ws.device_status() == lib.DLLM_DEV_BAD_INDEX | lib.DLLM_DEV_CAPACITY
    assert not guard[:B * N].any() and not guard[2 * B * N:].any()
    ko, vo = torch.full_like(kk, 7.0), torch.full_like(kk, 7.0)
    lib.dllm_kv8_read(k8, ks, v8, vs, idx, cnt, ko, vo, block, ws=ws)
    assert ws.device_status() == lib.DLLM_DEV_BAD_INDEX | lib.DLLM_DEV_CAPACITY
    assert torch.all(ko[3] == 7.0) and torch.all(ko[5] == 7.0) and torch.all(ko[8] == 7.0)
    assert torch.all(ko[0] == 1.0) and torch.all(ko[4] == 1.0)
    q = normal((9, H * hd), 1).to(BF)
    qo, kc = torch.full_like(q, 7.0), torch.full((3 * B, N, H, hd), 7.0, dtype=BF, device="cuda")
    g = torch.ones(hd, dtype=BF, device="cuda")
    lib.dllm_qk_norm_rope(q, kk, g, g, None, qo, kc[B:2 * B], idx, cnt, 1e-5, ws=ws)
    assert ws.device_status() == lib.DLLM_DEV_BAD_INDEX | lib.DLLM_DEV_CAPACITY
    assert torch.all(kc[:B] == 7.0) and torch.all(kc[2 * B:] == 7.0)
    assert torch.all(qo[3] == 7.0) and torch.all(qo[5] == 7.0)


# ------------------------------------------------------------------ attention

def attention_ref(q, K, V, vs, n, Hkv):
    """Oracle attention of q [R, Hq, hd] over the first n keys, with per-element bounds of the
    kernel's roundings (before the store) and the log-sum-exp.  vs [N, Hkv]: V scale of each key."""
    R, Hq, hd = q.shape
    o, tol = np.zeros((R, Hq, hd)), np.zeros((R, Hq, hd))
    lse = np.full((R, Hq), -np.inf)
    if n == 0:
        return o, tol, lse
    for h in range(Hq):
        g = h * Hkv // Hq
        k, v = K[:n, g], V[:n, g]
        s = q[:, h] @ k.T / math.sqrt(hd)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        l = p.sum(1, keepdims=True)
        o[:, h] = p @ v / l
        lse[:, h] = (m + np.log(l))[:, 0]
        # the score: hd/16 products of 16 added in fp32 with a truncating adder (2^-23 of the
        # largest partial sum each), its product with the scale and the reference (2^-24 each)
        mag = np.abs(q[:, h]) @ np.abs(k).T / math.sqrt(hd)
        ds = ((hd / 16 + 2) * 2.0 ** -23 * mag + 2.0 ** -22 * np.abs(s)).max(1, keepdims=True)
        # weights p_j * scale_j: 2^-11 of each, and 2^-25 of the largest one where they are
        # subnormal in f16; sums over n keys in fp32: n/16 additions of 2^-23 at most
        rel = 2.0 ** -11 + 2 * ds + n / 16 * 2.0 ** -23 + 2.0 ** -20
        w = (p * vs[:n, g]).max(1, keepdims=True)
        tol[:, h] = (rel * (p @ np.abs(v)) + 2.0 ** -25 * w * np.abs(v / vs[:n, g, None]).sum(0)) / l
    return o, tol, lse


def check_attention(lib, q, cache, block, counts, lens, stats=True):
    k8, ks, v8, vs = cache
    B, N, Hkv, hd = k8.shape
    k_cap = max(max(counts), 1)
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    kvl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o = torch.full_like(q, 7.0)
    Hq = q.shape[1] // hd
    m = torch.zeros(B * k_cap, Hq, device="cuda") if stats else None
    l = torch.zeros(B * k_cap, Hq, device="cuda") if stats else None
    ws = lib.dllm_attention_kv8(q, k8, ks, v8, vs, o, cnt, k_cap, block, kv_len=kvl, m=m, l=l)
    assert ws.device_status() == 0
    K, V = decoded(k8, ks, block), decoded(v8, vs, block)
    per_key = f64(vs).repeat(block, axis=2)[:, :, :N].transpose(0, 2, 1)
    off = 0
    for b, c in enumerate(counts):
        n = N if lens is None else lens[b]
        ref, tol, lse = attention_ref(f64(q[off:off + c]).reshape(c, Hq, hd), K[b], V[b], per_key[b], n,
                                      Hkv)
        got = f64(o[off:off + c]).reshape(c, Hq, hd)
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        assert np.all(np.abs(got - ref) <= tol), (b, np.max(np.abs(got - ref) - tol))
        if stats:
            gm, gl = f64(m[off:off + c]), f64(l[off:off + c])
            if n == 0:
                assert np.all(gm == -np.inf) and np.all(gl == 0)
            else:
                assert np.all((gl >= 1) & (gl < 2))
                assert np.all(np.abs(gm + np.log(gl) - lse) <= 2.0 ** -20 * np.abs(lse) + 2e-3)
        off += c
    assert torch.all(o[off:] == 7.0)
    return o


ATTN = [  # B, N, Hq, Hkv, hd, block, counts, lens
    (1, 1, 1, 1, 128, 16, [1], None),
    (2, 40, 2, 2, 64, 32, [3, 1], [40, 0]),
    (3, 333, 7, 1, 128, 64, [2, 0, 5], [333, 5, 17]),
    (2, 1000, 8, 2, 64, 16, [4, 4], [999, 129]),
    (1, 3000, 28, 4, 128, 128, [1], None),
    (4, 700, 4, 4, 128, 64, [16, 17, 1, 33], [700, 128, 1, 257]),
    (2, 513, 4, 4, 128, 32, [129, 300], [513, 384]),
    (1, 768, 4, 4, 128, 64, [77], None),
    (2, 400, 6, 2, 64, 64, [100, 257], [400, 130]),
    (3, 200, 14, 2, 128, 16, [103, 9, 40], [200, 0, 63]),
    (1, 1536, 2, 2, 128, 64, [1536], None),
]


@pytest.mark.parametrize("B,N,Hq,Hkv,hd,block,counts,lens", ATTN)
def test_attention_matches_oracle(lib, B, N, Hq, Hkv, hd, block, counts, lens):
    cache = filled(lib, B, N, Hkv, hd, block, 11)
    q = normal((B * max(counts), Hq * hd), 12, 2.0).to(BF)
    check_attention(lib, q, cache, block, counts, lens)


@pytest.mark.parametrize("rows", [2, 200])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_ignores_what_lies_past_the_length(lib, rows, hd):
    B, N, H, block = 2, 500, 2, 64
    cache = filled(lib, B, N, H, hd, block, 21)
    q = normal((B * rows, H * hd), 22).to(BF)
    lens = [131, 320]
    want = check_attention(lib, q, cache, block, [rows, rows], lens)
    for b, n in enumerate(lens):
        for i in (0, 2):
            cache[i].view(torch.uint8)[b, n:] = 0x7f            # NaN codes, and NaN scales of
            cache[i + 1][b, :, -(-n // block):] = math.nan      # the blocks without a live key
    got = torch.full_like(q, 7.0)
    lib.dllm_attention_kv8(q, *cache, got, torch.tensor([rows, rows], dtype=torch.int32, device="cuda"), rows,
                           block, kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows", [3, 200])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_over_scales_far_apart(lib, rows, hd):
    """V scales 2^40 apart between blocks, with queries that attend to the blocks of the small
    ones; K scales 2^20 apart; query rows from 2^-60 to 2^3."""
    B, N, H, block = 1, 300, 2, 16
    k8, ks, v8, vs = filled(lib, B, N, H, hd, block, 31)
    e = torch.arange(ks.shape[2], device="cuda")
    vs.copy_(torch.exp2(-(e * 7 % 41).float()).expand_as(vs))
    ks.copy_(torch.exp2(-6 - (e * 5 % 21).float()).expand_as(ks))
    q = normal((rows, H * hd), 32)
    # a row each aligned with one key, so that its block holds nearly all the weight
    for r in range(0, rows, 2):
        key = (r * 37) % N
        kk = k8[0, key].float()
        q[r] = (kk / kk.norm(dim=1, keepdim=True) * 40 / ks[0, :, key // block, None] / 448).flatten()
    q[1::2] *= torch.exp2(torch.linspace(-60, 3, q[1::2].shape[0], device="cuda"))[:, None]
    check_attention(lib, q.to(BF), (k8, ks, v8, vs), block, [rows], None)


@pytest.mark.parametrize("rows", [1, 130])
def test_attention_with_rising_scores(lib, rows):
    """Later keys with ever larger scores raise the reference maximum again and again."""
    B, N, H, hd, block = 1, 2000, 1, 128, 64
    k8, ks, v8, vs = filled(lib, B, N, H, hd, block, 41)
    ks.copy_(torch.exp2(torch.linspace(-14, -4, ks.shape[2], device="cuda").round()).expand_as(ks))
    q = normal((rows, H * hd), 42, 1.5).to(BF)
    check_attention(lib, q, (k8, ks, v8, vs), block, [rows], None)


def test_attention_of_non_finite_queries_stays_in_its_row(lib):
    B, N, H, hd, block = 1, 200, 1, 128, 64
    for rows in (4, 140):
        cache = filled(lib, B, N, H, hd, block, 51)
        q = normal((rows, H * hd), 52).to(BF)
        cnt = torch.tensor([rows], dtype=torch.int32, device="cuda")
        want, got = torch.zeros_like(q), torch.zeros_like(q)
        lib.dllm_attention_kv8(q, *cache, want, cnt, rows, block)
        q[1, 3] = math.nan
        q[2, 5] = math.inf
        lib.dllm_attention_kv8(q, *cache, got, cnt, rows, block)
        keep = [r for r in range(rows) if r not in (1, 2)]
        assert torch.equal(got[keep], want[keep]) and torch.isnan(got[1]).all()


def test_lengths_out_of_range_are_clamped_and_flagged(lib):
    B, N, H, hd, block = 2, 50, 1, 64, 16
    cache = filled(lib, B, N, H, hd, block, 61)
    q = normal((2, hd), 62).to(BF)
    o, ref = torch.zeros_like(q), torch.zeros_like(q)
    one = torch.ones(2, dtype=torch.int32, device="cuda")
    ws = lib.dllm_attention_kv8(q, *cache, o, one, 1, block,
                                kv_len=torch.tensor([99, -3], dtype=torch.int32, device="cuda"))
    assert ws.device_status() == lib.DLLM_DEV_BAD_SHAPE
    lib.dllm_attention_kv8(q, *cache, ref, one, 1, block,
                           kv_len=torch.tensor([50, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(o, ref) and torch.all(o[1] == 0)
    # no cached position at all: zeros
    empty = lib.kv8_cache(2, 0, H, hd, block)
    lib.dllm_attention_kv8(q, *empty, o, one, 1, block)
    assert torch.all(o == 0)


def test_attention_past_32_bit_offsets(lib):
    """A cache of more than 2^32 codes: the last sequence lies behind the 32-bit offsets."""
    B, N, H, hd, block = 9, 131072, 32, 128, 128
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    k8 = torch.zeros(B, N, H, hd, dtype=torch.uint8, device="cuda")
    v8 = torch.zeros(B, N, H, hd, dtype=torch.uint8, device="cuda")
    s = torch.full((B, H, N // block), 2.0 ** -6, device="cuda")
    n = 300
    rows = normal((n, H * hd), 1).to(BF)
    idx = torch.full((B, n), -1, dtype=torch.int32, device="cuda")
    idx[B - 1] = torch.arange(N - n, N, device="cuda")
    cnt = torch.zeros(B, dtype=torch.int32, device="cuda")
    cnt[B - 1] = n
    big = torch.zeros(B * n, H * hd, dtype=BF, device="cuda")
    big[:n] = rows
    lib.dllm_kv8_write(big, big, idx, cnt, k8, s, v8, s.clone(), block)
    out = torch.zeros_like(big)
    lib.dllm_kv8_read(k8, s, v8, s, idx, cnt, out, out.clone(), block)
    step = 2.0 ** -4 * rows.float().abs() + 2.0 ** -16
    assert torch.all((out[:n].float() - rows.float()).abs() <= step)
    q = normal((B, H * hd), 2).to(BF)
    one = torch.zeros(B, dtype=torch.int32, device="cuda")
    one[B - 1] = 1
    o, o2 = torch.zeros_like(q), torch.zeros_like(q)
    lib.dllm_attention_kv8(q, k8, s, v8, s, o, one, 1, block)
    # the same sequence as a cache of its own
    c = lambda t: t[B - 1:].contiguous()
    one1 = torch.ones(1, dtype=torch.int32, device="cuda")
    ws = lib.dllm_attention_kv8(q[:1], c(k8), c(s), c(v8), c(s), o2[:1], one1, 1, block)
    assert ws.device_status() == 0
    assert torch.allclose(o[0].float(), o2[0].float(), rtol=2.0 ** -7, atol=1e-5) and o[0].abs().sum() > 0


# ------------------------------------------------------------------ together

def chain(lib, st, ws, stream=None):
    lib.dllm_qk_norm_rope(st["q"], st["k"], st["g"], st["g"], st["rope"], st["qn"], st["kn"], st["idx"],
                          st["cnt"], 1e-5, stream=stream)
    lib.dllm_kv8_write(st["kn"], st["v"], st["idx"], st["cnt"], *st["cache"], st["block"], stream=stream)
    return lib.dllm_attention_kv8(st["qn"], *st["cache"], st["o"], st["cnt"], st["kcap"], st["block"], ws=ws,
                                  stream=stream)


def chain_state(lib, seed, counts=(50, 3), N=300, Hq=4, Hkv=2, hd=128, block=32):
    B = len(counts)
    idx, cnt, b_of, pos, k = rows_of(B, N, list(counts), seed)
    rope = torch.zeros(N, hd // 2, 2, device="cuda")
    lib.dllm_rope_table(rope, 1e4)
    R = B * k
    st = dict(idx=idx, cnt=cnt, rope=rope, kcap=k, block=block, cache=filled(lib, B, N, Hkv, hd, block, seed),
              q=normal((R, Hq * hd), seed + 1).to(BF), k=normal((R, Hkv * hd), seed + 2).to(BF),
              v=normal((R, Hkv * hd), seed + 3).to(BF), g=(1 + 0.1 * normal((hd,), seed + 4)).to(BF))
    for n, t in (("qn", "q"), ("kn", "k"), ("o", "q")):
        st[n] = torch.zeros_like(st[t])
    st.update(b_of=b_of, pos=pos)
    return st


def test_the_operators_together(lib):
    st = chain_state(lib, 71)
    before = [t.clone() for t in st["cache"]]
    ws = chain(lib, st, None)
    assert ws.device_status() == 0
    M, pos, b_of = len(st["pos"]), st["pos"], st["b_of"]
    # each stage against the oracle on what the stage before it stored
    ref = write_ref(before, st["kn"], st["v"], b_of, pos, st["block"])
    assert_cache(st["cache"], ref, st["block"])
    rk, mk = norm_ref(st["k"][:M], st["g"], pos, 1e4, 1e-5, 2)
    assert np.all(np.abs(f64(st["kn"][:M]) - rk) <= 2.0 ** -8 * np.abs(rk) + 2.0 ** -18 * mk)
    check_attention(lib, st["qn"], st["cache"], st["block"], [50, 3], None)
    # and the whole chain against the oracle's own: two roundings of q and k to bf16 move a
    # score by 2 * 2^-8 of sum |q k| at most, a code by one e4m3 step where it lies at a border
    o2 = torch.zeros_like(st["o"])
    lib.dllm_attention_kv8(st["qn"], *st["cache"], o2, st["cnt"], st["kcap"], st["block"])
    assert torch.equal(o2, st["o"])                      # deterministic


@pytest.mark.parametrize("counts", [(1, 1), (60, 7), (150, 300)])
def test_two_captured_chains_replay_beside_each_other(lib, counts):
    N = 320
    a, b = (chain_state(lib, s, counts, N) for s in (81, 91))
    ref = []
    for st in (a, b):
        st["ws"] = chain(lib, st, None)
        torch.cuda.synchronize()
        ref.append(st["o"].clone())
    graphs, streams = [], []
    for st in (a, b):
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            chain(lib, st, st["ws"])
        graphs.append(g)
        streams.append(s)
    for st in (a, b):
        st["o"].zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a["o"], ref[0]) and torch.equal(b["o"], ref[1])
    # replayed on other data: the graph reads its buffers anew
    a["q"].copy_(b["q"])
    graphs[0].replay()
    torch.cuda.synchronize()
    got = a["o"].clone()
    chain(lib, a, a["ws"])
    torch.cuda.synchronize()
    assert torch.equal(got, a["o"]) and not torch.equal(got, ref[0])


# ------------------------------------------------------------------ other sizes and streams

def test_norm_and_read_of_many_rows(lib):
    """Rows enough that a thread takes several, across sequences that end inside a run."""
    B, N, Hq, Hkv, hd, block = 7, 6000, 2, 1, 64, 128
    idx, cnt, b_of, pos, k = rows_of(B, N, [5000, 1, 0, 4999, 3333, 17, 4998], 5)
    M, R = len(pos), B * k
    assert R >= 2 * 8 * 8 * 148   # 8 rows per CTA, 8 CTAs on each SM, twice
    q, kk = normal((R, Hq * hd), 1).to(BF), normal((R, Hkv * hd), 2).to(BF)
    g = (1 + 0.1 * normal((hd,), 3)).to(BF)
    rope = torch.zeros(N, hd // 2, 2, device="cuda")
    lib.dllm_rope_table(rope, 1e4)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(kk, 7.0)
    lib.dllm_qk_norm_rope(q, kk, g, g, rope, qo, ko, idx, cnt, 1e-5)
    for x, y, H in ((q, qo, Hq), (kk, ko, Hkv)):
        ref, mag = norm_ref(x[:M], g, pos, 1e4, 1e-5, H)
        assert np.all(np.abs(f64(y[:M]) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * mag)
        assert torch.all(y[M:] == 7.0)
    cache = filled(lib, B, N, Hkv, hd, block, 6)
    k_out, v_out = torch.full_like(kk, 7.0), torch.full_like(kk, 7.0)
    lib.dllm_kv8_read(*cache, idx, cnt, k_out, v_out, block)
    for c, sc, y in ((cache[0], cache[1], k_out), (cache[2], cache[3], v_out)):
        assert np.array_equal(f64(y[:M]), decoded(c, sc, block)[b_of, pos].reshape(M, -1))
        assert torch.all(y[M:] == 7.0)


@pytest.mark.parametrize("block", [16, 64])
def test_write_of_long_lists(lib, block):
    """Lists that are searched rather than read whole, some of them short in a long buffer."""
    B, N, H, hd = 4, 2777, 2, 64
    idx, cnt, b_of, pos, k = rows_of(B, N, [1100, 3, 0, 2000], 8)
    kk, vv = normal((B * k, H * hd), 1, 2.0).to(BF), normal((B * k, H * hd), 2, 2.0).to(BF)
    cache = filled(lib, B, N, H, hd, block, 9)
    ref = write_ref(cache, kk, vv, b_of, pos, block)
    ws = lib.Workspace(256)
    lib.dllm_kv8_write(kk, vv, idx, cnt, *cache, block, ws=ws)
    assert ws.device_status() == 0
    assert_cache(cache, ref, block)


def test_kept_rows_at_much_larger_scales(lib):
    """Every code of a block, kept while its scale grows by 2^1 .. 2^40 (block 0: by nothing)."""
    N, H, hd, block = 41 * 16, 1, 128, 16
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    cache = lib.kv8_cache(1, N, H, hd, block)
    for i in (0, 2):
        cache[i].view(torch.uint8).copy_(codes.repeat(N * H * hd // 256).view(1, N, H, hd))
        cache[i + 1].fill_(2.0 ** -5)
    pos = np.arange(41) * 16 + np.arange(41) % 16
    idx = torch.from_numpy(pos.astype(np.int32))[None].cuda()
    x = torch.ones(41, hd, device="cuda") * 448 * 2.0 ** (torch.arange(41, device="cuda") - 5.0)[:, None]
    kk = x.to(BF)
    ref = write_ref(cache, kk, -kk, np.zeros(41, int), pos, block)
    lib.dllm_kv8_write(kk, -kk, idx, None, *cache, block)
    assert np.array_equal(f64(cache[1])[0, 0], 2.0 ** (np.arange(41) - 5.0))
    assert_cache(cache, ref, block)


@pytest.mark.parametrize("B,N,Hq,Hkv,hd,block,counts,lens", [
    (1, 1300, 8, 1, 128, 64, [2], None),               # 11 shares of 16 rows
    (1, 2600, 4, 1, 64, 32, [3], [2555]),              # 21
    (2, 9000, 4, 1, 128, 128, [1, 1], [9000, 130]),    # 64, most of the second's empty
    (1, 1900, 3, 1, 128, 64, [30], None),              # of 128 rows: 15
    (1, 3700, 2, 1, 64, 16, [50], [3600]),             # 29
    (2, 70000, 1, 1, 64, 64, [40, 7], [70000, 3]),     # 64, two CTAs per SM if there were fewer
])
def test_attention_over_many_shares(lib, B, N, Hq, Hkv, hd, block, counts, lens):
    q = normal((B * max(counts), Hq * hd), 5).to(BF)
    check_attention(lib, q, filled(lib, B, N, Hkv, hd, block, 6), block, counts, lens)


def test_attention_of_a_given_stream_without_a_workspace(lib):
    """The workspace that the call makes belongs to the call's stream."""
    st = chain_state(lib, 101, (1, 1), 4000)
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream, torch.cuda.default_stream(), 0):
        want, got = torch.zeros_like(st["o"]), torch.zeros_like(st["o"])
        args = (st["cnt"], st["kcap"], st["block"])
        lib.dllm_attention_kv8(st["q"], *st["cache"], want, *args)
        torch.cuda.synchronize()
        for _ in range(20):
            ws = lib.dllm_attention_kv8(st["q"], *st["cache"], got, *args, stream=s)
            del ws                                           # reused by the next call, in stream order
        torch.cuda.synchronize()
        assert torch.equal(got, want)
