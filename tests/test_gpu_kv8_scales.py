"""Attention over 8-bit caches whose V scales lie far apart: the softmax sum, which no
V scale may touch, and the weights, which f16 holds, against the oracle in 64 bits."""
import math

import numpy as np
import pytest
import torch

from _util import f64
from test_gpu_kv8 import BF, check_attention, decoded, filled, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,hd", [(1, 128), (3, 64), (130, 128), (200, 64)])
@pytest.mark.parametrize("block", [16, 64, 128])
@pytest.mark.parametrize("top", [0, 27, 60, 100])
def test_zero_blocks_beside_large_ones_keep_their_weight(lib, rows, hd, block, top):
    """Blocks of zero V rows get the smallest scale, 2^-100.  Their keys weigh as much as
    any others, whatever the scale (2^top) of the blocks beside them: output and statistics."""
    B, N, H = 1, 9000 if block == 128 else 700, 2   # (more than one block to a share of the keys)
    k8, ks, v8, vs = filled(lib, B, N, H, hd, block, 3)
    for i in range(vs.shape[2]):
        if i % 2:
            vs[:, :, i] = 2.0 ** top
        else:
            vs[:, :, i] = 2.0 ** -100
            v8.view(torch.uint8)[:, i * block:(i + 1) * block] = 0
    check_attention(lib, normal((rows, H * hd), 4).to(BF), (k8, ks, v8, vs), block, [rows], None)


@pytest.mark.parametrize("rows", [1, 130])
def test_only_blocks_of_zeros(lib, rows):
    """Zero rows only, or no row written at all (scale 0): zeros, and the scores' statistics."""
    B, N, H, hd, block = 1, 300, 1, 128, 32
    k8, ks, v8, vs = filled(lib, B, N, H, hd, block, 5)
    v8.view(torch.uint8).zero_()
    vs.fill_(2.0 ** -100)
    q = normal((rows, H * hd), 6).to(BF)
    o = check_attention(lib, q, (k8, ks, v8, vs), block, [rows], None)
    assert torch.all(o[:rows] == 0)
    cnt = torch.tensor([rows], dtype=torch.int32, device="cuda")
    got = []
    for scale in (2.0 ** -100, 0.0):
        vs.fill_(scale)
        st = [torch.full_like(q, 7.0)] + [torch.zeros(rows, H, device="cuda") for _ in range(2)]
        lib.dllm_attention_kv8(q, k8, ks, v8, vs, st[0], cnt, rows, block, m=st[1], l=st[2])
        got.append(st)
    lse = [m + torch.log(l) for _, m, l in got]
    assert torch.all(got[1][0] == 0) and torch.allclose(lse[0], lse[1], rtol=2.0 ** -20, atol=2.0 ** -20)


# ------------------------------------------------------------------ weights

def weight_bound(q, K, V, vs, width):
    """One head: the output [R, hd] of q [R, hd] over K, V [n, hd] (vs [n]: V's scales) and a bound
    of its error before the store.  Weights come in tiles of `width` keys.  With
    the largest weight * scale of a tile brought to 2^-6 or more, f16 holds the others to half a
    step, 2^-11 of each, or to 2^-25 where they are below 2^-14: 2^-25 / 2^-6 = 2^-19 of the largest.
    Where a tile's scales span more than six octaves its codes are first brought towards a common
    scale, by 2^-7 .. 2^1, and the largest product of weight and what is left of the scale to 2^8 or
    more: 2^-25 / 2^8 = 2^-33 of it."""
    n, hd = K.shape
    s = q @ K.T / math.sqrt(hd)
    p = np.exp(s - s.max(1, keepdims=True))
    l = p.sum(1, keepdims=True)
    mag = np.abs(q) @ np.abs(K).T / math.sqrt(hd)
    ds = ((hd / 16 + 2) * 2.0 ** -23 * mag + 2.0 ** -22 * np.abs(s)).max(1, keepdims=True)
    tol = (2.0 ** -11 + 2 * ds + n / 16 * 2.0 ** -23 + 2.0 ** -20) * (p @ np.abs(V))
    for t in range(0, n, width):
        e = np.log2(vs[t:t + width])
        mixed = e.max() - e.min() > 6
        unit = 2.0 ** (e - np.clip(e - e.max() + 1, -7, 1)) if mixed else 2.0 ** e
        tol += 2.0 ** (-33 if mixed else -19) * (p[:, t:t + width] * unit).max(1, keepdims=True) * (np.abs(V[t:t + width]) / unit[:, None]).sum(0)
    return p @ V / l, tol / l, p @ np.abs(V) / l


def check_weights(lib, q, cache, block, rows, where, tight=True):
    """Against the bound, which (tight) must itself be within 2^-9 of what the output is made of:
    half of what the store to bf16 may round."""
    k8, ks, v8, vs = cache
    B, N, H, hd = k8.shape
    o = torch.full_like(q, 7.0)
    cnt = torch.full((B,), rows, dtype=torch.int32, device="cuda")
    ws = lib.dllm_attention_kv8(q, k8, ks, v8, vs, o, cnt, rows, block)
    assert ws.device_status() == 0
    for b, h in where:
        one = lambda c, sc: decoded(c[b:b + 1, :, h:h + 1], sc[b:b + 1, h:h + 1], block)[0, :, 0]
        at = lambda t: f64(t.view(B, rows, H, hd)[b, :, h])
        ref, tol, size = weight_bound(at(q), one(k8, ks), one(v8, vs), f64(vs[b, h]).repeat(block)[:N],
                                      64 if rows > 16 else 16)   # (few rows: tiles of 16 keys)
        assert not tight or np.all(tol <= 2.0 ** -9 * size)
        err = np.abs(at(o) - ref) - (tol + 2.0 ** -8 * (np.abs(ref) + tol))
        assert np.all(err <= 0), (b, h, err.max())


UNITS = (74, 8)   # sequences and heads for which one CTA passes over all keys


def many(cache):
    """The cache of one sequence and head, as UNITS equal ones."""
    B, H = UNITS
    k8, ks, v8, vs = (t.view(torch.uint8) if i % 2 == 0 else t for i, t in enumerate(cache))
    code = lambda t: t.expand(B, -1, H, -1).contiguous().view(torch.float8_e4m3fn)
    scale = lambda t: t.expand(B, H, -1).contiguous()
    return code(k8), scale(ks), code(v8), scale(vs)


WHERE = [(0, 0), (UNITS[0] - 1, UNITS[1] - 1)]


@pytest.mark.parametrize("rows", [1, 130])
@pytest.mark.parametrize("block", [16, 64, 128])
@pytest.mark.parametrize("far", [9, 24, 30])
def test_a_scale_left_behind_by_an_outlier(lib, rows, block, far):
    """A row 2^far times larger than the others raises its block's scale and is then written anew
    at their size: the scale stays, the block's codes become small or zero."""
    N, hd = 1024, 128
    cache = lib.kv8_cache(1, N, 1, hd, block)
    k, v = normal((N, hd), 1).to(BF), (normal((N, hd), 2) + 0.3).to(BF)
    lib.dllm_kv8_write(k, v, None, None, *cache, block)
    idx = torch.tensor([[333]], dtype=torch.int32, device="cuda")
    row = v[333:334].clone()
    for x in (row * 2.0 ** far, row):
        lib.dllm_kv8_write(k[333:334], x, idx, None, *cache, block)
    vs = cache[3][0, 0]
    assert vs[333 // block] >= 2.0 ** (far - 1) * vs.min()
    q = normal((UNITS[0] * rows, UNITS[1] * hd), 3) * 0.1
    check_weights(lib, q.to(BF), many(cache), block, rows, WHERE)


@pytest.mark.parametrize("rows", [1, 130])
@pytest.mark.parametrize("block", [16, 64])
def test_a_heavy_key_with_one_large_channel(lib, rows, block):
    """The first of 16384 keys holds most of the weight, and one channel of its V row is 2000:
    the other keys' part in the other channels stays."""
    N, hd = 16384, 128
    cache = lib.kv8_cache(1, N, 1, hd, block)
    k, v = normal((N, hd), 1), normal((N, hd), 2) + 0.3
    v[0, 5] = 2000
    lib.dllm_kv8_write(k.to(BF), v.to(BF), None, None, *cache, block)
    k0 = k[0] / k[0].norm()
    q = normal((UNITS[0] * rows, UNITS[1] * hd), 3) * 0.05
    q += (k0 * 12 * math.sqrt(hd) / k[0].norm()).repeat(UNITS[1])
    check_weights(lib, q.to(BF), many(cache), block, rows, WHERE)


@pytest.mark.parametrize("rows", [1, 130])
@pytest.mark.parametrize("octaves,blocks", [(1, 78), (3, 25)])
@pytest.mark.parametrize("rising", [False, True])
def test_every_block_has_a_channel_of_its_own(lib, rows, octaves, blocks, rising):
    """V scales that fall (rise) from block to block, each block alone in its channel: every channel
    is as good as any other, whatever its size beside theirs."""
    hd, block = 128, 16
    N = blocks * block
    k8, ks, v8, vs = lib.kv8_cache(1, N, 1, hd, block)
    k8.copy_((normal((1, N, 1, hd), 1) * 100).clamp(-448, 448).to(torch.float8_e4m3fn))
    ks.fill_(2.0 ** -7)
    code = torch.zeros(1, N, 1, hd, device="cuda")
    for i in range(blocks):
        code[0, i * block:(i + 1) * block, 0, i] = 100 * normal((block,), 5 + i)
    v8.copy_(code.clamp(-448, 448).to(torch.float8_e4m3fn))
    e = octaves * torch.arange(blocks, device="cuda").float()
    vs.copy_(torch.exp2(e - e.max() if rising else -e).expand_as(vs))
    q = normal((UNITS[0] * rows, UNITS[1] * hd), 3) * 0.1
    check_weights(lib, q.to(BF), many((k8, ks, v8, vs)), block, rows, WHERE)


@pytest.mark.parametrize("rows", [1, 130])
@pytest.mark.parametrize("apart", [10, 20, 30, 60])
@pytest.mark.parametrize("first", [0, 10, 16, 40])
def test_heavy_keys_of_a_small_block_beside_light_ones_of_a_large(lib, rows, apart, first):
    """Within one tile: keys that hold the weight, in a block of scale 2^-apart, beside keys of
    2^-20 of their weight in a block of scale 1, each block alone in its channels; before it a
    tile whose products are 2^first larger than either's."""
    hd, block, N = 128, 16, 128
    k8, ks, v8, vs = lib.kv8_cache(1, N, 1, hd, block)
    kc, vc = torch.zeros(N, hd, device="cuda"), torch.zeros(N, hd, device="cuda")
    kc[64:80, 0] = 20                     # a score of 8 * 20 / sqrt(128) = 20.4 octaves
    kc[:, 1] = normal((N,), 19)           # (a fraction of an octave)
    for at, ch in ((0, 0), (64, 32), (80, 64), (96, 96)):
        end = {0: 64, 64: 80, 80: 96, 96: 128}[at]
        vc[at:end, ch:ch + 32] = 100 * normal((end - at, 32), 20 + at)
    k8.copy_(kc.view(1, N, 1, hd).to(torch.float8_e4m3fn))
    v8.copy_(vc.clamp(-448, 448).view(1, N, 1, hd).to(torch.float8_e4m3fn))
    ks.fill_(1.0)
    vs.fill_(1.0)
    vs[..., 4] = 2.0 ** -apart
    vs[..., :4] = 2.0 ** (first + max(0, 20 - apart))
    q = torch.zeros(UNITS[0] * rows, UNITS[1], hd, device="cuda")
    q[..., 0] = torch.linspace(8.0, 8.5, rows, device="cuda").repeat(UNITS[0])[:, None]
    q[..., 1] = 2
    check_weights(lib, q.flatten(1).to(BF), many((k8, ks, v8, vs)), block, rows, WHERE,
                  apart <= 30)   # (60: the small block's products are 2^-40 of the largest)


@pytest.mark.parametrize("rows", [1, 130])
@pytest.mark.parametrize("scales", [(48, -31, 109), (0, -62, 62), (0, -40, -62, 65, -10, 60)])
def test_scales_that_fall_far_and_rise_further(lib, rows, scales):
    """Blocks of a tile each, alone in their channels: the weights' reference falls by up to 2^64
    and rises by more than 2^126 at once; what was summed before keeps its bits."""
    hd, block = 128, 64
    N = block * len(scales)
    k8, ks, v8, vs = lib.kv8_cache(1, N, 1, hd, block)
    k8.copy_((normal((1, N, 1, hd), 1) * 100).clamp(-448, 448).to(torch.float8_e4m3fn))
    ks.fill_(2.0 ** -7)
    code = torch.zeros(1, N, 1, hd, device="cuda")
    for i in range(len(scales)):
        code[0, i * block:(i + 1) * block, 0, i * 20:(i + 1) * 20] = 100 * normal((block, 20), 5 + i)
    v8.copy_(code.clamp(-448, 448).to(torch.float8_e4m3fn))
    vs.copy_(torch.exp2(torch.tensor(scales, device="cuda").float()).expand_as(vs))
    # (products 2^83 below the largest are past what the weights hold)
    live = [i for i, e in enumerate(scales) if e > max(scales) - 75]
    assert len(live) >= 2
    v8.view(torch.uint8)[:, [n for n in range(N) if n // block not in live]] = 0
    q = normal((UNITS[0] * rows, UNITS[1] * hd), 3) * 0.1
    check_weights(lib, q.to(BF), many((k8, ks, v8, vs)), block, rows, WHERE)


@pytest.mark.parametrize("rows", [1, 3, 40])
@pytest.mark.parametrize("N", [100, 1000, 9000])
def test_values_at_the_end_of_the_range(lib, rows, N):
    """All V rows hold the largest values of bf16, so every mean is one of them: partial sums of
    several warps and key shares stay inside the floats' range."""
    hd, block = 128, 64
    k8, ks, v8, vs = filled(lib, 1, N, 1, hd, block, 7)
    want = torch.tensor([240.0, -240.0], device="cuda").repeat(hd // 2)   # 240 * 2^120 = 0.94 * 2^128
    v8.copy_(want.to(torch.float8_e4m3fn).expand_as(v8))
    vs.fill_(2.0 ** 120)
    q = normal((rows, hd), 8).to(BF)
    o = torch.zeros_like(q)
    cnt = torch.tensor([rows], dtype=torch.int32, device="cuda")
    lib.dllm_attention_kv8(q, k8, ks, v8, vs, o, cnt, rows, block)
    # weights off by 2^-11, the sums' few steps, and the store
    assert torch.all((o.double() / 2.0 ** 120 - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * 240)
