"""q/k norm, write and attention one after the other, against the oracle's chain in 64 bits from
the same inputs: what each stage rounds is followed through the stages behind it."""
import math

import numpy as np
import pytest

import oracle as O
from _util import f64
from test_gpu_kv8 import attention_ref, chain, chain_state, decoded, norm_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,block,Hq,Hkv,hd", [((50, 3), 32, 4, 2, 128), ((3, 2), 64, 2, 2, 128),
                                                    ((90, 300), 16, 6, 2, 64)])
def test_the_chain_against_the_oracles(lib, counts, block, Hq, Hkv, hd):
    st = chain_state(lib, 111, counts, 300, Hq, Hkv, hd, block)
    st["q"] *= 0.5
    before = [t.clone() for t in st["cache"]]
    ws = chain(lib, st, None)
    assert ws.device_status() == 0
    M, pos, b_of = len(st["pos"]), st["pos"], st["b_of"]
    # norms: fp32 inside (2^-18 of |a| + |b| at most), one rounding when stored
    near = {}
    for x, y, H in (("q", "qn", Hq), ("k", "kn", Hkv)):
        ref, mag = norm_ref(st[x][:M], st["g"], pos, 1e4, 1e-5, H)
        near[x] = (ref.reshape(M, H, hd), (2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * mag).reshape(M, H, hd))
        assert np.all(np.abs(f64(st[y][:M]) - ref) <= near[x][1].reshape(M, -1))
    # the cache: the oracle writes its own keys; scales lie between those of the ends of that
    # range, and codes between those of the ends at that scale
    k, dk = near["k"]
    K0, s0, s1 = decoded(before[0], before[1], block), f64(before[1]), f64(st["cache"][1])
    scales = []
    for x in (np.abs(k) - dk, np.abs(k) + dk):
        scales.append(s0.copy())
        O.kv8_write(K0.copy(), scales[-1], x, b_of, pos, block)
    assert np.all((scales[0] <= s1) & (s1 <= scales[1])) and np.mean(scales[0] == scales[1]) > 0.9
    at = s1.repeat(block, axis=2)[:, :, :K0.shape[1]].transpose(0, 2, 1)[..., None]

    def keys(x):
        K = K0.copy()
        K[b_of, pos] = x
        return O.e4m3_round(np.clip(K / at, -448, 448)) * at

    K = keys(k)
    dK = np.maximum(np.abs(keys(k - dk) - K), np.abs(keys(k + dk) - K))
    assert np.all(np.abs(decoded(*st["cache"][:2], block) - K) <= dK)
    V, vs = decoded(before[2], before[3], block), f64(before[3]).copy()
    O.kv8_write(V, vs, f64(st["v"][:M]).reshape(M, Hkv, hd), b_of, pos, block)
    assert np.array_equal(decoded(*st["cache"][2:], block), V)
    # attention: a score moved by d_j at most changes its weight by e^d_j - 1 of it, and with it
    # the sums above and below
    q, dq = near["q"]
    off = 0
    for b, c in enumerate(counts):
        rows = slice(off, off + c)
        per_key = vs[b].repeat(block, axis=1)[:, :V.shape[1]].T
        ref, tol, _ = attention_ref(q[rows], K[b], V[b], per_key, V.shape[1], Hkv)
        for h in range(Hq):
            g = h * Hkv // Hq
            qa, ka, kd, v = np.abs(q[rows, h]), np.abs(K[b][:, g]), dK[b][:, g], np.abs(V[b][:, g])
            d = (dq[rows, h] @ (ka + kd).T + qa @ kd.T) / math.sqrt(hd)
            s = q[rows, h] @ K[b][:, g].T / math.sqrt(hd)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            dp = p * np.expm1(d)
            moved = dp.sum(1, keepdims=True)
            assert np.all(moved < 0.5) and np.median(moved) < 0.25     # (the bound says something)
            # (the roundings of weights that have grown and sums that have shrunk: 1.5 / 0.5)
            lim = 3 * tol[:, h] + (dp @ v + np.abs(ref[:, h]) * moved) / (1 - moved)
            got = f64(st["o"][rows]).reshape(c, Hq, hd)[:, h]
            assert np.all(np.abs(got - ref[:, h]) <= lim + 2.0 ** -8 * (np.abs(ref[:, h]) + lim))
        off += c
