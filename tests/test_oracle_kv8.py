"""CPU pins of the oracle's 8-bit K/V cache: the e4m3 rounding against a list of every
code and against torch's conversion, the scale rule, the cache write against its
definition for the cases by hand, and the q/k norm in a layer."""
import numpy as np
import pytest
import torch

import oracle as O


def _codes():
    """Every finite non-negative e4m3 value, from the format's definition."""
    return np.array(sorted({(m / 8.0) * 2.0 ** -6 for m in range(8)}
                           | {(1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16)
                              for m in range(8) if not (e == 15 and m == 7)}))


def test_e4m3_round_picks_the_nearest_code():
    c = _codes()
    assert len(c) == 127 and c[-1] == 448.0 and c[1] == 2.0 ** -9
    assert np.array_equal(O.e4m3_round(c), c) and np.array_equal(O.e4m3_round(-c), -c)
    mid = (c[:-1] + c[1:]) / 2                       # ties: the code with an even last bit
    assert np.array_equal(O.e4m3_round(mid), np.where(np.arange(126) % 2 == 0, c[:-1], c[1:]))
    x = np.random.default_rng(0).uniform(0, 448, 5000) * 2.0 ** -np.arange(5000) ** 0.4
    best = c[np.argmin(np.abs(x[:, None] - c[None]), axis=1)]
    assert np.array_equal(O.e4m3_round(x), best)
    t = torch.from_numpy(x).float()
    assert np.array_equal(O.e4m3_round(t.double().numpy()),
                          t.to(torch.float8_e4m3fn).double().numpy())
    assert np.isnan(O.e4m3_round(np.array([np.nan, np.inf, -np.inf]))).all()


@pytest.mark.parametrize("a,s", [(0.0, 2.0 ** -100), (448.0, 1.0), (448.5, 2.0), (224.0, 0.5),
                                 (1.0, 2.0 ** -8), (1.75, 2.0 ** -8), (1.7578125, 2.0 ** -7),
                                 (3e38, 2.0 ** 120), (2.0 ** -130, 2.0 ** -100)])
def test_scale_is_the_smallest_power_of_two_that_covers(a, s):
    assert O.kv8_scale(a) == s


def test_write_keeps_grows_and_resets_scales():
    c = np.zeros((1, 5, 1, 2))                       # blocks of 4: the last one holds a token
    sc = np.zeros((1, 1, 2))
    w = lambda rows, pos: O.kv8_write(c, sc, np.array(rows, dtype=float)[:, None, :],
                                      np.zeros(len(pos), int), np.array(pos), 4)
    w([[1.0, -1.75]], [1])                           # a first row: its own scale
    assert sc[0, 0, 0] == 2.0 ** -8 and np.array_equal(c[0, 1, 0], [1.0, -1.75])
    w([[0.25, 0.1]], [2])                            # fits: the scale stays
    assert sc[0, 0, 0] == 2.0 ** -8 and np.array_equal(c[0, 2, 0], [0.25, 0.1015625])
    w([[500.0, 0.0]], [0])                           # grows: the kept rows at the new step
    assert sc[0, 0, 0] == 2.0
    assert np.array_equal(c[0, 1, 0], [1.0, -1.75]) and np.array_equal(c[0, 2, 0], [0.25, 0.1015625])
    w([[0.5, 0.0], [0.001, 0.0]], [1, 2])            # 0.001 / 2 is below half of 2^-9
    assert c[0, 2, 0, 0] == 0.0
    w([[1.0, 1.0]] * 4, [0, 1, 2, 3])                # whole block: a fresh scale
    assert sc[0, 0, 0] == 2.0 ** -8
    w([[np.nan, 3.0]], [4])                          # NaN stays and does not count
    assert sc[0, 0, 1] == 2.0 ** -7 and np.isnan(c[0, 4, 0, 0]) and c[0, 4, 0, 1] == 3.0
    before = c.copy()
    w([[1.0, 1.0]] * 4, [0, 1, 2, 3])                # again: nothing changes
    assert np.array_equal(before, c, equal_nan=True)


def _layer(rng, d, H, hd, F, **kw):
    m = lambda r, c: rng.normal(size=(r, c)) / np.sqrt(c)
    return O.LayerW(np.ones(d), m(H * hd, d), m(H * hd, d), m(H * hd, d), m(d, H * hd),
                    np.ones(d), m(F, d), m(F, d), m(d, F), **kw)


def test_qk_norm_makes_the_layer_blind_to_the_projections_scale():
    """With the norm (eps 0) scaling wq or wk by any factor changes nothing."""
    rng = np.random.default_rng(1)
    d, H, hd, F, N = 16, 2, 8, 24, 6
    cfg = O.ModelCfg(1, d, H, H, hd, F, 32, rms_eps=0.0, dtype="f32")
    w = _layer(rng, d, H, hd, F, q_norm=rng.normal(size=hd), k_norm=rng.normal(size=hd))
    x = rng.normal(size=(N, d))
    b, p = np.zeros(N, int), np.arange(N)
    run = lambda: O.layer_rows(cfg, w, x, b, p, np.zeros((1, N, H, hd)), np.zeros((1, N, H, hd)))
    y = run()
    w.wq, w.wk = 7.0 * w.wq, 0.01 * w.wk
    assert np.allclose(run(), y, rtol=1e-12, atol=1e-12)
    w.q_norm = 2.0 * w.q_norm
    assert not np.allclose(run(), y, rtol=1e-3)


def test_layer_over_an_8_bit_cache_attends_to_decoded_rows():
    rng = np.random.default_rng(2)
    d, H, hd, F, N, blk = 16, 2, 8, 24, 20, 16
    cfg = O.ModelCfg(1, d, H, H, hd, F, 32, dtype="f32")
    w = _layer(rng, d, H, hd, F)
    x = rng.normal(size=(N, d))
    b, p = np.zeros(N, int), np.arange(N)
    kc, vc = np.zeros((1, N, H, hd)), np.zeros((1, N, H, hd))
    ks, vs = np.zeros((1, H, 2)), np.zeros((1, H, 2))
    O.layer_rows(cfg, w, x, b, p, kc, vc, None, (ks, vs, blk))
    k0, v0 = np.zeros_like(kc), np.zeros_like(vc)
    O.layer_rows(cfg, w, x, b, p, k0, v0)
    # half a step of 4 significant bits, or of 2^-9 of the block's scale
    for c, c0, s in ((kc, k0, ks), (vc, v0, vs)):
        step = np.maximum(np.abs(c0) * 2.0 ** -4, np.repeat(s, blk, 2)[:, :, :N].transpose(0, 2, 1)[..., None] * 2.0 ** -10)
        assert np.all(np.abs(c - c0) <= step) and not np.array_equal(c, c0)
