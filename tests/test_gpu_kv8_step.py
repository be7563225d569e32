"""GPU parity of whole steps with q/k norms and with the K/V caches in 8 bits.

Each step starts from the GPU's own state (the oracle's caches are set to the values
that the GPU's hold), with the oracle's decisions forced on both sides."""
import numpy as np
import pytest
import torch

import oracle as O
import dllm_synth as SY
from _gpu import argmax_ok, to_dev
from _util import TOL, f64, max_abs_rel, oracle_cfg, oracle_policy, oracle_weights
from test_gpu_kv8 import decoded

pytestmark = pytest.mark.gpu


def shape_of(dtype="bf16", **kw):
    base = dict(dtype=dtype, n_layers=2, d=256, n_heads=4, n_kv_heads=2, head_dim=64, ffn=512,
                vocab=2048, batch=2, prompt_len=61, gen_len=100, block_len=32, n_unmask=5, ratio=0.25,
                alpha=0.5)
    return SY.with_(SY.TINY, **{**base, **kw})


class Case:
    def __init__(self, lib, shape, norms, block, **pol_kw):
        self.lib, self.s, self.block = lib, shape, block
        W = SY.model_weights(shape, seed=0, device="cpu")
        if norms:
            for i, L in enumerate(W["layers"]):
                for j, n in enumerate(("q_norm", "k_norm")):
                    g = 1.0 + 0.3 * SY.normal((shape.head_dim,), 1.0, 50 + 2 * i + j, "cpu", "f32")
                    L[n] = g.to(SY.torch_dtype(shape.dtype))
        self.model = lib.Model(lib.cfg_from_shape(shape), to_dev(W))
        self.ocfg, self.ow = oracle_cfg(shape), oracle_weights(W)
        B, N = shape.batch, shape.seq_len
        self.opol = oracle_policy(shape, kv8_block=block, **pol_kw)
        p = self.opol
        self.pol = lib.make_policy(p.score_layer, p.alpha, p.kind, p.mode, p.k, p.tau, p.n_unmask,
                                   p.gen_start, p.block_len, ffn_gate=p.ffn_gate, ffn_tau=p.ffn_tau,
                                   attn_update=p.attn_update, kv8_block=block)
        self.cache = lib.Cache(self.model.cfg, B, N, ffn_gate=p.ffn_gate, attn_update=p.attn_update,
                               kv8_block=block)
        self.ws = lib.Workspace(lib.dllm_step_workspace_size(self.model.cfg, B, N, self.pol))
        tok = SY.prompt_tokens(shape, seed=1)
        self.tokens = tok.cuda()
        self.st = O.empty_state(self.ocfg, f64(tok).astype(np.int64), block)

    def kv(self, c, s):
        return decoded(c, s, self.block) if self.block else f64(c)

    def pull(self):
        """The oracle's state <- the GPU's."""
        st, c = self.st, self.cache
        L = range(self.s.n_layers)
        none = [None] * self.s.n_layers
        st.k = [self.kv(c.k[l], (c.k_scale or none)[l]) for l in L]
        st.v = [self.kv(c.v[l], (c.v_scale or none)[l]) for l in L]
        if self.block:
            st.k_scale, st.v_scale = [f64(t) for t in c.k_scale], [f64(t) for t in c.v_scale]
        st.h_ref, st.conf, st.pred = f64(c.h_ref), f64(c.conf), f64(c.pred).astype(np.int64)
        st.tokens = f64(self.tokens).astype(np.int64)
        for name in ("ctx", "ffn", "q", "att_m", "att_l"):
            if getattr(c, name) is not None:
                setattr(st, name, [f64(t) for t in getattr(c, name)])

    def step(self, dense):
        self.pull()
        before = self.st.copy()
        out = O.step(self.ocfg, self.ow, self.st, self.opol, dense)
        kw = {}
        B = self.s.batch
        if not dense:
            a = np.full((B, self.s.k), -1, dtype=np.int32)
            for b, r in enumerate(out.idx):
                a[b, :len(r)] = r
            kw = dict(forced_idx=torch.from_numpy(a).cuda(),
                      forced_count=torch.tensor([len(r) for r in out.idx], dtype=torch.int32, device="cuda"))
            if self.opol.ffn_gate:
                f = np.zeros((self.s.n_layers, B * self.s.k), dtype=np.uint8)
                for l, sal in enumerate(out.ffn_salient):
                    f[l, :len(sal)] = sal
                kw["forced_ffn"] = torch.from_numpy(f).cuda()
        fu = torch.from_numpy(out.unmasked.astype(np.int32)).cuda()
        self.lib.dllm_step_ex(self.model, self.cache, self.tokens, self.pol, dense, self.ws,
                              forced_unmask_pos=fu, **kw)
        assert self.ws.device_status() == 0
        return out, before

    def check(self, out, before, dense):
        st, c, N = self.st, self.cache, self.s.seq_len
        # a stored code differs by one e4m3 step (1/8 of the value, 2^-9 of the scale) where the
        # bf16 path is off across a border; such steps at a share f of the codes, of random
        # sign, move what attention makes of them by 2^-3 sqrt(f), 2.2 % for f = 1/32 (the bf16
        # path is off by under 1/32 of a code's step on the average)
        tol = TOL[self.s.dtype] + (0.022 if self.block else 0.0)
        for l in range(self.s.n_layers):
            for t, s, o, b0 in ((c.k[l], c.k_scale, st.k[l], before.k[l]), (c.v[l], c.v_scale, st.v[l], before.v[l])):
                got = self.kv(t, s[l] if s else None)
                lim = tol * np.abs(o).max()
                if self.block:
                    sc = f64(s[l]).repeat(self.block, 2)[:, :, :N].transpose(0, 2, 1)[..., None]
                    lim = lim + np.abs(o) / 8 + 2.0 ** -9 * sc
                assert np.all(np.abs(got - o) <= lim), l
                if not dense and not self.block:
                    keep = np.ones((self.s.batch, N), bool)
                    for b, r in enumerate(out.idx):
                        keep[b, r] = False
                    assert np.array_equal(got[keep], b0[keep])
        conf, want = f64(c.conf), st.conf
        for b, r in enumerate(out.idx):
            for p in r:
                if want[b, p] != before.conf[b, p]:
                    assert abs(conf[b, p] - want[b, p]) <= 3 * tol * want.max() + 1e-7
        for l in range(self.s.n_layers):
            if self.opol.ffn_gate:
                assert max_abs_rel(f64(c.ctx[l]), st.ctx[l]) < 2 * tol
            if self.opol.attn_update:
                lse = lambda m, v: m + np.log(v)
                assert np.abs(lse(f64(c.att_m[l]), f64(c.att_l[l])) - lse(st.att_m[l], st.att_l[l])).max() < 0.1


CASES = [("f32", dict(), True, 0, {}), ("f32", dict(head_dim=10, n_heads=4, n_kv_heads=4), True, 0, {}),
         ("bf16", dict(), True, 0, {}), ("bf16", dict(head_dim=128, n_heads=2, n_kv_heads=2), True, 0, {}),
         ("bf16", dict(), False, 16, {}), ("bf16", dict(), True, 64, {}),
         ("bf16", dict(head_dim=128, n_heads=2, n_kv_heads=1), True, 32, {}),
         ("bf16", dict(head_dim=128, n_heads=2, n_kv_heads=2), False, 128, {}),
         ("bf16", dict(ratio=0.03), False, 64, {}), ("bf16", dict(score_layer=1), True, 16, dict(score_layer=1)),
         ("bf16", dict(), True, 32, dict(ffn_gate=True, ffn_tau=1e-3)),
         ("bf16", dict(), False, 32, dict(ffn_gate=True, ffn_tau=1e-3, attn_update=True)),
         ("bf16", dict(), True, 0, dict(ffn_gate=True, ffn_tau=1e-3, attn_update=True))]


@pytest.mark.parametrize("dtype,kw,norms,block,pol", CASES)
def test_steps_match_the_oracle(lib, dtype, kw, norms, block, pol):
    if kw.get("n_kv_heads") == 1 or kw.get("head_dim") == 10:
        kw = {**kw, "d": 256}
    run = Case(lib, shape_of(dtype, **kw), norms, block, **pol)
    for t in range(3):
        out, before = run.step(t == 0)
        run.check(out, before, t == 0)
    assert run.st is not None and (f64(run.tokens) != run.s.mask_id).sum() > run.s.batch * run.s.prompt_len


def test_partial_layer_with_norms(lib):
    shape = shape_of()
    run = Case(lib, shape, True, 0)
    B, N, d, k = shape.batch, shape.seq_len, shape.d, 7
    rng = np.random.default_rng(3)
    idx = np.stack([np.sort(rng.choice(N, k, replace=False)) for _ in range(B)]).astype(np.int32)
    x = SY.normal((B, N, d), 1.0, 9, "cuda", "bf16")
    kc = SY.normal((B, N, shape.n_kv_heads, shape.head_dim), 1.0, 10, "cuda", "bf16")
    vc = SY.normal((B, N, shape.n_kv_heads, shape.head_dim), 1.0, 11, "cuda", "bf16")
    ok, ov = f64(kc), f64(vc)
    b_of, p_of = np.repeat(np.arange(B), k), idx.reshape(-1).astype(int)
    want = O.layer_rows(run.ocfg, run.ow.layers[0], f64(x)[b_of, p_of], b_of, p_of, ok, ov)
    out = torch.zeros(B * k, d, dtype=torch.bfloat16, device="cuda")
    ws = lib.Workspace(lib.dllm_partial_layer_workspace_size(run.model.cfg, B, N, k))
    lib.dllm_partial_layer(run.model.cfg, run.model.layer(0), x, out, torch.from_numpy(idx).cuda(),
                           torch.full((B,), k, dtype=torch.int32, device="cuda"), kc, vc, ws, True)
    assert ws.device_status() == 0
    for got, ref in ((out, want), (kc, ok), (vc, ov)):
        assert max_abs_rel(f64(got), ref) < TOL["bf16"]


def test_graph_replay_and_generation_over_an_8_bit_cache(lib):
    shape = shape_of(ratio=0.2)
    runs = []
    for graph in (False, True):
        c = Case(lib, shape, True, 32)
        lib.dllm_step(c.model, c.cache, c.tokens, c.pol, True, c.ws)
        lib.dllm_step(c.model, c.cache, c.tokens, c.pol, False, c.ws)
        if graph:
            g = lib.StepGraph(c.model, c.cache, c.tokens, c.pol, c.ws)
            for _ in range(3):
                g.replay()
        else:
            for _ in range(3):
                lib.dllm_step(c.model, c.cache, c.tokens, c.pol, False, c.ws)
        torch.cuda.synchronize()
        runs.append([c.tokens] + [t.view(torch.uint8) for t in c.cache.k + c.cache.v] + c.cache.k_scale
                    + c.cache.v_scale + [c.cache.conf])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    c = Case(lib, shape, False, 64)
    ws = lib.Workspace(lib.dllm_generate_workspace_size(c.model.cfg, 2, shape.seq_len, c.pol))
    # 100 positions, 5 a step, no step across a block of 32: 3 * ceil(32 / 5) + ceil(4 / 5)
    flags = lib.dllm_generate(c.model, c.cache, c.tokens, c.pol, 22, ws)
    torch.cuda.synchronize()
    assert flags[0] and not any(flags[1:]) and not (c.tokens == shape.mask_id).any()


def test_step_refuses_an_8_bit_cache_it_cannot_use(lib):
    shape = shape_of()
    c = Case(lib, shape, False, 32)
    go = lambda: lib.dllm_step(c.model, c.cache, c.tokens, c.pol, True, c.ws)
    for bad in (8, 48, 256, -16):
        c.pol.kv8_block = bad
        with pytest.raises(lib.DllmError) as e:
            go()
        assert e.value.status == 1
    c.pol.kv8_block = 32
    plain = lib.Cache(c.model.cfg, 2, shape.seq_len)           # a bf16 cache: no scales
    with pytest.raises(lib.DllmError):
        lib.dllm_step(c.model, plain, c.tokens, c.pol, True, c.ws)
    f = Case(lib, shape_of("f32"), False, 0)
    f.pol.kv8_block = 32
    ws = lib.Workspace(lib.dllm_step_workspace_size(f.model.cfg, 2, shape.seq_len, f.pol))
    with pytest.raises(lib.DllmError) as e:
        lib.dllm_step(f.model, f.cache, f.tokens, f.pol, True, ws)
    assert e.value.status == 2
    L = c.model.layer(0)
    L.q_norm = c.cache.h_ref.data_ptr()                        # one gain without the other
    with pytest.raises(lib.DllmError):
        go()


def test_steps_of_long_sequences(lib):
    """More rows per sequence than the write reads as one list, from a step's own row maps."""
    run = Case(lib, shape_of(prompt_len=700, gen_len=600, batch=1, d=256, ratio=0.9), True, 64)
    assert run.s.k > 1024
    for t in range(2):
        out, before = run.step(t == 0)
        run.check(out, before, t == 0)
