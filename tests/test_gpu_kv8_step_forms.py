"""The forms of a step over 8-bit caches: what a partial step may not touch, bit for bit, the
second skip point, response-only steps, refreshes, and tokens in host memory."""
import numpy as np
import pytest
import torch

import oracle as O
from _util import f64, max_abs_rel
from test_gpu_kv8 import decoded
from test_gpu_kv8_step import Case, shape_of

pytestmark = pytest.mark.gpu


def held(cache):
    return [[t.view(torch.uint8).clone() if t.element_size() == 1 else t.clone() for t in (c, s)]
            for c, s in zip(cache.k + cache.v, cache.k_scale + cache.v_scale)]


def check_kept(run, before, rows_of_layer):
    """Of each layer's K and V: blocks without a recomputed row as they were; in the others the
    rows that were kept, at the scale before bit for bit, at a larger one rounded once."""
    L, N, blk = run.s.n_layers, run.s.seq_len, run.block
    grown = 0
    for i, ((c0, s0), (c1, s1)) in enumerate(zip(before, held(run.cache))):
        rows = rows_of_layer(i % L)
        for b in range(run.s.batch):
            new = np.zeros(-(-N // blk) * blk, bool)
            new[rows[b]] = True
            touched = new.reshape(-1, blk).any(1)
            kept = torch.from_numpy(~new[:N]).cuda()
            same = torch.from_numpy(~touched).cuda()
            assert torch.equal(s0[b][:, same], s1[b][:, same])
            scale0, scale1 = (s[b].repeat_interleave(blk, 1)[:, :N].T for s in (s0, s1))   # [N, H]
            equal = (scale0 == scale1) & kept[:, None]
            assert torch.equal(c0[b][equal], c1[b][equal])
            grew = f64(((scale0 != scale1) & kept[:, None]).float()) > 0
            assert np.all(f64(scale1)[grew] > f64(scale0)[grew])
            old, got = decoded(c0[b:b + 1], s0[b:b + 1], blk)[0], decoded(c1[b:b + 1], s1[b:b + 1], blk)[0]
            at = f64(scale1)[..., None]
            assert np.array_equal(got[grew], (O.e4m3_round(old / at) * at)[grew])
            grown += int(grew.sum())
    return grown


@pytest.mark.parametrize("block,kw,pol", [
    (16, dict(ratio=0.06), {}), (64, dict(ratio=0.03), {}), (128, dict(), {}),
    (32, dict(ratio=0.1, n_layers=3, score_layer=1), dict(score_layer=1)),
    (16, dict(ratio=0.1), dict(ffn_gate=True, ffn_tau=1e-3, attn_update=True))])
def test_what_a_partial_step_keeps(lib, block, kw, pol):
    run = Case(lib, shape_of(**kw), True, block, **pol)
    run.step(True)
    grown = 0
    for _ in range(4):
        before = held(run.cache)
        out, _ = run.step(False)
        # (layers below the score layer run on every row)
        whole = [np.arange(run.s.seq_len)] * run.s.batch
        grown += check_kept(run, before, lambda l: out.idx if l >= run.opol.score_layer else whole)
    assert grown > 0   # (both ways of keeping a row were met)


def test_response_only_steps(lib):
    shape = shape_of(ratio=0.2, prompt_len=96, gen_len=64)
    run = Case(lib, shape, False, 32, select_from=96)
    run.pol.select_from = 96
    run.step(True)
    prompt = [t[:, :96].clone() if t.dim() == 4 else t[:, :, :3].clone() for x in held(run.cache) for t in x]
    for _ in range(3):
        before = held(run.cache)
        out, b4 = run.step(False)
        assert all(r.min() >= 96 for r in out.idx)
        run.check(out, b4, False)
        check_kept(run, before, lambda l: out.idx)
    # the prompt ends with a block: none of its codes and scales moved
    after = [t[:, :96] if t.dim() == 4 else t[:, :, :3] for x in held(run.cache) for t in x]
    assert all(torch.equal(a, b) for a, b in zip(prompt, after))


def test_second_skip_point(lib):
    shape, k2 = shape_of(n_layers=4, ratio=0.2), 10
    run = Case(lib, shape, True, 16, score_layer2=2, k2=k2)
    run.pol.score_layer2, run.pol.k2 = 2, k2
    B, N = shape.batch, shape.seq_len
    run.cache = lib.Cache(run.model.cfg, B, N, second_ref=True, kv8_block=16)
    run.ws = lib.Workspace(lib.dllm_step_workspace_size(run.model.cfg, B, N, run.pol))

    def pad(rows, width):
        a = np.full((B, width), -1, dtype=np.int32)
        for b, r in enumerate(rows):
            a[b, :len(r)] = r
        return torch.from_numpy(a).cuda(), torch.tensor([len(r) for r in rows], dtype=torch.int32, device="cuda")

    for t in range(4):
        run.pull()
        run.st.h_ref2 = f64(run.cache.h_ref2)
        before, b4 = held(run.cache), run.st.copy()
        out = O.step(run.ocfg, run.ow, run.st, run.opol, t == 0)
        io = dict(forced_unmask_pos=torch.from_numpy(out.unmasked.astype(np.int32)).cuda())
        if t:
            io["forced_idx"], io["forced_count"] = pad(out.idx, shape.k)
            io["forced_idx2"], io["forced_count2"] = pad(out.idx2, k2)
        lib.dllm_step_ex(run.model, run.cache, run.tokens, run.pol, t == 0, run.ws, **io)
        assert run.ws.device_status() == 0
        run.check(out, b4, t == 0)
        assert max_abs_rel(f64(run.cache.h_ref2), run.st.h_ref2) < 0.02 + 0.022   # (as Case.check)
        if t:
            assert all(len(a) < len(b) for a, b in zip(out.idx2, out.idx))
            check_kept(run, before, lambda l: out.idx if l < 2 else out.idx2)


def state_of(c):
    return [c.tokens] + [t for x in held(c.cache) for t in x] + [c.cache.conf, c.cache.pred, c.cache.h_ref]


@pytest.mark.parametrize("on_block", [False, True])
def test_generation_with_refreshes_equals_its_steps(lib, on_block):
    shape = shape_of(ratio=0.2)
    runs = [Case(lib, shape, True, 32) for _ in range(2)]
    for c in runs:
        c.pol.refresh_every = 0 if on_block else 3
        c.pol.refresh_on_block = int(on_block)
    g, s = runs
    T = 9
    ws = lib.Workspace(lib.dllm_generate_workspace_size(g.model.cfg, shape.batch, shape.seq_len, g.pol))
    flags = lib.dllm_generate(g.model, g.cache, g.tokens, g.pol, T, ws)
    # blocks of 32 positions at 5 a step: the first ends with the seventh step
    assert flags == ([t in (0, 7) for t in range(T)] if on_block else [t % 3 == 0 for t in range(T)])
    for dense in flags:
        lib.dllm_step(s.model, s.cache, s.tokens, s.pol, dense, s.ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(state_of(g), state_of(s)))


def test_tokens_in_host_memory(lib):
    shape = shape_of(ratio=0.2)
    h, d = [Case(lib, shape, True, 64) for _ in range(2)]
    B, N = shape.batch, shape.seq_len
    ws = lib.Workspace(lib.dllm_step_host_workspace_size(h.model.cfg, B, N, h.pol))
    tokens = h.tokens.cpu().pin_memory()
    for t in range(3):
        lib.dllm_step_host(h.model, h.cache, tokens, h.pol, t == 0, ws)
        lib.dllm_step(d.model, d.cache, d.tokens, d.pol, t == 0, d.ws)
    torch.cuda.synchronize()
    h.tokens.copy_(tokens)
    assert all(torch.equal(a, b) for a, b in zip(state_of(h), state_of(d)))
