"""Host-side checks of steps over 8-bit K/V caches (CPU): a cache and a policy that do not
belong together are refused before anything is launched."""
import ctypes as C

import pytest
import torch

import dllm_synth as SY
from test_abi import lib  # noqa: F401  (builds the library)

INVALID = 1


def case(S, cache_block, policy_block):
    s = SY.with_(SY.TINY, dtype="bf16", n_layers=2, d=256, n_heads=4, n_kv_heads=2, head_dim=64, ffn=512,
                 vocab=2048, batch=2, prompt_len=61, gen_len=100, block_len=32, n_unmask=5, ratio=0.25)
    model = S.Model(S.cfg_from_shape(s), SY.model_weights(s, seed=0, device="cpu"))
    pol = S.make_policy(0, 0.5, 0, 0, s.k, 0.0, s.n_unmask, s.prompt_len, s.block_len, kv8_block=policy_block)
    cache = S.Cache(model.cfg, s.batch, s.seq_len, device="cpu", kv8_block=cache_block)
    ws = S.Workspace(256 + S.dllm_generate_workspace_size(model.cfg, s.batch, s.seq_len, pol)
                     + S.dllm_step_host_workspace_size(model.cfg, s.batch, s.seq_len, pol), "cpu")
    ws.buf = ws.buf[-ws.buf.data_ptr() % 256:]   # (aligned as device memory is)
    ws.nbytes = ws.buf.numel()
    return model, pol, cache, ws, SY.prompt_tokens(s, seed=1)


@pytest.mark.parametrize("entry,cache_block,policy_block", [
    (e, c, p) for e in ("step", "step_ex", "generate", "step_host")
    for c, p in ((64, 0), (64, 16), (16, 64), (0, 32))
    if c or e != "step_host"])   # (a plain cache: refused by the step itself, after the tokens' copy)
def test_a_cache_of_another_block_is_refused(lib, entry, cache_block, policy_block):  # noqa: F811
    import sparse_token_recompute_b200 as S
    model, pol, cache, ws, tokens = case(S, cache_block, policy_block)
    go = {"step": lambda: S.dllm_step(model, cache, tokens, pol, True, ws, stream=0),
          "step_ex": lambda: S.dllm_step_ex(model, cache, tokens, pol, False, ws, stream=0),
          "generate": lambda: S.dllm_generate(model, cache, tokens, pol, 2, ws, stream=0),
          "step_host": lambda: S.dllm_step_host(model, cache, tokens, pol, True, ws, stream=0)}[entry]
    with pytest.raises(S.DllmError) as e:
        go()
    assert e.value.status == INVALID


def test_scales_without_a_block_are_refused_by_the_library(lib):  # noqa: F811
    """A caller of the C entry point: the cache names scales, the policy does not know of them."""
    import sparse_token_recompute_b200 as S
    model, pol, cache, ws, tokens = case(S, 64, 0)
    io = S.StepIO()
    go = lambda: S._step_ex(C.byref(model.cfg), C.byref(model.s), C.byref(cache.s), tokens.data_ptr(),
                            *tokens.shape, C.byref(pol), 1, C.byref(io), ws.ptr, ws.nbytes, None)
    assert go() == INVALID
    cache.v_scale = None
    cache._refresh()
    assert go() == INVALID


def test_codes_are_not_a_cache_of_the_other_calls(lib):  # noqa: F811
    """Layer and attention calls over plain caches read two or four bytes per element."""
    import sparse_token_recompute_b200 as S
    model, pol, cache, ws, tokens = case(S, 64, 64)
    B, N = tokens.shape
    k8, v8 = cache.k[0], cache.v[0]
    q = torch.zeros(B * 4, 256, dtype=torch.bfloat16)
    x, o = torch.zeros_like(cache.h_ref), torch.zeros_like(q)
    idx, cnt = torch.zeros(B, 4, dtype=torch.int32), torch.ones(B, dtype=torch.int32)
    ml = torch.zeros(B * 4, 4)
    for a, b in ((k8, v8), (k8.view(torch.uint8), v8), (v8.to(torch.bfloat16), v8)):
        for go in (lambda: S.dllm_partial_layer(model.cfg, model.layer(0), x, o, idx, cnt, a, b, ws, True, stream=0),
                   lambda: S.dllm_attention_bf16(q, a, b, o, cnt, 4, ws=ws, stream=0),
                   lambda: S.dllm_attention_stats_bf16(q, a, b, o, ml, ml, cnt, 4, ws=ws, stream=0),
                   lambda: S.dllm_attention_bf16_noalloc(q, a, b, o, cnt, 4, stream=0),
                   lambda: S.dllm_attention_update_bf16(q, o, ml, ml, cnt, 4, a, b, a, b, cnt, 4, 2, ws=ws, stream=0)):
            with pytest.raises(TypeError):
                go()
