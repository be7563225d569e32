"""Host-side checks of the 8-bit K/V cache operators (CPU): what the C entry points
refuse before they touch the GPU, and what the binding refuses before it calls them."""
import ctypes as C

import pytest
import torch

from test_abi import lib  # noqa: F401  (builds the library)

BUF = (C.c_uint8 * 8192)()
P = (C.addressof(BUF) + 255) & ~255   # an aligned address; never dereferenced on the host


def _norm(S, **kw):
    a = dict(q=P, ldq=256, k=P, ldk=128, kin=0, qg=P, kg=P, rope=P, qo=P, ldqo=256, ko=P, ldko=128,
             kout=0, idx=P, count=P, k_cap=4, B=2, N=8, Hq=2, Hkv=1, hd=128, eps=1e-5, dtype=1,
             ws=None, nb=0)
    a.update(kw)
    return S._qk_norm(*a.values(), None)


@pytest.mark.parametrize("kw,st", [
    (dict(B=-1), 1), (dict(N=-1), 1), (dict(k_cap=0), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1),
    (dict(dtype=7), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(Hq=3, Hkv=2), 2), (dict(hd=96), 2), (dict(hd=258, dtype=0), 2), (dict(hd=63, dtype=0), 2),
    (dict(B=1 << 20, k_cap=1 << 20), 2), (dict(idx=None, count=None, k_cap=9), 5),
    (dict(q=None), 1), (dict(ko=None), 1), (dict(qg=None), 1), (dict(q=P + 2), 1), (dict(rope=P + 8), 1),
    (dict(ldq=248), 1), (dict(ldq=260), 1), (dict(ldko=64), 1), (dict(ws=P, nb=100), 3),
    (dict(ws=P + 16, nb=512), 3), (dict(B=0), 0), (dict(N=0), 0)])
def test_norm_refusals(lib, kw, st):  # noqa: F811
    import sparse_token_recompute_b200 as S
    assert _norm(S, **kw) == st


def _write(S, **kw):
    a = dict(k=P, ldk=256, v=P, ldv=256, idx=P, count=P, k_cap=4, B=2, N=100, H=2, hd=128, block=64,
             k8=P, ks=P, v8=P, vs=P, ws=None, nb=0)
    a.update(kw)
    return S._kv8_write(*a.values(), None)


@pytest.mark.parametrize("kw,st", [
    (dict(B=-1), 1), (dict(k_cap=0), 1), (dict(H=0), 1), (dict(hd=96), 2), (dict(block=48), 2),
    (dict(block=8), 2), (dict(block=256), 2), (dict(block=0), 2), (dict(k=None), 1), (dict(vs=None), 1),
    (dict(k8=P + 8), 1), (dict(ks=P + 2), 1), (dict(idx=P + 1), 1), (dict(ldk=128), 1),
    (dict(ldv=260), 1), (dict(idx=None, count=None, k_cap=101), 5), (dict(ws=P, nb=8), 3),
    (dict(N=0), 0), (dict(B=0), 0)])
def test_write_refusals(lib, kw, st):  # noqa: F811
    import sparse_token_recompute_b200 as S
    assert _write(S, **kw) == st


def _read(S, **kw):
    a = dict(k8=P, ks=P, v8=P, vs=P, idx=P, count=P, k_cap=4, B=2, N=100, H=2, hd=128, block=64,
             k=P, ldk=256, v=P, ldv=256, ws=None, nb=0)
    a.update(kw)
    return S._kv8_read(*a.values(), None)


@pytest.mark.parametrize("kw,st", [
    (dict(k_cap=-3), 1), (dict(hd=32), 2), (dict(block=100), 2), (dict(v8=None), 1), (dict(v=P + 4), 1),
    (dict(ldk=255), 1), (dict(ws=P, nb=255), 3), (dict(B=0), 0)])
def test_read_refusals(lib, kw, st):  # noqa: F811
    import sparse_token_recompute_b200 as S
    assert _read(S, **kw) == st


def _attn(S, **kw):
    a = dict(q=P, k8=P, ks=P, v8=P, vs=P, o=P, m=None, l=None, count=P, kv_len=P, B=2, k_cap=4,
             N=100, Hq=4, Hkv=2, hd=128, block=64, ws=P, nb=1 << 20)
    a.update(kw)
    return S._attn_kv8(*a.values(), None)


@pytest.mark.parametrize("kw,st", [
    (dict(B=-1), 1), (dict(N=-1), 1), (dict(k_cap=0), 1), (dict(Hq=3), 2), (dict(hd=80), 2),
    (dict(block=24), 2), (dict(B=1 << 16, k_cap=1 << 16), 2), (dict(q=None), 1), (dict(o=None), 1),
    (dict(m=P), 1), (dict(l=P), 1), (dict(k8=None), 1), (dict(o=P + 2), 1), (dict(kv_len=P + 2), 1),
    (dict(ws=None), 3), (dict(ws=P + 8), 3), (dict(nb=64), 3), (dict(N=4096, nb=256), 3),
    (dict(B=0), 0)])
def test_attention_refusals(lib, kw, st):  # noqa: F811
    import sparse_token_recompute_b200 as S
    assert _attn(S, **kw) == st


def test_rope_table_refusals(lib):  # noqa: F811
    import sparse_token_recompute_b200 as S
    assert S._rope_table(P, -1, 64, 1e4, None) == 1
    assert S._rope_table(P, 4, 63, 1e4, None) == 1
    assert S._rope_table(P, 4, 64, 0.0, None) == 1
    assert S._rope_table(P + 4, 4, 64, 1e4, None) == 1
    assert S._rope_table(None, 0, 64, 1e4, None) == 0


def test_sizes(lib):  # noqa: F811
    import sparse_token_recompute_b200 as S
    assert S.dllm_kv8_scale_count(2, 100, 3, 64) == 12
    assert S.dllm_kv8_scale_count(2, 100, 3, 48) == 0
    # no key shares where the rows alone fill the GPU; shares for one row over many keys
    assert S.dllm_attention_kv8_workspace_size(32, 308, 1536, 32, 32, 128) == 256
    assert S.dllm_attention_kv8_workspace_size(1, 1, 16384, 28, 4, 128) > 256
    k8, ks, v8, vs = S.kv8_cache(2, 100, 3, 64, 16, device="cpu")
    assert k8.shape == (2, 100, 3, 64) and ks.shape == (2, 3, 7) and float(vs.abs().sum()) == 0


def test_the_binding_refuses_what_the_library_would_misread(lib):  # noqa: F811
    import sparse_token_recompute_b200 as S
    B, N, H, hd, blk, k = 2, 40, 2, 64, 16, 3
    c = S.kv8_cache(B, N, H, hd, blk, device="cpu")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    idx = torch.zeros(B, k, dtype=torch.int32)
    cnt = torch.zeros(B, dtype=torch.int32)
    R = B * k
    w = lambda k=bf(R, H * hd), v=bf(R, H * hd), idx=idx, cnt=cnt, c=c, blk=blk: S.dllm_kv8_write(
        k, v, idx, cnt, *c, blk)
    for kw, err in [(dict(k=torch.zeros(R, H * hd)), TypeError), (dict(k=bf(R, H * hd + 8)), ValueError),
                    (dict(v=bf(H * hd, R).t()), ValueError), (dict(k=bf(R - 1, H * hd)), ValueError),
                    (dict(idx=idx.long()), TypeError), (dict(idx=idx[:1]), ValueError),
                    (dict(cnt=cnt.float()), TypeError), (dict(cnt=torch.zeros(3, dtype=torch.int32)), ValueError),
                    (dict(blk=32), ValueError), (dict(c=(c[0].float(), *c[1:])), TypeError),
                    (dict(c=(c[0].transpose(1, 2), *c[1:])), ValueError),
                    (dict(c=(c[0], c[1].double(), *c[2:])), TypeError),
                    (dict(k=bf(1, H * hd).expand(R, H * hd)), ValueError)]:
        with pytest.raises(err):
            w(**kw)
    with pytest.raises(ValueError):
        S.dllm_kv8_read(*c, idx, cnt, bf(R, H * hd), bf(R, 64), blk)
    q = bf(R, 4 * hd)
    with pytest.raises(ValueError):
        S.dllm_attention_kv8(q, *c, bf(R, 2 * hd), cnt, k, blk)
    with pytest.raises(ValueError):
        S.dllm_attention_kv8(q, *c, bf(R, 4 * hd), cnt, k + 1, blk)
    with pytest.raises(ValueError):
        S.dllm_attention_kv8(bf(R, 4 * hd + 8), *c, bf(R, 4 * hd + 8), cnt, k, blk)
    with pytest.raises(TypeError):
        S.dllm_attention_kv8(q.half(), *c, q, cnt, k, blk)
    g, kk = bf(hd), bf(R, 2 * hd)
    rope = torch.zeros(N, hd // 2, 2)
    n = lambda q=q, kk=kk, g=g, rope=rope, qo=q, ko=kk: S.dllm_qk_norm_rope(q, kk, g, g, rope, qo, ko, idx,
                                                                         cnt, 1e-5)
    for kw, err in [(dict(q=q.half()), TypeError), (dict(kk=kk.float()), TypeError),
                    (dict(rope=rope.double()), TypeError), (dict(rope=rope[:, :5]), ValueError),
                    (dict(g=g.float()), TypeError), (dict(qo=bf(R, 5 * hd)), ValueError),
                    (dict(ko=bf(B, N + 1, 2, hd), rope=rope), ValueError), (dict(ko=bf(B, N, 1, hd)), ValueError)]:
        with pytest.raises(err):
            n(**kw)
    with pytest.raises(ValueError):
        S.dllm_qk_norm_rope(q, kk, g, g, rope, q, kk, None, None, 1e-5)


def test_more_positions_than_the_kernels_count_are_refused(lib):  # noqa: F811
    import sparse_token_recompute_b200 as S
    far = (1 << 30) + 1
    assert _norm(S, N=far) == _write(S, N=far) == _read(S, N=far) == _attn(S, N=far) == 2
    assert _attn(S, B=1, k_cap=1 << 20, Hq=1 << 11, Hkv=1, hd=64) == 2   # 2^31 rows of heads
    assert S.dllm_attention_kv8_workspace_size(1, 1, far, 4, 4, 64) == 256
