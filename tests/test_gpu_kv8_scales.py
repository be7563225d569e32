"""Attention over 8-bit caches whose V scales lie far apart: the softmax sum, which no
V scale may touch, and the weights, which f16 holds, against the oracle in 64 bits."""
import pytest
import torch

from test_gpu_kv8 import BF, check_attention, filled, normal

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
