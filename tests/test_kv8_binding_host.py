"""What the binding of the q/k norm says when the number of positions is nowhere (CPU)."""
import pytest
import torch

from test_abi import lib  # noqa: F401  (builds the library)


def test_norm_without_a_number_of_positions(lib):  # noqa: F811
    """Compact keys, no table and no N: nothing says how many positions there are."""
    import sparse_token_recompute_b200 as S
    q, k, g = (torch.zeros(6, 256, dtype=torch.bfloat16), torch.zeros(6, 128, dtype=torch.bfloat16),
               torch.ones(64, dtype=torch.bfloat16))
    cnt = torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="N"):
        S.dllm_qk_norm_rope(q, k, g, g, None, q, k, None, cnt, 1e-5)
