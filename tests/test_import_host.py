"""The package without torch (CPU): the library handle, its structures, size queries and
plans need none, and only calls that take tensors import it."""
import os
import subprocess
import sys

from test_abi import lib  # noqa: F401  (builds the library)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys


class NoTorch:
    def find_spec(self, name, path=None, target=None):
        if name == "torch" or name.startswith("torch."):
            raise ImportError("torch is not there")


sys.meta_path.insert(0, NoTorch())
import sparse_token_recompute_b200 as S
from sparse_token_recompute_b200 import *
assert "torch" not in sys.modules
assert S.version() >= 101 and S.status_string(0) == "ok"
cfg = S.make_cfg(1, 256, 4, 4, 64, 512, 1024, 5e5, 1e-5, 1023, "bf16")
pol = S.make_policy(k=32, n_unmask=8, gen_start=64, block_len=64, kv8_block=64)
assert S.dllm_step_workspace_size(cfg, 1, 128, pol) > 0
assert S.dllm_kv8_scale_count(2, 100, 3, 64) == 12
assert S.dllm_attention_kv8_workspace_size(1, 1, 16384, 28, 4, 128) > 256
assert S.dllm_attention_plan_info(1, 4, 128, 4, 64)["ctas"] > 0
assert callable(S.dllm_kv8_write) and callable(dllm_attention_kv8) and callable(kv8_cache)
assert S.DLLM_ERR_INVALID_ARG == DLLM_ERR_INVALID_ARG
"""


def test_the_package_loads_without_torch(lib):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
