"""Python binding of libdllm.so, the sm_100a selected-token denoising step.

Argument marshalling only: every step of the path runs in the library's
CUDA kernels.  Tensors are torch CUDA tensors (device memory and streams);
they are passed as raw pointers through ctypes.  If the shared library is
missing, importing this package raises: there is no fallback path.

The functions carry the C names (``dllm_score``, ``dllm_select``,
``dllm_unmask``, ``dllm_partial_layer``, ``dllm_step`` ...); ``Model``,
``Cache`` and ``Workspace`` hold the ctypes structs and the torch-owned
buffers the calls need.
"""
from __future__ import annotations

import ctypes as C
import json
import operator
import os
from typing import Dict, List, Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdllm.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m sparse_token_recompute_b200.build` "
        "(there is no CPU or eager fallback)")

_lib = C.CDLL(LIB_PATH)

DLLM_OK, DLLM_ERR_INVALID_ARG = 0, 1
DLLM_F32, DLLM_BF16 = 0, 1
DLLM_SCORE_COS, DLLM_SCORE_ES_L1 = 0, 1
DLLM_SELECT_TOPK, DLLM_SELECT_THRESH = 0, 1
DLLM_DEV_TIMEOUT, DLLM_DEV_CAPACITY, DLLM_DEV_BAD_INDEX, DLLM_DEV_BAD_SHAPE = 1, 2, 4, 8


class _Torch:
    """Stands for torch until a call needs it: structures, sizes and plans do without."""

    def __getattr__(self, name):
        global torch
        import torch
        return getattr(torch, name)


torch = _Torch()

vp = C.c_void_p


class ModelCfg(C.Structure):
    _fields_ = [("n_layers", C.c_int), ("d", C.c_int), ("n_heads", C.c_int),
                ("n_kv_heads", C.c_int), ("head_dim", C.c_int), ("ffn", C.c_int),
                ("vocab", C.c_int), ("rope_theta", C.c_float), ("rms_eps", C.c_float),
                ("mask_id", C.c_int), ("dtype", C.c_int)]


class LayerW(C.Structure):
    _fields_ = [(n, vp) for n in ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w_gate",
                                  "w_up", "w_down", "q_norm", "k_norm")]


class ModelW(C.Structure):
    _fields_ = [("embed", vp), ("layers", C.POINTER(LayerW)), ("final_norm", vp),
                ("lm_head", vp)]


class CacheS(C.Structure):
    _fields_ = [("k", C.POINTER(vp)), ("v", C.POINTER(vp)), ("h_ref", vp), ("conf", vp),
                ("pred", vp), ("h_ref2", vp), ("ctx", C.POINTER(vp)), ("ffn", C.POINTER(vp)),
                ("q", C.POINTER(vp)), ("att_m", C.POINTER(vp)), ("att_l", C.POINTER(vp)),
                ("k_scale", C.POINTER(vp)), ("v_scale", C.POINTER(vp))]


class Policy(C.Structure):
    _fields_ = [("score_layer", C.c_int), ("alpha", C.c_float), ("kind", C.c_int),
                ("mode", C.c_int), ("k", C.c_int), ("tau", C.c_float), ("n_unmask", C.c_int),
                ("gen_start", C.c_int), ("block_len", C.c_int), ("select_from", C.c_int),
                ("unmask_tau", C.c_float), ("refresh_every", C.c_int),
                ("refresh_on_block", C.c_int), ("score_layer2", C.c_int), ("k2", C.c_int),
                ("ffn_gate", C.c_int), ("ffn_tau", C.c_float), ("attn_update", C.c_int),
                ("kv8_block", C.c_int)]


class StepIO(C.Structure):
    _fields_ = [("forced_idx", vp), ("forced_count", vp), ("forced_unmask_pos", vp),
                ("idx_out", vp), ("count_out", vp), ("pos_out", vp), ("scores_out", vp),
                ("forced_idx2", vp), ("forced_count2", vp), ("idx2_out", vp),
                ("count2_out", vp), ("scores2_out", vp), ("ffn_rows_out", vp),
                ("forced_ffn", vp)]


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_i, _f, _sz = C.c_int, C.c_float, C.c_size_t
_status_string = _sig("dllm_status_string", C.c_char_p, [_i])
_version = _sig("dllm_version", _i, [])
_score = _sig("dllm_score", _i, [vp, vp, _i, _i, _i, _i, vp, vp, _i, _i, vp, vp, vp, _f, _i,
                                 vp, vp])
_select_ws = _sig("dllm_select_workspace_size", _sz, [_i, _i])
_select = _sig("dllm_select", _i, [vp, _i, _i, _i, _i, _f, vp, vp, _i, vp, _sz, vp])
_unmask = _sig("dllm_unmask", _i, [vp, vp, vp, _i, _i, _i, _i, _i, _i, vp, vp])
_unmask_tau = _sig("dllm_unmask_tau", _i, [vp, vp, vp, _i, _i, _i, _i, _i, _i, _f, vp, _i, vp])
_unmask_cap = _sig("dllm_unmask_capacity", _i, [C.POINTER(Policy)])
_select_range = _sig("dllm_select_range", _i, [vp, _i, _i, _i, _i, _i, _f, vp, vp, _i, vp, _sz,
                                               vp])
_layer_ws = _sig("dllm_partial_layer_workspace_size", _sz, [C.POINTER(ModelCfg), _i, _i, _i])
_layer = _sig("dllm_partial_layer", _i, [C.POINTER(ModelCfg), C.POINTER(LayerW), vp, _i, vp,
                                         vp, vp, _i, _i, _i, vp, vp, vp, _sz, vp])
_step_ws = _sig("dllm_step_workspace_size", _sz, [C.POINTER(ModelCfg), _i, _i,
                                                  C.POINTER(Policy)])
_step = _sig("dllm_step", _i, [C.POINTER(ModelCfg), C.POINTER(ModelW), C.POINTER(CacheS), vp,
                               _i, _i, C.POINTER(Policy), _i, vp, vp, vp, vp, vp, vp, vp, vp,
                               _sz, vp])
_step_ex = _sig("dllm_step_ex", _i, [C.POINTER(ModelCfg), C.POINTER(ModelW), C.POINTER(CacheS),
                                     vp, _i, _i, C.POINTER(Policy), _i, C.POINTER(StepIO), vp,
                                     _sz, vp])
_gen_ws = _sig("dllm_generate_workspace_size", _sz, [C.POINTER(ModelCfg), _i, _i,
                                                     C.POINTER(Policy)])
_gen = _sig("dllm_generate", _i, [C.POINTER(ModelCfg), C.POINTER(ModelW), C.POINTER(CacheS), vp,
                                  _i, _i, C.POINTER(Policy), _i, vp, C.POINTER(C.c_uint8), vp,
                                  _sz, vp])
_step_host_ws = _sig("dllm_step_host_workspace_size", _sz, [C.POINTER(ModelCfg), _i, _i,
                                                            C.POINTER(Policy)])
_step_host = _sig("dllm_step_host", _i, [C.POINTER(ModelCfg), C.POINTER(ModelW),
                                         C.POINTER(CacheS), vp, _i, _i, C.POINTER(Policy), _i,
                                         vp, vp, _sz, vp])
_devstat = _sig("dllm_get_device_status", _i, [vp, vp, C.POINTER(C.c_int32)])
_attn_noalloc = _sig("dllm_attention_bf16_noalloc", _i, [vp, vp, vp, vp, vp, _i, _i, _i, _i, _i,
                                                         _i, vp])
_attn_ws = _sig("dllm_attention_workspace_size", _sz, [_i])
_attn_stats = _sig("dllm_attention_stats_bf16", _i, [vp, vp, vp, vp, vp, vp, vp, _i, _i, _i, _i,
                                                     _i, _i, vp, _sz, vp])
_attn_upd_ws = _sig("dllm_attention_update_workspace_size", _sz, [_i])
_attn_upd = _sig("dllm_attention_update_bf16", _i, [vp, vp, vp, vp, vp, _i, _i, vp, vp, vp, vp,
                                                    vp, _i, _i, _i, _i, vp, _sz, vp])
_attn = _sig("dllm_attention_bf16", _i, [vp, vp, vp, vp, vp, _i, _i, _i, _i, _i, _i, vp, _sz,
                                         vp])


class _Int:
    """A C int argument of the calls whose host time matters: ctypes passes a Python int as it
    is, without the c_int instance (about 0.1 us each) that the type itself makes."""
    from_param = operator.index


_rope_table = _sig("dllm_rope_table", _i, [vp, _i, _i, _f, vp])
_n = _Int
_qk_norm = _sig("dllm_qk_norm_rope", _i, [vp, _n, vp, _n, _n, vp, vp, vp, vp, _n, vp, _n, _n, vp,
                                          vp, _n, _n, _n, _n, _n, _n, _f, _n, vp, _sz, vp])
_kv8_scales = _sig("dllm_kv8_scale_count", _sz, [_i, _i, _i, _i])
_kv8_write = _sig("dllm_kv8_write", _i, [vp, _n, vp, _n, vp, vp, _n, _n, _n, _n, _n, _n, vp, vp,
                                         vp, vp, vp, _sz, vp])
_kv8_read = _sig("dllm_kv8_read", _i, [vp, vp, vp, vp, vp, vp, _n, _n, _n, _n, _n, _n, vp, _n,
                                       vp, _n, vp, _sz, vp])
_attn_kv8_ws = _sig("dllm_attention_kv8_workspace_size", _sz, [_i, _i, _i, _i, _i, _i])
_attn_kv8 = _sig("dllm_attention_kv8", _i, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, _n, _n, _n,
                                            _n, _n, _n, _n, vp, _sz, vp])
_gemm_ws = _sig("dllm_gemm_workspace_size", _sz, [_i, _i, _i, _i])
_gemm = _sig("dllm_gemm_bf16", _i, [vp, vp, vp, _i, _i, _i, _i, _i, vp, _sz, vp])
_gemm_stall = _sig("dllm_selftest_gemm_stall", _i, [vp, vp, vp, _i, _i, _i, vp, _sz, vp])
_gemm_plan = _sig("dllm_gemm_plan_info", _i, [_i, _i, _i, vp, _i, _i, vp])
_attn_plan = _sig("dllm_attention_plan_info", _i, [_i, _i, _i, _i, _i, _i, vp])
_prof_enable = _sig("dllm_profile_enable", None, [_i])
_prof_reset = _sig("dllm_profile_reset", None, [])
_prof_read = _sig("dllm_profile_read", _sz, [C.c_char_p, _sz])


class DllmError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


def status_string(st: int) -> str:
    return _status_string(int(st)).decode()


def version() -> int:
    return int(_version())


def _check(st: int, where: str):
    if st != DLLM_OK:
        raise DllmError(st, where)


def ptr(t) -> Optional[int]:
    """Device (or host) address of a tensor; None stays NULL."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(t) -> int:
    if t.dtype == torch.bfloat16:
        return DLLM_BF16
    if t.dtype == torch.float32:
        return DLLM_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


# ----------------------------------------------------------------- workspace

def _empty_bytes(nbytes: int, device):
    # 256-byte alignment: torch's caching allocator returns at least 512-byte aligned blocks
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


class Workspace:
    """A caller-owned scratch buffer (torch memory) passed to the library."""

    def __init__(self, nbytes: int, device="cuda"):
        self.buf = _empty_bytes(nbytes, device)
        self.buf[:256].zero_()
        self.nbytes = self.buf.numel()

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    def device_status(self, stream=None) -> int:
        v = C.c_int32(0)
        _devstat(self.ptr, _stream(stream), C.byref(v))
        return int(v.value)


# ----------------------------------------------------------------- thin calls

def dllm_score(h_cur, h_ref, conf, masked, scores, alpha: float, kind: int = DLLM_SCORE_COS,
               logits=None, logit_pos=None, pred=None, stream=None):
    B, N, d = h_cur.shape
    Mm = V = 0
    if logits is not None:
        _, Mm, V = logits.shape
    st = _score(ptr(h_cur), ptr(h_ref), B, N, d, _dtype_code(h_cur), ptr(logits), ptr(logit_pos),
                Mm, V, ptr(conf), ptr(pred), ptr(masked), float(alpha), int(kind), ptr(scores),
                _stream(stream))
    _check(st, "dllm_score")


def dllm_select(scores, idx, count, mode: int, k: int, tau: float = 0.0, ws: Workspace = None,
                stream=None):
    B, N = scores.shape
    k_cap = idx.shape[1]
    st = _select(ptr(scores), B, N, int(mode), int(k), float(tau), ptr(idx), ptr(count), k_cap,
                 ws.ptr if ws else None, ws.nbytes if ws else 0, _stream(stream))
    _check(st, "dllm_select")


def dllm_select_range(scores, idx, count, lo: int, mode: int, k: int, tau: float = 0.0,
                      ws: Workspace = None, stream=None):
    B, N = scores.shape
    k_cap = idx.shape[1]
    st = _select_range(ptr(scores), B, N, int(lo), int(mode), int(k), float(tau), ptr(idx),
                       ptr(count), k_cap, ws.ptr if ws else None, ws.nbytes if ws else 0,
                       _stream(stream))
    _check(st, "dllm_select_range")


def dllm_select_workspace_size(B: int, N: int) -> int:
    return int(_select_ws(B, N))


def dllm_unmask(conf, pred, tokens, mask_id: int, gen_start: int, block_len: int, n_unmask: int,
                pos_out=None, stream=None):
    B, N = tokens.shape
    st = _unmask(ptr(conf), ptr(pred), ptr(tokens), B, N, int(mask_id), int(gen_start),
                 int(block_len), int(n_unmask), ptr(pos_out), _stream(stream))
    _check(st, "dllm_unmask")


def dllm_unmask_tau(conf, pred, tokens, mask_id: int, gen_start: int, block_len: int,
                    n_unmask: int, tau: float, pos_out=None, stream=None):
    B, N = tokens.shape
    pos_cap = pos_out.shape[1] if pos_out is not None else max(n_unmask, block_len)
    st = _unmask_tau(ptr(conf), ptr(pred), ptr(tokens), B, N, int(mask_id), int(gen_start),
                     int(block_len), int(n_unmask), float(tau), ptr(pos_out), int(pos_cap),
                     _stream(stream))
    _check(st, "dllm_unmask_tau")


def dllm_unmask_capacity(pol: "Policy") -> int:
    return int(_unmask_cap(C.byref(pol)))


def dllm_gemm_workspace_size(M, N, K, splits=0) -> int:
    return int(_gemm_ws(M, N, K, splits))


def dllm_gemm_bf16(A, Bm, Cm, accumulate=False, splits=0, ws: Workspace = None, stream=None):
    M, K = A.shape
    N = Bm.shape[0]
    if ws is None:
        ws = Workspace(dllm_gemm_workspace_size(M, N, K, splits), A.device)
    st = _gemm(ptr(A), ptr(Bm), ptr(Cm), M, N, K, int(bool(accumulate)), int(splits), ws.ptr,
               ws.nbytes, _stream(stream))
    _check(st, "dllm_gemm_bf16")
    return ws


GEMM_KINDS = {"plain": 0, "residual": 1, "swiglu": 2, "qkv": 3, "lmhead": 4}


def dllm_gemm_plan_info(kind: str, M: int, K: int, seg_cols, head_dim: int = 0) -> Dict[str, int]:
    """The host-side launch plan of one projection GEMM (no GPU work)."""
    segs = (C.c_int32 * len(seg_cols))(*[int(c) for c in seg_cols])
    out = (C.c_int32 * 5)()
    st = _gemm_plan(GEMM_KINDS[kind], int(M), int(K), C.cast(segs, C.c_void_p), len(seg_cols),
                    int(head_dim), C.cast(out, C.c_void_p))
    _check(st, "dllm_gemm_plan_info")
    return {"bn": out[0], "splits": out[1], "tiles_n": out[2], "grid": out[3], "pair": out[4]}


def dllm_attention_plan_info(B: int, k_cap: int, N: int, n_heads: int, head_dim: int,
                             in_step: bool = True) -> Dict[str, int]:
    """The host-side launch plan of the exact partial attention (no GPU work)."""
    out = (C.c_int32 * 3)()
    st = _attn_plan(int(B), int(k_cap), int(N), int(n_heads), int(head_dim), int(bool(in_step)),
                    C.cast(out, C.c_void_p))
    _check(st, "dllm_attention_plan_info")
    return {"tiles_per_cta": out[0], "key_shares": out[1], "ctas": out[2]}


def dllm_selftest_gemm_stall(A, Bm, Cm, ws: Workspace = None, stream=None):
    """The CTA-pair GEMM with one stage signal withheld: ends with DLLM_DEV_TIMEOUT
    in ws's device status (after the 2 s wait limit); C is undefined."""
    M, K = A.shape
    N = Bm.shape[0]
    if ws is None:
        ws = Workspace(dllm_gemm_workspace_size(M, N, K, 1), A.device)
    st = _gemm_stall(ptr(A), ptr(Bm), ptr(Cm), M, N, K, ws.ptr, ws.nbytes, _stream(stream))
    _check(st, "dllm_selftest_gemm_stall")
    return ws


def _no_codes(where: str, *tensors):
    """The calls over plain K/V: one-byte codes (kv8_cache) would be read past their end."""
    for t in tensors:
        if t.element_size() == 1:
            raise TypeError(f"{where}: K/V of {t.dtype}, wanted rows of the model's dtype")


def dllm_attention_workspace_size(B: int) -> int:
    return int(_attn_ws(B))


def dllm_attention_bf16(q, k_cache, v_cache, o, count, k_cap: int, ws: Workspace = None,
                        stream=None):
    _no_codes("dllm_attention_bf16", k_cache, v_cache)
    B, N, Hkv, hd = k_cache.shape
    Hq = q.shape[1] // hd
    if ws is None:
        ws = Workspace(dllm_attention_workspace_size(B), q.device)
    st = _attn(ptr(q), ptr(k_cache), ptr(v_cache), ptr(o), ptr(count), B, int(k_cap), N, Hq, Hkv,
               hd, ws.ptr, ws.nbytes, _stream(stream))
    _check(st, "dllm_attention_bf16")
    return ws


def dllm_attention_stats_bf16(q, k_cache, v_cache, o, m, l, count, k_cap: int,
                              ws: Workspace = None, stream=None):
    """dllm_attention_bf16 plus each row's softmax statistics m, l [B*k_cap, Hq] (f32)."""
    _no_codes("dllm_attention_stats_bf16", k_cache, v_cache)
    B, N, Hkv, hd = k_cache.shape
    Hq = q.shape[1] // hd
    if ws is None:
        ws = Workspace(dllm_attention_workspace_size(B), q.device)
    st = _attn_stats(ptr(q), ptr(k_cache), ptr(v_cache), ptr(o), ptr(m), ptr(l), ptr(count), B,
                     int(k_cap), N, Hq, Hkv, hd, ws.ptr, ws.nbytes, _stream(stream))
    _check(st, "dllm_attention_stats_bf16")
    return ws


def dllm_attention_update_bf16(q, o, m, l, r_count, r_cap: int, k_new, v_new, k_old, v_old,
                               a_count, a_cap: int, n_kv_heads: int, ws: Workspace = None,
                               stream=None):
    """Incremental attention of stable rows (see include/dllm.h); q/o [B*r_cap, Hq*hd],
    m/l [B*r_cap, Hq] updated in place; changed keys [B*a_cap, Hkv, hd]."""
    _no_codes("dllm_attention_update_bf16", k_new, v_new, k_old, v_old)
    B = r_count.shape[0]
    hd = k_new.shape[-1]
    Hq = q.shape[1] // hd
    if ws is None:
        ws = Workspace(int(_attn_upd_ws(B)), q.device)
    st = _attn_upd(ptr(q), ptr(o), ptr(m), ptr(l), ptr(r_count), B, int(r_cap), ptr(k_new),
                   ptr(v_new), ptr(k_old), ptr(v_old), ptr(a_count), int(a_cap), Hq,
                   int(n_kv_heads), hd, ws.ptr, ws.nbytes, _stream(stream))
    _check(st, "dllm_attention_update_bf16")
    return ws


DLLM_NOALLOC_MAX_SEQS = 4096


def dllm_attention_bf16_noalloc(q, k_cache, v_cache, o, count, k_cap: int, stream=None):
    """Partial attention without a workspace, for callers that cannot allocate
    device memory (memory carved into fixed pools, operators handed only their
    tensors); its scratch is a fixed array inside the library shared by all calls."""
    _no_codes("dllm_attention_bf16_noalloc", k_cache, v_cache)
    B, N, Hkv, hd = k_cache.shape
    Hq = q.shape[1] // hd
    st = _attn_noalloc(ptr(q), ptr(k_cache), ptr(v_cache), ptr(o), ptr(count), B, int(k_cap), N,
                       Hq, Hkv, hd, _stream(stream))
    _check(st, "dllm_attention_bf16_noalloc")


# ----------------------------------------------------------------- 8-bit K/V cache
#
# A call for a handful of rows costs the GPU a few microseconds, so the checks below are
# written to cost little when they pass: each function compares what it needs at once and
# looks for the reason only when something does not fit.

def _bad(checks, device):
    """Raises the error of the first failing check of [(name, tensor, dtypes, shape)]: shape
    None entries are any size; ("rows", w) wants a 2-D tensor of w contiguous elements per
    row."""
    for name, t, dtypes, shape in checks:
        if t is None:
            continue
        if t.dtype not in dtypes:
            raise TypeError(f"{name}: dtype {t.dtype}, wanted {' or '.join(map(str, dtypes))}")
        if shape[0] == "rows":
            if t.dim() != 2 or t.shape[1] != shape[1] or (shape[1] > 1 and t.stride(1) != 1) or (
                    t.shape[0] > 1 and t.stride(0) < shape[1]):
                raise ValueError(f"{name}: shape {tuple(t.shape)} strides {t.stride()}, wanted "
                                 f"rows of {shape[1]} contiguous elements that do not overlap")
        elif not t.is_contiguous():
            raise ValueError(f"{name}: not contiguous")
        elif len(shape) != t.dim() or any(w is not None and w != h for w, h in zip(shape, t.shape)):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, wanted {shape}")
    for name, t, _, _ in checks:
        if t is not None and (t.get_device() < 0 or t.get_device() != device):
            raise ValueError(f"{name}: on {t.device}, wanted a CUDA tensor on the others' device")
    raise ValueError("arguments that do not fit together")


_CODES = _F32 = _I32 = _BF16 = None


def _dtypes():
    """The types above, which the calls below compare with (set by the first of them)."""
    global _CODES, _F32, _I32, _BF16
    _CODES = (torch.float8_e4m3fn, torch.uint8)
    _F32, _I32, _BF16 = torch.float32, torch.int32, torch.bfloat16


def _kv8_checks(k8, k_scale, v8, v_scale, B, N, H, hd, nblk):
    f32 = (_F32,)
    return [("k8", k8, _CODES, (B, N, H, hd)), ("v8", v8, _CODES, (B, N, H, hd)),
            ("k_scale", k_scale, f32, (B, H, nblk)), ("v_scale", v_scale, f32, (B, H, nblk))]


def _cache_fits(k8, ks, v8, vs, shape, scales, dev):
    return (k8.dtype in _CODES and v8.dtype in _CODES and ks.dtype is _F32 and vs.dtype is _F32
            and v8.shape == shape and ks.shape == scales and vs.shape == scales
            and k8.is_contiguous() and v8.is_contiguous() and ks.is_contiguous()
            and vs.is_contiguous() and dev >= 0 and v8.get_device() == dev
            and ks.get_device() == dev and vs.get_device() == dev)


def _rows_fit(t, dtype, width, dev):
    """Rows and row stride of a 2-D tensor of `width` contiguous elements per row; stride 0 if
    it is none."""
    sh = t.shape
    if t.dtype is not dtype or len(sh) != 2 or sh[1] != width or t.get_device() != dev:
        return 0, 0
    if t.is_contiguous():
        return sh[0], width
    a, b = t.stride()
    return sh[0], a if (b == 1 or width == 1) and a >= width else 0


def _cache_rows_fit(t, dtype, shape, dev):
    """1 if the tensor is a contiguous cache of that shape, else 0."""
    return int(t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == dev)


def _lists_fit(idx, count, B, rows, dev):
    """k_cap of idx [B, k_cap] / count [B] over compact tensors of `rows` rows; 0 if they do
    not fit."""
    k_cap = rows // B if B else 1
    if idx is not None:
        sh = idx.shape
        if len(sh) != 2 or sh[0] != B or idx.dtype is not _I32 or not idx.is_contiguous() or (
                idx.get_device() != dev):
            return 0
        k_cap = sh[1]
    if count is not None and (count.shape != (B,) or count.dtype is not _I32
                              or not count.is_contiguous() or count.get_device() != dev):
        return 0
    return k_cap if rows >= B * k_cap else 0


def _list_checks(idx, count, B):
    i32 = (_I32,)
    return [("idx", idx, i32, (B, None)), ("count", count, i32, (B,))]


def _stream_context(stream, device):
    """The stream of a call as torch's current one (None: it is already)."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _launch(dev: int, fn, args, ws, stream, where: str):
    """fn(*args, workspace, bytes, stream) on device `dev`, which is made current for the call."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    p, n = (None, 0) if ws is None else (ws.buf.data_ptr(), ws.nbytes)
    if ws is not None and ws.buf.get_device() != dev:
        raise ValueError(f"{where}: the workspace is on {ws.buf.device}")
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, p, n, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, p, n, stream)
    if st:
        raise DllmError(st, where)


def dllm_rope_table(table, theta: float, stream=None):
    """table [N, head_dim/2, 2] float32 <- cos, sin of the rotation angles."""
    if _F32 is None:
        _dtypes()
    dev = table.get_device()
    if (table.dtype is not _F32 or dev < 0 or table.dim() != 3 or table.shape[2] != 2
            or not table.is_contiguous()):
        _bad([("table", table, (_F32,), (None, None, 2))], dev)
    with torch.cuda.device(dev):
        st = _rope_table(ptr(table), table.shape[0], 2 * table.shape[1], float(theta),
                         _stream(stream))
    _check(st, "dllm_rope_table")


def dllm_qk_norm_rope(q, k, q_gain, k_gain, rope, q_out, k_out, idx, count, eps: float,
                      N: int = None, ws: Workspace = None, stream=None):
    """Per-head RMS norm of q and k rows and their rotation (see include/dllm.h).  q, q_out:
    [rows, n_heads*head_dim]; k, k_out: [rows, n_kv_heads*head_dim] compact rows, or a
    [B, N, n_kv_heads, head_dim] cache whose rows at the positions are meant; rope: a
    dllm_rope_table or None; idx [B, k_cap] and count [B] as for dllm_partial_layer.  The
    number of positions N comes from a cache or the table."""
    if _F32 is None:
        _dtypes()
    code, dt, dev, hd = _dtype_code(q), q.dtype, q.get_device(), q_gain.shape[0]
    if idx is None and count is None:
        raise ValueError("idx or count: the number of sequences is theirs")
    B = (idx if idx is not None else count).shape[0]
    wq, sk = q.shape[1], k.shape
    k_in, k_to = len(sk) == 4, k_out.dim() == 4
    if N is None:
        if rope is None and not (k_in or k_to):
            raise ValueError("N: the number of positions, which neither a cache nor a table gives")
        N = sk[1] if k_in else k_out.shape[1] if k_to else rope.shape[0]
    wk = sk[2] * hd if k_in else sk[1]
    rows, ldq = _rows_fit(q, dt, wq, dev)
    n, ldqo = _rows_fit(q_out, dt, wq, dev)
    rows = n if n < rows else rows
    if k_in:
        ldk = _cache_rows_fit(k, dt, (B, N, wk // hd, hd), dev)
    else:
        n, ldk = _rows_fit(k, dt, wk, dev)
        rows = n if n < rows else rows
    if k_to:
        ldko = _cache_rows_fit(k_out, dt, (B, N, wk // hd, hd), dev)
    else:
        n, ldko = _rows_fit(k_out, dt, wk, dev)
        rows = n if n < rows else rows
    k_cap = _lists_fit(idx, count, B, rows, dev)
    if not (ldq and ldqo and ldk and ldko and k_cap and dev >= 0 and wq % hd == 0 and wk % hd == 0
            and q_gain.dtype is dt and k_gain.dtype is dt and k_gain.shape == (hd,)
            and q_gain.dim() == 1 and q_gain.get_device() == dev and k_gain.get_device() == dev
            and q_gain.is_contiguous() and k_gain.is_contiguous()
            and (rope is None or (rope.dtype is _F32 and rope.get_device() == dev
                                  and rope.is_contiguous() and rope.shape[1:] == (hd // 2, 2)
                                  and rope.shape[0] >= N))):
        if wq % hd or wk % hd:
            raise ValueError(f"rows of {wq} and {wk} elements for heads of {hd}")
        if rope is not None and rope.dim() == 3 and rope.shape[0] < N:
            raise ValueError(f"rope: {rope.shape[0]} positions, wanted {N}")
        _bad([("q", q, (dt,), ("rows", wq)), ("q_out", q_out, (dt,), ("rows", wq)),
              ("k", k, (dt,), (B, N, wk // hd, hd) if k_in else ("rows", wk)),
              ("k_out", k_out, (dt,), (B, N, wk // hd, hd) if k_to else ("rows", wk)),
              ("q_gain", q_gain, (dt,), (hd,)), ("k_gain", k_gain, (dt,), (hd,)),
              ("rope", rope, (_F32,), (None, hd // 2, 2))]
             + _list_checks(idx, count, B), dev)
    _launch(dev, _qk_norm, (q.data_ptr(), ldq, k.data_ptr(), ldk, k_in, q_gain.data_ptr(),
                            k_gain.data_ptr(), ptr(rope), q_out.data_ptr(), ldqo,
                            k_out.data_ptr(), ldko, k_to, ptr(idx), ptr(count), k_cap, B, N,
                            wq // hd, wk // hd, hd, eps, code), ws, stream, "dllm_qk_norm_rope")


def dllm_kv8_scale_count(B: int, N: int, n_kv_heads: int, block: int) -> int:
    return int(_kv8_scales(B, N, n_kv_heads, block))


def kv8_cache(B: int, N: int, n_kv_heads: int, head_dim: int, block: int, device="cuda"):
    """An empty 8-bit cache: codes [B, N, n_kv_heads, head_dim] (float8_e4m3fn) and scales
    [B, n_kv_heads, ceil(N/block)] of zeros, as (k8, k_scale, v8, v_scale)."""

    def code():
        return torch.zeros(B, N, n_kv_heads, head_dim, dtype=torch.uint8,
                           device=device).view(torch.float8_e4m3fn)

    def scale():
        return torch.zeros(B, n_kv_heads, -(-N // block), device=device)
    return code(), scale(), code(), scale()


def _kv8_rows_call(fn, where, k, v, idx, count, k8, k_scale, v8, v_scale, block, ws, stream, reads):
    if _F32 is None:
        _dtypes()
    shape = k8.shape
    B, N, H, hd = shape
    nblk, dev, w = -(-N // max(block, 1)), k8.get_device(), H * hd
    rows, ldk = _rows_fit(k, _BF16, w, dev)
    n, ldv = _rows_fit(v, _BF16, w, dev)
    rows = n if n < rows else rows
    k_cap = _lists_fit(idx, count, B, rows, dev)
    if not (ldk and ldv and k_cap and _cache_fits(k8, k_scale, v8, v_scale, shape, (B, H, nblk), dev)):
        if ldk and ldv and B and rows < B * (idx.shape[1] if idx is not None else 1):
            raise ValueError(f"compact tensors of {rows} rows for {B} sequences")
        bf = (_BF16,)
        _bad([("k", k, bf, ("rows", w)), ("v", v, bf, ("rows", w))]
             + _kv8_checks(k8, k_scale, v8, v_scale, B, N, H, hd, nblk)
             + _list_checks(idx, count, B), dev)
    lists = (ptr(idx), ptr(count), k_cap, B, N, H, hd, block)
    cache = (k8.data_ptr(), k_scale.data_ptr(), v8.data_ptr(), v_scale.data_ptr())
    kv = (k.data_ptr(), ldk, v.data_ptr(), ldv)
    _launch(dev, fn, cache + lists + kv if reads else kv + lists + cache, ws, stream, where)


def dllm_kv8_write(k, v, idx, count, k8, k_scale, v8, v_scale, block: int, ws: Workspace = None,
                   stream=None):
    """K/V rows [rows, n_kv_heads*head_dim] bf16 into the 8-bit cache at the positions idx
    [B, k_cap] (None: row j at position j), count [B] of them (None: all)."""
    _kv8_rows_call(_kv8_write, "dllm_kv8_write", k, v, idx, count, k8, k_scale, v8, v_scale, block,
                   ws, stream, False)


def dllm_kv8_read(k8, k_scale, v8, v_scale, idx, count, k_out, v_out, block: int,
                  ws: Workspace = None, stream=None):
    """Rows of the 8-bit cache as bf16 compact rows [rows, n_kv_heads*head_dim]."""
    _kv8_rows_call(_kv8_read, "dllm_kv8_read", k_out, v_out, idx, count, k8, k_scale, v8, v_scale,
                   block, ws, stream, True)


def dllm_attention_kv8_workspace_size(B, k_cap, N, n_heads, n_kv_heads, head_dim) -> int:
    return int(_attn_kv8_ws(B, k_cap, N, n_heads, n_kv_heads, head_dim))


def dllm_attention_kv8(q, k8, k_scale, v8, v_scale, o, count, k_cap: int, block: int, kv_len=None,
                       m=None, l=None, ws: Workspace = None, stream=None):
    """Attention of compact query rows [B*k_cap, n_heads*head_dim] over the 8-bit cache (the
    first kv_len[b] positions of each sequence); returns the workspace, to be kept for the
    next call of these sizes."""
    if _F32 is None:
        _dtypes()
    bf16, shape, dev = _BF16, k8.shape, k8.get_device()
    B, N, H, hd = shape
    R, wq = q.shape
    nblk, Hq = -(-N // max(block, 1)), wq // hd
    if not (q.dtype is bf16 and o.dtype is bf16 and o.shape[1:] == (wq,) and R >= B * k_cap
            and o.shape[0] >= B * k_cap and q.is_contiguous() and o.is_contiguous()
            and q.get_device() == dev and o.get_device() == dev and wq % hd == 0
            and _lists_fit(None, count, B, R, dev) and (kv_len is None or _lists_fit(None, kv_len, B, R, dev))
            and (m is None or (m.dtype is _F32 and m.shape[1:] == (Hq,) and m.is_contiguous()
                               and m.shape[0] >= B * k_cap and m.get_device() == dev))
            and (l is None or (l.dtype is _F32 and l.shape[1:] == (Hq,) and l.is_contiguous()
                               and l.shape[0] >= B * k_cap and l.get_device() == dev))
            and _cache_fits(k8, k_scale, v8, v_scale, shape, (B, H, nblk), dev)):
        if wq % hd:
            raise ValueError(f"rows of {wq} elements for heads of {hd}")
        for name, t in (("q", q), ("o", o), ("m", m), ("l", l)):
            if t is not None and t.shape[0] < B * k_cap:
                raise ValueError(f"{name}: {t.shape[0]} rows for {B} sequences of {k_cap}")
        bf, f32 = (bf16,), (_F32,)
        _bad([("q", q, bf, (None, wq)), ("o", o, bf, (None, wq)), ("m", m, f32, (None, Hq)),
              ("l", l, f32, (None, Hq))] + _kv8_checks(k8, k_scale, v8, v_scale, B, N, H, hd, nblk)
             + _list_checks(None, count, B) + _list_checks(None, kv_len, B), dev)
    if ws is None:  # (allocated for, and its status cleared on, the stream of the call)
        with _stream_context(stream, k8.device):
            ws = Workspace(dllm_attention_kv8_workspace_size(B, k_cap, N, Hq, H, hd), k8.device)
    _launch(dev, _attn_kv8, (q.data_ptr(), k8.data_ptr(), k_scale.data_ptr(), v8.data_ptr(),
                             v_scale.data_ptr(), o.data_ptr(), ptr(m), ptr(l), ptr(count),
                             ptr(kv_len), B, k_cap, N, Hq, H, hd, block), ws, stream,
            "dllm_attention_kv8")
    return ws


def profile_enable(on: bool = True):
    _prof_enable(int(bool(on)))


def profile_reset():
    _prof_reset()


def profile_read() -> Dict[str, List[float]]:
    n = _prof_read(None, 0)
    buf = C.create_string_buffer(int(n))
    _prof_read(buf, n)
    return json.loads(buf.value.decode())


# ----------------------------------------------------------------- model / cache

def make_cfg(n_layers, d, n_heads, n_kv_heads, head_dim, ffn, vocab, rope_theta, rms_eps,
             mask_id, dtype) -> ModelCfg:
    return ModelCfg(n_layers, d, n_heads, n_kv_heads, head_dim, ffn, vocab, float(rope_theta),
                    float(rms_eps), mask_id, DLLM_BF16 if dtype == "bf16" else DLLM_F32)


def cfg_from_shape(s) -> ModelCfg:
    return make_cfg(s.n_layers, s.d, s.n_heads, s.n_kv_heads, s.head_dim, s.ffn, s.vocab,
                    s.rope_theta, s.rms_eps, s.mask_id, s.dtype)


def layer_struct(L: Dict[str, object]) -> LayerW:
    return LayerW(*(ptr(L[n]) for n in ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm",
                                        "w_gate", "w_up", "w_down")),
                  ptr(L.get("q_norm")), ptr(L.get("k_norm")))


class Model:
    """Weights (torch CUDA tensors, dict layout of ``dllm_synth.model_weights``) plus
    the ctypes structs that point at them."""

    def __init__(self, cfg: ModelCfg, W: Dict[str, object]):
        self.cfg = cfg
        self.W = W
        n = len(W["layers"])
        self._layers = (LayerW * max(n, 1))(*[layer_struct(L) for L in W["layers"]])
        self.s = ModelW(ptr(W["embed"]), self._layers, ptr(W["final_norm"]), ptr(W["lm_head"]))

    def layer(self, i: int) -> LayerW:
        return self._layers[i]


class Cache:
    """Per-layer K/V caches, hidden reference, cached confidence and argmax (torch memory).
    kv8_block > 0: the K/V caches in 8 bits (float8_e4m3fn codes and their scales)."""

    def __init__(self, cfg: ModelCfg, B: int, N: int, device="cuda", second_ref: bool = False,
                 ffn_gate: bool = False, attn_update: bool = False, kv8_block: int = 0):
        dt = torch.bfloat16 if cfg.dtype == DLLM_BF16 else torch.float32
        kv = (B, N, cfg.n_kv_heads, cfg.head_dim)
        self.k_scale = self.v_scale = None
        self.kv8_block = int(kv8_block)
        if kv8_block:
            layers = [kv8_cache(*kv, kv8_block, device) for _ in range(cfg.n_layers)]
            self.k, self.k_scale, self.v, self.v_scale = ([c[i] for c in layers] for i in range(4))
        else:
            self.k = [torch.zeros(kv, dtype=dt, device=device) for _ in range(cfg.n_layers)]
            self.v = [torch.zeros(kv, dtype=dt, device=device) for _ in range(cfg.n_layers)]
        self.h_ref = torch.zeros(B, N, cfg.d, dtype=dt, device=device)
        # reference of the second skip point (policies with score_layer2 > 0)
        self.h_ref2 = torch.zeros(B, N, cfg.d, dtype=dt, device=device) if second_ref else None
        # DyLLM FFN gate: per layer, attention outputs and FFN outputs of every row
        q = cfg.n_heads * cfg.head_dim
        self.ctx = [torch.zeros(B, N, q, dtype=dt, device=device)
                    for _ in range(cfg.n_layers)] if ffn_gate else None
        self.ffn = [torch.zeros(B, N, cfg.d, dtype=dt, device=device)
                    for _ in range(cfg.n_layers)] if ffn_gate else None
        # approximate attention: per layer each row's query and softmax statistics
        self.q = [torch.zeros(B, N, q, dtype=dt, device=device)
                  for _ in range(cfg.n_layers)] if attn_update else None
        self.att_m = [torch.zeros(B, N, cfg.n_heads, dtype=torch.float32, device=device)
                      for _ in range(cfg.n_layers)] if attn_update else None
        self.att_l = [torch.zeros(B, N, cfg.n_heads, dtype=torch.float32, device=device)
                      for _ in range(cfg.n_layers)] if attn_update else None
        self.conf = torch.zeros(B, N, dtype=torch.float32, device=device)
        self.pred = torch.zeros(B, N, dtype=torch.int32, device=device)
        self._refresh()

    def _refresh(self):
        L = max(len(self.k), 1)
        self._kp = (vp * L)(*[ptr(t) for t in self.k])
        self._vp = (vp * L)(*[ptr(t) for t in self.v])
        self._cp = (vp * L)(*[ptr(t) for t in self.ctx]) if self.ctx else None
        self._fp = (vp * L)(*[ptr(t) for t in self.ffn]) if self.ffn else None
        self._qp = (vp * L)(*[ptr(t) for t in self.q]) if self.q else None
        self._mp = (vp * L)(*[ptr(t) for t in self.att_m]) if self.att_m else None
        self._lp = (vp * L)(*[ptr(t) for t in self.att_l]) if self.att_l else None
        self._ksp = (vp * L)(*[ptr(t) for t in self.k_scale]) if self.k_scale else None
        self._vsp = (vp * L)(*[ptr(t) for t in self.v_scale]) if self.v_scale else None
        self.s = CacheS(self._kp, self._vp, ptr(self.h_ref), ptr(self.conf), ptr(self.pred),
                        ptr(self.h_ref2), self._cp, self._fp, self._qp, self._mp, self._lp,
                        self._ksp, self._vsp)


def make_policy(score_layer=0, alpha=0.5, kind=DLLM_SCORE_COS, mode=DLLM_SELECT_TOPK, k=1,
                tau=0.0, n_unmask=1, gen_start=0, block_len=32, select_from=0, unmask_tau=0.0,
                refresh_every=0, refresh_on_block=False, score_layer2=0, k2=0, ffn_gate=False,
                ffn_tau=0.0, attn_update=False, kv8_block=0) -> Policy:
    return Policy(score_layer, float(alpha), kind, mode, k, float(tau), n_unmask, gen_start,
                  block_len, int(select_from), float(unmask_tau), int(refresh_every),
                  int(bool(refresh_on_block)), int(score_layer2), int(k2), int(bool(ffn_gate)),
                  float(ffn_tau), int(bool(attn_update)), int(kv8_block))


def dllm_partial_layer_workspace_size(cfg: ModelCfg, B: int, N: int, k_cap: int) -> int:
    return int(_layer_ws(C.byref(cfg), B, N, k_cap))


def dllm_partial_layer(cfg: ModelCfg, lw: LayerW, x_in, x_out, idx, count, k_cache, v_cache,
                       ws: Workspace, x_in_is_full: bool, stream=None):
    _no_codes("dllm_partial_layer", k_cache, v_cache)
    B, k_cap = idx.shape
    N = k_cache.shape[1]
    st = _layer(C.byref(cfg), C.byref(lw), ptr(x_in), int(bool(x_in_is_full)), ptr(x_out),
                ptr(idx), ptr(count), k_cap, B, N, ptr(k_cache), ptr(v_cache), ws.ptr, ws.nbytes,
                _stream(stream))
    _check(st, "dllm_partial_layer")


def _same_block(cache: Cache, pol: Policy, where: str):
    """An 8-bit cache steps under policies of its own block: another one's scales lie elsewhere."""
    if cache.kv8_block and cache.kv8_block != pol.kv8_block:
        raise DllmError(DLLM_ERR_INVALID_ARG, f"{where}: a cache with blocks of {cache.kv8_block} under "
                                              f"policy.kv8_block {pol.kv8_block}")


def dllm_step_workspace_size(cfg: ModelCfg, B: int, N: int, pol: Policy) -> int:
    return int(_step_ws(C.byref(cfg), B, N, C.byref(pol)))


def dllm_step(model: Model, cache: Cache, tokens, pol: Policy, dense: bool, ws: Workspace,
              forced_idx=None, forced_count=None, forced_unmask_pos=None, idx_out=None,
              count_out=None, pos_out=None, scores_out=None, stream=None):
    B, N = tokens.shape
    _same_block(cache, pol, "dllm_step")
    st = _step(C.byref(model.cfg), C.byref(model.s), C.byref(cache.s), ptr(tokens), B, N,
               C.byref(pol), int(bool(dense)), ptr(forced_idx), ptr(forced_count),
               ptr(forced_unmask_pos), ptr(idx_out), ptr(count_out), ptr(pos_out),
               ptr(scores_out), ws.ptr, ws.nbytes, _stream(stream))
    _check(st, "dllm_step")


def dllm_generate_workspace_size(cfg: ModelCfg, B: int, N: int, pol: Policy) -> int:
    return int(_gen_ws(C.byref(cfg), B, N, C.byref(pol)))


def dllm_generate(model: Model, cache: Cache, tokens, pol: Policy, n_steps: int, ws: Workspace,
                  pos_log=None, stream=None):
    """n_steps steps with the policy's refresh schedule; returns the per-step
    dense flags (host list of bool).  pos_log: device [n_steps, B, capacity]."""
    B, N = tokens.shape
    _same_block(cache, pol, "dllm_generate")
    flags = (C.c_uint8 * max(int(n_steps), 1))()
    st = _gen(C.byref(model.cfg), C.byref(model.s), C.byref(cache.s), ptr(tokens), B, N,
              C.byref(pol), int(n_steps), ptr(pos_log), flags, ws.ptr, ws.nbytes,
              _stream(stream))
    _check(st, "dllm_generate")
    return [bool(flags[t]) for t in range(int(n_steps))]


def dllm_step_ex(model: Model, cache: Cache, tokens, pol: Policy, dense: bool, ws: Workspace,
                 stream=None, **io):
    """dllm_step with the second skip point; keyword tensors fill dllm_step_io
    (forced_idx, forced_count, forced_unmask_pos, idx_out, count_out, pos_out,
    scores_out, forced_idx2, forced_count2, idx2_out, count2_out, scores2_out,
    ffn_rows_out, forced_ffn)."""
    B, N = tokens.shape
    _same_block(cache, pol, "dllm_step_ex")
    s = StepIO(*[ptr(io.get(name)) for name, _ in StepIO._fields_])
    unknown = set(io) - {name for name, _ in StepIO._fields_}
    if unknown:
        raise TypeError(f"unknown dllm_step_io fields: {sorted(unknown)}")
    st = _step_ex(C.byref(model.cfg), C.byref(model.s), C.byref(cache.s), ptr(tokens), B, N,
                  C.byref(pol), int(bool(dense)), C.byref(s), ws.ptr, ws.nbytes,
                  _stream(stream))
    _check(st, "dllm_step_ex")


def dllm_step_host_workspace_size(cfg: ModelCfg, B: int, N: int, pol: Policy) -> int:
    return int(_step_host_ws(C.byref(cfg), B, N, C.byref(pol)))


def dllm_step_host(model: Model, cache: Cache, tokens_host, pol: Policy, dense: bool,
                   ws: Workspace, pos_host=None, stream=None):
    """One step whose tokens live in HOST memory (the C entry point copies them
    in, runs the step and copies tokens and revealed positions back, all on the
    stream; the host tensors hold the results after the stream synchronises).
    tokens_host [B, N] int32 and pos_host [B, capacity] int32: CPU tensors,
    preferably pinned."""
    B, N = tokens_host.shape
    _same_block(cache, pol, "dllm_step_host")
    st = _step_host(C.byref(model.cfg), C.byref(model.s), C.byref(cache.s), ptr(tokens_host), B,
                    N, C.byref(pol), int(bool(dense)), ptr(pos_host), ws.ptr, ws.nbytes,
                    _stream(stream))
    _check(st, "dllm_step_host")


class StepGraph:
    """One ``dllm_step`` captured into a CUDA graph and replayed.

    Every launch of a step depends only on device data (the index lists and
    row counts are produced on the device), so a step with fixed buffers can
    be recorded once and replayed for each later step, removing the per-launch
    host cost.  Capture once after an eager call of the same step (which sets
    the kernels' shared-memory attributes); buffers must stay at the same
    addresses for the life of the graph.
    """

    def __init__(self, model: Model, cache: Cache, tokens, pol: Policy, ws: Workspace,
                 dense: bool = False, pos_out=None):
        profile_enable(False)  # per-launch timing events cannot be read back from a graph
        self.stream = torch.cuda.Stream()
        self.graph = torch.cuda.CUDAGraph()
        self.stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(self.graph, stream=self.stream):
            dllm_step(model, cache, tokens, pol, dense, ws, pos_out=pos_out,
                      stream=self.stream)
        torch.cuda.current_stream().wait_stream(self.stream)

    def replay(self):
        self.graph.replay()


__all__ = [n for n in dir() if n.startswith(("dllm_", "DLLM_"))] + ["StepGraph",

    "kv8_cache", "Model", "Cache", "Workspace", "ModelCfg", "LayerW", "Policy", "make_cfg", "cfg_from_shape",
    "make_policy", "profile_enable", "profile_reset", "profile_read", "status_string", "version",
    "DllmError", "LIB_PATH"]
