"""Cases, plain forms and exact values of the 8-bit K/V cache operators.

Four operators that a step over an 8-bit cache uses one after the other:

qk_norm  per-head RMS norm of queries and keys and their position rotation
write    selected K/V rows into the e4m3 cache (one power-of-two scale per
         sequence, kv head and block of tokens)
read     rows of the cache back to bf16
attn     attention of compact query rows over the cache

Rows are packed by sequence as everywhere in the library: sequence b holds
count[b] rows, at positions idx[b, 0 .. count[b]) in ascending order (rows
behind the last sequence are left as they were).
"""
import math

import torch

own = False  # True: run() calls the library; False: the plain form

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -100
EPS = 1e-5
THETA = 5.0e5


# ------------------------------------------------------------------ cases

def _case(op, B, k, N, Hq, Hkv, hd, block=64, dtype="bf16", dense=False, ragged=True, name=None):
    c = dict(op=op, B=B, k=k, N=N, Hq=Hq, Hkv=Hkv, hd=hd, block=block, dtype=dtype, dense=dense,
             ragged=ragged)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token for each of 8 sequences, grouped heads (28 query, 4 kv): the latency of a call
        _case("qk_norm", 8, 1, 2048, 28, 4, 128, ragged=False, name="norm 7B one row"),
        # the rows that a 20 % step recomputes for 32 sequences
        _case("qk_norm", 32, 308, 1536, 32, 32, 128, name="norm 8B r20"),
        # an fp32 model (exact-arithmetic checks), odd sizes
        _case("qk_norm", 3, 333, 1000, 6, 2, 64, dtype="f32", name="norm f32 odd"),
        # one new token per sequence into a cache that holds the others
        _case("write", 8, 1, 2048, 28, 4, 128, ragged=False, name="write 7B one row"),
        # a 20 % step's rows, scattered over every block of the cache
        _case("write", 32, 308, 1536, 32, 32, 128, name="write 8B r20"),
        # a dense step or refresh: every row of every sequence
        _case("write", 32, 1536, 1536, 32, 32, 128, dense=True, ragged=False, name="write 8B dense"),
        # the rows whose K/V a step is about to change, before it does (short blocks)
        _case("read", 8, 103, 2048, 28, 4, 128, block=32, name="read 7B r5"),
        # a whole layer's cache back to bf16
        _case("read", 32, 1536, 1536, 32, 32, 128, dense=True, ragged=False, name="read 8B all"),
        # one query row per sequence over a long cache, lengths of their own
        _case("attn", 8, 1, 16384, 28, 4, 128, name="attn 7B one row long"),
        # one sequence's 10 % step
        _case("attn", 1, 77, 768, 32, 32, 128, ragged=False, name="attn 8B B1 r10"),
        # the 20 % step of 32 sequences
        _case("attn", 32, 308, 1536, 32, 32, 128, ragged=False, name="attn 8B r20"),
        # head_dim 64, short blocks, odd lengths, one of them zero
        _case("attn", 3, 45, 1013, 12, 4, 64, block=16, name="attn hd64 odd"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_norm", "write", "read", "attn"])
    hd = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 32])
    G = rng.choice([1, 1, 4, 7, 8]) if Hkv <= 8 else 1
    # bf16 model widths are multiples of 128
    if (Hkv * hd) % 128:
        Hkv *= 2
    B = _log(rng, 1, 32)
    N = _log(rng, 33, 16384)
    k = _log(rng, 1, min(N, 2048))
    block = rng.choice([16, 32, 64, 128])
    dtype = "f32" if op == "qk_norm" and rng.random() < 0.25 else "bf16"
    dense = op in ("write", "read") and rng.random() < 0.3
    while True:  # no larger than the largest listed case of the operator
        rows = B * (N if dense else k)
        if op == "attn":
            big = max(B * Hkv * G * k * N / 4.8e8, B * N * Hkv * hd / 2.0e8)
        elif op == "qk_norm":
            big = max(rows * Hkv * (G + 1) * hd * (2 if dtype == "f32" else 1) / 8.0e7,
                      B * N * hd / 1.0e8)
        else:
            big = max(rows * Hkv * hd / 2.0e8, B * N * Hkv * hd / 2.0e8)
        if big <= 1.0:
            break
        if B > 1:
            B = max(1, B // 2)
        elif k > 64 and not dense:
            k //= 2
        else:
            N = max(33, N // 2)
            k = min(k, N)
    if dense:
        k = N
    return _case(op, B, k, N, Hkv * G, Hkv, hd, block, dtype, dense, not dense and rng.random() < 0.7)


# ------------------------------------------------------------------ inputs

def _rows(case, gen):
    """(idx [B, k], count [B], count as a list): ascending positions; a ragged case has other
    counts per sequence (the last of several has none where there is more than one row)."""
    B, k, N = case["B"], case["k"], case["N"]
    if case["ragged"] and k > 1:
        u = torch.rand(B, generator=torch.Generator().manual_seed(gen.initial_seed() & 0xFFFFFF))
        counts = [max(0, k - int(float(x) * k * 0.3)) for x in u]
        if B > 2:
            counts[-1] = 0
    else:
        counts = [k] * B
    pick = torch.rand(B, N, generator=gen, device="cuda").argsort(1)[:, :k]
    idx = torch.full((B, k), -1, dtype=torch.int32, device="cuda")
    for b, c in enumerate(counts):
        idx[b, :c] = pick[b, :c].sort().values.to(torch.int32)
    return idx, torch.tensor(counts, dtype=torch.int32, device="cuda"), counts


def _normal(shape, gen, dtype):
    """Activations: N(0, 1) with a few channels of the last axis several times larger."""
    x = torch.randn(shape, generator=gen, device="cuda")
    ch = 1.0 + 7.0 * (torch.rand(shape[-1], generator=gen, device="cuda") < 0.05)
    return (x * ch).to(dtype)


def _new_cache(case, gen):
    """An 8-bit cache that holds N rows per sequence: codes of N(0, 1) rows at each block's own scale."""
    B, N, H, hd, blk = (case[x] for x in ("B", "N", "Hkv", "hd", "block"))
    nb = -(-N // blk)
    s = torch.exp2(torch.randint(-7, -3, (B, H, nb), generator=gen, device="cuda").float())
    x = torch.randn((B, N, H, hd), generator=gen, device="cuda")
    x = x / s.repeat_interleave(blk, 2)[:, :, :N].permute(0, 2, 1)[..., None]
    return x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    B, k, N, Hq, Hkv, hd = (case[x] for x in ("B", "k", "N", "Hq", "Hkv", "hd"))
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    st = {"case": case}
    if case["dense"]:
        st["idx"] = st["count"] = None
    else:
        st["idx"], st["count"], counts = _rows(case, gen)
    R = B * k
    if case["op"] == "qk_norm":
        st["q"] = _normal((R, Hq * hd), gen, dt)
        st["k"] = _normal((R, Hkv * hd), gen, dt)
        st["q_gain"] = (1 + 0.1 * torch.randn(hd, generator=gen, device="cuda")).to(dt)
        st["k_gain"] = (1 + 0.1 * torch.randn(hd, generator=gen, device="cuda")).to(dt)
        inv = THETA ** (-2.0 * torch.arange(hd // 2, device="cuda", dtype=torch.float64) / hd)
        ang = torch.arange(N, device="cuda", dtype=torch.float64)[:, None] * inv
        st["rope"] = torch.stack([ang.cos(), ang.sin()], -1).float()
        st["q_out"] = torch.zeros_like(st["q"])
        st["k_out"] = torch.zeros_like(st["k"])
        return st
    st["k8"], st["ks"] = _new_cache(case, gen)
    st["v8"], st["vs"] = _new_cache(case, gen)
    if case["op"] == "write":
        st["k"] = _normal((R, Hkv * hd), gen, dt)
        st["v"] = _normal((R, Hkv * hd), gen, dt)
    elif case["op"] == "read":
        st["k_out"] = torch.zeros(R, Hkv * hd, dtype=dt, device="cuda")
        st["v_out"] = torch.zeros(R, Hkv * hd, dtype=dt, device="cuda")
    else:
        st["q"] = _normal((R, Hq * hd), gen, dt)
        st["o"] = torch.zeros_like(st["q"])
        lens = [N] * B
        if case["ragged"]:
            u = torch.rand(B, generator=torch.Generator().manual_seed(int(seed) + 3))
            lens = [N - int(float(x) * N * 0.3) for x in u]
            if B > 2:
                lens[0] = 0
        st["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms

def _places(st):
    """For the padded rows [B, k]: which exist, their compact row (R for the others), their position."""
    c = st["case"]
    B, k = c["B"], c["k"]
    j = torch.arange(k, device="cuda")
    if st["count"] is None:
        there = torch.ones(B, k, dtype=torch.bool, device="cuda")
        return there, torch.arange(B * k, device="cuda").view(B, k), j.expand(B, k)
    n = st["count"].long()
    there = j < n[:, None]
    row = torch.where(there, (n.cumsum(0) - n)[:, None] + j, B * k)
    return there, row, torch.where(there, st["idx"].long(), 0)


def _padded(x, row):
    """Compact rows [R, w] as [B, k, w] in 32 bits (what does not exist: the last row, unused)."""
    return x[row.clamp(max=x.shape[0] - 1)].float()


def _put(out, row, there, y):
    """Compact rows of `out` <- the padded y where they exist."""
    R = out.shape[0]
    buf = torch.cat([out, out[:1]])
    buf[row.reshape(-1)] = y.reshape(-1, out.shape[1]).to(out.dtype)
    out.copy_(buf[:R])
    return out


def _plain_norm(st):
    c = st["case"]
    there, row, pos = _places(st)
    cs = st["rope"][pos]
    outs = []
    for x, g, out in ((st["q"], st["q_gain"], st["q_out"]), (st["k"], st["k_gain"], st["k_out"])):
        y = _padded(x, row).unflatten(-1, (-1, c["hd"]))
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * g.float()
        a, b = y.chunk(2, -1)
        co, si = cs[..., None, :, 0], cs[..., None, :, 1]
        outs.append(_put(out, row, there, torch.cat([a * co - b * si, b * co + a * si], -1)))
    return outs


def _pow2_scale(a):
    """Smallest power of two s >= 2^-100 with a <= 448 s."""
    m, e = torch.frexp(a)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(a > 0, torch.ldexp(torch.ones_like(a), e), 0.0).clamp(min=MIN_SCALE)


def _plain_write(st):
    c = st["case"]
    B, N, H, hd, blk = (c[x] for x in ("B", "N", "Hkv", "hd", "block"))
    nb = -(-N // blk)
    there, row, pos = _places(st)
    new = torch.zeros(B, nb * blk + 1, dtype=torch.bool, device="cuda")
    at = torch.where(there, pos, nb * blk)
    new.scatter_(1, at, True)
    new = new[:, :nb * blk].view(B, nb, blk)
    tokens = (N - torch.arange(nb, device="cuda") * blk).clamp(max=blk)
    n_new = new.sum(-1)
    whole, some = (n_new == tokens)[:, None], (n_new > 0)[:, None]
    per_tok = lambda s: s.repeat_interleave(blk, 2)[:, :, :N].transpose(1, 2)[..., None]
    kept = ~new.view(B, -1)[:, :N, None, None]
    for x, c8, sc in ((st["k"], st["k8"], st["ks"]), (st["v"], st["v8"], st["vs"])):
        full = torch.zeros(B, nb * blk + 1, H * hd, device="cuda")
        full.scatter_(1, at[..., None].expand(-1, -1, H * hd), _padded(x, row))
        full = full[:, :nb * blk]
        a = torch.where(full.isfinite() & new.view(B, -1, 1), full.abs(), 0.0)
        a = a.view(B, nb, blk, H, hd).amax((2, 4)).transpose(1, 2)
        s = torch.where(some & (whole | (a > E4M3_MAX * sc)), _pow2_scale(a), sc)
        y = full[:, :N].view(B, N, H, hd) / per_tok(s)
        del full
        y = torch.where(y.isfinite(), y, math.nan)
        old = c8.float() * torch.where(per_tok(s) > 0, per_tok(sc) / per_tok(s), 1.0)
        c8.copy_(torch.where(kept, old, y).to(torch.float8_e4m3fn))
        sc.copy_(s)
    return [st["k8"], st["ks"], st["v8"], st["vs"]]


def _decoded(c8, sc, blk):
    N = c8.shape[1]
    return c8.float() * sc.repeat_interleave(blk, 2)[:, :, :N].transpose(1, 2)[..., None]


def _plain_read(st):
    c = st["case"]
    there, row, pos = _places(st)
    outs = []
    for c8, sc, out in ((st["k8"], st["ks"], st["k_out"]), (st["v8"], st["vs"], st["v_out"])):
        x = _decoded(c8, sc, c["block"]).flatten(2)
        x = x.gather(1, pos[..., None].expand(-1, -1, x.shape[2]))
        outs.append(_put(out, row, there, x))
    return outs


def _plain_attn(st):
    c = st["case"]
    B, N, Hq, Hkv, hd = (c[x] for x in ("B", "N", "Hq", "Hkv", "hd"))
    there, row, _ = _places(st)
    q = _padded(st["q"], row).view(B, -1, Hkv, Hq // Hkv, hd).permute(0, 2, 3, 1, 4)
    live = torch.arange(N, device="cuda") < st["len"][:, None]
    K = _decoded(st["k8"], st["ks"], c["block"]).permute(0, 2, 3, 1)
    V = _decoded(st["v8"], st["vs"], c["block"]).permute(0, 2, 1, 3)
    V = torch.where(live[:, None, :, None], V, 0.0)
    s = q.flatten(2, 3) @ K / math.sqrt(hd)
    s = s.masked_fill_(~live[:, None, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m.isfinite(), m, 0.0)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.where(l > 0, (p @ V) / l, 0.0)
    o = o.view(B, Hkv, Hq // Hkv, -1, hd).permute(0, 3, 1, 2, 4).flatten(2)
    return [_put(st["o"], row, there, o)]


# ------------------------------------------------------------------ the framework's calls

def _own(st):
    import sparse_token_recompute_b200 as S
    c = st["case"]
    op = c["op"]
    if op == "qk_norm":
        S.dllm_qk_norm_rope(st["q"], st["k"], st["q_gain"], st["k_gain"], st["rope"], st["q_out"],
                            st["k_out"], st["idx"], st["count"], EPS)
        return [st["q_out"], st["k_out"]]
    if op == "write":
        S.dllm_kv8_write(st["k"], st["v"], st["idx"], st["count"], st["k8"], st["ks"], st["v8"],
                         st["vs"], c["block"])
        return [st["k8"], st["ks"], st["v8"], st["vs"]]
    if op == "read":
        S.dllm_kv8_read(st["k8"], st["ks"], st["v8"], st["vs"], st["idx"], st["count"],
                        st["k_out"], st["v_out"], c["block"])
        return [st["k_out"], st["v_out"]]
    # a program keeps its workspace from call to call
    st["ws"] = S.dllm_attention_kv8(st["q"], st["k8"], st["ks"], st["v8"], st["vs"], st["o"],
                                    st["count"], c["k"], c["block"], kv_len=st["len"],
                                    ws=st.get("ws"))
    return [st["o"]]


def run(st):
    if own:
        return _own(st)
    return {"qk_norm": _plain_norm, "write": _plain_write, "read": _plain_read,
            "attn": _plain_attn}[st["case"]["op"]](st)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    rows, es = c["B"] * c["k"] * (0.85 if c["ragged"] and c["k"] > 1 else 1.0), 4 if c["dtype"] == "f32" else 2
    kv = c["Hkv"] * c["hd"]
    if c["op"] == "qk_norm":
        n = rows * (c["Hq"] + c["Hkv"]) * c["hd"]
        return {"bytes": 2 * n * es + rows * (c["hd"] * 4 + 4), "flops": 8 * n}
    blocks = c["B"] * c["Hkv"] * -(-c["N"] // c["block"])
    if c["op"] in ("write", "read"):
        return {"bytes": rows * (kv * 2 * 3 + 4) + 2 * 4 * min(blocks, rows * c["Hkv"]),
                "flops": rows * kv * 2 * 2}
    keys = c["B"] * c["N"] * (0.85 if c["ragged"] else 1.0)
    return {"bytes": keys * kv * 2 + blocks * 8 + 2 * rows * c["Hq"] * c["hd"] * 2,
            "flops": 4.0 * rows * (keys / c["B"]) * c["Hq"] * c["hd"]}


# ------------------------------------------------------------------ exact values

def _e4m3_64(y):
    """y (64 bits, |y| <= 448) rounded to e4m3: 4 significant bits, none finer than 2^-9, ties to even."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -60)))
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return torch.round(y / step) * step


def _list_rows(st):
    """[(sequence, compact row range, positions)] from the host's view of the row lists."""
    c = st["case"]
    if st["count"] is None:
        return [(b, slice(b * c["k"], (b + 1) * c["k"]), torch.arange(c["k"], device="cuda"))
                for b in range(c["B"])]
    got, at = [], 0
    for b, n in enumerate(st["count"].tolist()):
        got.append((b, slice(at, at + n), st["idx"][b, :n].long()))
        at += n
    return got


def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    op, hd, blk = case["op"], case["hd"], case["block"]
    lists = _list_rows(st)
    if op == "qk_norm":
        outs = []
        for x, g in ((st["q"], st["q_gain"]), (st["k"], st["k_gain"])):
            z = torch.zeros(x.shape, dtype=f64, device="cuda")
            for _, rows, pos in lists:
                w = torch.view_as_complex(st["rope"][pos].to(f64))[:, None, :]
                y = x[rows].to(f64).view(len(pos), x.shape[1] // hd, hd)
                y = y * (y.square().sum(-1, keepdim=True) / hd + EPS).rsqrt() * g.to(f64)
                r = torch.complex(y[..., :hd // 2], y[..., hd // 2:]) * w
                z[rows] = torch.cat([r.real, r.imag], -1).flatten(1)
            outs.append(z)
        return outs
    if op == "write":
        outs = []
        for x, c8, sc in ((st["k"], st["k8"], st["ks"]), (st["v"], st["v8"], st["vs"])):
            code, scale = c8.to(f64), sc.to(f64)
            N = code.shape[1]
            nb = scale.shape[2]
            for b, rows, pos in lists:
                if not len(pos):
                    continue
                y = x[rows].to(f64).view(len(pos), -1, hd)
                which = pos // blk
                a = torch.zeros(nb, y.shape[1], dtype=f64, device="cuda")
                a.scatter_reduce_(0, which[:, None].expand(-1, y.shape[1]), y.abs().amax(-1), "amax")
                n = torch.bincount(which, minlength=nb)
                size = torch.tensor([min(blk, N - i * blk) for i in range(nb)], device="cuda")
                fresh = torch.exp2(torch.ceil(torch.log2(a / E4M3_MAX))).clamp(min=MIN_SCALE)
                s0 = scale[b].T.clone()
                change = (n > 0)[:, None] & ((n == size)[:, None] | (a > E4M3_MAX * s0))
                s1 = torch.where(change, fresh, s0)
                tok = torch.arange(N, device="cuda") // blk
                code[b] = _e4m3_64(code[b] * (s0 / s1)[tok][..., None])
                code[b, pos] = _e4m3_64(y / s1[which][..., None])
                scale[b] = s1.T
            outs += [code, scale]
        return outs
    if op == "read":
        outs = []
        for c8, sc in ((st["k8"], st["ks"]), (st["v8"], st["vs"])):
            z = torch.zeros(case["B"] * case["k"], case["Hkv"] * hd, dtype=f64, device="cuda")
            for b, rows, pos in lists:
                z[rows] = (c8[b][pos].to(f64) * sc[b].T[pos // blk][..., None].to(f64)).flatten(1)
            outs.append(z)
        return outs
    z = torch.zeros(st["q"].shape, dtype=f64, device="cuda")
    G = case["Hq"] // case["Hkv"]
    for (b, rows, pos), n in zip(lists, st["len"].tolist()):
        if not len(pos) or not n:
            continue
        tok = torch.arange(n, device="cuda") // blk
        K = st["k8"][b, :n].to(f64) * st["ks"][b].T[tok][..., None].to(f64)
        V = st["v8"][b, :n].to(f64) * st["vs"][b].T[tok][..., None].to(f64)
        q = st["q"][rows].to(f64).view(len(pos), case["Hkv"], G, hd)
        p = torch.softmax(torch.einsum("rhgd,nhd->rhgn", q, K) * hd ** -0.5, -1)
        z[rows] = torch.einsum("rhgn,nhd->rhgd", p, V).flatten(1)
    return [z]
