"""Cases of the training and serving operators around Condensate attention.

Three operators: the per-head query/key norm with the position rotation and
the move into the [B, H, n, d] layout the attention reads ("norm_rope"), its
backward pass ("norm_rope_backward"), and the backward pass of the attention
over the sets C_i of the prefill ("prefill_backward").  `run` computes each
in plain torch (own = False) or through the package's entry points
(own = True) on the same state.
"""
import math

import torch

own = False  # whether run() calls the package's kernels

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def _rope(name, op, B, n, Hq, Hkv, d, dtype, rot=None, norm=True,
          interleaved=False, cache=0, far=0, base=10000.0):
    """One norm_rope case.  cache > 0: K and V rows are appended to caches of
    that many rows, at their end.  far > 0: positions are drawn up to it."""
    return {"name": name, "op": op, "B": B, "n": n, "Hq": Hq, "Hkv": Hkv,
            "d": d, "dtype": dtype, "rot": d if rot is None else rot,
            "norm": norm, "interleaved": interleaved, "cache": cache,
            "far": far, "base": base}


def _bwd(name, B, nq, L, Hq, Hkv, d, W, k, dtype, o_dtype, adaptive=False):
    """One prefill_backward case: the last nq of L positions; adaptive:
    per-query windows drawn from [64, 256]."""
    return {"name": name, "op": "prefill_backward", "B": B, "nq": nq, "L": L,
            "Hq": Hq, "Hkv": Hkv, "d": d, "W": W, "k": k, "dtype": dtype,
            "o_dtype": o_dtype, "adaptive": adaptive}


def listed():
    return [
        # one decoded token of one sequence, appended to its cache: latency
        _rope("rope_decode_1", "norm_rope", 1, 1, 32, 8, 128, "bf16",
              cache=4096, far=1 << 20, base=1e6),
        # one decoded token for each sequence of a batch
        _rope("rope_decode_48", "norm_rope", 48, 1, 32, 8, 128, "bf16",
              cache=512, far=131072, base=1e6),
        # an odd fp32 chunk with a partial, interleaved rotation
        _rope("rope_f32_odd", "norm_rope", 3, 1001, 10, 5, 64, "f32", rot=32,
              interleaved=True),
        # a training batch of the GPT-2-small shape
        _rope("rope_gpt2s_8k", "norm_rope", 4, 8192, 12, 12, 64, "bf16"),
        # the 32K Llama-shaped prefill, the largest
        _rope("rope_llama_32k", "norm_rope", 1, 32768, 32, 32, 128, "bf16",
              base=500000.0),
        # gradients of a short odd fp32 sequence
        _rope("rope_bwd_f32_odd", "norm_rope_backward", 1, 333, 6, 3, 128,
              "f32"),
        # gradients of the GPT-2-small training batch
        _rope("rope_bwd_gpt2s_8k", "norm_rope_backward", 4, 8192, 12, 12, 64,
              "bf16"),
        # gradients of a grouped-query training sequence
        _rope("rope_bwd_gqa_16k", "norm_rope_backward", 1, 16384, 32, 8, 128,
              "bf16", base=500000.0),
        # the tiny fp32 prefill: latency
        _bwd("bwd_tiny_f32", 1, 512, 512, 1, 1, 64, 64, 16, "f32", "f32"),
        # the last, odd chunk of a longer sequence, fp32 output gradients
        _bwd("bwd_chunk_odd", 2, 777, 5001, 8, 2, 64, 100, 17, "bf16", "f32"),
        # a training batch of the GPT-2-small shape
        _bwd("bwd_gpt2s_8k", 2, 8192, 8192, 12, 12, 64, 64, 32, "bf16",
             "bf16"),
        # two of the 32K prefill's heads on one kv head, per-query windows
        _bwd("bwd_adaptive_32k", 1, 32768, 32768, 2, 1, 128, 256, 64, "bf16",
             "bf16", adaptive=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo),
                                                          math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_backward", "prefill_backward",
                     "prefill_backward"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op != "prefill_backward":
        B = rng.choice([1, 1, 2, 3, 16])
        size = 4 if dtype == "f32" else 2
        row = (Hq + 2 * Hkv) * d * size
        most = min(32768, (1 << 29) // (row * B))
        n = _log(rng, 1, most)
        decode = op == "norm_rope" and n <= 4
        c = _rope("", op, B, n, Hq, Hkv, d, dtype,
                  rot=rng.choice([d, d, d // 2]),
                  norm=rng.random() < 0.8 or op != "norm_rope",
                  interleaved=rng.random() < 0.3,
                  cache=_log(rng, 8, 2048) if decode else 0,
                  far=1 << 20 if decode else 0)
    else:
        k = rng.choice([0, 8, 16, 31, 32, 64, 100])
        W = _log(rng, 8, 256)
        adaptive = rng.random() < 0.25
        if adaptive:
            W = 256
        B = rng.choice([1, 1, 2])
        most = min(32768, (1 << 29) // (B * Hq * (1 + W + k) * d))
        nq = _log(rng, 33, most)
        L = nq if rng.random() < 0.7 else nq + _log(rng, 1, 4000)
        c = _bwd("", B, nq, L, Hq, Hkv, d, W, k, dtype,
                 rng.choice(["bf16", "bf16", "f32"]) if dtype == "bf16"
                 else "f32", adaptive)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _prepare_rope(c, seed):
    g = _gen(seed)
    t = TYPES[c["dtype"]]
    B, n, Hq, Hkv, d = (c[x] for x in ("B", "n", "Hq", "Hkv", "d"))
    # the fused projection's output; q, k, v are its parts
    qkv = _normal(g, B, n, Hq + 2 * Hkv, d, dtype=t, scale=1.7)
    s = {"op": c["op"], "q": qkv[:, :, :Hq], "k": qkv[:, :, Hq:Hq + Hkv],
         "v": qkv[:, :, Hq + Hkv:], "interleaved": c["interleaved"],
         "eps": 1e-6, "Hq": Hq, "Hkv": Hkv, "qw": None, "kw": None,
         "positions": None, "cache": c["cache"]}
    if c["norm"]:
        s["qw"] = (1 + 0.2 * _normal(g, d)).to(t)
        s["kw"] = (1 + 0.2 * _normal(g, d)).to(t)
    rot = c["rot"]
    e = torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot
    s["inv_freq"] = (c["base"] ** -e).float()
    if c["far"]:
        p = torch.randint(0, c["far"] - n, (B, 1), generator=g, device=DEV)
        s["positions"] = (p + torch.arange(n, device=DEV)).to(torch.int32)
    if c["cache"]:
        Lc = c["cache"] + n
        s["Kc"] = _normal(g, B, Hkv, Lc, d, dtype=t)
        s["Vc"] = _normal(g, B, Hkv, Lc, d, dtype=t)
    if c["op"] == "norm_rope_backward":
        s["dQ"] = _normal(g, B, Hq, n, d, dtype=t, scale=0.02)
        s["dK"] = _normal(g, B, Hkv, n, d, dtype=t, scale=0.02)
        s["dV"] = _normal(g, B, Hkv, n, d, dtype=t, scale=0.02)
    return s


def _sets(Q, K, win, k, C_max):
    """The sets C_i, ascending and padded with -1, from a plain scoring."""
    B, Hq, nq, _ = Q.shape
    Hkv, L = K.shape[1], K.shape[2]
    big = 1 << 30
    idx = torch.empty(B, Hq, nq, C_max, dtype=torch.int32, device=DEV)
    pos = torch.arange(L - nq, L, device=DEV)
    j = torch.arange(L, device=DEV)
    off = torch.arange(int(win.max()), device=DEV)
    step = max(1, (1 << 28) // L)
    for b in range(B):
        for h in range(Hq):
            Kh = K[b, h // (Hq // Hkv)].float()
            for r in range(0, nq, step):
                i = pos[r:r + step, None]
                w = win[b, r:r + step, None]
                x = Q[b, h, r:r + step].float() @ Kh.T
                x.masked_fill_((j < 1) | (j > i - w), -math.inf)
                parts = [torch.where(i - w >= 0, 0, big)]
                if k > 0:
                    v, at = x.topk(min(k, L), dim=1)
                    parts.append(torch.where(v == -math.inf, big, at))
                inside = (off < w) & (off <= i)
                parts.append(torch.where(inside, i - off, big))
                row = torch.cat(parts, 1).sort(1).values[:, :C_max]
                row = torch.where(row == big, -1, row).to(torch.int32)
                idx[b, h, r:r + step, :row.shape[1]] = row
                idx[b, h, r:r + step, row.shape[1]:] = -1
    return idx


def _prepare_bwd(c, seed):
    g = _gen(seed)
    t = TYPES[c["dtype"]]
    B, nq, L, Hq, Hkv, d, W, k = (c[x] for x in ("B", "nq", "L", "Hq", "Hkv",
                                                 "d", "W", "k"))
    G = Hq // Hkv
    Q = _normal(g, B, Hq, nq, d)
    K = _normal(g, B, Hkv, L, d)
    V = _normal(g, B, Hkv, L, d, dtype=t)
    # keys that whole blocks of queries look for: eight for each block of
    # 128 queries, near three times the block's mean
    for r in range(128, nq, 128):
        hi = L - nq + r - W
        if hi > 8:
            at = torch.randint(1, hi, (8,), generator=g, device=DEV)
            m = Q[:, ::G, r:r + 128].mean(2, keepdim=True)
            K[:, :, at] = 3 * m + 0.1 * _normal(g, B, Hkv, 8, d)
    Q, K = Q.to(t), K.to(t)
    if c["adaptive"]:
        r = torch.rand(B, nq, generator=g, device=DEV)
        win = torch.floor(64 + 192 * r + 0.5).to(torch.int32)
    else:
        win = torch.full((B, nq), W, dtype=torch.int32, device=DEV)
    idx = _sets(Q, K, win, k, min(L, 1 + W + k))
    return {"op": c["op"], "Q": Q, "K": K, "V": V,
            "dO": _normal(g, B, Hq, nq, d, dtype=TYPES[c["o_dtype"]],
                          scale=0.02),
            "idx": idx, "count": (idx >= 0).sum(-1, dtype=torch.int32),
            "W": W, "k": k, "W_i": win if c["adaptive"] else None}


def prepare(case, seed):
    if case["op"] == "prefill_backward":
        return _prepare_bwd(case, seed)
    return _prepare_rope(case, seed)


# -------------------------------------------------------------- plain forms
def _cos_sin(s, n, B):
    """cos and sin [B, n, 1, rot / 2]; the angles in 64 bits."""
    p = s["positions"]
    if p is None:
        p = torch.arange(n, device=DEV)[None].expand(B, n)
    a = p[:, :, None, None].double() * s["inv_freq"].double()
    return a.cos().float(), a.sin().float()


def _rotate(y, cos, sin, interleaved):
    """The rotation of the leading 2 * cos.shape[-1] elements of each row."""
    h = cos.shape[-1]
    x, rest = y[..., :2 * h], y[..., 2 * h:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
    else:
        a, b = x[..., :h], x[..., h:]
    p, q = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        x = torch.stack([p, q], -1).flatten(-2)
    else:
        x = torch.cat([p, q], -1)
    return torch.cat([x, rest], -1)


def _plain_rope(s):
    B, n = s["q"].shape[:2]
    t = s["q"].dtype
    cos, sin = _cos_sin(s, n, B)

    def one(x, w):
        y = x.float()
        if w is not None:
            r = torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"])
            y = y * r * w.float()
        y = _rotate(y, cos, sin, s["interleaved"])
        return y.transpose(1, 2).contiguous().to(t)

    Q, K = one(s["q"], s["qw"]), one(s["k"], s["kw"])
    V = s["v"].transpose(1, 2).contiguous()
    if s["cache"]:
        s["Kc"][:, :, -n:] = K
        s["Vc"][:, :, -n:] = V
        return Q, s["Kc"], s["Vc"]
    return Q, K, V


def _plain_rope_backward(s):
    B, n = s["q"].shape[:2]
    t = s["q"].dtype
    cos, sin = _cos_sin(s, n, B)

    def one(x, w, dy):
        # the rotation's transpose is the rotation by the negative angle
        gy = _rotate(dy.transpose(1, 2).float(), cos, -sin, s["interleaved"])
        if w is None:
            return gy.to(t), None
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
        xh = x * r
        gw = (gy * xh).sum((0, 1, 2))
        gx = gy * w.float()
        gx = r * (gx - xh * (gx * xh).mean(-1, keepdim=True))
        return gx.to(t), gw.to(w.dtype)

    dq, dqw = one(s["q"], s["qw"], s["dQ"])
    dk, dkw = one(s["k"], s["kw"], s["dK"])
    dv = s["dV"].transpose(1, 2)
    return torch.cat([dq, dk, dv], 2), dqw, dkw


def _plain_backward(s):
    """Gathers the rows of every set, recomputes the probabilities, and adds
    the keys' gradients up by index."""
    Q, K, V, dO, idx = (s[x] for x in ("Q", "K", "V", "dO", "idx"))
    B, Hq, nq, d = Q.shape
    Hkv, L = K.shape[1], K.shape[2]
    C = idx.shape[-1]
    scale = 1 / math.sqrt(d)
    live = idx >= 0
    bh = torch.arange(B * Hq, device=DEV)
    base = (bh // Hq * Hkv + bh % Hq // (Hq // Hkv)) * L
    flat = (idx.clamp(min=0) + base.view(B, Hq, 1, 1)).view(-1)
    q, g = (x.float().reshape(-1, 1, d) for x in (Q, dO))
    rows = K.float().view(-1, d)[flat].view(-1, C, d)
    x = (rows @ q.transpose(1, 2)).squeeze(-1) * scale
    x = x.masked_fill(~live.view(-1, C), -math.inf)
    p = torch.exp(x - x.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    vals = V.float().view(-1, d)[flat].view(-1, C, d)
    dp = (vals @ g.transpose(1, 2)).squeeze(-1)
    del vals
    ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
    dQ = (ds[:, None] @ rows).view(B, Hq, nq, d)
    del rows
    dK = torch.zeros(B * Hkv * L, d, device=DEV)
    dK.index_add_(0, flat, (ds[..., None] * q).view(-1, d))
    dV = torch.zeros(B * Hkv * L, d, device=DEV)
    dV.index_add_(0, flat, (p[..., None] * g).view(-1, d))
    t = Q.dtype
    return dQ.to(t), dK.view(K.shape).to(t), dV.view(V.shape).to(t)


# ----------------------------------------------------------------- one pass
def run(s):
    if own:
        import sparse_transformer_attention_b200 as ca
        if s["op"] == "prefill_backward":
            return ca.condensate_attn_prefill_backward(
                s["Q"], s["K"], s["V"], s["dO"], s["idx"], s["count"],
                s["W"], s["k"], W_i=s["W_i"])
        rope = dict(q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"],
                    positions=s["positions"], interleaved=s["interleaved"])
        if s["op"] == "norm_rope":
            if not s["cache"]:
                return ca.condensate_attn_norm_rope(
                    s["q"], s["k"], s["v"], s["inv_freq"], **rope)
            n = s["q"].shape[1]
            Q, _, _ = ca.condensate_attn_norm_rope(
                s["q"], s["k"], s["v"], s["inv_freq"],
                K=s["Kc"][:, :, -n:], V=s["Vc"][:, :, -n:], **rope)
            return Q, s["Kc"], s["Vc"]
        Hq, Hkv = s["Hq"], s["Hkv"]
        B, n, _, d = s["q"].shape
        dqkv = torch.empty(B, n, Hq + 2 * Hkv, d, dtype=s["q"].dtype,
                           device=DEV)
        _, _, _, dqw, dkw = ca.condensate_attn_norm_rope_backward(
            s["dQ"], s["dK"], s["dV"], s["q"], s["k"], s["inv_freq"],
            dq=dqkv[:, :, :Hq], dk=dqkv[:, :, Hq:Hq + Hkv],
            dv=dqkv[:, :, Hq + Hkv:], **rope)
        return dqkv, dqw, dkw
    if s["op"] == "norm_rope":
        return _plain_rope(s)
    if s["op"] == "norm_rope_backward":
        return _plain_rope_backward(s)
    return _plain_backward(s)


# ------------------------------------------------------------------- floors
def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    d, B, Hq, Hkv = c["d"], c["B"], c["Hq"], c["Hkv"]
    if c["op"] == "prefill_backward":
        nq, L, k = c["nq"], c["L"], c["k"]
        W = 160 if c["adaptive"] else c["W"]
        o = 4 if c["o_dtype"] == "f32" else 2
        # |C_i| = min(i + 1, 1 + W + k); the Top-k part, min(k, i - W) when
        # positive, is what has to be read of the index rows
        i0, m = L - nq, 1 + W + k
        short = min(nq, max(0, m - i0))
        size_sum = short * (2 * i0 + short + 1) // 2 + (nq - short) * m
        listed_sum = sum(min(k, max(0, i - W)) for i in range(i0, L))
        rows = B * Hq * nq
        return {"bytes": 2 * (rows + 2 * B * Hkv * L) * d * size
                + rows * d * o + B * Hq * 4 * (listed_sum + nq),
                "flops": 10 * d * B * Hq * size_sum}
    n = c["n"]
    elems = B * n * (Hq + 2 * Hkv) * d
    reads = elems
    if c["op"] == "norm_rope_backward" and c["norm"]:
        reads += B * n * (Hq + Hkv) * d
    # a norm (4) and a rotation (6 for each pair) for each element of q and k
    ops = 10 if c["op"] == "norm_rope" else 20
    return {"bytes": (elems + reads) * size,
            "flops": ops * B * n * (Hq + Hkv) * d}


# ------------------------------------------------------------ 64-bit values
def _exact_angles(s, B, n):
    p = s["positions"].double() if s["positions"] is not None else \
        torch.arange(n, device=DEV, dtype=torch.float64).repeat(B, 1)
    return torch.einsum("bn,f->bnf", p, s["inv_freq"].double())[:, None]


def _as_complex(x, h, interleaved):
    """The rotated part of x [B, H, n, d] as complex numbers."""
    x = x[..., :2 * h]
    x = x.unflatten(-1, (h, 2)) if interleaved else \
        x.unflatten(-1, (2, h)).transpose(-1, -2)
    return torch.view_as_complex(x.contiguous())


def _turned(x, turn, interleaved):
    """x with its leading pairs multiplied by the unit numbers `turn`."""
    h = turn.shape[-1]
    z = torch.view_as_real(_as_complex(x, h, interleaved) * turn)
    z = z if interleaved else z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), x[..., 2 * h:]], -1)


def _exact_rope(s):
    B, n = s["q"].shape[:2]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       _exact_angles(s, B, n))

    def one(x, w):
        x = x.double().permute(0, 2, 1, 3)
        if w is not None:
            norm = x.square().sum(-1, keepdim=True) / x.shape[-1] + s["eps"]
            x = x / norm.sqrt() * w.double()
        return _turned(x, turn, s["interleaved"])

    Q, K = one(s["q"], s["qw"]), one(s["k"], s["kw"])
    V = s["v"].double().permute(0, 2, 1, 3)
    if s["cache"]:
        keep = slice(0, s["Kc"].shape[2] - n)
        K = torch.cat([s["Kc"][:, :, keep].double(), K], 2)
        V = torch.cat([s["Vc"][:, :, keep].double(), V], 2)
    return Q, K, V


def _exact_rope_backward(s):
    B, n = s["q"].shape[:2]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       -_exact_angles(s, B, n))

    def one(x, w, dy):
        g = _turned(dy.double(), turn, s["interleaved"])
        if w is None:
            return g, None
        x = x.double().permute(0, 2, 1, 3)
        d = x.shape[-1]
        a = x.square().sum(-1, keepdim=True) / d + s["eps"]
        gw = torch.einsum("bhnc,bhnc->c", g, x / a.sqrt())
        u = g * w.double()
        # y = x a^(-1/2):  dx = u a^(-1/2) - x (u . x) a^(-3/2) / d
        dot = (u * x).sum(-1, keepdim=True)
        return u / a.sqrt() - x * dot / (a * a.sqrt() * d), gw

    dq, dqw = one(s["q"], s["qw"], s["dQ"])
    dk, dkw = one(s["k"], s["kw"], s["dK"])
    return torch.cat([dq, dk, s["dV"].double()], 1).permute(0, 2, 1, 3), \
        dqw, dkw


def _exact_backward(s):
    """Dense rows with everything outside the sets masked, head by head."""
    Q, K, V, dO, idx = (s[x] for x in ("Q", "K", "V", "dO", "idx"))
    B, Hq, nq, d = Q.shape
    Hkv, L = K.shape[1], K.shape[2]
    out = [torch.zeros(x.shape, dtype=torch.float64, device=DEV)
           for x in (Q, K, V)]
    step = max(1, (1 << 27) // L)
    for b in range(B):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            Kd, Vd = K[b, g].double(), V[b, g].double()
            for r in range(0, nq, step):
                at = slice(r, r + step)
                Qd, Gd = Q[b, h, at].double(), dO[b, h, at].double()
                member = torch.zeros(Qd.shape[0], L + 1, dtype=torch.bool,
                                     device=DEV)
                ix = idx[b, h, at].long()
                member.scatter_(1, torch.where(ix < 0, L, ix), True)
                S = (Qd @ Kd.T / d ** 0.5).masked_fill(~member[:, :L],
                                                       -math.inf)
                P = torch.softmax(S, 1)
                O = P @ Vd
                dS = P * (Gd @ Vd.T - (Gd * O).sum(1, keepdim=True)) / d ** 0.5
                out[0][b, h, at] = dS @ Kd
                out[1][b, g] += dS.T @ Qd
                out[2][b, g] += P.T @ Gd
    return tuple(out)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm_rope":
        return _exact_rope(s)
    if s["op"] == "norm_rope_backward":
        return _exact_rope_backward(s)
    return _exact_backward(s)
