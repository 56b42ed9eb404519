"""Backward pass of the prefill against the plain 64-bit form over the same
sets (tests/block_plain.py holds the bounds)."""
import pytest
import torch

import block_plain as plain
import sparse_transformer_attention_b200 as ca

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(B, nq, L, Hq, Hkv, d, dtype, o_dtype, seed=0, popular=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    Q, K, V = rnd(B, Hq, nq, d), rnd(B, Hkv, L, d), rnd(B, Hkv, L, d)
    if popular:  # keys that every row selects
        Q += 1.0
        at = torch.randperm(max(1, L - nq // 2 - 1), generator=g,
                            device="cuda")[:popular] + 1
        K[:, :, at.clamp(max=L - 1)] += 2.0
    dO = rnd(B, Hq, nq, d)
    return ((scale * Q).to(dtype), K.to(dtype), V.to(dtype), dO.to(o_dtype))


def run(Q, K, V, dO, W, k, W_i=None, W_h=None, k_h=None):
    """(sets, gradients) through the forward and the backward entry point,
    with a clean status word behind the backward."""
    _, idx, cnt = ca.condensate_attn_prefill(Q, K, V, W, k, W_i=W_i, W_h=W_h,
                                             k_h=k_h, o_dtype=dO.dtype)
    B, Hq, nq, d = Q.shape
    ws = torch.empty(ca.condensate_attn_prefill_backward_workspace_size(
        Q.dtype, dO.dtype, B, nq, K.shape[2], Hq, K.shape[1], d, k),
        dtype=torch.uint8, device="cuda").fill_(0xFF)
    outs = [torch.full_like(x, float("nan")) for x in (Q, K, V)]
    got = ca.condensate_attn_prefill_backward(
        Q, K, V, dO, idx, cnt, W, k, W_i=W_i, W_h=W_h, dQ=outs[0],
        dK=outs[1], dV=outs[2], workspace=ws)
    assert ca.condensate_attn_status(ws) == ca.CA_OK
    return idx, cnt, got


def check(Q, K, V, dO, idx, got):
    want = plain.attention_backward(Q, K, V, dO, idx)
    for x, (y, b), nm in zip(got, want, ("dQ", "dK", "dV")):
        assert torch.isfinite(x).all(), nm
        plain.check(x, y, b, nm)


CASES = [
    # B, nq, L, Hq, Hkv, d, W, k, dtype, o_dtype
    (1, 1, 1, 1, 1, 64, 1, 0, F32, F32),
    (1, 1, 1, 1, 1, 128, 64, 16, BF, BF),
    (1, 2, 2, 2, 1, 64, 1, 1, BF, F32),
    (1, 1, 500, 8, 1, 128, 16, 8, BF, BF),
    (2, 65, 65, 2, 2, 64, 1, 0, BF, BF),
    (1, 130, 130, 2, 1, 64, 1, 5, F32, F32),
    (1, 97, 97, 4, 4, 128, 200, 16, BF, BF),
    (1, 81, 81, 1, 1, 64, 64, 16, BF, BF),
    (1, 300, 300, 8, 1, 64, 33, 31, BF, BF),
    (3, 129, 129, 6, 3, 128, 16, 128, BF, F32),
    (1, 512, 512, 1, 1, 64, 64, 16, F32, F32),
    (2, 200, 777, 4, 1, 64, 50, 33, BF, BF),
    (1, 333, 1001, 2, 2, 128, 100, 64, F32, F32),
    (1, 700, 700, 4, 2, 64, 64, 32, BF, BF),
    (1, 257, 900, 2, 1, 128, 256, 100, BF, BF),
    (1, 64, 70000, 2, 1, 64, 64, 32, BF, BF),
    (1, 300, 70000, 2, 1, 64, 64, 32, BF, BF),   # three sort passes
    (1, 250, 300, 2, 1, 64, 20, 17, F32, BF),
]
IDS = lambda c: "-".join(str(x).replace("torch.", "") for x in c)  # noqa: E731


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_against_formula(case):
    B, nq, L, Hq, Hkv, d, W, k, dt, odt = case
    x = make(B, nq, L, Hq, Hkv, d, dt, odt)
    idx, _, got = run(*x, W, k)
    check(*x, idx, got)


@pytest.mark.parametrize("dt,d,G,popular,k", [
    (BF, 64, 2, 16, 16), (BF, 128, 8, 3, 32), (F32, 64, 1, 8, 8),
    (BF, 64, 1, 70, 32)])
def test_keys_that_every_row_selects(dt, d, G, popular, k):
    """A few keys (and the anchor) with lists as long as the sequence: many
    ranges each, next to keys with none."""
    x = make(1, 600, 600, 2 * G, 2, d, dt, dt, popular=popular, scale=0.5)
    idx, _, got = run(*x, 32, k)
    check(*x, idx, got)


@pytest.mark.parametrize("dt,d", [(BF, 64), (BF, 128), (F32, 64)])
def test_windows_of_each_query(dt, d):
    """W_i from 1 to beyond the sequence, one row's window far larger than
    its neighbours'."""
    x = make(2, 300, 400, 4, 2, d, dt, dt)
    g = torch.Generator(device="cuda").manual_seed(1)
    W_i = torch.randint(1, 90, (2, 300), generator=g, device="cuda",
                        dtype=torch.int32)
    W_i[0, 250] = 390
    W_i[1, 299] = 5000
    W_i[1, 17] = 1
    idx, _, got = run(*x, 1, 20, W_i=W_i)
    check(*x, idx, got)


@pytest.mark.parametrize("dt", [BF, F32])
def test_windows_and_sizes_of_each_head(dt):
    x = make(1, 260, 300, 4, 2, 64, dt, dt)
    W_h = torch.tensor([1, 64, 17, 400], dtype=torch.int32, device="cuda")
    k_h = torch.tensor([24, 0, 7, 24], dtype=torch.int32, device="cuda")
    idx, _, got = run(*x, 1, 24, W_h=W_h, k_h=k_h)
    check(*x, idx, got)


@pytest.mark.parametrize("dt,odt,d", [
    (BF, BF, 64), (BF, BF, 128), (BF, F32, 64), (BF, F32, 128),
    (F32, F32, 64), (F32, F32, 128)])
@pytest.mark.parametrize("L,per_query", [(270, False), (270, True),
                                         (1100, False), (1100, True)])
def test_many_heads(dt, odt, d, L, per_query):
    """42 heads of keys: more tiles and entries than an SM's share, where
    other tests have too few for all SMs; keys that every row selects; keys
    before any window."""
    x = make(3, 260, L, 28, 14, d, dt, odt, popular=3, scale=0.5)
    W_i = None
    if per_query:
        g = torch.Generator(device="cuda").manual_seed(3)
        W_i = torch.randint(1, 80, (3, 260), generator=g, device="cuda",
                            dtype=torch.int32)
    idx, _, got = run(*x, 40, 64, W_i=W_i)
    check(*x, idx, got)


@pytest.mark.parametrize("dt", [BF, F32])
def test_peaked_scores(dt):
    """Scores up to the hundreds: probabilities of nearly one and of zero."""
    x = make(1, 200, 200, 2, 1, 64, dt, dt, scale=16.0)
    idx, _, got = run(*x, 16, 16)
    check(*x, idx, got)


def test_keys_nobody_attends_to():
    """With k = 0 and a chunk at the end, early keys but the anchor get
    zeros, written over whatever was there."""
    x = make(1, 100, 1000, 2, 2, 64, BF, BF)
    idx, _, got = run(*x, 30, 0)
    check(*x, idx, got)
    assert (got[1][:, :, 1:871] == 0).all() and (got[2][:, :, 1:871] == 0).all()


def test_equal_bits_streams_and_graphs():
    Q, K, V, dO = make(1, 500, 500, 4, 2, 64, BF, BF, popular=20, scale=0.5)
    W, k = 40, 24
    idx, cnt, want = run(Q, K, V, dO, W, k)
    f = ca.condensate_attn_prefill_backward
    for _ in range(3):
        got = f(Q, K, V, dO, idx, cnt, W, k)
        assert all(torch.equal(x, y) for x, y in zip(want, got))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = f(Q, K, V, dO, idx, cnt, W, k, stream=side)
    got2 = f(Q, K, V, dO, idx, cnt, W, k)  # at the same time, own workspace
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert all(torch.equal(x, y) for x, y in zip(want, got2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = f(Q, K, V, dO, idx, cnt, W, k)
    keep = dO.clone()
    dO.copy_(torch.randn_like(dO))
    graph.replay()
    for x, y in zip(f(Q, K, V, dO, idx, cnt, W, k), held):
        assert torch.equal(x, y)
    dO.copy_(keep)
    graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(want, held))


def test_bad_sets_are_reported():
    """Positions outside a row's candidates and counts that do not fit are
    skipped and reported; the call stays inside its buffers."""
    Q, K, V, dO = make(1, 200, 200, 2, 1, 64, BF, BF)
    W, k = 20, 8
    idx, cnt, want = run(Q, K, V, dO, W, k)
    ws = torch.empty(ca.condensate_attn_prefill_backward_workspace_size(
        BF, BF, 1, 200, 200, 2, 1, 64, k), dtype=torch.uint8, device="cuda")

    def status(i, c):
        got = ca.condensate_attn_prefill_backward(Q, K, V, dO, i, c, W, k,
                                                  workspace=ws)
        assert all(torch.isfinite(x).all() for x in got)
        return ca.condensate_attn_status(ws)

    assert status(idx, cnt) == ca.CA_OK
    for value in (-1, 0, 195, 1 << 30, -(1 << 31)):
        bad = idx.clone()
        bad[0, 1, 199, 3] = value
        assert status(bad, cnt) == 7  # CA_ERR_DEVICE_ARG
    for value in (-5, 0, 12, 500, (1 << 31) - 1):
        bad = cnt.clone()
        bad[0, 0, 150] = value
        assert status(idx, bad) == 7
    assert status(idx, cnt) == ca.CA_OK


def test_gradients_against_differences():
    """Kernel gradients along a direction against central differences of the
    64-bit forward over the same sets (h = 2^-12; the third derivative of a
    softmax of scores of order one leaves far under 1e-4 of the magnitudes)."""
    Q, K, V, dO = make(1, 90, 120, 4, 2, 64, F32, F32)
    idx, _, got = run(Q, K, V, dO, 16, 8)
    gen = torch.Generator(device="cuda").manual_seed(5)
    h = 2.0 ** -12
    x = [t.double() for t in (Q, K, V)]
    for n in range(3):
        u = torch.randn(x[n].shape, generator=gen, device="cuda").double()
        f = []
        for s in (h, -h):
            y = list(x)
            y[n] = x[n] + s * u
            f.append((plain.attention(*y, idx) * dO.double()).sum())
        num = (f[0] - f[1]) / (2 * h)
        prod = got[n].double() * u
        assert abs(num - prod.sum()) <= 1e-4 * prod.abs().sum()


def test_autograd_attention_is_the_two_entry_points():
    Q, K, V, dO = make(2, 150, 150, 4, 2, 64, BF, F32)
    W_i = torch.randint(1, 60, (2, 150), device="cuda", dtype=torch.int32)
    leaves = [t.clone().requires_grad_() for t in (Q, K, V)]
    O, idx, cnt = ca.attention(*leaves, 60, 12, W_i=W_i)
    O2, idx2, cnt2 = ca.condensate_attn_prefill(Q, K, V, 60, 12, W_i=W_i)
    assert torch.equal(O, O2) and torch.equal(idx, idx2)
    O.backward(dO)
    want = ca.condensate_attn_prefill_backward(Q, K, V, dO, idx2, cnt2, 60,
                                               12, W_i=W_i)
    assert all(torch.equal(t.grad, y) for t, y in zip(leaves, want))
    for t in leaves:
        t.grad = None
    O, _, _ = ca.attention(*leaves, 60, 12, W_i=W_i)
    O.sum().backward()  # an expanded gradient
    want = ca.condensate_attn_prefill_backward(
        Q, K, V, torch.ones_like(O), idx2, cnt2, 60, 12, W_i=W_i)
    assert all(torch.equal(t.grad, y) for t, y in zip(leaves, want))


@pytest.mark.parametrize("il,norm", [(False, True), (True, False)])
def test_layer_from_fused_projection(il, norm):
    """qkv_attention, fp32, whole chain against 64-bit autograd over the same
    sets.  Each stage is held to its own bounds above; together they stay
    within 2^-13 of the gradients' norms (score errors of some 100 U times
    scores of order ten)."""
    B, n, Hq, Hkv, d, W, k = 2, 120, 4, 2, 64, 16, 12
    g = torch.Generator(device="cuda").manual_seed(2)
    qkv = torch.randn(B, n, (Hq + 2 * Hkv) * d, generator=g, device="cuda")
    inv = 10000.0 ** (-torch.arange(0, d, 2, device="cuda") / d)
    w = [1 + 0.2 * torch.randn(d, generator=g, device="cuda")
         for _ in range(2)] if norm else [None, None]
    leaves = [t.clone().requires_grad_() for t in (qkv, *w) if t is not None]
    G = torch.randn(B, Hq, n, d, generator=g, device="cuda")
    O = ca.qkv_attention(leaves[0], Hq, Hkv, W, k, inv, *(leaves[1:] or w),
                         interleaved=il)
    O.backward(G)

    x = qkv.view(B, n, Hq + 2 * Hkv, d)
    q, kk, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    Q, K, V = ca.condensate_attn_norm_rope(q, kk, v, inv, *w, interleaved=il)
    _, idx, _ = ca.condensate_attn_prefill(Q, K, V, W, k)
    dl = [t.detach().double().requires_grad_() for t in leaves]
    ang = plain.angles(torch.arange(n, device="cuda").repeat(B, 1), inv)
    xd = dl[0].view(B, n, Hq + 2 * Hkv, d)
    wd = dl[1:] or [None, None]

    def one(t, wt):
        if wt is not None:
            t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * wt
        f = ang.shape[-1]
        c, s = ang.cos()[:, :, None], ang.sin()[:, :, None]
        a, b = (t[..., 0::2], t[..., 1::2]) if il else (t[..., :f], t[..., f:])
        y, z = a * c - b * s, b * c + a * s
        t = torch.stack([y, z], -1).flatten(-2) if il else torch.cat([y, z], -1)
        return t.transpose(1, 2)

    Od = plain.attention(one(xd[:, :, :Hq], wd[0]),
                         one(xd[:, :, Hq:Hq + Hkv], wd[1]),
                         xd[:, :, Hq + Hkv:].transpose(1, 2), idx)
    Od.backward(G.double())
    assert (O - Od).norm() <= 2.0 ** -13 * Od.norm()
    for t, y in zip(leaves, dl):
        assert (t.grad - y.grad).norm() <= 2.0 ** -13 * y.grad.norm()


def test_decode_from_projection_rows():
    """One token at a time: its K and V rows appended to the cache, then the
    decode that reads it, against the prefill's last row."""
    B, L, Hq, Hkv, d, W, k = 2, 300, 8, 2, 64, 32, 16
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(B, L, Hq + 2 * Hkv, d, generator=g, device="cuda").to(BF)
    parts = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    inv = 10000.0 ** (-torch.arange(0, d, 2, device="cuda") / d)
    Q, K, V = ca.condensate_attn_norm_rope(*parts, inv)
    Kc, Vc = K.clone(), V.clone()
    Kc[:, :, -1], Vc[:, :, -1] = 0, 0
    last = [t[:, -1:] for t in parts]
    q, _, _ = ca.condensate_attn_norm_rope(
        *last, inv, pos0=L - 1, K=Kc[:, :, -1:], V=Vc[:, :, -1:])
    assert torch.equal(Kc, K) and torch.equal(Vc, V)
    assert torch.equal(q, Q[:, :, -1:])
    o, idx, cnt = ca.condensate_attn_decode(q[:, :, 0].contiguous(), Kc, Vc,
                                            W, k)
    O, idx2, cnt2 = ca.condensate_attn_prefill(Q[:, :, -1:].contiguous(), K,
                                               V, W, k)
    assert torch.equal(idx, idx2[:, :, 0]) and torch.equal(cnt, cnt2[:, :, 0])
    assert (o - O[:, :, 0]).abs().max() <= 1e-2


def test_offsets_beyond_32_bits():
    """8 kv heads x 2.1 M keys x 128: the last head's rows lie behind element
    2^31.  The sets are made here; the last head is compared whole, at the
    keys that its rows list and see."""
    H, L, nq, d, W, k = 8, 2_100_000, 16, 128, 16, 8
    g = torch.Generator(device="cuda").manual_seed(6)
    K, V = (torch.empty(1, H, L, d, dtype=BF, device="cuda").normal_(
        generator=g) for _ in range(2))
    Q, dO = (torch.randn(1, H, nq, d, generator=g, device="cuda").to(BF)
             for _ in range(2))
    far = torch.randint(1, L - nq - W, (1, H, nq, k), generator=g,
                        device="cuda")
    far[..., 0] = L - nq - W - 1  # every row's
    far = far.sort(-1).values
    i = torch.arange(L - nq, L, device="cuda").view(1, 1, nq, 1)
    win = (i - W + 1 + torch.arange(W, device="cuda")).expand(1, H, nq, W)
    idx = torch.cat([torch.zeros_like(far[..., :1]), far, win],
                    -1).to(torch.int32).contiguous()
    cnt = torch.full((1, H, nq), 1 + k + W, dtype=torch.int32, device="cuda")
    dQ, dK, dV = ca.condensate_attn_prefill_backward(Q, K, V, dO, idx, cnt, W,
                                                     k)
    # the listed and seen keys of the last head, and the sets over them
    keys = torch.unique(idx[0, -1].long())
    at = torch.searchsorted(keys, idx[:, -1:].long())
    part = lambda t: t[:, -1:, keys].contiguous()  # noqa: E731
    last = lambda t: t[:, -1:]  # noqa: E731
    want = plain.attention_backward(last(Q), part(K), part(V), last(dO), at)
    got = last(dQ), part(dK), part(dV)
    for x, (y, b), nm in zip(got, want, ("dQ", "dK", "dV")):
        plain.check(x, y, b, nm)
    other = torch.ones(L, dtype=torch.bool, device="cuda")
    other[keys] = False
    assert not dK[0, -1][other].any() and not dV[0, -1][other].any()


@pytest.mark.parametrize("dt,d,nq,W,k,heads", [
    (BF, 64, 700, 64, 32, 2), (BF, 128, 300, 40, 64, 2),
    (F32, 64, 300, 20, 16, 2), (BF, 64, 260, 40, 64, 42)])
def test_debug_build(dt, d, nq, W, k, heads):
    """The index-checking build: no check fires, and equal bits."""
    from sparse_transformer_attention_b200 import binding, build
    x = make(1, nq, nq, 2 * heads, heads, d, dt, dt, popular=8, scale=0.5)
    idx, cnt, want = run(*x, W, k)
    prev = binding.use_library(build.build(debug=True))
    try:
        assert binding.load().condensate_attn_build_flags() == 1
        idx2, cnt2, got = run(*x, W, k)  # asserts a clean status word
    finally:
        binding.use_library(prev)
    assert torch.equal(idx, idx2) and torch.equal(cnt, cnt2)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dt,odt,d", [
    (BF, BF, 64), (BF, F32, 64), (BF, BF, 128), (F32, F32, 64)])
@pytest.mark.parametrize("nq,L,heads", [(200, 777, 1), (300, 300, 1),
                                        (260, 270, 42)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite_where_others_attend(dt, odt, d, nq, L, heads, value):
    """A key (a row) that is not finite reaches the gradients of the rows that
    attend to it (the keys that it attends to) and no others: those keep their
    bits, next to it in the same tile as anywhere."""
    W, k = 40, 16
    Q, K, V, dO = make(1, nq, L, 2 * heads, heads, d, dt, odt)
    idx, cnt, base = run(Q, K, V, dO, W, k)

    def grads(q, kk, v, g):
        return ca.condensate_attn_prefill_backward(q, kk, v, g, idx, cnt, W, k)

    def same(x, y, attended, what):
        assert torch.equal(x[~attended], y[~attended]), what
        assert not torch.isfinite(x[attended]).all(-1).any(), what

    p0 = L - nq
    for j in (1, p0 + 100, p0 + 104, L - 2):
        attended = (idx == j).any(-1)  # [1, Hq, nq]
        attended[:, 2:] = False        # the other kv heads' keys stay
        for n in (1, 2):
            x = [Q, K, V, dO]
            x[n] = x[n].clone()
            x[n][0, 0, j] = value
            got = grads(*x)
            # dQ of another row of the head may only stay; rows that attend
            # to an infinite key with a score of -inf may stay, too
            if n == 1 and value == float("inf"):
                assert torch.equal(got[0][~attended], base[0][~attended]), j
            else:
                same(got[0], base[0], attended, ("dQ", n, j))
    for i in (0, 100, nq - 1):
        keys = torch.zeros(L + 1, dtype=torch.bool, device="cuda")
        at = idx[0, 0, i].long()
        keys[torch.where(at < 0, L, at)] = True
        attended = torch.zeros(1, heads, L, dtype=torch.bool, device="cuda")
        attended[0, 0] = keys[:L]
        for n in (0, 3):
            x = [Q, K, V, dO]
            x[n] = x[n].clone()
            x[n][0, 0, i] = value
            got = grads(*x)
            rows = torch.ones(2 * heads, nq, dtype=torch.bool, device="cuda")
            rows[0, i] = False
            assert torch.equal(got[0][0][rows], base[0][0][rows]), (n, i)
            for y in (1, 2):
                assert torch.equal(got[y][~attended], base[y][~attended]), \
                    (n, i, y)
            if n == 3:
                same(got[2], base[2], attended, ("dV", n, i))
            if value != value:
                same(got[1], base[1], attended, ("dK", n, i))


def test_refusals():
    Q, K, V, dO = make(1, 64, 64, 2, 1, 64, BF, BF)
    _, idx, cnt = ca.condensate_attn_prefill(Q, K, V, 16, 4)
    f = ca.condensate_attn_prefill_backward
    with pytest.raises(ValueError):
        f(Q, K[:, :, :32], V, dO, idx, cnt, 16, 4)
    with pytest.raises(ValueError):
        f(Q.transpose(1, 2), K, V, dO, idx, cnt, 16, 4)
    with pytest.raises(TypeError):
        f(Q, K.float(), V, dO, idx, cnt, 16, 4)
    with pytest.raises(TypeError):
        f(Q, K, V, dO, idx.long(), cnt, 16, 4)
    with pytest.raises(TypeError):
        f(Q, K, V, dO.half(), idx, cnt, 16, 4)
    with pytest.raises(ValueError):
        f(Q, K, V, dO, idx, cnt, 16, 4,
          W_i=torch.ones(1, 63, dtype=torch.int32, device="cuda"))
    with pytest.raises(ca.CondensateError):   # C_max below 1 + W + k
        f(Q, K, V, dO, idx, cnt, 20, 4)
    with pytest.raises(ca.CondensateError):   # window below 1
        f(Q, K, V, dO, idx, cnt, 0, 4)
    with pytest.raises(ca.CondensateError):   # k above the prefill's
        f(Q, K, V, dO, idx, cnt, 16, 129)
    with pytest.raises(ca.CondensateError):   # workspace too small
        f(Q, K, V, dO, idx, cnt, 16, 4,
          workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
