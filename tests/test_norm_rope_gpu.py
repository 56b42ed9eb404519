"""Per-head norm with position rotation, and its backward pass, against the
plain 64-bit form (tests/block_plain.py holds the bounds)."""
import pytest
import torch

import block_plain as plain
import sparse_transformer_attention_b200 as ca

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(B, n, Hq, Hkv, d, dtype, rot, norm=True, w_dtype=None, seed=0,
         far=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (1.5 * rnd(B, n, Hq + 2 * Hkv, d)).to(dtype)
    w = [(1 + 0.3 * rnd(d)).to(w_dtype or dtype) if norm else None
         for _ in range(2)]
    inv = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda").double() /
                       max(rot, 1))).float() if rot else None
    pos = None
    if far:
        pos = torch.randint(far - 1000, far, (B, n), generator=g,
                            device="cuda").to(torch.int32)
    return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], inv, w, pos


def ang_of(q, inv, pos, pos0=0):
    B, n = q.shape[:2]
    if pos is None:
        pos = torch.arange(pos0, pos0 + n, device="cuda").repeat(B, 1)
    if inv is None:
        inv = torch.empty(0, device="cuda")
    return plain.angles(pos, inv)


CASES = [
    # B, n, Hq, Hkv, d, dtype, rot, interleaved, norm, far
    (1, 1, 1, 1, 64, BF, 64, False, True, None),
    (1, 1, 32, 8, 128, BF, 128, False, True, 1 << 20),
    (5, 1, 6, 3, 128, F32, 128, True, True, 131072),
    (2, 3, 5, 5, 64, BF, 16, True, True, None),
    (3, 97, 7, 1, 64, F32, 32, False, True, None),
    (1, 700, 12, 12, 64, BF, 64, False, True, None),
    (2, 333, 8, 2, 128, BF, 96, False, True, (1 << 31) - 1),
    (1, 130, 3, 3, 128, F32, 48, False, False, None),
    (2, 50, 9, 3, 64, BF, 0, False, True, None),
    (1, 41, 4, 2, 128, BF, 128, True, False, None),
    (1, 5000, 2, 1, 64, BF, 64, False, True, None),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(
    str(x).replace("torch.", "") for x in c))
def test_forward_and_backward(case):
    B, n, Hq, Hkv, d, dtype, rot, il, norm, far = case
    q, k, v, inv, (qw, kw), pos = make(B, n, Hq, Hkv, d, dtype, rot, norm,
                                       far=far)
    a = dict(q_weight=qw, k_weight=kw, eps=1e-5, positions=pos,
             interleaved=il)
    Q, K, V = ca.condensate_attn_norm_rope(q, k, v, inv, **a)
    ang = ang_of(q, inv, pos)
    for x, w, y, nm in ((q, qw, Q, "Q"), (k, kw, K, "K")):
        plain.check(y, *plain.norm_rope(x, w, 1e-5, ang, il), nm)
    assert torch.equal(V, v.transpose(1, 2))

    g = torch.Generator(device="cuda").manual_seed(9)
    dQ, dK, dV = (torch.randn(y.shape, generator=g, device="cuda").to(dtype)
                  for y in (Q, K, V))
    fused = torch.full((B, n, Hq + 2 * Hkv, d), float("nan"), dtype=dtype,
                       device="cuda")
    parts = dict(dq=fused[:, :, :Hq], dk=fused[:, :, Hq:Hq + Hkv],
                 dv=fused[:, :, Hq + Hkv:])
    *_, dqw, dkw = ca.condensate_attn_norm_rope_backward(dQ, dK, dV, q, k,
                                                         inv, **a, **parts)
    for x, w, dy, dx, dw, H, nm in (
            (q, qw, dQ, parts["dq"], dqw, Hq, "q"),
            (k, kw, dK, parts["dk"], dkw, Hkv, "k")):
        # a lane adds the rows of at most this many tokens' heads in one run
        chain = (B * n // (592 * 8) + 1) * H
        ex, bx, ew, bw = plain.norm_rope_backward(dy, x, w, 1e-5, ang, il,
                                                  chain)
        plain.check(dx, ex, bx, "d" + nm)
        assert (dw is None) == (w is None)
        if w is not None:
            plain.check(dw, ew, bw, "dw of " + nm)
    assert torch.equal(parts["dv"], dV.transpose(1, 2))


def test_cache_rows_only():
    """K and V go to rows of a longer cache; the others stay as they were."""
    q, k, v, inv, (qw, kw), _ = make(3, 4, 8, 2, 64, BF, 64)
    Kc = torch.full((3, 2, 50, 64), -7.0, dtype=BF, device="cuda")
    Vc = Kc.clone()
    a = dict(q_weight=qw, k_weight=kw, pos0=20)
    Q, K, V = ca.condensate_attn_norm_rope(q, k, v, inv, K=Kc[:, :, 20:24],
                                           V=Vc[:, :, 20:24], **a)
    Q2, K2, V2 = ca.condensate_attn_norm_rope(q, k, v, inv, **a)
    assert torch.equal(Q, Q2)
    for c, y in ((Kc, K2), (Vc, V2)):
        assert torch.equal(c[:, :, 20:24], y)
        assert (c[:, :, :20] == -7).all() and (c[:, :, 24:] == -7).all()


def test_in_place_and_parts_left_out():
    q, k, v, inv, (qw, kw), _ = make(2, 33, 4, 2, 128, BF, 128)
    Q, K, V = ca.condensate_attn_norm_rope(q, k, v, inv, qw, kw)
    q2 = q.clone()
    ca.condensate_attn_norm_rope(q2, None, None, inv, qw,
                                 Q=q2.transpose(1, 2))
    assert torch.equal(q2.transpose(1, 2), Q)
    Q3, K3, V3 = ca.condensate_attn_norm_rope(q, k, None, inv, qw, kw)
    assert V3 is None and torch.equal(Q3, Q) and torch.equal(K3, K)


def test_broadcast_input_rows():
    """Rows read through zero strides, and their gradients row by row."""
    q, k, v, inv, (qw, kw), _ = make(1, 20, 4, 2, 64, F32, 64)
    qe = q[:, :1].expand(3, 20, 4, 64)
    ke, ve = k.expand(3, 20, 2, 64), v.expand(3, 20, 2, 64)
    Q, K, V = ca.condensate_attn_norm_rope(qe, ke, ve, inv, qw, kw)
    ang = ang_of(qe, inv, None)
    plain.check(Q, *plain.norm_rope(qe, qw, 1e-6, ang, False), "Q")
    plain.check(K, *plain.norm_rope(ke, kw, 1e-6, ang, False), "K")
    base = q[:, :1].clone().requires_grad_()
    Qg, _, _ = ca.norm_rope(base.expand(3, 20, 4, 64), ke, ve, inv, qw, kw)
    Qg.sum().backward()
    dx, bx, _, _ = plain.norm_rope_backward(
        torch.ones_like(Q), qe, qw, 1e-6, ang, False, 8)
    # the 60 row gradients are added by autograd in fp32
    add = 60 * plain.U * dx.abs().sum((0, 1), keepdim=True)
    plain.check(base.grad, dx.sum((0, 1), keepdim=True),
                bx.sum((0, 1), keepdim=True) + add, "broadcast")


def test_weight_types_and_zero_rows():
    """bf16 rows with fp32 weights; a row of zeros is finite (eps)."""
    q, k, v, inv, (qw, kw), _ = make(1, 9, 2, 2, 128, BF, 64, w_dtype=F32)
    q[:, 3] = 0
    Q, _, _ = ca.condensate_attn_norm_rope(q, k, v, inv, qw, kw)
    assert (Q[:, :, 3] == 0).all()
    ang = ang_of(q, inv, None)
    plain.check(Q, *plain.norm_rope(q, qw, 1e-6, ang, False), "Q")
    dy = torch.ones_like(Q)
    dq, _, _, dqw, _ = ca.condensate_attn_norm_rope_backward(
        dy, None, None, q, None, inv, qw)
    assert dqw.dtype == F32
    dx, bx, dw, bw = plain.norm_rope_backward(dy, q, qw, 1e-6, ang, False, 2)
    plain.check(dq, dx, bx, "dq")
    plain.check(dqw, dw, bw, "dqw")


def test_only_one_norm_and_one_weight_gradient():
    q, k, v, inv, (qw, kw), _ = make(2, 40, 4, 2, 64, BF, 64)
    kw = kw.clone().requires_grad_()
    Q, K, V = ca.norm_rope(q, k, v, inv, None, kw)
    ang = ang_of(q, inv, None)
    plain.check(Q, *plain.norm_rope(q, None, 1e-6, ang, False), "Q")
    K.float().sum().backward()
    _, _, dw, bw = plain.norm_rope_backward(torch.ones_like(K), k,
                                            kw.detach(), 1e-6, ang, False, 4)
    plain.check(kw.grad, dw, bw, "dkw")


def test_gradients_against_differences():
    """The kernel's gradients along a direction against central differences
    of the 64-bit form: step h = 2^-10 of values near one leaves h^2 / 6 of a
    third derivative, under 1e-5 of the sums' magnitudes here."""
    B, n, Hq, Hkv, d = 1, 17, 2, 1, 64
    q, k, v, inv, (qw, kw), _ = make(B, n, Hq, Hkv, d, F32, 64)
    ang = ang_of(q, inv, None)
    gen = torch.Generator(device="cuda").manual_seed(3)
    dQ = torch.randn(B, Hq, n, d, generator=gen, device="cuda")
    dq, _, _, dqw, _ = ca.condensate_attn_norm_rope_backward(
        dQ, None, None, q, None, inv, qw)

    def loss(x, w):
        return (plain.norm_rope(x, w, 1e-6, ang, False)[0] * dQ.double()).sum()

    h = 2.0 ** -10
    for x, grad, f in ((q, dq, lambda t: loss(t, qw)),
                       (qw, dqw, lambda t: loss(q, t))):
        u = torch.randn(x.shape, generator=gen, device="cuda").double()
        num = (f(x.double() + h * u) - f(x.double() - h * u)) / (2 * h)
        ana = (grad.double() * u).sum()
        assert abs(num - ana) <= 1e-5 * (grad.double() * u).abs().sum()


def test_offsets_beyond_32_bits():
    """180,000 tokens of 96 heads x 128: the last tokens lie behind element
    2^31 of the projection."""
    n, Hq, Hkv, d = 180_000, 32, 32, 128
    x = torch.empty(1, n, Hq + 2 * Hkv, d, dtype=BF, device="cuda").normal_()
    w = torch.ones(d, dtype=BF, device="cuda")
    inv = 10000.0 ** (-torch.arange(0, d, 2, device="cuda") / d)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    Q, K, V = ca.condensate_attn_norm_rope(q, k, v, inv, w, w)
    dq, dk, dv, _, _ = ca.condensate_attn_norm_rope_backward(
        Q, K, V, q, k, inv, w, w)
    at = slice(n - 40, n)
    pos = torch.arange(n - 40, n, device="cuda").view(1, 40)
    ang = plain.angles(pos, inv)
    for a, A, da in ((q, Q, dq), (k, K, dk)):
        plain.check(A[:, :, at], *plain.norm_rope(a[:, at], w, 1e-6, ang,
                                                  False))
        dx, bx, _, _ = plain.norm_rope_backward(A[:, :, at], a[:, at], w,
                                                1e-6, ang, False, 1)
        plain.check(da[:, at], dx, bx)
    assert torch.equal(V[:, :, at], v[:, at].transpose(1, 2))
    assert torch.equal(dv[:, at], v[:, at])


def test_equal_bits_streams_and_graphs():
    """The same call twice, on a side stream, and captured and replayed with
    new inputs in the same buffers."""
    q, k, v, inv, (qw, kw), _ = make(2, 900, 6, 2, 64, BF, 64)
    dQ = torch.randn(2, 6, 900, 64, device="cuda").to(BF)
    dK, dV = (torch.randn(2, 2, 900, 64, device="cuda").to(BF)
              for _ in range(2))

    def both(stream=None):
        return (*ca.condensate_attn_norm_rope(q, k, v, inv, qw, kw,
                                              stream=stream),
                *ca.condensate_attn_norm_rope_backward(
                    dQ, dK, dV, q, k, inv, qw, kw, stream=stream))

    want = both()
    for got in (both(), both()):
        assert all(torch.equal(x, y) for x, y in zip(want, got))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    keep = q.clone()
    q.copy_(torch.randn_like(q))
    graph.replay()
    for x, y in zip(both(), held):
        assert torch.equal(x, y)
    q.copy_(keep)
    graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(want, held))


def test_refusals():
    q, k, v, inv, (qw, kw), _ = make(2, 8, 4, 2, 64, BF, 64)
    f = ca.condensate_attn_norm_rope
    with pytest.raises(ValueError):
        f(q, k[:, :, :, :32], v, inv)                 # another d
    with pytest.raises(TypeError):
        f(q, k.float(), v, inv)                       # another type
    with pytest.raises(ValueError):
        f(q.transpose(2, 3), k, v, inv)               # d not innermost
    with pytest.raises(TypeError):
        f(q, k, v, inv.double())
    with pytest.raises(TypeError):
        f(q, k, v, inv, qw, kw.float())               # weights differ
    with pytest.raises(ValueError):
        f(q, k, v, inv, qw.cpu())
    with pytest.raises(ca.CondensateError):           # rot not 16 | rot
        f(q, k, v, inv[:12])
    with pytest.raises(ca.CondensateError):           # rot > d
        f(q, k, v, inv.repeat(2))
    with pytest.raises(ca.CondensateError):           # folded output rows
        f(q, k, v, inv, K=torch.empty(2, 1, 8, 64, dtype=BF, device="cuda")
          .expand(2, 2, 8, 64))
    with pytest.raises(ca.CondensateError):           # rows off 16 bytes
        base = torch.empty(2 * 8 * 4 * 64 + 8, dtype=BF, device="cuda")
        f(base[1:1 + 2 * 8 * 4 * 64].view(2, 8, 4, 64), None, None, inv)
    with pytest.raises(ValueError):
        ca.condensate_attn_norm_rope_backward(
            torch.empty(2, 4, 8, 64, dtype=BF, device="cuda"), None, None,
            None, None, inv, qw)                      # q missing
    with pytest.raises(ca.CondensateError):           # workspace too small
        ca.condensate_attn_norm_rope_backward(
            torch.zeros(2, 4, 8, 64, dtype=BF, device="cuda"), None, None, q,
            None, inv, qw,
            workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
