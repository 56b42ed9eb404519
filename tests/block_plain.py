"""Plain 64-bit forms of the operators around the attention, and bounds on
what fp32 arithmetic may add to their results (elementwise, from the
magnitudes of what is summed).  Half a step of the output's type comes on
top: finfo(t).eps / 2 of the value."""
import math

import torch

U = 2.0 ** -24  # fp32 unit roundoff


def half_step(t):
    return torch.finfo(t).eps / 2


def angles(positions, inv_freq):
    return positions.double()[:, :, None] * inv_freq.double()  # [B, n, f]


def rotate(x, ang, interleaved, sign=1.0):
    """x [B, n, H, d] float64, the leading 2 f elements turned by ang."""
    f = ang.shape[-1]
    c, s = ang.cos()[:, :, None], sign * ang.sin()[:, :, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * f:2], x[..., 1:2 * f:2]
        y[..., 0:2 * f:2], y[..., 1:2 * f:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :f], x[..., f:2 * f]
        y[..., :f], y[..., f:2 * f] = a * c - b * s, b * c + a * s
    return y


def pair_mag(x, f, interleaved):
    """|a| + |b| at both places of each pair, |x| at the others."""
    y = x.abs()
    z = y.clone()
    if interleaved:
        t = y[..., 0:2 * f:2] + y[..., 1:2 * f:2]
        z[..., 0:2 * f:2], z[..., 1:2 * f:2] = t, t
    else:
        t = y[..., :f] + y[..., f:2 * f]
        z[..., :f], z[..., f:2 * f] = t, t
    return z


def norm_rope(x, w, eps, ang, interleaved):
    """(y [B, H, n, d], bound).  The bound: a sum of d <= 128 squares by lane
    and shuffle tree (14 U, half of it after the root), mean, eps and rsqrt
    (6 U), two products (2 U); cos and sin from a rounded argument |x| <= pi
    (4 U) with 2 ulp (4 U); product and fma (2 U): under 32 U of |a| + |b|."""
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    y = rotate(x, ang, interleaved)
    bound = 32 * U * pair_mag(x, ang.shape[-1], interleaved)
    return y.transpose(1, 2), bound.transpose(1, 2)


def norm_rope_backward(dy, x, w, eps, ang, interleaved, chain):
    """(dx, bound, dw, bound): dy [B, H, n, d], dx token-major.  g errs by
    less than 12 U of its pair's magnitudes; mean(w g xh) adds its own sum of
    d terms (14 U) and the error of r (10 U, once in xh and once outside), so
    each of the two terms of dx is within 64 U of its magnitudes; a weight's
    gradient adds up rows in runs of at most `chain` and then trees of 5 + 8
    + 19 + 5 more."""
    g = rotate(dy.transpose(1, 2).double(), ang, interleaved, -1.0)
    mag = pair_mag(dy.transpose(1, 2).double(), ang.shape[-1], interleaved)
    if w is None:
        return g, 12 * U * mag, None, None
    x, w = x.double(), w.double()
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    xh = x * r
    dx = r * (w * g - xh * (w * g * xh).mean(-1, keepdim=True))
    wm = w.abs() * mag
    bx = 64 * U * r * (wm + xh.abs() * (wm * xh.abs()).mean(-1, keepdim=True))
    dw = (g * xh).sum((0, 1, 2))
    bw = (64 + chain + 37) * U * (mag * xh.abs()).sum((0, 1, 2))
    return dx, bx, dw, bw


def member_mask(idx, L):
    ix = idx.long()
    m = torch.zeros(*ix.shape[:-1], L + 1, dtype=torch.bool, device=idx.device)
    m.scatter_(-1, torch.where(ix < 0, L, ix), True)
    return m[..., :L]


def attention(Q, K, V, idx):
    """O [B, Hq, nq, d] float64 over the listed sets."""
    G = Q.shape[1] // K.shape[1]
    Kd, Vd = (x.double().repeat_interleave(G, 1) for x in (K, V))
    S = Q.double() @ Kd.transpose(-1, -2) / math.sqrt(Q.shape[-1])
    S = S.masked_fill(~member_mask(idx, K.shape[2]), -math.inf)
    return torch.softmax(S, -1) @ Vd


def attention_backward(Q, K, V, dO, idx):
    """((dQ, bound), (dK, bound), (dV, bound)).

    Rounding, to first order, with C the largest set: a score errs by
    (d + 4) 2 U sum|q k| / sqrt(d) + 4 U |s| (2 U: tensor-core sums may
    truncate); p by twice the row's largest such error and (4 C + 64) U for
    the exponentials, the running maximum's rescales and the sum; dP by
    (d + 4) 2 U sum|dO v|; D by the sum of its terms' errors.  dS is taken as
    e dP - D e, so its terms count with |dP| + |D|.  bf16 operands of a
    matrix product hold p and dS in two parts (2^-16 relative), and so do the
    terms of p's normaliser (2^-16 more); an fp32 dO beside bf16 inputs as
    well (2^-16 in dP; in dV its lo part meets p's hi part only, 2^-16 more).  The sums over rows or keys add (their length + 8)
    2 U of their magnitudes."""
    d, L = Q.shape[-1], K.shape[2]
    B, Hkv = K.shape[:2]
    G = Q.shape[1] // Hkv
    rep = lambda x: x.double().repeat_interleave(G, 1)  # noqa: E731
    Qd, Gd, Kd, Vd = Q.double(), dO.double(), rep(K), rep(V)
    T = lambda x: x.transpose(-1, -2)  # noqa: E731
    sc = 1 / math.sqrt(d)
    m = member_mask(idx, L)
    S = Qd @ T(Kd) * sc
    eS = (2 * (d + 4) * U * (Qd.abs() @ T(Kd.abs())) * sc + 4 * U * S.abs())
    eS = (eS * m).amax(-1, keepdim=True)
    P = torch.softmax(S.masked_fill(~m, -math.inf), -1)
    dP = Gd @ T(Vd)
    D = (P * dP).sum(-1, keepdim=True)
    dS = P * (dP - D) * sc
    C = idx.shape[-1]
    split = 2.0 ** -15 if Q.dtype == torch.bfloat16 else 0.0
    planes = split / 2 if dO.dtype == torch.float32 else 0.0
    rp = 2 * eS + (4 * C + 64) * U + split
    edP = (2 * (d + 4) * U + planes) * (Gd.abs() @ T(Vd.abs()))
    eD = (P * (edP + rp * dP.abs())).sum(-1, keepdim=True)
    edS = sc * P * (rp * (dP.abs() + D.abs()) + edP + eD)
    mag = sc * P * (dP.abs() + D.abs())
    group = lambda x: x.unflatten(1, (Hkv, G)).sum(2)  # noqa: E731
    dQ = dS @ Kd
    bQ = (edS + 2 * (C + 8) * U * mag) @ Kd.abs()
    n = m.sum(-2).unflatten(1, (Hkv, G)).sum(2)[..., None]  # rows of a key
    dK, dV = group(T(dS) @ Qd), group(T(P) @ Gd)
    bK = group(T(edS) @ Qd.abs()) + 2 * (n + 8) * U * group(T(mag) @ Qd.abs())
    bV = group(T((rp + 2 * planes) * P) @ Gd.abs()) + 2 * (n + 8) * U * \
        group(T(P) @ Gd.abs())
    return (dQ, bQ), (dK, bK), (dV, bV)


def check(got, want, bound, what=""):
    """|got - want| <= bound + half a step of got's type, elementwise."""
    err = (got.double() - want).abs()
    # second-order terms: the bounds are first-order, take 1 + 2^-6 of them
    tol = 1.015625 * bound + half_step(got.dtype) * (want.abs() + bound)
    bad = ~(err <= tol)
    assert not bad.any(), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst ratio "
        f"{float((err / tol.clamp(min=1e-300)).max()):.3g}, first at "
        f"{bad.nonzero()[0].tolist()}")
