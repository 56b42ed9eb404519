"""Host-side checks of the operators around the attention (no GPU needed):
arguments refused before anything is launched, workspace sizes, and the
binding's own checks."""
import ctypes

import pytest
import torch

import sparse_transformer_attention_b200 as ca
from sparse_transformer_attention_b200 import binding
from sparse_transformer_attention_b200.binding import CaNormRope, CaRows

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced
P = ctypes.c_void_p
INV, UNS, ALI, WS = (binding.CA_ERR_INVALID_ARG, binding.CA_ERR_UNSUPPORTED,
                     binding.CA_ERR_ALIGNMENT, binding.CA_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    from sparse_transformer_attention_b200 import build
    build.build()
    return binding.load()


def _grids(over, name, n_grids=3, heads=(8, 2, 2), n=10, d=64):
    out = []
    for i in range(n_grids):
        r = dict(data=FAKE, stride_b=n * 12 * d, stride_t=12 * d, stride_h=d)
        r.update(over.get(f"{name}{i}", {}))
        out.append(CaRows(r["data"], r["stride_b"], r["stride_t"],
                          r["stride_h"]))
    return (CaRows * n_grids)(*out)


def _params(over):
    p = dict(q_weight=FAKE, k_weight=FAKE, w_dtype=1, eps=1e-6, inv_freq=FAKE,
             rot_dim=64, interleaved=0, positions=None, pos0=0)
    p.update({k: v for k, v in over.items() if k in p})
    return CaNormRope(*p.values())


def _sizes(over):
    a = dict(dtype=1, B=2, n=10, Hq=8, Hkv=2, d=64)
    a.update({k: v for k, v in over.items() if k in a})
    return list(a.values())


def _forward(lib, over):
    p = _params(over)
    return lib.condensate_attn_norm_rope(
        None if over.get("in") == 0 else _grids(over, "in"), *_sizes(over),
        None if over.get("p") == 0 else ctypes.byref(p),
        None if over.get("out") == 0 else _grids(over, "out"), None)


def _backward(lib, over):
    p = _params(over)
    ws = over.get("ws", FAKE)
    return lib.condensate_attn_norm_rope_backward(
        None if over.get("out") == 0 else _grids(over, "out"),
        None if over.get("x") == 0 else _grids(over, "x"), *_sizes(over),
        None if over.get("p") == 0 else ctypes.byref(p),
        None if over.get("in") == 0 else _grids(over, "in"),
        P(over.get("dqw", FAKE)), P(over.get("dkw", FAKE)), P(ws),
        over.get("ws_bytes", 16), None)


COMMON = [
    ({"in": 0}, INV), ({"out": 0}, INV), ({"p": 0}, INV),
    ({"B": 0}, INV), ({"n": 0}, INV), ({"Hq": 0}, INV), ({"Hkv": 0}, INV),
    ({"in0": {"data": None}}, INV), ({"out1": {"data": None}}, INV),
    ({"dtype": 5}, UNS), ({"w_dtype": 3}, UNS), ({"d": 96}, UNS),
    ({"rot_dim": -16}, INV), ({"rot_dim": 80}, INV), ({"rot_dim": 24}, UNS),
    ({"inv_freq": None}, INV), ({"eps": -1.0}, INV),
    ({"eps": float("nan")}, INV), ({"pos0": (1 << 31) - 5}, INV),
    ({"in0": {"data": FAKE + 2}}, ALI), ({"out2": {"stride_h": 60}}, ALI),
    ({"in1": {"stride_t": -64}}, INV), ({"q_weight": FAKE + 2}, ALI),
    ({"inv_freq": FAKE + 1}, ALI), ({"positions": FAKE + 2}, ALI),
]


@pytest.mark.parametrize("over,code", COMMON + [
    ({"out0": {"stride_h": 0}}, INV), ({"out1": {"stride_t": 0}}, INV),
    ({"out2": {"stride_b": 0}}, INV)])
def test_norm_rope_refusals(lib, over, code):
    assert _forward(lib, over) == code


@pytest.mark.parametrize("over,code", COMMON + [
    ({"in0": {"stride_h": 0}}, INV), ({"x": 0}, INV),
    ({"x1": {"data": None}}, INV), ({"x0": {"data": FAKE + 4}}, ALI),
    ({"q_weight": None}, INV),        # its gradient asked for without it
    ({"dqw": FAKE + 1}, ALI), ({"ws": 0}, WS), ({}, WS),
    ({"ws": FAKE + 8, "ws_bytes": 1 << 24}, ALI)])
def test_norm_rope_backward_refusals(lib, over, code):
    assert _backward(lib, over) == code


def _prefill_backward(lib, **over):
    a = dict(Q=FAKE, K=FAKE, V=FAKE, dtype=1, dO=FAKE, o_dtype=0, B=1,
             nq=1000, L=1000, Hq=8, Hkv=2, d=128, W=64, k=16, W_i=0, W_h=0,
             idx=FAKE, cnt=FAKE, C_max=81, dQ=FAKE, dK=FAKE, dV=FAKE,
             ws=FAKE, ws_bytes=16)
    a.update(over)
    ptr = {"Q", "K", "V", "dO", "W_i", "W_h", "idx", "cnt", "dQ", "dK", "dV",
           "ws"}
    return lib.condensate_attn_prefill_backward(
        *(P(v) if n in ptr else v for n, v in a.items()), None)


@pytest.mark.parametrize("over,code", [
    *(({n: 0}, INV) for n in ("Q", "K", "V", "dO", "idx", "cnt", "dQ", "dK",
                              "dV", "B", "nq", "Hq", "Hkv", "C_max", "W")),
    ({"ws": 0}, WS), ({}, WS), ({"L": 999}, INV), ({"k": -1}, INV),
    ({"C_max": 80}, INV), ({"Hq": 7}, INV), ({"d": 96}, UNS),
    ({"dtype": 2}, UNS), ({"o_dtype": 2}, UNS), ({"Hq": 6, "Hkv": 2}, UNS),
    ({"k": 129, "C_max": 1000}, UNS), ({"dO": FAKE + 8}, ALI),
    ({"idx": FAKE + 4}, ALI), ({"W_i": FAKE + 2}, ALI),
    ({"ws": FAKE + 4}, ALI),
    # 2^31 slots of one kv head: 8 x 3,000,000 x 128
    ({"nq": 3000000, "L": 3000000, "Hq": 8, "Hkv": 1, "k": 127,
      "C_max": 192}, UNS),
])
def test_prefill_backward_refusals(lib, over, code):
    assert _prefill_backward(lib, **over) == code


@pytest.mark.parametrize("out", ["dQ", "dK", "dV", "ws"])
@pytest.mark.parametrize("other", ["Q", "K", "V", "dO", "idx", "cnt", "W_i",
                                   "W_h", "dQ", "dK", "dV", "ws"])
def test_prefill_backward_refuses_overlap(lib, out, other):
    """Results that begin in another grid's last 16 bytes, and the reverse."""
    if out == other:
        return
    names = ("Q", "K", "V", "dO", "idx", "cnt", "W_i", "W_h", "dQ", "dK",
             "dV", "ws")
    at = {n: (i + 1) << 40 for i, n in enumerate(names)}
    need = ca.condensate_attn_prefill_backward_workspace_size(
        torch.bfloat16, torch.float32, 1, 1000, 1000, 8, 2, 128, 16)
    rows, keys = 8 * 1000, 2 * 1000
    size = dict(Q=rows * 256, K=keys * 256, V=keys * 256, dO=rows * 512,
                idx=rows * 81 * 4, cnt=rows * 4, W_i=4000, W_h=32,
                dQ=rows * 256, dK=keys * 256, dV=keys * 256, ws=need)
    for a, b in ((out, other), (other, out)):
        over = dict(at)
        over[a] = at[b] + size[b] // 16 * 16 - 16
        assert _prefill_backward(lib, ws_bytes=need, **over) == INV


def test_workspace_sizes(lib):
    f = ca.condensate_attn_prefill_backward_workspace_size
    b = torch.bfloat16
    base = f(b, b, 1, 1000, 1000, 8, 2, 64, 16)
    # at least p and dS of every slot
    assert base > 8 * 1000 * 17 * 8
    assert f(b, b, 2, 1000, 1000, 8, 2, 64, 16) > base
    for bad in ((0, 1000, 1000, 8, 2, 64, 16), (1, 0, 1000, 8, 2, 64, 16),
                (1, 1000, 999, 8, 2, 64, 16), (1, 1000, 1000, 7, 2, 64, 16),
                (1, 1000, 1000, 8, 2, 96, 16), (1, 1000, 1000, 8, 2, 64, 129),
                (1, 3000000, 3000000, 8, 1, 64, 127)):
        assert f(b, b, *bad) == 0
    g = lib.condensate_attn_norm_rope_workspace_size
    assert g(64) > 0 and g(128) == 2 * g(64) and g(96) == 0


def test_binding_refuses_cpu_tensors(lib):
    x = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError):
        ca.condensate_attn_norm_rope(x, x, x, None)
    with pytest.raises(ValueError):
        ca.condensate_attn_norm_rope_backward(x, None, None, None, None, None)
    y = torch.zeros(1, 2, 4, 64)
    i = torch.zeros(1, 2, 4, 8, dtype=torch.int32)
    with pytest.raises(ValueError):
        ca.condensate_attn_prefill_backward(y, y, y, y, i, i[..., 0], 4, 2)
    with pytest.raises(ValueError):
        ca.qkv_attention(torch.zeros(1, 4, 100), 2, 1, 4, 2, None)


def test_packed_structures():
    """The binding's packed bytes have the header's layout."""
    from sparse_transformer_attention_b200 import block
    rows = (CaRows * 3)(*(CaRows(16 * i + 16, 3 * i, 3 * i + 1, 3 * i + 2)
                          for i in range(3)))
    packed = block._ROWS3.pack(*(x for r in rows for x in (
        r.data, r.stride_b, r.stride_t, r.stride_h)))
    assert packed == bytes(rows)
    p = CaNormRope(16, 32, 1, 0.5, 48, 64, 1, 80, -7)
    packed = block._PARAMS.pack(16, 32, 1, 0.5, 48, 64, 1, 80, -7)
    assert len(packed) == ctypes.sizeof(p)
    assert bytes(CaNormRope.from_buffer_copy(packed)) == bytes(p)
