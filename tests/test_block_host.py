"""Layer norm, rotary positions and the gated feed-forward block without a GPU: the C entries refuse bad
arguments before touching the device, the torch conveniences refuse mismatched tensors before any C call,
and the layer's sub-layers order their calls."""
import contextlib
import types

import pytest
import torch

from deformable_slide_attention_b200 import abi, build, layer

P = 1 << 24  # fake, 16-byte aligned addresses: validation fails before any device access
INV, UNS, SMALL = 1, 2, 3
BF16, F32 = abi.DSA3D_BF16, abi.DSA3D_F32


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def ptrs(n):
    return [P * (i + 1) for i in range(n)]


def swap(p, i, v):
    q = list(p)
    q[i] = v
    return q


def test_layer_norm_refusals():
    p = ptrs(7)  # x, add, weight, bias, y, h, stats

    def call(p=p, rows=10, C=64, eps=1e-5, dtype=BF16):
        return abi.dsa3d_layer_norm(*p, rows, C, eps, dtype, 0)
    assert call(swap(p, 0, 0)) == INV and call(swap(p, 4, 0)) == INV
    assert call(swap(p, 1, 0)) == INV      # h without add
    assert call(swap(p, 5, 0)) == INV      # add without h
    assert call(swap(p, 2, 0)) == INV      # bias without weight
    assert call(swap(p, 0, P + 8)) == INV  # misaligned
    assert call(swap(p, 2, P * 3 + 2)) == INV
    assert call(swap(p, 4, P)) == INV      # y over x
    assert call(swap(p, 4, P + 64)) == INV
    assert call(swap(p, 5, P + 64)) == INV  # h beside x's start
    assert call(swap(p, 6, P + 64)) == INV  # stats inside x
    assert call(dtype=5) == INV and call(rows=-1) == INV and call(C=0) == INV
    assert call(eps=-1.0) == INV and call(eps=float("nan")) == INV and call(eps=float("inf")) == INV
    assert call(C=16392) == UNS and call(C=8193) == UNS and call(rows=1 << 31) == UNS
    assert abi.dsa3d_layer_norm(0, 0, 0, 0, 0, 0, 0, 0, 64, 1e-5, BF16, 0) == 0  # no rows: nothing to do


def test_layer_norm_backward_refusals():
    need = abi.dsa3d_layer_norm_backward_workspace_bytes(10, 64, BF16)
    assert need > 0 and need % 512 == 0
    assert abi.dsa3d_layer_norm_backward_workspace_bytes(0, 64, BF16) == 0
    assert abi.dsa3d_layer_norm_backward_workspace_bytes(10, 0, BF16) == 0
    p = ptrs(9)  # h, weight, stats, dy, add, dx, dw, db, ws

    def call(p=p, n=need, rows=10, C=64, dtype=BF16):
        return abi.dsa3d_layer_norm_backward(*p, n, rows, C, dtype, 0)
    for i in (0, 2, 3, 5, 8):
        assert call(swap(p, i, 0)) == INV, i
    for i in (1, 6, 7):  # the weight and its two gradients come together
        assert call(swap(p, i, 0)) == INV, i
    assert call(n=need - 1) == SMALL
    assert call(swap(p, 5, P)) == INV and call(swap(p, 5, P * 5 + 16)) == INV  # dx over h, beside add's start
    assert call(swap(p, 7, P * 7)) == INV and call(swap(p, 8, P * 4)) == INV   # db over dw, workspace over dy
    assert call(C=16392) == UNS and call(dtype=9) == INV


ROT = dict(first=0, rows=24, F=2, Hp=3, Wp=4, heads=2, dh=32, axes=(12, 10, 10), start=(0.0,) * 3,
           step=(1.0,) * 3, base=10000.0, ld=(64, 64, 64, 64), dtype=BF16, p=tuple(ptrs(4)))


@pytest.mark.parametrize("fn", [abi.dsa3d_rotary3d, abi.dsa3d_rotary3d_backward])
def test_rotary3d_refusals(fn):
    def call(**kw):
        a = {**ROT, **kw}
        return fn(*a["p"], *a["ld"], a["first"], a["rows"], a["F"], a["Hp"], a["Wp"], a["heads"], a["dh"],
                  a["axes"], a["start"], a["step"], a["base"], 1, a["dtype"], 0)
    assert call(p=(0, P, P * 2, P * 3)) == INV and call(p=(P, 0, P * 2, P * 3)) == INV
    assert call(p=(P, P * 2, P * 3, 0)) == INV and call(p=(P + 1, P * 2, P * 3, P * 4)) == INV
    assert call(first=1) == INV and call(first=25, rows=0) == INV and call(rows=-1) == INV  # past the grid
    assert call(axes=(12, 10, 12)) == INV   # more than dh
    assert call(axes=(11, 10, 10)) == INV and call(axes=(0, 0, 0)) == INV and call(axes=(-2, 10, 10)) == INV
    assert call(base=0.0) == INV and call(base=float("nan")) == INV and call(base=float("inf")) == INV
    assert call(start=(float("nan"), 0.0, 0.0)) == INV and call(step=(1.0, 1e300, 1.0)) == INV
    assert call(dh=33, axes=(12, 10, 10)) == UNS and call(dh=258, ld=(516,) * 4) == UNS
    assert call(heads=0) == INV and call(Wp=0) == INV and call(dtype=3) == INV
    assert call(F=1 << 20, Hp=1 << 10, Wp=2) == UNS
    assert call(ld=(63, 64, 64, 64)) == INV            # tokens overlap
    assert call(ld=(1 << 41, 64, 64, 64)) == UNS
    assert call(p=(P, P * 2, P * 2, P * 4)) == INV     # q_out over k
    assert call(p=(P, P * 2, P + 64, P * 4)) == INV    # q_out beside q's start
    assert call(p=(P, P * 2, P, P * 4), ld=(64, 64, 96, 64)) == INV   # in place with another stride
    assert call(p=(P, P * 2, P * 3, P * 3 + 64)) == INV               # the outputs overlap
    # rows of one packed buffer: interleaved rows that overlap by one head
    assert call(p=(P, P * 2, P * 3, P * 3 + 64), ld=(64, 64, 192, 192)) == INV
    assert call(rows=0, p=(0, 0, 0, 0)) == 0


def test_gated_ffn_refusals():
    rows, C, hid = 10, 64, 96
    need = abi.dsa3d_gated_ffn_workspace_bytes(rows, C, hid, BF16)
    assert need >= rows * hid * 2
    assert abi.dsa3d_gated_ffn_workspace_bytes(0, C, hid, BF16) == 0
    assert abi.dsa3d_gated_ffn_workspace_bytes(rows, C, 0, BF16) == 0
    p = ptrs(7)  # x, wg, wu, wd, add, y, ws

    def call(p=p, n=need, rows=rows, C=C, hid=hid, act=abi.DSA3D_SILU, dtype=BF16):
        return abi.dsa3d_gated_ffn(*p, n, rows, C, hid, act, dtype, 0)
    for i in (0, 1, 2, 3, 5, 6):
        assert call(swap(p, i, 0)) == INV, i
    assert call(swap(p, 3, P * 4 + 8)) == INV
    assert call(n=0) == SMALL and call(act=2) == INV and call(dtype=2) == INV
    assert call(swap(p, 5, P)) == INV and call(swap(p, 5, P * 5 + 64)) == INV  # y over x, beside add's start
    assert call(swap(p, 6, P * 2)) == INV                                     # workspace over a weight
    assert call(rows=-1) == INV and call(C=0) == INV and call(hid=(1 << 20) + 1) == UNS
    assert abi.dsa3d_gated_ffn(0, 0, 0, 0, 0, 0, 0, 0, 0, C, hid, 0, BF16, 0) == 0


def test_gated_ffn_backward_refusals():
    rows, C, hid = 10, 64, 96
    need = abi.dsa3d_gated_ffn_backward_workspace_bytes(rows, C, hid, BF16)
    p = ptrs(10)  # x, wg, wu, wd, dy, dx, dwg, dwu, dwd, ws

    def call(p=p, n=need, act=abi.DSA3D_GELU, dtype=BF16):
        return abi.dsa3d_gated_ffn_backward(*p, n, rows, C, hid, act, dtype, 0)
    for i in range(10):
        assert call(swap(p, i, 0)) == INV, i
    for i in range(5, 10):  # outputs and workspace over an input, and over each other
        assert call(swap(p, i, P * 3)) == INV, i
        assert call(swap(p, i, P * (5 + (i - 4) % 5 + 1))) == INV, i
    assert call(n=64) == SMALL and call(act=-1) == INV and call(dtype=2) == INV
    # a full-size call's workspace covers 65536 tokens
    assert abi.dsa3d_gated_ffn_backward_workspace_bytes(1 << 20, C, hid, BF16) == \
        abi.dsa3d_gated_ffn_backward_workspace_bytes(1 << 17, C, hid, BF16)


# ---- the torch conveniences ---------------------------------------------------------------------------
@pytest.fixture()
def calls(monkeypatch):
    log = []
    for name in ("dsa3d_layer_norm", "dsa3d_layer_norm_backward", "dsa3d_rotary3d", "dsa3d_rotary3d_backward",
                 "dsa3d_gated_ffn", "dsa3d_gated_ffn_backward"):
        monkeypatch.setattr(abi, name, lambda *a, _n=name: log.append((_n, a)) or 0)
    monkeypatch.setattr(abi, "_on_device", lambda *a: None)
    monkeypatch.setattr(abi, "_on_stream", lambda *a: contextlib.nullcontext())
    monkeypatch.setattr(abi, "_current_stream_handle", lambda ref: 0)
    return log


def test_conveniences_pass_what_they_check(calls):
    x, w = torch.zeros(6, 8, dtype=torch.bfloat16), torch.zeros(8)
    y, h, stats = abi.layer_norm(x, w, w)
    assert h is x and stats.shape == (2, 6) and y.dtype == x.dtype
    y, h, stats = abi.layer_norm(x, add=x, want_stats=False)
    assert h.shape == x.shape and h is not x and stats is None
    dx, dw, db = abi.layer_norm_backward(x, w, torch.zeros(2, 6), x)
    assert dw.dtype == torch.float32 and db.shape == (8,)
    assert abi.layer_norm_backward(x, None, torch.zeros(2, 6), x, add=x)[1:] == (None, None)
    qkv = torch.zeros(6, 3, 2, 32)
    q, k = abi.rotary3d(qkv[:, 0], qkv[:, 1], (1, 2, 3), (12, 10, 10))
    assert q.is_contiguous() and q.shape == (6, 2, 32)
    assert calls[-1][1][4:8] == (192, 192, 64, 64)  # token strides: read packed, written contiguous
    assert abi.rotary3d_backward(q, None, (1, 2, 3), (12, 10, 10))[1] is None
    abi.rotary3d(q, k, (1, 2, 3), (12, 10, 10), out=(q, k))
    wg, wd = torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(16, 8, dtype=torch.bfloat16)
    assert abi.gated_ffn(x, wg, wg, wd, add=y).shape == x.shape
    assert [t.shape for t in abi.gated_ffn_backward(x, wg, wg, wd, x)] == [x.shape, wg.shape, wg.shape, wd.shape]
    assert [c[0] for c in calls] == ["dsa3d_layer_norm"] * 2 + ["dsa3d_layer_norm_backward"] * 2 + \
        ["dsa3d_rotary3d", "dsa3d_rotary3d_backward", "dsa3d_rotary3d", "dsa3d_gated_ffn", "dsa3d_gated_ffn_backward"]


def test_conveniences_refuse_before_any_call(calls):
    x, w, st = torch.zeros(6, 8, dtype=torch.bfloat16), torch.zeros(8), torch.zeros(2, 6)
    q = torch.zeros(6, 2, 32)
    wg, wd = torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(16, 8, dtype=torch.bfloat16)
    dims, axes = (1, 2, 3), (12, 10, 10)
    bad = [
        lambda: abi.layer_norm(x[0], w, w), lambda: abi.layer_norm(x.t(), w, w),
        lambda: abi.layer_norm(x, w[:7], w), lambda: abi.layer_norm(x, w.double(), w),
        lambda: abi.layer_norm(x, w, w, add=x[:5]), lambda: abi.layer_norm(x, w, w, add=x.float()),
        lambda: abi.layer_norm(x, w, w, out=x.float()),
        lambda: abi.layer_norm_backward(x, w, st[:1], x), lambda: abi.layer_norm_backward(x, w, st, x.float()),
        lambda: abi.layer_norm_backward(x, w[:3], st, x),
        lambda: abi.rotary3d(x, None, dims, axes), lambda: abi.rotary3d(q, q[:5], dims, axes),
        lambda: abi.rotary3d(q, q.to(torch.bfloat16), dims, axes), lambda: abi.rotary3d(q, q, dims, (12, 10)),
        lambda: abi.rotary3d(q, q.transpose(1, 2).contiguous().transpose(1, 2), dims, axes),
        lambda: abi.rotary3d(q, q, dims, axes, out=(q, None)),
        lambda: abi.rotary3d(q[:1].expand(6, 2, 32), None, dims, axes),  # one token's storage for six
        lambda: abi.gated_ffn(x, wg, wg, wd.t(), ), lambda: abi.gated_ffn(x, wg, wg[:, :8], wd),
        lambda: abi.gated_ffn(x, wg.float(), wg, wd), lambda: abi.gated_ffn(x, wg, wg, wd, activation="relu"),
        lambda: abi.gated_ffn(x, wg, wg, wd, add=x[:2]), lambda: abi.gated_ffn(x, wg, wg, wd, workspace=torch.zeros(4)),
        lambda: abi.gated_ffn_backward(x, wg, wg, wd, x[:, :4]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
        assert calls == [], i
    for f in (lambda: abi.layer_norm(x.half()), lambda: abi.rotary3d(q.half(), None, dims, axes),
              lambda: abi.gated_ffn(x.half(), wg, wg, wd)):
        with pytest.raises(TypeError):
            f()


# ---- the layer ------------------------------------------------------------------------------------------
def test_feed_forward_orders_its_calls():
    log = []

    def norm(x, w, b, eps, add=None):
        log.append("layer_norm")
        h = x if add is None else x + add
        return h * 2, h, "stats"

    def ffn(n, g, u, d, activation, add):
        log.append("gated_ffn " + activation)
        return n * 3 + add

    def ffn_bwd(n, g, u, d, dy, activation):
        log.append("gated_ffn_backward " + activation)
        return dy * 5, g, u, d

    def norm_bwd(h, w, stats, dn, add):
        log.append("layer_norm_backward")
        assert stats == "stats"
        return dn * 7 + add, w, w

    ops = types.SimpleNamespace(layer_norm=norm, gated_ffn=ffn, gated_ffn_backward=ffn_bwd, layer_norm_backward=norm_bwd)
    x, a = torch.ones(2, 3), torch.full((2, 3), 2.0)
    wts = layer.FeedForwardWeights(*(torch.full((1,), float(i)) for i in range(5)))
    y, ctx = layer.feed_forward(x, wts, activation="gelu", add=a, ops=ops)
    assert torch.equal(y, (x + a) * 7)  # norm doubles, the block triples, plus h
    g = layer.feed_forward_backward(ctx, x, ops=ops)
    assert torch.equal(g["x"], x * 36)  # 5 * 7 through the block and the norm, 1 along the residual
    assert set(g) == {"x", "norm_weight", "norm_bias", "gate_weight", "up_weight", "down_weight"}
    assert log == ["layer_norm", "gated_ffn gelu", "gated_ffn_backward gelu", "layer_norm_backward"]


def test_layer_turns_q_and_k_and_turns_their_gradients_back():
    log = []
    N, H, DH = 6, 2, 4

    def rotary3d(q, k, dims, axes, **kw):
        log.append(("rotary3d", tuple(axes), kw["base"], kw["interleaved"]))
        return q + 1, k + 2

    def rotary3d_backward(dq, dk, dims, axes, out=None, **kw):
        log.append(("rotary3d_backward", tuple(axes), kw["base"], kw["interleaved"]))
        return dq * 10, dk * 100

    ops = types.SimpleNamespace(
        rotary3d=rotary3d, rotary3d_backward=rotary3d_backward,
        offset_head=lambda *a, **k: torch.zeros(H, N, 3),
        forward=lambda q, k, v, off, dims, window: (q + k, None),
        dwconv3d=lambda x, w, b, dims, add=None, out=None: out,
        backward=lambda q, k, v, off, lse, dout, dims, window: (dout, dout, dout, off),
        offset_head_backward=lambda x, *a, **k: (x * 0, None, None, None, None),
        dwconv3d_backward=lambda x, w, dy, dims: (x * 0, None, None))
    q = torch.zeros(N, H, DH)
    wts = layer.LayerWeights(*[None] * 6)
    rot = layer.Rotary((2, 2, 0), base=100.0, interleaved=False)
    out, ctx = layer.forward(torch.zeros(N, H * DH), q, q, q, wts, (1, 2, 3), (1, 1, 1), ops=ops, rotary=rot)
    assert torch.equal(out, q + 3)
    g = layer.backward(ctx, q + 1, ops=ops)
    assert torch.equal(g["q"], q + 10) and torch.equal(g["k"], q + 100) and torch.equal(g["v"], q + 1)
    assert log == [("rotary3d", (2, 2, 0), 100.0, False), ("rotary3d_backward", (2, 2, 0), 100.0, False)]
