"""The transformer block's operators on the GPU (layer norm, rotary positions, the gated feed-forward
block) against their formulas in 64 bits, element by element, within derived bounds
(tests/block_reference.py); then streams, captured graphs, in-place forms and the layer's sub-layers."""
import math

import pytest
import torch

from deformable_slide_attention_b200 import abi, layer
from tests import block_reference as ref
from tests.block_reference import check

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("gpu_lib")]

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return torch.empty(shape, device="cuda").normal_(mean, std, generator=g).to(dtype)


# ---- layer norm --------------------------------------------------------------------------------------
NORM_SHAPES = [(1, 1), (3, 2), (5, 7), (1, 8), (37, 32), (513, 64), (130, 100), (9, 258), (4099, 1001),
               (777, 2048), (2500, 512), (33, 4096), (5, 8191), (7, 8200), (2, 16384), (0, 64),
               # the backward's ring: four rows per step, blocks of 512 threads; element-wise rows, four in flight
               (40000, 64), (400, 4096), (400, 8192), (150000, 5)]


def _norm_inputs(rows, C, dtype, seed):
    g = _gen(seed)
    x = _randn(g, rows, C, std=2.0) + _randn(g, rows, 1, std=3.0)
    return (g, x.to(dtype), _randn(g, C, std=0.3, mean=1.0), _randn(g, C, std=0.3))


@pytest.mark.parametrize("rows,C", NORM_SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("add,affine", [(False, True), (True, True), (True, False)])
def test_layer_norm_and_backward(rows, C, dtype, add, affine):
    td = DT[dtype]
    g, x, w, b = _norm_inputs(rows, C, td, rows * 31 + C)
    if not affine:
        w = b = None
    a = _randn(g, rows, C, dtype=td) if add else None
    eps = 1e-5
    y, h, stats = abi.layer_norm(x, w, b, eps, add=a)
    (ry, rh, rs), (ey, es) = ref.layer_norm(x, w, b, eps, a)
    assert torch.equal(h, rh) and (add or h is x)
    check("y", y, ry, ey)
    check("stats", stats, rs, es)
    dy, more = _randn(g, rows, C, dtype=td), (_randn(g, rows, C, dtype=td) if add else None)
    got = abi.layer_norm_backward(h, w, stats, dy, add=more)
    want, bound = ref.layer_norm_backward(h, w, stats, dy, more)
    check("dx", got[0], want[0], bound[0])
    if affine:
        check("dw", got[1], want[1], bound[1])
        check("db", got[2], want[2], bound[2])
        again = abi.layer_norm_backward(h, w, stats, dy, add=more)
        assert all(torch.equal(p, q) for p, q in zip(got, again))  # a fixed order of summation
    else:
        assert got[1] is None and got[2] is None


def test_layer_norm_gradient_against_differences():
    """The formula's gradient of sum(y * dy) against central differences of the 64-bit forward, at
    steps whose cubic term is below 1e-6, and the kernel's against the formula's."""
    g, x, w, b = _norm_inputs(4, 12, torch.float32, 5)
    dy = _randn(g, 4, 12)
    _, _, stats = abi.layer_norm(x, w, b, 1e-5)
    dx, dw, db = abi.layer_norm_backward(x, w, stats, dy)

    def f(xx, ww, bb):
        m = xx.mean(1, keepdim=True)
        r = ((xx - m).square().mean(1, keepdim=True) + 1e-5).rsqrt()
        return (((xx - m) * r * ww + bb) * dy.double()).sum().item()

    args = [x.double(), w.double(), b.double()]
    for got, k in ((dx, 0), (dw, 1), (db, 2)):
        flat = args[k].view(-1)
        for i in range(0, flat.numel(), 5):
            old = flat[i].item()
            flat[i] = old + 1e-4
            up = f(*args)
            flat[i] = old - 1e-4
            down = f(*args)
            flat[i] = old
            assert abs((up - down) / 2e-4 - got.view(-1)[i].item()) < 2e-5 * max(1.0, got.abs().max().item())


@pytest.mark.parametrize("C", [64, 63])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_norm_rows_do_not_touch_each_other(C, dtype):
    """A constant row (variance 0) gives the bias exactly; a row with an infinity or a NaN is not finite,
    and the rows beside it are what they are without it."""
    g, x, w, b = _norm_inputs(9, C, DT[dtype], 3)
    x[4] = 2.5
    y0, _, s0 = abi.layer_norm(x, w, b)
    assert torch.equal(y0[4], b.to(DT[dtype])) and s0[0, 4].item() == 2.5
    x[2, 1], x[6, C - 1] = float("inf"), float("nan")
    y, _, _ = abi.layer_norm(x, w, b)
    keep = [0, 1, 3, 4, 5, 7, 8]
    assert torch.equal(y[keep], y0[keep])
    assert not torch.isfinite(y[2]).any() and not torch.isfinite(y[6]).any()


def test_layer_norm_in_place_sum_and_gradient():
    """The C entries' in-place forms: h over x, h over add, dx over add."""
    g, x, w, b = _norm_inputs(70, 128, torch.bfloat16, 4)
    a = _randn(g, 70, 128, dtype=torch.bfloat16)
    y0, h0, stats = abi.layer_norm(x, w, b, add=a)
    st = torch.cuda.current_stream().cuda_stream
    for over in (0, 1):
        xs, as_ = x.clone(), a.clone()
        h, y = (xs, as_)[over], torch.empty_like(x)
        assert abi.dsa3d_layer_norm(xs.data_ptr(), as_.data_ptr(), w.data_ptr(), b.data_ptr(), y.data_ptr(),
                                    h.data_ptr(), None, 70, 128, 1e-5, abi.DSA3D_BF16, st) == 0
        assert torch.equal(y, y0) and torch.equal(h, h0)
    dy = _randn(g, 70, 128, dtype=torch.bfloat16)
    dx0, dw0, db0 = abi.layer_norm_backward(h0, w, stats, dy, add=a)
    dx, dw, db = a.clone(), torch.empty_like(w), torch.empty_like(w)
    n = abi.dsa3d_layer_norm_backward_workspace_bytes(70, 128, abi.DSA3D_BF16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert abi.dsa3d_layer_norm_backward(h0.data_ptr(), w.data_ptr(), stats.data_ptr(), dy.data_ptr(),
                                         dx.data_ptr(), dx.data_ptr(), dw.data_ptr(), db.data_ptr(),
                                         ws.data_ptr(), n, 70, 128, abi.DSA3D_BF16, st) == 0
    assert torch.equal(dx, dx0) and torch.equal(dw, dw0) and torch.equal(db, db0)


# ---- rotary positions ------------------------------------------------------------------------------------
ROT_CASES = [  # dims, first, rows, heads, dh, axes
    ((4, 5, 6), 0, 120, 2, 32, (12, 10, 10)), ((1, 1, 1), 0, 1, 1, 2, (2, 0, 0)),
    ((3, 7, 9), 41, 77, 3, 64, (20, 22, 22)), ((2, 3, 5), 29, 1, 5, 128, (44, 42, 42)),
    ((2, 3, 5), 7, 0, 2, 32, (12, 10, 10)), ((2, 4, 4), 3, 20, 2, 48, (16, 16, 8)),
    ((2, 4, 4), 0, 32, 7, 128, (32, 48, 48)), ((1, 6, 6), 5, 30, 4, 64, (0, 16, 16)),
    ((5, 2, 3), 0, 30, 2, 30, (6, 8, 10)), ((3, 2, 2), 1, 9, 9, 256, (128, 64, 64)),
    ((256, 68, 120), 2088959 - 40, 41, 2, 64, (24, 20, 20))]


@pytest.mark.parametrize("case", range(len(ROT_CASES)))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("backward", [False, True])
def test_rotary3d(case, dtype, interleaved, backward):
    dims, first, rows, heads, dh, axes = ROT_CASES[case]
    g = _gen(case)
    q, k = (_randn(g, rows, heads, dh, dtype=DT[dtype]) for _ in range(2))
    kw = dict(first=first, start=(100000.0 if case % 2 else 0.0, -1.5, 0.0), step=(1.0, 0.5, 2.0),
              base=10000.0 if case % 3 else 500.0, interleaved=interleaved)
    call = abi.rotary3d_backward if backward else abi.rotary3d
    got = call(q, k, dims, axes, **kw)
    for name, x, o in (("q", q, got[0]), ("k", k, got[1])):
        want, bound = ref.rotary(x, dims, axes, backward=backward, **kw)
        check(name, o, want, bound)
        assert torch.equal(o[..., sum(axes):], x[..., sum(axes):])
    alone, none = call(q, None, dims, axes, **kw)
    assert none is None and torch.equal(alone, got[0])
    qi, ki = q.clone(), k.clone()
    call(qi, ki, dims, axes, out=(qi, ki), **kw)
    assert torch.equal(qi, got[0]) and torch.equal(ki, got[1])


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_rotary3d_reads_and_writes_packed_projections(interleaved, pad):
    """q and k as views of a packed [rows][3 heads dh + pad] projection, results written into another:
    aligned or not, the same values as contiguous ones, and nothing else of the buffers changes."""
    dims, axes, heads, dh = (2, 3, 7), (12, 10, 10), 3, 32
    rows, width = 42, 3 * heads * dh + pad
    g = _gen(8)
    src = _randn(g, rows, width, dtype=torch.bfloat16)
    dst = torch.full((rows, width), 7.0, dtype=torch.bfloat16, device="cuda")
    cut = lambda t, i: t[:, i * heads * dh:(i + 1) * heads * dh].unflatten(1, (heads, dh))
    q, k = cut(src, 0), cut(src, 1)
    want = abi.rotary3d(q.contiguous(), k.contiguous(), dims, axes, interleaved=interleaved)
    got = abi.rotary3d(q, k, dims, axes, interleaved=interleaved)
    abi.rotary3d(q, k, dims, axes, interleaved=interleaved, out=(cut(dst, 0), cut(dst, 2)))
    for a, b, c in zip(want, got, (cut(dst, 0), cut(dst, 2))):
        check("strided read", b, a.double(), ref.half_step(torch.bfloat16) * a.double().abs() * 2)
        assert torch.equal(b, c)
    assert bool((cut(dst, 1) == 7.0).all()) and bool((dst[:, 3 * heads * dh:] == 7.0).all())


def test_rotary3d_keeps_scores_and_undoes_itself():
    """The backward undoes the forward; a rotated q . k depends on the positions' difference only; dims
    past the rotated ones keep their bits, infinities and NaN too."""
    g = _gen(1)
    dims, axes, heads, dh = (3, 4, 5), (16, 24, 24), 2, 64
    q, k = _randn(g, 60, heads, dh), _randn(g, 60, heads, dh)
    qr, kr = abi.rotary3d(q, k, dims, axes)
    qb, _ = abi.rotary3d_backward(qr, kr, dims, axes)
    assert (qb - q).abs().max().item() < 64 * 2.0 ** -24 * q.abs().max().item()
    q2, k2 = abi.rotary3d(q, k, dims, axes, start=(7.0, 3.0, 11.0))
    same = (qr * kr).sum(-1) - (q2 * k2).sum(-1)  # one token's q and k: the shift drops out
    assert same.abs().max().item() < 40 * 2.0 ** -24 * 2 * (q.abs() * k.abs()).sum(-1).max().item() + 1e-5
    x = _randn(g, 60, heads, dh, dtype=torch.bfloat16)
    x[..., 40], x[..., 47] = float("inf"), float("nan")
    for inter in (True, False):
        y, _ = abi.rotary3d(x, None, dims, (8, 16, 16), interleaved=inter)
        assert torch.equal(y[..., 40:].view(torch.int16), x[..., 40:].contiguous().view(torch.int16))
        assert torch.isfinite(y[..., :40]).all()


# ---- gated feed-forward -------------------------------------------------------------------------------------
FFN_SHAPES = [(1, 1, 1), (3, 5, 7), (1, 64, 160), (7, 64, 160), (65, 40, 72), (130, 258, 685), (200, 512, 1024),
              (129, 128, 264), (1000, 72, 200), (16, 2048, 1032), (300, 1000, 520), (1, 2048, 1001), (700, 131, 257),
              (150, 64, 259), (2, 64, 160), (3, 520, 1032), (4, 2048, 40), (4, 8, 4104), (5, 2048, 1032), (8, 520, 264),
              (9, 264, 520), (257, 64, 2048), (0, 64, 96)]


def _ffn_inputs(rows, C, hidden, dtype, seed, std=1.0):
    g = _gen(seed)
    x = _randn(g, rows, C, dtype=dtype, std=std)
    w = [_randn(g, C, hidden, dtype=dtype, std=C ** -0.5) for _ in range(2)]
    return g, x, (*w, _randn(g, hidden, C, dtype=dtype, std=hidden ** -0.5))


@pytest.mark.parametrize("rows,C,hidden", FFN_SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_ffn_and_backward(rows, C, hidden, dtype, act):
    td = DT[dtype]
    g, x, w = _ffn_inputs(rows, C, hidden, td, rows + C + hidden, std=2.0)
    a, dy = _randn(g, rows, C, dtype=td), _randn(g, rows, C, dtype=td)
    for add in (None, a):
        y = abi.gated_ffn(x, *w, activation=act, add=add)
        check("y", y, *ref.gated_ffn(x, *w, act, add))
    inplace = a.clone()
    assert torch.equal(abi.gated_ffn(x, *w, activation=act, add=inplace, out=inplace), y)
    got = abi.gated_ffn_backward(x, *w, dy, activation=act)
    want, bound = ref.gated_ffn_backward(x, *w, dy, act)
    for name, o, r, e in zip(("dx", "dgate", "dup", "ddown"), got, want, bound):
        check(name, o, r, e)
    again = abi.gated_ffn_backward(x, *w, dy, activation=act)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("C,hidden", [(64, 136), (61, 131)])
@pytest.mark.parametrize("rows", [1000, 513])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gated_ffn_in_chunks(dtype, rows, C, hidden):
    """The smallest documented workspaces (chunks of 256 tokens): the forward and dx are the same but for
    the order of their sums, the weight gradients are within their bounds; less is refused."""
    td = DT[dtype]
    g, x, w = _ffn_inputs(rows, C, hidden, td, 6)
    dy = _randn(g, rows, C, dtype=td)
    code = abi._dtype_code(x)
    small = torch.empty(abi.dsa3d_gated_ffn_workspace_bytes(256, C, hidden, code), dtype=torch.uint8, device="cuda")
    check("y", abi.gated_ffn(x, *w, workspace=small), *ref.gated_ffn(x, *w, "silu", None))
    up = lambda n: (n + 255) // 256 * 256
    small = torch.empty(abi.dsa3d_gated_ffn_backward_workspace_bytes(256, C, hidden, code) +
                        12 * up(C) * up(hidden) + 1024, dtype=torch.uint8, device="cuda")
    got = abi.gated_ffn_backward(x, *w, dy, workspace=small)
    want, bound = ref.gated_ffn_backward(x, *w, dy, "silu")
    for name, o, r, e in zip(("dx", "dgate", "dup", "ddown"), got, want, bound):
        check(name, o, r, e)
    with pytest.raises(abi.Dsa3dError):
        abi.gated_ffn_backward(x, *w, dy, workspace=small[:1024])


def test_gated_ffn_large_values_stay_finite():
    """Gates of +-30 and beyond: silu and gelu saturate, their derivatives too."""
    g, x, w = _ffn_inputs(64, 64, 128, torch.float32, 9, std=30.0)
    dy = _randn(g, 64, 64)
    for act in ("silu", "gelu"):
        y = abi.gated_ffn(x, *w, activation=act)
        assert torch.isfinite(y).all()
        for t in abi.gated_ffn_backward(x, *w, dy, activation=act):
            assert torch.isfinite(t).all()


# ---- sizes past 32 bits, chunks ------------------------------------------------------------------------
def test_rows_past_32_bits_of_elements():
    """1,100,000 x 4096 bf16 (4.5 billion elements per tensor): first, middle and last rows of the norm, its
    dx and the rotation, against the same rows computed alone (the norm's rows do not depend on the launch)."""
    N, C = 1100000, 4096
    g = _gen(31)
    x = torch.empty(N, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w, b = _randn(g, C, mean=1.0), _randn(g, C)
    rows = torch.tensor([0, 1, 524287, 524288, 1048575, 1048576, N - 2, N - 1], device="cuda")
    y, _, stats = abi.layer_norm(x, w, b)
    xs = x[rows].contiguous()
    (ry, _, rs), (ey, es) = ref.layer_norm(xs, w, b, 1e-5, None)
    check("y", y[rows], ry, ey)
    check("stats", stats[:, rows], rs, es)
    dx, _, _ = abi.layer_norm_backward(x, w, stats, y, add=x)
    want, bound = ref.layer_norm_backward(xs, w, stats[:, rows].contiguous(), y[rows].contiguous(), xs)
    check("dx", dx[rows], want[0], bound[0])
    del dx
    kw = dict(start=(0.0,) * 3, step=(1.0,) * 3, base=10000.0, interleaved=True)
    q, _ = abi.rotary3d(x.view(N, 32, 128), None, (256, 68, 120), (44, 42, 42), out=(y.view(N, 32, 128), None), **kw)
    for i, r in enumerate(rows.tolist()):
        want, bound = ref.rotary(xs[i:i + 1].view(1, 32, 128), (256, 68, 120), (44, 42, 42), first=r, backward=False, **kw)
        check("rotary", q[r:r + 1], want, bound)
    del x, y, q
    torch.cuda.empty_cache()


def test_gated_ffn_of_more_tokens_than_a_chunk():
    """66,000 tokens: a chunk of 65,536 and a short one, whole in memory for the reference."""
    g, x, w = _ffn_inputs(66000, 32, 72, torch.bfloat16, 14)
    dy = _randn(g, 66000, 32, dtype=torch.bfloat16)
    check("y", abi.gated_ffn(x, *w, add=dy), *ref.gated_ffn(x, *w, "silu", dy))
    got = abi.gated_ffn_backward(x, *w, dy)
    want, bound = ref.gated_ffn_backward(x, *w, dy, "silu")
    for name, o, r, e in zip(("dx", "dgate", "dup", "ddown"), got, want, bound):
        check(name, o, r, e)


def test_no_wait_ran_out():
    """The bounded waits of the kernels above recorded nothing."""
    assert abi.dsa3d_check_device(torch.cuda.current_stream().cuda_stream) == 0


# ---- streams, graphs, sub-layers -------------------------------------------------------------------------------
def _run_all(x, q, w, b, f, dims, axes, stream=None):
    y, h, stats = abi.layer_norm(x, w, b, add=x, stream=stream)
    dx, dw, db = abi.layer_norm_backward(h, w, stats, y, add=x, stream=stream)
    qr, kr = abi.rotary3d(q, q, dims, axes, stream=stream)
    z = abi.gated_ffn(y, *f, add=x, stream=stream)
    return (y, h, stats, dx, dw, db, qr, kr, z, *abi.gated_ffn_backward(y, *f, z, stream=stream))


def _all_inputs(dtype=torch.bfloat16):
    dims, axes = (2, 8, 20), (12, 10, 10)
    g, x, f = _ffn_inputs(320, 64, 192, dtype, 12)
    return x, _randn(g, 320, 2, 32, dtype=dtype), _randn(g, 64, mean=1.0), _randn(g, 64), f, dims, axes


def test_on_another_stream_and_from_two_streams_at_once():
    args = _all_inputs()
    want = _run_all(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [_run_all(*args, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_beside_the_attention_on_another_stream():
    """The feed-forward block and the attention, both with tensor memory of their own, on two streams at
    once, several times over: each as when it runs alone."""
    from deformable_slide_attention_b200 import inputs
    dims, heads, dh, window = (16, 32, 32), 4, 64, (3, 7, 7)
    _, inp = inputs.custom(*dims, heads, dh, window, "bf16", seed=9, scale=2.0)
    d = {k: v.cuda() for k, v in inp.items()}
    g, x, w = _ffn_inputs(6000, 512, 1032, torch.bfloat16, 3)
    dy = _randn(g, 6000, 512, dtype=torch.bfloat16)

    def attention():
        out, lse = abi.forward(d["q"], d["k"], d["v"], d["offsets"], dims, window)
        return (out, *abi.backward(d["q"], d["k"], d["v"], d["offsets"], lse, d["dout"], dims, window)[:3])

    def block():
        return (abi.gated_ffn(x, *w), *abi.gated_ffn_backward(x, *w, dy))
    want = attention(), block()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        for s, f, ref_ in zip(streams, (attention, block), want):
            with torch.cuda.stream(s):
                got.append((f(), ref_))
    torch.cuda.synchronize()
    for r, ref_ in got:
        assert all(torch.equal(a, b) for a, b in zip(r, ref_))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C,hidden", [(300, 72, 136), (70, 61, 77), (6, 64, 96)])
def test_gated_ffn_rows_do_not_touch_each_other(dtype, rows, C, hidden):
    """A token with a NaN or an infinity: its own y and dx are not finite, every other row's are what they
    are without it."""
    g, x, w = _ffn_inputs(rows, C, hidden, DT[dtype], 2)
    dy = _randn(g, rows, C, dtype=DT[dtype])
    y0, dx0 = abi.gated_ffn(x, *w), abi.gated_ffn_backward(x, *w, dy)[0]
    x[1, 2], x[rows - 2, C - 1] = float("nan"), float("inf")
    y, dx = abi.gated_ffn(x, *w), abi.gated_ffn_backward(x, *w, dy)[0]
    keep = [r for r in range(rows) if r not in (1, rows - 2)]
    assert torch.equal(y[keep], y0[keep]) and torch.equal(dx[keep], dx0[keep])
    assert not torch.isfinite(y[1]).any() and not torch.isfinite(y[rows - 2]).any()


def test_captured_and_replayed_with_new_inputs():
    args = _all_inputs()
    _run_all(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _run_all(*args)
    for seed in (1, 2):
        args[0].copy_(_randn(_gen(seed), *args[0].shape))
        args[1].copy_(_randn(_gen(seed + 9), *args[1].shape))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(kept, _run_all(*args)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_feed_forward_sublayer(dtype):
    """layer.feed_forward (x + FFN(norm(x))) and its backward against automatic differentiation of the
    formula in 64 bits: relative 2-norm error, a rounding of the norm's output and of each part."""
    td, (rows, C, hidden) = DT[dtype], (150, 64, 176)
    g, x, f = _ffn_inputs(rows, C, hidden, td, 21)
    wts = layer.FeedForwardWeights(_randn(g, C, std=0.2, mean=1.0), _randn(g, C, std=0.2), *f)
    dy = _randn(g, rows, C, dtype=td)
    y, ctx = layer.feed_forward(x, wts, activation="gelu")
    grads = layer.feed_forward_backward(ctx, dy)
    leaves = [t.double().requires_grad_() for t in (x, wts.norm_weight, wts.norm_bias, *f)]
    n = torch.nn.functional.layer_norm(leaves[0], (C,), leaves[1], leaves[2], 1e-5)
    want = leaves[0] + (torch.nn.functional.gelu(n @ leaves[3]) * (n @ leaves[4])) @ leaves[5]
    ref_grads = torch.autograd.grad(want, leaves, dy.double())
    tol = 4 * ref.half_step(td) + 200 * ref.F32
    names = ("x", "norm_weight", "norm_bias", "gate_weight", "up_weight", "down_weight")
    for name, a, b in [("y", y, want.detach())] + [(m, grads[m], r) for m, r in zip(names, ref_grads)]:
        err = ((a.double() - b).norm() / b.norm()).item()
        assert err <= tol, (name, err, tol)


@pytest.mark.parametrize("interleaved", [True, False])
def test_block_forward_and_backward(interleaved):
    """A whole transformer block as a user writes it: norm, packed projection, rotary positions inside
    layer.forward, deformable attention with its convolution, residual sum, feed-forward sub-layer, and
    the backward pass through all of it; fp32, against the same chain with the new operators replaced by
    64-bit formulas and their derivatives (the attention's own calls are shared)."""
    dims, window, heads, dh = (2, 4, 6), (1, 3, 3), 2, 32
    C, N = heads * dh, math.prod(dims)
    g = _gen(77)
    x = _randn(g, N, C)
    wq = [_randn(g, C, C, std=C ** -0.5) for _ in range(3)]
    nw, nb = _randn(g, C, std=0.2, mean=1.0), _randn(g, C, std=0.2)
    K = math.prod(window)
    wts = layer.LayerWeights(_randn(g, C, *window, std=K ** -0.5), _randn(g, C), _randn(g, C, *window, std=K ** -0.5),
                             _randn(g, C), _randn(g, C, heads * 3, std=0.1), _randn(g, heads * 3, std=0.1))
    ffn = layer.FeedForwardWeights(nw, nb, _randn(g, C, 160, std=0.1), _randn(g, C, 160, std=0.1),
                                   _randn(g, 160, C, std=0.1))
    rot = layer.Rotary(axes=(12, 10, 10), interleaved=interleaved)
    dout = _randn(g, N, C)
    # forward
    n, _, stats = abi.layer_norm(x, nw, nb)
    q, k, v = ((n @ w).view(N, heads, dh) for w in wq)
    att, ctx = layer.forward(n, q, k, v, wts, dims, window, rotary=rot)
    y, fctx = layer.feed_forward(att.view(N, C), ffn, add=x)
    # backward
    fg = layer.feed_forward_backward(fctx, dout)
    ag = layer.backward(ctx, fg["x"].view(N, heads, dh))
    dn = ag["x"] + sum(ag[m].reshape(N, C) @ w.t() for m, w in zip("qkv", wq))
    dx, dnw, dnb = abi.layer_norm_backward(x, nw, stats, dn, add=fg["x"])
    # the same with 64-bit formulas
    kw = dict(first=0, start=(0.0,) * 3, step=(1.0,) * 3, base=10000.0, interleaved=interleaved)
    (rn, _, rs), _ = ref.layer_norm(x, nw, nb, 1e-5, None)
    qr, kr = (ref.rotary((rn.float() @ w).view(N, heads, dh), dims, rot.axes, backward=False, **kw)[0].float()
              for w in wq[:2])
    att2, ctx2 = layer.forward(rn.float(), qr, kr, (rn.float() @ wq[2]).view(N, heads, dh), wts, dims, window)
    h = x.double() + att2.view(N, C).double()
    leaves = [t.double().requires_grad_() for t in (h, nw, nb, ffn.gate_weight, ffn.up_weight, ffn.down_weight)]
    m = torch.nn.functional.layer_norm(leaves[0], (C,), leaves[1], leaves[2], 1e-5)
    y2 = leaves[0] + (torch.nn.functional.silu(m @ leaves[3]) * (m @ leaves[4])) @ leaves[5]
    rg = torch.autograd.grad(y2, leaves, dout.double())
    ag2 = layer.backward(ctx2, rg[0].float().view(N, heads, dh))
    dq, dk = (ref.rotary(ag2[m_], dims, rot.axes, backward=True, **kw)[0].float() for m_ in "qk")
    dn2 = ag2["x"] + sum(d.reshape(N, C) @ w.t() for d, w in zip((dq, dk, ag2["v"]), wq))
    (dx2, dnw2, dnb2), _ = ref.layer_norm_backward(x, nw, rs.float(), dn2, rg[0].float())
    for name, a, b in (("y", y, y2), ("dgate", fg["gate_weight"], rg[3]), ("ddown", fg["down_weight"], rg[5]),
                       ("dx", dx, dx2), ("dnw", dnw, dnw2), ("dnb", dnb, dnb2), ("dq", ag["q"], dq)):
        err = ((a.double() - b.double()).norm() / b.double().norm()).item()
        assert err <= 1e-4, (name, err)  # fp32 chain of six operators; offsets near a cell's edge move little
