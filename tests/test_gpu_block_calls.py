"""Calls of the transformer block's operators that their documentation allows beside the plain ones: one
workspace for calls of every length, chunks of tokens whose split sums differ from chunk to chunk."""
import pytest
import torch

from deformable_slide_attention_b200 import abi
from tests import block_reference as ref
from tests.block_reference import check
from tests.test_block_contracts_host import WORKSPACE_WIDTHS, check_workspace_never_shrinks

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("gpu_lib")]

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g).to(dtype)


def _ffn_inputs(rows, C, hidden, dtype, seed):
    g = _gen(seed)
    x, a, dy = (_randn(g, rows, C, dtype=dtype) for _ in range(3))
    w = (_randn(g, C, hidden, dtype=dtype, std=C ** -0.5), _randn(g, C, hidden, dtype=dtype, std=C ** -0.5),
         _randn(g, hidden, C, dtype=dtype, std=hidden ** -0.5))
    return x, w, a, dy


def _check_grads(got, want_bound):
    for name, o, r, e in zip(("dx", "dgate", "dup", "ddown"), got, *want_bound):
        check(name, o, r, e)


# ---- workspaces --------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [abi.DSA3D_F32, abi.DSA3D_BF16])
@pytest.mark.parametrize("C,hidden", WORKSPACE_WIDTHS + [(256, 2048), (4096, 512), (8, 20000)])
def test_feed_forward_workspace_never_shrinks_on_this_gpu(C, hidden, dtype):
    check_workspace_never_shrinks(C, hidden, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,hidden", [(256, 2048), (264, 640), (61, 131)])
def test_one_workspace_for_calls_of_every_length(C, hidden, dtype):
    """The longest call's workspace: shorter ones give what they give with their own."""
    x, w, a, dy = _ffn_inputs(700, C, hidden, DT[dtype], 21)
    code = abi._dtype_code(x)
    buf = torch.empty(max(f(700, C, hidden, code) for f in (abi.dsa3d_gated_ffn_workspace_bytes,
                                                            abi.dsa3d_gated_ffn_backward_workspace_bytes)),
                      dtype=torch.uint8, device="cuda")
    for rows in (1, 2, 3, 4, 5, 8, 9, 16, 100, 128, 129, 256, 257, 513, 700):
        xs, ad, ds = x[:rows], a[:rows], dy[:rows]
        assert torch.equal(abi.gated_ffn(xs, *w, add=ad, workspace=buf), abi.gated_ffn(xs, *w, add=ad)), rows
        got, own = abi.gated_ffn_backward(xs, *w, ds, workspace=buf), abi.gated_ffn_backward(xs, *w, ds)
        assert all(torch.equal(p, q) for p, q in zip(got, own)), rows


# Workspaces for 256, 1024 and 2560 tokens: chunks of as many tokens or some more, and a shorter last one.  With
# 148 SMs 2560 tokens by 2048 columns leave 6 of 80 tiles to the last round, in eight parts each; 1024 make 32
# tiles of two parts: the shorter chunk has more sums.
@pytest.mark.parametrize("tokens", [256, 1024, 2560])
@pytest.mark.parametrize("C", [2048, 2044, 2041])
def test_gated_ffn_in_chunks_with_split_tails(C, tokens):
    rows, hidden = 3600, 2048
    x, w, a, dy = _ffn_inputs(rows, C, hidden, torch.bfloat16, C + tokens)
    size = abi.dsa3d_gated_ffn_workspace_bytes(tokens, C, hidden, abi.DSA3D_BF16)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    check("y", abi.gated_ffn(x, *w, add=a, workspace=ws), *ref.gated_ffn(x, *w, "silu", a))
    size = abi.dsa3d_gated_ffn_backward_workspace_bytes(tokens, C, hidden, abi.DSA3D_BF16)
    ws = torch.empty(size + 12 * 2048 * 2048 + 1024, dtype=torch.uint8, device="cuda")
    _check_grads(abi.gated_ffn_backward(x, *w, dy, workspace=ws), ref.gated_ffn_backward(x, *w, dy, "silu"))


@pytest.mark.parametrize("tokens", [256, 300, 1024])
def test_gated_ffn_f32_in_chunks_with_split_sums(tokens):
    rows, C, hidden = 1500, 130, 1030
    x, w, a, dy = _ffn_inputs(rows, C, hidden, torch.float32, tokens)
    size = abi.dsa3d_gated_ffn_workspace_bytes(tokens, C, hidden, abi.DSA3D_F32)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    check("y", abi.gated_ffn(x, *w, add=a, workspace=ws), *ref.gated_ffn(x, *w, "silu", a))
    size = abi.dsa3d_gated_ffn_backward_workspace_bytes(tokens, C, hidden, abi.DSA3D_F32)
    ws = torch.empty(size + 12 * 256 * 1280 + 1024, dtype=torch.uint8, device="cuda")
    _check_grads(abi.gated_ffn_backward(x, *w, dy, workspace=ws), ref.gated_ffn_backward(x, *w, dy, "silu"))


# ---- rotary positions ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("base", [0.25, 1.0, 2.0])
def test_rotary_bases_near_one(base, backward):
    q = _randn(_gen(3), 60, 2, 64)
    kw = dict(first=0, start=(1000.0, 0.0, -3.5), step=(1.0, 0.5, 2.0), base=base, interleaved=True)
    call = abi.rotary3d_backward if backward else abi.rotary3d
    got, _ = call(q, None, (3, 4, 5), (16, 24, 24), **kw)
    check("q", got, *ref.rotary(q, (3, 4, 5), (16, 24, 24), backward=backward, **kw))


# ---- shards of tensors whose rows are no multiple of 16 bytes -------------------------------------------------
def _shard(t, first):
    """The rows from `first` on, where they lie; the same values in a tensor of their own."""
    return t[first:], t[first:].clone()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [5, 61, 62, 60, 1001])
@pytest.mark.parametrize("first", [1, 2, 3])
def test_layer_norm_of_a_shard_of_odd_rows(C, first, dtype):
    td = DT[dtype]
    g = _gen(C * 4 + first)
    (x, x0), (a, a0), (dy, dy0), (out, _) = (_shard(_randn(g, 50 + first, C, dtype=td), first) for _ in range(4))
    w, b = _randn(g, C), _randn(g, C)
    y, h, stats = abi.layer_norm(x, w, b, add=a, out=out)
    assert y.data_ptr() == out.data_ptr()
    (ry, rh, rs), (ey, es) = ref.layer_norm(x0, w, b, 1e-5, a0)
    check("y", y, ry, ey)
    check("stats", stats, rs, es)
    assert torch.equal(h, rh)
    got = abi.layer_norm_backward(x, w, stats, dy, add=a)
    want, bound = ref.layer_norm_backward(x0, w, stats, dy0, a0)
    for name, o, r, e in zip(("dx", "dw", "db"), got, want, bound):
        check(name, o, r, e)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,hidden", [(61, 131), (62, 130), (60, 132), (60, 64), (64, 131)])
@pytest.mark.parametrize("rows", [1, 140])
def test_gated_ffn_of_shards_of_odd_rows(rows, C, hidden, dtype):
    """Every tensor starts at the second row of a larger one (of 16-byte rows that changes nothing)."""
    td = DT[dtype]
    shards = [_shard(t, 1) for t in (lambda x, w, a, dy: (x, *w, a, dy))(*_ffn_inputs(rows + 1, C, hidden, td, rows))]
    x, wg, wu, wd, a, dy = (t for t, _ in shards)
    w = [_shard(torch.cat([t[:1], t, t[:1]]), 1)[0][:n] for t, n in ((wg, C), (wu, C), (wd, hidden))]
    own = [t.clone() for t in (x, *w, a, dy)]
    out = torch.zeros(rows + 1, C, dtype=td, device="cuda")
    y = abi.gated_ffn(x, *w, add=a, out=out[1:])
    check("y", y, *ref.gated_ffn(own[0], *own[1:4], "silu", own[4]))
    assert not out[0].any()
    got = abi.gated_ffn_backward(x, *w, dy)
    _check_grads(got, ref.gated_ffn_backward(own[0], *own[1:4], own[5], "silu"))


# ---- last: the device's record ----------------------------------------------------------------------------
def test_no_wait_ran_out_in_any_test_before():
    """Nothing that ran since the record was last read (streams, graphs and chunks among it) gave up a wait."""
    torch.cuda.synchronize()
    assert abi.dsa3d_check_device(torch.cuda.current_stream().cuda_stream) == 0
