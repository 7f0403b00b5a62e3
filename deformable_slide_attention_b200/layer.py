"""The 3D-DSA layer of MegaSlide-DiT (arXiv 2607.22696, the 3D-DSA definition, Eq. 1) composed
from the library's calls:

    offsets = OffsetNet(X)                           (depthwise conv + pointwise layer)
    out     = DWConv3D(X) + Attention(q, k, v, offsets)

forward() returns out [N][heads][dh] and a context; backward() takes dO and returns the
gradients with respect to X (the offset network's and the convolution's parts, summed), q, k, v
and every weight.  q, k and v come from the caller (the paper's W_q, W_k, W_v projections of X,
like the layer norm and residual around the operator, are outside the operator), so their
gradients are returned for the caller to carry back through those projections.  Every step runs
in the library's CUDA kernels; this module only orders the calls and adds the two dX parts.

With rotary=Rotary(...), forward() first turns q and k by their tokens' (frame, row, column)
positions, and backward() turns dq and dk back.

feed_forward() and feed_forward_backward() are the block's other sub-layer:

    h = x (+ add)        y = h + FFN(LayerNorm(h))        FFN(n) = (act(n Wg) * (n Wu)) Wd
"""
from __future__ import annotations

import dataclasses

from . import abi


@dataclasses.dataclass
class LayerWeights:
    """fp32 weights: conv_weight [C][kt][kh][kw] and conv_bias [C] (the DWConv3D term);
    off_dw_weight [C][kt][kh][kw], off_dw_bias [C], off_pw_weight [C][heads*(K)*3] and
    off_pw_bias [heads*(K)*3] (the offset network; K = kt*kh*kw with per-tap offsets)."""
    conv_weight: object
    conv_bias: object
    off_dw_weight: object
    off_dw_bias: object
    off_pw_weight: object
    off_pw_bias: object


@dataclasses.dataclass(frozen=True)
class Rotary:
    """Rotary positions of q and k (abi.rotary3d): head dims per axis (frames, rows, columns), the
    positions' start and step per axis, the base of the frequencies and the pairing of dims."""
    axes: tuple
    start: tuple = (0.0, 0.0, 0.0)
    step: tuple = (1.0, 1.0, 1.0)
    base: float = 10000.0
    interleaved: bool = True

    def _args(self):
        return dict(start=self.start, step=self.step, base=self.base, interleaved=self.interleaved)


@dataclasses.dataclass
class FeedForwardWeights:
    """norm_weight and norm_bias [C] fp32 (None: a norm without them); gate_weight, up_weight [C][hidden]
    and down_weight [hidden][C] in the activations' dtype."""
    norm_weight: object
    norm_bias: object
    gate_weight: object
    up_weight: object
    down_weight: object


def forward(x, q, k, v, wts: LayerWeights, dims, window, per_tap=False, ops=abi, rotary=None):
    """x [N][C] with C = heads*dh; q, k, v [N][heads][dh].  Returns (out [N][heads][dh], ctx).
    With rotary (a Rotary), q and k are turned by their positions first and may then be views of a
    packed projection (strided tokens)."""
    heads = q.shape[1]
    if rotary is not None:
        q, k = ops.rotary3d(q, k, dims, rotary.axes, **rotary._args())
    offsets = ops.offset_head(x, wts.off_dw_weight, wts.off_dw_bias, wts.off_pw_weight,
                              wts.off_pw_bias, dims, heads, per_tap=per_tap)
    fwd = ops.forward_taps if per_tap else ops.forward
    out, lse = fwd(q, k, v, offsets, dims, window)
    flat = out.view(out.shape[0], -1)
    ops.dwconv3d(x, wts.conv_weight, wts.conv_bias, dims, add=flat, out=flat)  # out += DWConv3D(x)
    return out, (x, q, k, v, offsets, lse, wts, tuple(dims), tuple(window), per_tap, rotary)


def backward(ctx, dout, ops=abi):
    """dout [N][heads][dh] -> dict of gradients: x, q, k, v, conv_weight, conv_bias,
    off_dw_weight, off_dw_bias, off_pw_weight, off_pw_bias (and offsets, the attention's)."""
    x, q, k, v, offsets, lse, wts, dims, window, per_tap, rotary = ctx
    heads = q.shape[1]
    bwd = ops.backward_taps if per_tap else ops.backward
    dq, dk, dv, doff = bwd(q, k, v, offsets, lse, dout, dims, window)
    if rotary is not None:
        dq, dk = ops.rotary3d_backward(dq, dk, dims, rotary.axes, out=(dq, dk), **rotary._args())
    dx_off, d_odw, d_odb, d_opw, d_opb = ops.offset_head_backward(
        x, wts.off_dw_weight, wts.off_dw_bias, wts.off_pw_weight, doff, dims, heads, per_tap=per_tap)
    dx_conv, d_cw, d_cb = ops.dwconv3d_backward(x, wts.conv_weight, dout.view(dout.shape[0], -1), dims)
    dx = (dx_off.float() + dx_conv.float()).to(x.dtype)
    return {"x": dx, "q": dq, "k": dk, "v": dv, "offsets": doff, "conv_weight": d_cw,
            "conv_bias": d_cb, "off_dw_weight": d_odw, "off_dw_bias": d_odb,
            "off_pw_weight": d_opw, "off_pw_bias": d_opb}


def feed_forward(x, wts: FeedForwardWeights, eps=1e-5, activation="silu", add=None, ops=abi):
    """h = x (+ add, another branch's output to be summed first); y = h + FFN(LayerNorm(h)).
    x [N][C].  Returns (y [N][C], ctx)."""
    n, h, stats = ops.layer_norm(x, wts.norm_weight, wts.norm_bias, eps, add=add)
    y = ops.gated_ffn(n, wts.gate_weight, wts.up_weight, wts.down_weight, activation=activation, add=h)
    return y, (h, n, stats, wts, activation)


def feed_forward_backward(ctx, dy, ops=abi):
    """dy [N][C] -> dict of gradients: x (that of h: of x and of add alike), norm_weight, norm_bias,
    gate_weight, up_weight, down_weight."""
    h, n, stats, wts, activation = ctx
    dn, d_gate, d_up, d_down = ops.gated_ffn_backward(n, wts.gate_weight, wts.up_weight, wts.down_weight, dy,
                                                      activation=activation)
    dx, d_nw, d_nb = ops.layer_norm_backward(h, wts.norm_weight, stats, dn, add=dy)
    return {"x": dx, "norm_weight": d_nw, "norm_bias": d_nb, "gate_weight": d_gate, "up_weight": d_up,
            "down_weight": d_down}
