"""The operators of the transformer block around 3D Deformable Slide Attention, as cases to measure:

  layer_norm    y = (h - mean) rstd w + b over the channels of each token, h = x (+ add), and its
                backward pass (dx, the channel sums dw and db);
  rotary3d      the rotation of q and k by their (frame, row, column) positions, and its inverse
                (the backward pass);
  gated_ffn     y = (act(x Wg) * (x Wu)) Wd (+ add), and its backward pass from x and dy alone.

run() computes a case in plain torch operations where ``own`` is false, and through
deformable_slide_attention_b200.abi where it is true.  Sizes are those of the workloads in
deformable_slide_attention_b200/inputs.py (C = heads x dh channels, N = F x H' x W' tokens), with
feed-forward widths of about 8/3 C and 4 C.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases -----------------------------------------------------------------------------------
def _ln(direction, rows, C, dtype, add=False, affine=True):
    return {"op": "layer_norm", "dir": direction, "rows": rows, "C": C, "dtype": dtype, "add": add,
            "affine": affine}


def _rot(direction, F, Hp, Wp, first, rows, heads, dh, at, ay, ax, dtype, interleaved, t0=0.0, step=1.0):
    return {"op": "rotary3d", "dir": direction, "F": F, "Hp": Hp, "Wp": Wp, "first": first, "rows": rows,
            "heads": heads, "dh": dh, "at": at, "ay": ay, "ax": ax, "dtype": dtype,
            "interleaved": interleaved, "t0": t0, "step": step}


def _ffn(direction, rows, C, hidden, dtype, act="silu", add=False):
    return {"op": "gated_ffn", "dir": direction, "rows": rows, "C": C, "hidden": hidden, "dtype": dtype,
            "act": act, "add": add}


def listed():
    return [
        # the tiny fp32 workload's tokens and channels: the call's latency
        {"name": "ln-fwd-tiny", **_ln("fwd", 256, 64, "f32")},
        # a 720p clip between two sub-layers: the residual sum, then its norm
        {"name": "ln-fwd-720p-add", **_ln("fwd", 115200, 2048, "bf16", add=True)},
        # the same place in the backward pass: dx joins the residual branch's gradient
        {"name": "ln-bwd-720p-add", **_ln("bwd", 115200, 2048, "bf16", add=True)},
        # a ragged token count and an odd channel count, which no wide load fits
        {"name": "ln-bwd-odd", **_ln("bwd", 4099, 1001, "f32")},
        # one new token of the long 1080p video, past its 256 frames' start: the call's latency
        {"name": "rotary-fwd-token", **_rot("fwd", 256, 68, 120, 2088959, 1, 32, 128, 44, 42, 42, "bf16",
                                            True, t0=4096.0)},
        # a 720p clip's q and k, read out of the packed q, k, v projection
        {"name": "rotary-fwd-720p", **_rot("fwd", 32, 45, 80, 0, 115200, 16, 128, 44, 42, 42, "bf16", True)},
        # one rank's share of the 1080p tokens (a shard that starts inside a frame), dq and dk back,
        # pairs split in halves, a part of the head left unrotated, positions at half resolution
        {"name": "rotary-bwd-1080p-shard", **_rot("bwd", 256, 68, 120, 65280 + 17, 65273, 32, 128, 32, 40, 40,
                                                  "bf16", False, step=0.5)},
        # one token through the 1080p model's block: its three weights are read once
        {"name": "ffn-fwd-token", **_ffn("fwd", 1, 4096, 10944, "bf16", add=True)},
        # four frames of 720p
        {"name": "ffn-fwd-720p", **_ffn("fwd", 14400, 2048, 8192, "bf16", add=True)},
        # the small workload's tokens, trained
        {"name": "ffn-bwd-small", **_ffn("bwd", 16384, 512, 2048, "bf16", act="gelu")},
        # four frames of 720p, trained, with a hidden width off the tile sizes
        {"name": "ffn-bwd-720p", **_ffn("bwd", 14400, 2048, 5464, "bf16")},
        # a frame of fp32 tokens, trained, sizes that no tile and no wide load fits
        {"name": "ffn-bwd-f32-odd", **_ffn("bwd", 1001, 258, 685, "f32")},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size over the logarithm of [lo, hi]: any, a multiple of 8 or a multiple of 64."""
    n = _log(rng, lo, hi)
    step = rng.choice([1, 8, 64])
    return min(hi, max(lo, n // step * step))


def draw(rng):
    kind = rng.choice(["layer_norm", "rotary3d", "gated_ffn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    direction = rng.choice(["fwd", "bwd"])
    if kind == "layer_norm":
        C = _size(rng, 8, 8192)
        rows = _log(rng, 1, max(2, min(115200, 115200 * 1024 // C)))
        return _ln(direction, rows, C, dtype, add=rng.random() < 0.5, affine=rng.random() < 0.8)
    if kind == "rotary3d":
        dh = rng.choice([32, 64, 128])
        heads = rng.randint(1, 32)
        F, Hp, Wp = _log(rng, 1, 256), _log(rng, 1, 68), _log(rng, 1, 120)
        N = F * Hp * Wp
        first = rng.randint(0, N - 1)
        rows = _log(rng, 1, max(1, min(N - first, 65280 * 2048 // (heads * dh))))
        ax = 2 * rng.randint(0, dh // 6)
        ay = 2 * rng.randint(0, dh // 6)
        at = 2 * rng.randint(1, dh // 2 - (ax + ay) // 2)
        if rng.random() < 0.5:
            at = dh - ax - ay
        return _rot(direction, F, Hp, Wp, first, rows, heads, dh, at, ay, ax, dtype, rng.random() < 0.5,
                    t0=float(rng.choice([0, 0, 1000, 100000])), step=rng.choice([1.0, 1.0, 0.5]))
    if dtype == "f32":
        C, hidden = _size(rng, 16, 512), _size(rng, 32, 2048)
        rows = _log(rng, 1, max(2, min(4096, (1 << 31) // (C * hidden))))
    else:
        C, hidden = _size(rng, 16, 4096), _size(rng, 32, 10944)
        rows = _log(rng, 1, max(2, min(16384, 14400 * 2048 * 4096 // (C * hidden))))
    return _ffn(direction, rows, C, hidden, dtype, act=rng.choice(["silu", "gelu"]), add=rng.random() < 0.5)


# ---- what a user has in hand -----------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 2654435761 % (1 << 62) + 1)
    td = _DT[case["dtype"]]

    def normal(*shape, dtype=td, std=1.0, mean=0.0):
        return torch.empty(shape, device=dev).normal_(mean, std, generator=gen).to(dtype)

    s = dict(case)
    if case["op"] == "layer_norm":
        rows, C = case["rows"], case["C"]
        # a residual stream: tokens of different scale and mean
        x = normal(rows, C) * (0.5 + 2 * torch.rand(rows, 1, device=dev, generator=gen)) + normal(rows, 1)
        s["x"] = x.to(td)
        del x
        s["weight"] = normal(C, dtype=torch.float32, std=0.2, mean=1.0) if case["affine"] else None
        s["bias"] = normal(C, dtype=torch.float32, std=0.2) if case["affine"] else None
        s["addend"] = normal(rows, C) if case["add"] else None
        if case["dir"] == "bwd":
            s["dy"] = normal(rows, C)
            x32 = s["x"].double() if rows * C < (1 << 24) else s["x"].float()
            mean = x32.mean(1)
            rstd = torch.rsqrt((x32 - mean[:, None]).square_().mean(1) + 1e-5)
            s["stats"] = torch.stack([mean, rstd]).float()
    elif case["op"] == "rotary3d":
        rows, heads, dh = case["rows"], case["heads"], case["dh"]
        if case["dir"] == "fwd":  # q and k where a packed projection wrote them
            qkv = normal(rows, 3, heads, dh)
            s["q"], s["k"] = qkv[:, 0], qkv[:, 1]
        else:  # the attention's dq and dk
            s["q"], s["k"] = normal(rows, heads, dh), normal(rows, heads, dh)
    else:
        rows, C, hidden = case["rows"], case["C"], case["hidden"]
        s["x"] = normal(rows, C)
        s["wg"] = normal(C, hidden, std=C ** -0.5)
        s["wu"] = normal(C, hidden, std=C ** -0.5)
        s["wd"] = normal(hidden, C, std=hidden ** -0.5)
        s["addend"] = normal(rows, C) if case["add"] and case["dir"] == "fwd" else None
        if case["dir"] == "bwd":
            s["dy"] = normal(rows, C)
    return s


# ---- one pass ----------------------------------------------------------------------------------------
def run(s):
    if own:
        return _RUN_OWN[s["op"], s["dir"]](s)
    return _RUN_PLAIN[s["op"], s["dir"]](s)


def _own_ln_fwd(s):
    from deformable_slide_attention_b200 import abi
    y, h, stats = abi.layer_norm(s["x"], s["weight"], s["bias"], eps=1e-5, add=s["addend"])
    return (y, stats) if s["addend"] is None else (y, stats, h)


def _own_ln_bwd(s):
    from deformable_slide_attention_b200 import abi
    return abi.layer_norm_backward(s["x"], s["weight"], s["stats"], s["dy"], add=s["addend"])


def _own_rot(s, call):
    return call(s["q"], s["k"], (s["F"], s["Hp"], s["Wp"]), (s["at"], s["ay"], s["ax"]), first=s["first"],
                start=(s["t0"], 0.0, 0.0), step=(1.0, s["step"], s["step"]), base=10000.0,
                interleaved=s["interleaved"])


def _own_rot_fwd(s):
    from deformable_slide_attention_b200 import abi
    return _own_rot(s, abi.rotary3d)


def _own_rot_bwd(s):
    from deformable_slide_attention_b200 import abi
    return _own_rot(s, abi.rotary3d_backward)


def _own_ffn_fwd(s):
    from deformable_slide_attention_b200 import abi
    return abi.gated_ffn(s["x"], s["wg"], s["wu"], s["wd"], activation=s["act"], add=s["addend"])


def _own_ffn_bwd(s):
    from deformable_slide_attention_b200 import abi
    return abi.gated_ffn_backward(s["x"], s["wg"], s["wu"], s["wd"], s["dy"], activation=s["act"])


def _plain_ln_fwd(s):
    x = s["x"]
    h = x if s["addend"] is None else (x.float() + s["addend"].float()).to(x.dtype)
    h32 = h.float()
    mean = h32.mean(1, keepdim=True)
    c = h32 - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5)
    y = c * rstd
    if s["weight"] is not None:
        y = y * s["weight"] + s["bias"]
    out = (y.to(x.dtype), torch.stack([mean[:, 0], rstd[:, 0]]))
    return out if s["addend"] is None else (*out, h)


def _plain_ln_bwd(s):
    mean, rstd = s["stats"][0][:, None], s["stats"][1][:, None]
    dy = s["dy"].float()
    xhat = (s["x"].float() - mean) * rstd
    g = dy if s["weight"] is None else dy * s["weight"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if s["addend"] is not None:
        dx = dx + s["addend"].float()
    dx = dx.to(s["x"].dtype)
    if s["weight"] is None:
        return dx, None, None
    return dx, (dy * xhat).sum(0), dy.sum(0)


def _angles(s, dev):
    """Rotation angles [rows][pairs] in 64 bits: position x base^(-2j / axis size)."""
    n = s["first"] + torch.arange(s["rows"], device=dev)
    pos = (s["t0"] + (n // (s["Hp"] * s["Wp"])).double(),
           s["step"] * (n // s["Wp"] % s["Hp"]).double(),
           s["step"] * (n % s["Wp"]).double())
    freq = [10000.0 ** (-2.0 * torch.arange(a // 2, device=dev, dtype=torch.float64) / max(a, 1))
            for a in (s["at"], s["ay"], s["ax"])]
    return torch.cat([p[:, None] * f for p, f in zip(pos, freq)], 1)


def _plain_rot(s, sign):
    ang = _angles(s, s["q"].device)
    cos, sin = torch.cos(ang).float()[:, None], (sign * torch.sin(ang)).float()[:, None]
    R = s["at"] + s["ay"] + s["ax"]

    def rotate(x):
        x32 = x.float()
        if s["interleaved"]:
            a, b = x32[..., 0:R:2], x32[..., 1:R:2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = x32[..., :R // 2], x32[..., R // 2:R]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([r, x32[..., R:]], -1).to(x.dtype)

    return rotate(s["q"]), rotate(s["k"])


def _act(g, name):
    """The activation and its derivative."""
    if name == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    cdf = 0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5


def _plain_ffn_fwd(s):
    x = s["x"].float()
    a, _ = _act(x @ s["wg"].float(), s["act"])
    y = (a * (x @ s["wu"].float())) @ s["wd"].float()
    if s["addend"] is not None:
        y = y + s["addend"].float()
    return y.to(s["x"].dtype)


def _plain_ffn_bwd(s):
    td = s["x"].dtype
    x, dy = s["x"].float(), s["dy"].float()
    wg, wu, wd = s["wg"].float(), s["wu"].float(), s["wd"].float()
    g, u = x @ wg, x @ wu
    a, da = _act(g, s["act"])
    dh = dy @ wd.t()
    dg, du = dh * u * da, dh * a
    dx = dg @ wg.t() + du @ wu.t()
    return dx.to(td), (x.t() @ dg).to(td), (x.t() @ du).to(td), ((a * u).t() @ dy).to(td)


_RUN_OWN = {("layer_norm", "fwd"): _own_ln_fwd, ("layer_norm", "bwd"): _own_ln_bwd,
            ("rotary3d", "fwd"): _own_rot_fwd, ("rotary3d", "bwd"): _own_rot_bwd,
            ("gated_ffn", "fwd"): _own_ffn_fwd, ("gated_ffn", "bwd"): _own_ffn_bwd}
_RUN_PLAIN = {("layer_norm", "fwd"): _plain_ln_fwd, ("layer_norm", "bwd"): _plain_ln_bwd,
              ("rotary3d", "fwd"): lambda s: _plain_rot(s, 1.0),
              ("rotary3d", "bwd"): lambda s: _plain_rot(s, -1.0),
              ("gated_ffn", "fwd"): _plain_ffn_fwd, ("gated_ffn", "bwd"): _plain_ffn_bwd}


# ---- what a pass cannot do without ---------------------------------------------------------------------
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    rows = case["rows"]
    if case["op"] == "layer_norm":
        C = case["C"]
        if case["dir"] == "fwd":  # x, y (and the addend and the sum), weights, statistics
            return {"bytes": (4 if case["add"] else 2) * rows * C * es + 8 * C * case["affine"] + 8 * rows,
                    "flops": 8 * rows * C}
        # x, dy, dx (and the addend), weight, dw, db, statistics
        return {"bytes": (4 if case["add"] else 3) * rows * C * es + 12 * C * case["affine"] + 8 * rows,
                "flops": (14 if case["affine"] else 10) * rows * C}
    if case["op"] == "rotary3d":  # q and k, in and out
        R = case["at"] + case["ay"] + case["ax"]
        return {"bytes": 4 * rows * case["heads"] * case["dh"] * es, "flops": 6 * rows * case["heads"] * R}
    C, hidden = case["C"], case["hidden"]
    if case["dir"] == "fwd":  # x, y (and the addend), three weights; three products
        return {"bytes": ((3 if case["add"] else 2) * rows * C + 3 * C * hidden) * es,
                "flops": 6 * rows * C * hidden}
    # x, dy, dx, three weights and their gradients; gate, up, dh, two for dx, three weight gradients
    return {"bytes": (3 * rows * C + 6 * C * hidden) * es, "flops": 16 * rows * C * hidden}


# ---- from the definition, in 64 bits ---------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer_norm":
        return _exact_ln(s)
    if case["op"] == "rotary3d":
        return _exact_rot(s)
    if case["rows"] * case["C"] * case["hidden"] > (1 << 34):
        return None  # minutes of 64-bit products
    return _exact_ffn(s)


def _exact_ln(s):
    td, C = s["x"].dtype, s["C"]
    if s["dir"] == "fwd":
        h = s["x"].double()
        if s["addend"] is not None:
            h = (h + s["addend"].double()).to(td).double()  # the sum is kept in the I/O type
        m1 = h.sum(1) / C
        h2 = h - m1[:, None]
        rstd = (h2.square().sum(1) / C + 1e-5) ** -0.5
        y = torch.einsum("nc,n->nc", h2, rstd)
        if s["weight"] is not None:
            y.mul_(s["weight"].double()).add_(s["bias"].double())
        out = (y, torch.stack([m1, rstd]))
        return out if s["addend"] is None else (*out, h)
    # with the given statistics, dx_i = sum_j dy_j w_j d y_j / d x_i of the normalised row
    mean, rstd = s["stats"].double()
    xhat = s["x"].double().sub_(mean[:, None]).mul_(rstd[:, None])
    dy = s["dy"].double()
    dw = torch.einsum("nc,nc->c", dy, xhat) if s["affine"] else None
    db = dy.sum(0) if s["affine"] else None
    if s["affine"]:
        dy.mul_(s["weight"].double())
    along = torch.einsum("nc,nc->n", dy, xhat) / C
    level = torch.einsum("nc->n", dy) / C
    dx = dy.sub_(level[:, None]).sub_(xhat.mul_(along[:, None])).mul_(rstd[:, None])
    if s["addend"] is not None:
        dx.add_(s["addend"].double())
    return dx, dw, db


def _exact_rot(s):
    """The rotation as a product of complex numbers, pair by pair."""
    dev, R = s["q"].device, s["at"] + s["ay"] + s["ax"]
    n = torch.arange(s["first"], s["first"] + s["rows"], device=dev, dtype=torch.int64)
    x = n % s["Wp"]
    y = torch.div(n - x, s["Wp"], rounding_mode="floor") % s["Hp"]
    t = torch.div(n, s["Wp"] * s["Hp"], rounding_mode="floor")
    parts = []
    for size, p in ((s["at"], s["t0"] + t.double()), (s["ay"], s["step"] * y.double()),
                    (s["ax"], s["step"] * x.double())):
        j = torch.arange(0, size, 2, device=dev, dtype=torch.float64)
        parts.append(torch.outer(p, torch.exp(-j / max(size, 1) * math.log(10000.0))))
    theta = torch.cat(parts, -1)
    turn = torch.polar(torch.ones_like(theta), theta if s["dir"] == "fwd" else -theta)[:, None]

    def rotate(v):
        w = v.double()
        if s["interleaved"]:
            z = torch.view_as_complex(w[..., :R].reshape(*w.shape[:-1], R // 2, 2).contiguous()) * turn
            w = torch.cat([torch.view_as_real(z).reshape(*w.shape[:-1], R), w[..., R:]], -1)
        else:
            z = torch.complex(w[..., :R // 2].contiguous(), w[..., R // 2:R].contiguous()) * turn
            w = torch.cat([z.real, z.imag, w[..., R:]], -1)
        return w

    return rotate(s["q"]), rotate(s["k"])


def _exact_ffn(s):
    """The formula in 64 bits; its gradients by automatic differentiation."""
    train = s["dir"] == "bwd"
    v = [s[k].double().requires_grad_(train) for k in ("x", "wg", "wu", "wd")]
    g = v[0].mm(v[1])
    if s["act"] == "silu":
        a = g * torch.sigmoid(g)
    else:
        a = 0.5 * g * torch.erfc(-g / math.sqrt(2.0))
    y = (a * v[0].mm(v[2])).mm(v[3])
    if not train:
        return y if s["addend"] is None else y + s["addend"].double()
    return torch.autograd.grad(y, v, s["dy"].double())
