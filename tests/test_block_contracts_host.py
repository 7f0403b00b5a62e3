"""Contracts of the transformer block's operators that need no GPU: what kernels that start early may
read how, workspace sizes, and refusals."""
import glob
import os
import re

import pytest

from deformable_slide_attention_b200 import abi, build

CSRC = os.path.join(os.path.dirname(build.__file__), "csrc")


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def _kernels():
    """(name, parameters, body, file) of every __global__ function, comments removed."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            src = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s+)?(\w+)\(", src):
            at, depth = m.end(), 1
            while depth:
                depth += {"(": 1, ")": -1}.get(src[at], 0)
                at += 1
            begin = src.index("{", at)
            end, depth = begin + 1, 1
            while depth:
                depth += {"{": 1, "}": -1}.get(src[end], 0)
                end += 1
            yield m.group(1), src[m.end():at - 1], src[begin:end], os.path.basename(path)


def test_early_started_kernels_read_their_predecessors_data_by_ordinary_loads():
    """A kernel that waits for its predecessor inside (prior_kernel_done) is resident while that one still
    writes: its data is not read-only for the kernel's life, which __ldg and const __restrict__ promise, and
    a load under that promise may be moved over the wait."""
    early = [k for k in _kernels() if "prior_kernel_done()" in k[2]]
    assert {k[0] for k in early} >= {"dsa3d_norm_reduce_kernel", "dsa3d_ffn_rows_kernel", "dsa3d_ffn_rows_join_kernel",
                                     "dsa3d_ffn_join_kernel", "dsa3d_ffn_tail_kernel"}
    for name, params, body, path in early:
        after = body[body.index("prior_kernel_done()"):]
        assert "__ldg(" not in after, (path, name)
        assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", params + body), (path, name)


# C, hidden: few-token paths (16-byte rows), odd widths, summed axes long enough to be cut
WORKSPACE_WIDTHS = [(4096, 10944), (2048, 8192), (512, 2048), (64, 136), (61, 131), (1001, 4099)]


def check_workspace_never_shrinks(C, hidden, dtype):
    """A workspace sized once for the longest call is enough for every shorter one."""
    rows = sorted({*range(0, 20), 100, 127, 128, 129, 255, 256, 257, *range(300, 5000, 97), *range(512, 20000, 256),
                   *range(20000, 65536, 2999), 65280, 65535, 65536, 65537, 100000, 1 << 21, (1 << 31) - 1})
    for size in (abi.dsa3d_gated_ffn_workspace_bytes, abi.dsa3d_gated_ffn_backward_workspace_bytes):
        sizes = [size(r, C, hidden, dtype) for r in rows]
        for i in range(1, len(rows)):
            assert sizes[i] >= sizes[i - 1], (size.__name__, rows[i - 1], sizes[i - 1], rows[i], sizes[i])


@pytest.mark.parametrize("dtype", [abi.DSA3D_F32, abi.DSA3D_BF16])
@pytest.mark.parametrize("C,hidden", WORKSPACE_WIDTHS)
def test_feed_forward_workspace_never_shrinks(C, hidden, dtype):
    check_workspace_never_shrinks(C, hidden, dtype)


# ---- refusals (fake, 16-byte aligned addresses: validation fails before any device access) -----------------
INV, UNS = 1, 2
ROT = dict(first=0, rows=24, F=2, Hp=3, Wp=4, heads=2, dh=32, axes=(12, 10, 10), start=(0.0,) * 3, step=(1.0,) * 3,
           base=10000.0, ld=(64,) * 4, p=tuple((i + 1) << 40 for i in range(4)))


def rotary(fn, **kw):
    a = {**ROT, **kw}
    return fn(*a["p"], *a["ld"], a["first"], a["rows"], a["F"], a["Hp"], a["Wp"], a["heads"], a["dh"], a["axes"],
              a["start"], a["step"], a["base"], 1, abi.DSA3D_BF16, 0)


@pytest.mark.parametrize("fn", [abi.dsa3d_rotary3d, abi.dsa3d_rotary3d_backward])
def test_rotary_strides_whose_product_with_the_rows_passes_64_bits_are_refused(fn):
    """Offsets are 64-bit sums: (2^31 - 1) tokens 2^40 elements apart would wrap around them."""
    grid = dict(F=1 << 15, Hp=1 << 8, Wp=255)
    rows = grid["F"] * grid["Hp"] * grid["Wp"]
    for i in range(4):
        ld = [64] * 4
        ld[i] = 1 << 40
        assert rotary(fn, **grid, rows=rows, ld=tuple(ld)) == UNS, i
    assert rotary(fn, **grid, rows=rows, ld=(1 << 33,) * 4) == UNS
    assert rotary(fn, **grid, rows=rows, ld=(64, 1 << 31, 64, 64)) == UNS


@pytest.mark.parametrize("fn", [abi.dsa3d_rotary3d, abi.dsa3d_rotary3d_backward])
def test_rotary_bases_below_one_whose_angles_cannot_be_reduced_are_refused(fn):
    """Below a base of 1 frequencies grow with the pair: base^(-10/12) for the last of 12 dims.  Positions
    times the largest frequency stay within the 2^40 that positions alone do; past it fp64 keeps no angle, and
    frequencies of infinity would give NaN."""
    for base in (1e-300, 5e-324, 1e-30):
        assert rotary(fn, base=base) == INV, base
    far = (2.0 ** 39, 0.0, 0.0)
    assert rotary(fn, base=0.1, start=far) == INV
    assert rotary(fn, base=1e-300, axes=(0, 2, 12)) == INV


def _at(i):
    return (i + 1) << 40


def test_alignment_follows_the_rows():
    """16 bytes, or what the rows of a tensor keep (a shard that starts at any of them): less is refused."""
    p = [_at(i) for i in range(7)]  # x, add, weight, bias, y, h, stats
    for C, dtype, less in ((61, abi.DSA3D_BF16, 1), (62, abi.DSA3D_BF16, 2), (60, abi.DSA3D_BF16, 4),
                           (64, abi.DSA3D_BF16, 8), (61, abi.DSA3D_F32, 2), (62, abi.DSA3D_F32, 4),
                           (64, abi.DSA3D_F32, 8)):
        for i in (0, 1, 4, 5):
            q = list(p)
            q[i] += less
            assert abi.dsa3d_layer_norm(*q, 10, C, 1e-5, dtype, 0) == INV, (C, dtype, i)
        b = [_at(i) for i in range(9)]  # h, weight, stats, dy, add, dx, dw, db, ws
        for i in (0, 3, 4, 5):
            q = list(b)
            q[i] += less
            assert abi.dsa3d_layer_norm_backward(*q, 1 << 30, 10, C, dtype, 0) == INV, (C, dtype, i)
        f = [_at(i) for i in range(7)]  # x, wg, wu, wd, add, y, ws
        for i, widths in ((0, (C, 64)), (3, (C, 64)), (4, (C, 64)), (5, (C, 64)), (1, (64, C)), (2, (64, C)), (6, (64, C))):
            q = list(f)
            q[i] += 8 if i == 6 else less
            assert abi.dsa3d_gated_ffn(*q, 1 << 30, 10, *widths, 0, dtype, 0) == INV, (C, dtype, i)
        f = [_at(i) for i in range(10)]  # x, wg, wu, wd, dy, dx, dwg, dwu, dwd, ws
        for i, widths in ((0, (C, 64)), (3, (C, 64)), (4, (C, 64)), (5, (C, 64)), (8, (C, 64)), (1, (64, C)), (2, (64, C)),
                          (6, (64, C)), (7, (64, C)), (9, (64, C))):
            q = list(f)
            q[i] += 8 if i == 9 else less
            assert abi.dsa3d_gated_ffn_backward(*q, 1 << 30, 10, *widths, 0, dtype, 0) == INV, (C, dtype, i)
