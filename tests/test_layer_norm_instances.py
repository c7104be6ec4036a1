"""Every instance of the layer norm's kernels: that the rule on width and types
reaches each one in the library and that the widths below run each (on the CPU),
and those widths against the formula in 64 bits, by few rows and by more rows
than the launches take at once.

Bounds: of r, y, dx and dresidual as in test_layer_norm_gpu.py.  The weights'
gradients, which here are sums over thousands of rows: an element passes at most
84 additions (9 rows of a lane, 3 lane groups, 8 waves, 32 partial rows of a
thread, 32 of a workgroup), each off by 2^-24 of the sum of absolute values, and
h is off by at most 44 * 2^-24 of 1 + |h| (half of the 46 additions of the
variance's sum, the roundings of r, of its difference from a mean that lies
below the deviation here, and of three products): 128 * 2^-24 of the sum of
|dy| (1 + |h|).
"""
import re
import subprocess

import pytest
import torch

import model_reference as ref
import selective_state_space_30_amd as ssm
from test_layer_norm_gpu import DEV, TYPES

BF16, F32 = torch.bfloat16, torch.float32
NAMES = {BF16: "unsigned short", F32: "float"}


def shape_of(dim, types, backward):
    """Lanes of a row's group, pieces a lane, threads, whether they fill the row
    (the rule of ssm_layer_norm.hip)."""
    n = 4 if types == "f32" else 8
    if types == "f32":
        alone, shared = (7, 5) if backward else (8, 6)
    else:
        alone, shared = 4, 2 if backward and types != "bf16" else 3
    pieces = -(-dim // n)
    per = lambda lanes: -(-pieces // lanes)  # noqa: E731
    lanes = next((k for k in (64, 32, 16, 8)
                  if pieces % k == 0 and dim % n == 0 and per(k) <= alone), 0)
    if not lanes:
        lanes = 8
        while lanes < 64 and per(lanes) > 1:
            lanes *= 2
        if per(lanes) > alone:
            while lanes < 512 and per(lanes) > shared:
                lanes *= 2
    return n, lanes, per(lanes), 256 if lanes <= 64 else lanes, per(lanes) * lanes * n == dim


def instance(dim, types, backward):
    n, _, per, threads, whole = shape_of(dim, types, backward)
    return (types, "bwd" if backward else "fwd", n, per, whole,
            (256 if threads <= 256 else 512) if backward else 0)


def built():
    out = subprocess.run(["nm", "-C", ssm.LIB_PATH], stdout=subprocess.PIPE, text=True,
                         check=True).stdout
    kinds = {tuple(NAMES[t] for t in k): name for name, k in TYPES.items()}
    found = set()
    for which, args in re.findall(r"layer_norm_(fwd|bwd)_kernel<([^>]*)>", out):
        t = [a.strip() for a in args.split(",")]
        found.add((kinds[tuple(t[:3])], which, int(t[3]), int(t[4]), t[5] == "true",
                   int(t[6]) if which == "bwd" else 0))
    return found


# widths: of 8 to 64 lanes and of 2, 4 and 8 waves, filled and not, at each
# number of pieces
WIDE = [40, 64, 100, 128, 192, 250, 256, 384, 700, 1024, 1100, 1536, 1800, 2048, 2560, 3500, 4096,
        5000, 6144, 7001, 8192, 9001, 12288, 13000, 16384]
WIDTHS = {"bf16": WIDE, "wide": WIDE, "down": WIDE,
          "f32": [9, 32, 40, 64, 96, 128, 160, 192, 224, 256, 300, 320, 384, 448, 512, 600, 640,
                  768, 896, 900, 1024, 1100, 1280, 1400, 1536, 1700, 1792, 1900, 2048, 2300, 2560,
                  2700, 3500, 4096, 5120, 5500, 6144, 7001, 8192, 9001, 10240, 11000, 12288, 13000,
                  14336, 15000, 16384]}


def rows_for(types, dim):
    """More rows than the forward pass takes at once (4 waves a SIMD), so more
    than the backward pass does; the last round is not full."""
    _, lanes, _, threads, _ = shape_of(dim, types, False)
    most = 256 * 1024 // threads * (threads // lanes)
    return most + most // 5 + 1


CASES = [(t, rows, dim) for t in TYPES for dim in WIDTHS[t] for rows in (5, rows_for(t, dim))]


def reachable():
    return {instance(dim, t, b) for t in TYPES for b in (False, True) for dim in range(1, 16385)}


def test_each_instance_is_reached():
    assert built() == reachable()


def test_each_instance_has_a_case():
    assert {instance(dim, t, b) for t, _, dim in CASES for b in (False, True)} == reachable()


def make(types, rows, dim):
    xt, rt, yt = TYPES[types]
    gen = torch.Generator(device=DEV)
    gen.manual_seed(rows + 3 * dim)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    inp = {"x": (1.5 * r(rows, dim)).to(xt), "residual": (2 * r(rows, dim) + 0.7).to(rt),
           "weight": 1 + 0.2 * r(dim), "bias": r(dim)}
    return inp, r(rows, dim).to(rt), r(rows, dim).to(yt)


def check(got, want, what):
    tol = 2.0 ** -8 + 1e-5 if got.dtype == BF16 else 2e-5
    assert got.shape == want.shape, what
    over = (got.double() - want).abs() / (want.abs() + want.pow(2).mean().sqrt())
    assert torch.isfinite(got).all() and over.max() <= tol, "%s: %g" % (what, over.max())


def weights_bound(inp, dy):
    r = inp["x"].double() + inp["residual"].double()
    h = (r - r.mean(-1, keepdim=True)) * (r.var(-1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    return 128 * 2.0 ** -24 * (dy.double().abs() * (1 + h.abs())).sum(0)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s_%dx%d" % c)
def test_layer_norm(case):
    types, rows, dim = case
    inp, dr, dy = make(types, rows, dim)
    r, y = ssm.ssm_layer_norm_fwd(**inp, dtype=TYPES[types][2])
    got = ssm.ssm_layer_norm_bwd(**inp, dr=dr, dy=dy)
    wr, wy = ref.layer_norm(**inp)
    want = ref.layer_norm_gradients(**inp, dr=dr, dy=dy)
    check(r, wr, "r")
    check(y, wy, "y")
    bound = weights_bound(inp, dy)
    assert set(got) == set(want)
    for n in want:
        if n in ("dweight", "dbias"):
            over = (got[n].double() - want[n]).abs() - bound - 2.0 ** -24 * want[n].abs()
            assert over.max() <= 0, "%s: %g over the bound" % (n, over.max())
        else:
            check(got[n], want[n], n)
