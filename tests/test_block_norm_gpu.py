"""The block norm (ssm_block_norm_fwd, _bwd) against its formula in 64 bits.

Tolerances on |g - r| / (|r| + rms(r)): an output is rounded once, 2^-8 of
|r| in bf16 (half of torch.finfo's eps), and everything before is fp32 with a handful of roundings and
sums of up to 16384 terms (tree and strided sums: below 64 * 2^-24 = 4e-6
relative to the root sum of squares).  bf16: 2^-8 + 1e-5; fp32, and the
weights' gradients, which are sums over rows of such terms: 2e-5.
"""
import pytest
import torch

import linattn_reference as ref
import selective_state_space_30_amd as ssm
from parity_metrics import report, scaled_max_err

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("x", "w_post", "z", "scale", "residual", "w_pre")


def check(got, want, what):
    tol = 2.0 ** -8 + 1e-5 if got.dtype == BF16 else 2e-5
    assert scaled_max_err(got, want) <= tol, "%s: %s" % (what, report(got, want))


def make(dtype, rows, dim, parts, wide=False, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    all_ = {"x": (1.5 * r(rows, dim)).to(dtype), "w_post": 1 + 0.2 * r(dim),
            "z": r(rows, dim).to(dtype), "scale": 0.5 + 0.1 * r(dim),
            "residual": (2 * r(rows, dim)).to(F32 if wide else dtype), "w_pre": 1 + 0.2 * r(dim)}
    inp = {n: (t if n == "x" or n in parts else None) for n, t in all_.items()}
    dr = r(rows, dim).to(F32 if wide and "residual" in parts else dtype)
    dy = r(rows, dim).to(dtype) if "w_pre" in parts else None
    return inp, dr, dy


ALL = ("w_post", "z", "scale", "residual", "w_pre")
CASES = [
    # dtype, rows, dim, groups, parts, wide
    (BF16, 1, 64, 1, ALL, False),
    (BF16, 5, 2560, 1, ("residual", "w_pre"), False),
    (BF16, 3, 5120, 80, ("w_post", "z"), False),
    (BF16, 7, 768, 1, ALL, True),
    (BF16, 4, 1536, 24, ALL, True),
    (BF16, 3, 1000, 5, ALL, False),       # parts of 200: no power of two of pieces
    (BF16, 2, 960, 80, ALL, False),       # parts of 12 elements: single ones
    (BF16, 2, 1537, 1, ALL, False),       # odd width
    (BF16, 2, 1539, 3, ALL, True),
    (BF16, 2, 8192, 1, ALL, True),
    (BF16, 2, 16384, 1, ALL, False),
    (BF16, 2, 8192, 2, ALL, False),
    (BF16, 1, 1, 1, ALL, False),
    (BF16, 3, 130, 130, ALL, False),      # parts of one element
    (BF16, 9, 100, 1, (), False),         # nothing: r = x
    (BF16, 9, 100, 1, ("z",), False),
    (F32, 1, 64, 1, ALL, False),
    (F32, 1030, 192, 1, ALL, False),      # more rows than workgroups keep sums
    (F32, 5, 2560, 20, ALL, False),
    (F32, 2, 1537, 1, ("w_post", "residual", "w_pre"), False),
    (F32, 2, 8190, 3, ALL, False),
    (F32, 2, 16384, 1, ALL, False),
    (F32, 2, 16383, 1, ALL, False),
    (F32, 3, 300, 1, ("scale", "residual"), False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s_%dx%d_g%d_%s_%d" % (
    "bf16" if c[0] == BF16 else "f32", c[1], c[2], c[3], "".join(p[0] + p[-1] for p in c[4]), c[5]))
def test_block_norm(case):
    dtype, rows, dim, groups, parts, wide = case
    inp, dr, dy = make(dtype, rows, dim, parts, wide, seed=rows + dim)
    d = {n: None if t is None else t.to(DEV) for n, t in inp.items()}
    h = {n: None if t is None else t.double() for n, t in inp.items()}
    r, y = ssm.ssm_block_norm_fwd(**d, groups=groups)
    wr, wy = ref.block_norm(**h, groups=groups)
    assert r.dtype == (dtype if d["residual"] is None else d["residual"].dtype)
    check(r, wr, "r")
    assert (y is None) == (wy is None)
    if y is not None:
        check(y, wy, "y")
    got = ssm.ssm_block_norm_bwd(**d, groups=groups, dr=dr.to(DEV),
                                 dy=None if dy is None else dy.to(DEV))
    want = ref.block_norm_gradients(h, groups, 1e-5, dr.double(),
                                    None if dy is None else dy.double())
    assert set(got) == set(want)
    for n in want:
        check(got[n], want[n], n)


def test_without_gradient_of_r():
    inp, _, dy = make(BF16, 6, 256, ALL, seed=3)
    d = {n: t.to(DEV) for n, t in inp.items()}
    got = ssm.ssm_block_norm_bwd(**d, dy=dy.to(DEV))
    want = ref.block_norm_gradients({n: t.double() for n, t in inp.items()}, 1, 1e-5, None,
                                    dy.double())
    for n in want:
        check(got[n], want[n], n)


def test_rows_of_zeros_and_large_values():
    """A row of zeros divides by sqrt(eps); large and small rows keep their
    scale."""
    inp, dr, dy = make(F32, 4, 320, ALL, seed=5)
    inp["x"][0] = 0
    inp["residual"][0] = 0
    inp["x"][1] *= 1e15
    inp["x"][2] *= 1e-12
    d = {n: t.to(DEV) for n, t in inp.items()}
    r, y = ssm.ssm_block_norm_fwd(**d, groups=5)
    wr, wy = ref.block_norm(**{n: t.double() for n, t in inp.items()}, groups=5)
    for i in range(4):
        check(r[i], wr[i], "r of row %d" % i)
        check(y[i], wy[i], "y of row %d" % i)
    got = ssm.ssm_block_norm_bwd(**d, groups=5, dr=dr.to(DEV), dy=dy.to(DEV))
    want = ref.block_norm_gradients({n: t.double() for n, t in inp.items()}, 5, 1e-5,
                                    dr.double(), dy.double())
    for i in range(4):
        check(got["dx"][i], want["dx"][i], "dx of row %d" % i)


def test_slices_in_place_and_leading_dimensions():
    gen = torch.Generator().manual_seed(8)
    for off in (0, 3):
        wide = torch.randn(2, 3, off + 2 * 512 + 5, generator=gen).to(BF16).to(DEV)
        x, z = wide[..., off:off + 512], wide[..., off + 512:off + 1024]
        res = torch.randn(2, 3, 512, generator=gen).to(DEV)
        w = torch.rand(512, generator=gen).to(DEV)
        r, y = ssm.ssm_block_norm_fwd(x, w_post=w, z=z, residual=res, w_pre=w, groups=8)
        r2, y2 = ssm.ssm_block_norm_fwd(x.contiguous(), w_post=w, z=z.contiguous(), residual=res,
                                        w_pre=w, groups=8)
        # the same sums in another order where single elements are taken
        assert torch.allclose(r, r2, rtol=1e-5, atol=1e-5)
        assert torch.allclose(y.float(), y2.float(), rtol=2.0 ** -7, atol=1e-5)
        inplace = res.clone()
        r3, y3 = ssm.ssm_block_norm_fwd(x, w_post=w, z=z, residual=inplace, w_pre=w, groups=8,
                                        r=inplace)
        assert r3 is inplace and torch.equal(r3, r) and torch.equal(y3, y)


def test_no_rows():
    x = torch.zeros(0, 64, dtype=BF16, device=DEV)
    w = torch.ones(64, device=DEV)
    r, y = ssm.ssm_block_norm_fwd(x, w_post=w, w_pre=w)
    assert r.shape == x.shape and y.shape == x.shape
    got = ssm.ssm_block_norm_bwd(x, w_post=w, w_pre=w, dy=x)
    assert got["dx"].shape == x.shape
    assert (got["dw_post"] == 0).all() and (got["dw_pre"] == 0).all()


def test_deterministic():
    inp, dr, dy = make(BF16, 2000, 640, ALL, True, seed=6)
    d = {n: t.to(DEV) for n, t in inp.items()}
    a, b = (ssm.ssm_block_norm_bwd(**d, groups=10, dr=dr.to(DEV), dy=dy.to(DEV)) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)
