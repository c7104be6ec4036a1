"""The layer norm with the residual sum before it (ssm_layer_norm_fwd, _bwd)
against its formula in 64 bits.

Tolerances on |g - r| / (|r| + rms(r)): an output is rounded once, 2^-8 of |r|
in bf16, and everything before is fp32 with a handful of roundings and sums of
up to 16384 terms (tree and strided sums: below 64 * 2^-24 = 4e-6 relative to
the root sum of squares).  bf16: 2^-8 + 1e-5; fp32, and the weights'
gradients, which are sums over rows of such terms: 2e-5.
"""
import pytest
import torch

import model_reference as ref
import selective_state_space_30_amd as ssm
from parity_metrics import report, scaled_max_err

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": (BF16, BF16, BF16), "wide": (BF16, F32, BF16), "f32": (F32, F32, F32),
         "down": (F32, F32, BF16)}


def check(got, want, what):
    tol = 2.0 ** -8 + 1e-5 if got.dtype == BF16 else 2e-5
    assert got.shape == want.shape, what
    assert scaled_max_err(got, want) <= tol, "%s: %s" % (what, report(got, want))


def make(types, rows, dim, parts, seed=0):
    xt, rt, yt = TYPES[types]
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    inp = {"x": (1.5 * r(rows, dim)).to(xt)}
    inp["weight"] = 1 + 0.2 * r(dim) if "w" in parts else None
    inp["bias"] = r(dim) if "b" in parts else None
    inp["residual"] = (2 * r(rows, dim) + 0.7).to(rt) if "r" in parts else None
    dr = r(rows, dim).to(rt if "r" in parts else xt) if "d" in parts else None
    return inp, dr, r(rows, dim).to(yt)


CASES = []
# a row held by 8, 16, 32 and 64 lanes and by 2, 4 and 8 waves, with whole and
# broken pieces, at every number of pieces a lane
for t in TYPES:
    CASES += [(t, 1, 1, "wbrd"), (t, 3, 7, "wbrd"), (t, 5, 64, "wbrd"), (t, 9, 65, "wbrd"),
              (t, 17, 200, "wbrd"), (t, 6, 319, "wbrd"), (t, 4, 512, "wbrd"), (t, 7, 768, "wbrd"),
              (t, 5, 1537, "wbrd"), (t, 5, 2048, "wbrd"), (t, 3, 2560, "wbrd"),
              (t, 2, 4099, "wbrd"), (t, 3, 5120, "wbrd"), (t, 2, 8192, "wbrd"),
              (t, 2, 12289, "wbrd"), (t, 2, 16384, "wbrd"),
              (t, 9000, 40, "wbrd"), (t, 2100, 264, "wbrd"), (t, 1500, 1030, "wbrd")]
CASES = [c for c in CASES if c[0] != "down" or c[3]]
for parts in ("", "w", "b", "r", "wr", "bd", "wb"):
    CASES += [("bf16", 70, 300, parts), ("f32", 70, 300, parts)]
CASES += [("wide", 70, 300, "r"), ("wide", 33, 2560, "wr"), ("down", 70, 300, "wb"),
          ("down", 33, 2560, "wbd")]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s_%dx%d_%s" % c)
def test_layer_norm(case):
    types, rows, dim, parts = case
    inp, dr, dy = make(types, rows, dim, parts, seed=rows + dim)
    d = {n: None if t is None else t.to(DEV) for n, t in inp.items()}
    yt = TYPES[types][2]
    r, y = ssm.ssm_layer_norm_fwd(**d, dtype=yt)
    wr, wy = ref.layer_norm(**inp)
    assert y.dtype == yt
    if "r" in parts:
        assert r.dtype == TYPES[types][1]
        check(r, wr, "r")
    else:
        assert r is d["x"]
    check(y, wy, "y")
    got = ssm.ssm_layer_norm_bwd(**d, dr=None if dr is None else dr.to(DEV), dy=dy.to(DEV))
    want = ref.layer_norm_gradients(**inp, dr=dr, dy=dy)
    assert set(got) == set(want)
    for n in want:
        check(got[n], want[n], n)
    if "r" in parts and TYPES[types][0] == TYPES[types][1]:
        assert got["dresidual"] is got["dx"]


def test_rows_of_one_value_and_far_means():
    """Rows whose variance is 0 divide by sqrt(eps); rows far from 0 lose what
    their inputs' 24 bits lose, and no more: an error of r of 2^-24 max|r| (of
    the sum) and one as large of the mean, over the row's deviation, and a
    gradient that it enters once more by h."""
    inp, dr, dy = make("f32", 5, 320, "wbrd", seed=5)
    inp["x"][0], inp["residual"][0] = 3.0, -1.0
    inp["x"][1], inp["residual"][1] = 0.0, 0.0
    inp["x"][2] += 3000.0
    inp["x"][3] *= 1e15
    inp["x"][4] *= 1e-12
    inp["residual"][4] *= 1e-12
    d = {n: t.to(DEV) for n, t in inp.items()}
    r, y = ssm.ssm_layer_norm_fwd(**d)
    got = ssm.ssm_layer_norm_bwd(**d, dr=dr.to(DEV), dy=dy.to(DEV))
    wr, wy = ref.layer_norm(**inp)
    want = ref.layer_norm_gradients(**inp, dr=dr, dy=dy)
    assert torch.equal(y[0].cpu(), inp["bias"]) and torch.equal(y[1].cpu(), inp["bias"])
    for i in range(5):
        far = 3 * 2.0 ** -24 * 3010 / 2.0 * 4 if i == 2 else 0.0
        for g, w in ((r, wr), (y, wy), (got["dx"], want["dx"])):
            assert scaled_max_err(g[i], w[i]) <= 2e-5 + far, "row %d" % i


@pytest.mark.parametrize("dim", [7, 320, 1000, 1537, 5000, 16384])
def test_rows_of_one_value_are_their_bias(dim):
    """Whatever the value.  A sum takes at most 32 additions in a lane, 9 over
    lanes and waves and a division, each off by 2^-24: the mean is off by
    42 * 2^-24 of the value, what is left of that after its own mean by 42 * 2^-24
    of it, over at least sqrt(eps) and at least 2^-10 of what was taken away."""
    values = torch.tensor([0.1, 1.0 / 3, -777.7, 3e4, 1e-30, 123456.7, 1e20, -3e25])
    x = values.unsqueeze(1).expand(len(values), dim).contiguous()
    w, b = torch.full((dim,), 1.5), torch.linspace(-1, 1, dim)
    _, y = ssm.ssm_layer_norm_fwd(x.to(DEV), w.to(DEV), b.to(DEV))
    far = (values.abs().unsqueeze(1) * 42 ** 2 * 2.0 ** -48 / 1e-5 ** 0.5).clamp(max=42 * 2.0 ** -14)
    assert ((y.cpu() - b).abs() <= 1.5 * far + 2.0 ** -23).all()
    # dy of ones: 1.5 less its mean is what the sum's rounding leaves
    got = ssm.ssm_layer_norm_bwd(torch.ones(1, dim, device=DEV), w.to(DEV),
                                 dy=torch.ones(1, dim, device=DEV))
    assert got["dx"].abs().max() <= 1.5 / 1e-5 ** 0.5 * 64 * 2.0 ** -24


def test_not_finite_stays_in_its_row():
    inp, dr, dy = make("bf16", 40, 200, "wbrd", seed=6)
    inp["x"][3, 5], inp["residual"][9, 0] = float("nan"), float("inf")
    d = {n: t.to(DEV) for n, t in inp.items()}
    r, y = ssm.ssm_layer_norm_fwd(**d)
    got = ssm.ssm_layer_norm_bwd(**d, dr=dr.to(DEV), dy=dy.to(DEV))
    bad = torch.zeros(40, dtype=torch.bool)
    bad[[3, 9]] = True
    assert (~torch.isfinite(r)).sum() == 2
    for t in (y, got["dx"]):
        assert torch.equal(t.isnan().any(1).cpu(), bad)
    assert torch.isfinite(got["dbias"]).all() and got["dweight"].isnan().all()


@pytest.mark.parametrize("types", ["bf16", "wide"])
def test_slices_in_place_and_leading_dimensions(types):
    gen = torch.Generator().manual_seed(8)
    rt = TYPES[types][1]
    for off in (0, 3):
        wide = torch.randn(2, 3, off + 517, generator=gen).to(BF16).to(DEV)
        x = wide[..., off:off + 512]
        res = torch.randn(2, 3, 600, generator=gen).to(rt).to(DEV)[..., off:off + 512]
        w, b = torch.rand(512, generator=gen).to(DEV), torch.rand(512, generator=gen).to(DEV)
        r, y = ssm.ssm_layer_norm_fwd(x, w, b, residual=res)
        r2, y2 = ssm.ssm_layer_norm_fwd(x.contiguous(), w, b, residual=res.contiguous())
        assert torch.equal(r, r2) and torch.equal(y, y2)
        inplace = res.contiguous()
        r3, y3 = ssm.ssm_layer_norm_fwd(x, w, b, residual=inplace, r=inplace)
        assert r3 is inplace and torch.equal(r3, r) and torch.equal(y3, y)
        dy = torch.randn(2, 3, 512, generator=gen).to(BF16).to(DEV)
        a = ssm.ssm_layer_norm_bwd(x, w, b, residual=res, dy=dy)
        c = ssm.ssm_layer_norm_bwd(x.contiguous(), w, b, residual=res.contiguous(), dy=dy)
        assert all(torch.equal(a[n], c[n]) for n in a)


@pytest.mark.parametrize("types", ["bf16", "wide", "f32"])
@pytest.mark.parametrize("dim", [1, 3, 37, 1001, 5003, 16383])
def test_in_place_where_pieces_overlap(types, dim):
    """A row's last piece begins inside the one before, which another lane or
    wave may have written already."""
    inp, _, _ = make(types, 700, dim, "wbr", seed=9)
    x, res, w, b = (inp[n].to(DEV) for n in ("x", "residual", "weight", "bias"))
    r, y = ssm.ssm_layer_norm_fwd(x, w, b, residual=res)
    for _ in range(3):
        inplace = res.clone()
        r2, y2 = ssm.ssm_layer_norm_fwd(x, w, b, residual=inplace, r=inplace)
        assert r2 is inplace and torch.equal(r2, r) and torch.equal(y2, y)


def test_from_r_alone():
    """A caller that kept the sum in fp32 gives it as x: the same gradient."""
    inp, dr, dy = make("wide", 50, 640, "wbrd", seed=12)
    d = {n: t.to(DEV) for n, t in inp.items()}
    r, _ = ssm.ssm_layer_norm_fwd(**d)
    a = ssm.ssm_layer_norm_bwd(**d, dr=dr.to(DEV), dy=dy.to(DEV))
    b = ssm.ssm_layer_norm_bwd(r, d["weight"], d["bias"], dr=dr.to(DEV), dy=dy.to(DEV))
    assert torch.equal(a["dresidual"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])
    assert torch.equal(a["dbias"], b["dbias"])


def test_given_outputs_and_rows_behind_them():
    inp, dr, dy = make("bf16", 6, 100, "wbrd", seed=3)
    d = {n: t.to(DEV) for n, t in inp.items()}
    nan = lambda *s, dtype=BF16: torch.full(s, float("nan"), dtype=dtype, device=DEV)  # noqa: E731
    r, y, dx, ds = (nan(9, 100) for _ in range(4))
    dw, db = nan(102, dtype=F32), nan(102, dtype=F32)
    ssm.ssm_layer_norm_fwd(**d, r=r[:6], y=y[:6])
    got = ssm.ssm_layer_norm_bwd(**d, dr=dr.to(DEV), dy=dy.to(DEV), out=dict(
        dx=dx[:6], dresidual=ds[:6], dweight=dw[1:101], dbias=db[1:101]))
    assert torch.equal(got["dx"], got["dresidual"]) and got["dresidual"] is not got["dx"]
    for t in (r, y, dx, ds):
        assert t[6:].isnan().all() and torch.isfinite(t[:6]).all()
    for t in (dw, db):
        assert t[0].isnan() and t[101].isnan() and torch.isfinite(t[1:101]).all()


def test_no_rows():
    x = torch.zeros(0, 64, dtype=BF16, device=DEV)
    w = torch.ones(64, device=DEV)
    r, y = ssm.ssm_layer_norm_fwd(x, w, w, residual=x)
    assert r.shape == x.shape and y.shape == x.shape
    got = ssm.ssm_layer_norm_bwd(x, w, w, residual=x, dy=x)
    assert got["dx"].shape == x.shape
    assert (got["dweight"] == 0).all() and (got["dbias"] == 0).all()


def test_deterministic_whatever_the_workspace_holds():
    inp, dr, dy = make("wide", 3000, 640, "wbrd", seed=6)
    d = {n: t.to(DEV) for n, t in inp.items()}
    a = ssm.ssm_layer_norm_bwd(**d, dr=dr.to(DEV), dy=dy.to(DEV))
    size = ssm.ssm_layer_norm_bwd_workspace_size(3000, 640)
    for fill in (0, 255):
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        b = ssm.ssm_layer_norm_bwd(**d, dr=dr.to(DEV), dy=dy.to(DEV), workspace=ws)
        assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.slow
def test_offsets_past_32_bits():
    """Over 2^31 elements: the last rows are those of a call of their own."""
    rows, dim = 270000, 8192
    x = torch.randn(1000, dim, device=DEV).to(BF16).repeat(270, 1)
    assert x.numel() > 2 ** 31
    w, b = torch.rand(dim, device=DEV), torch.rand(dim, device=DEV)
    _, y = ssm.ssm_layer_norm_fwd(x, w, b)
    _, last = ssm.ssm_layer_norm_fwd(x[-1000:], w, b)
    assert torch.equal(y[-1000:], last) and torch.equal(y[:1000], last)
    del y
    dx = ssm.ssm_layer_norm_bwd(x, w, b, dy=x)["dx"]
    last = ssm.ssm_layer_norm_bwd(x[-1000:], w, b, dy=x[-1000:])["dx"]
    assert torch.equal(dx[-1000:], last) and torch.equal(dx[:1000], last)
    assert rows == dx.shape[0]
