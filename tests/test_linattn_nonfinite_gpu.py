"""An infinity or NaN in one token reaches the results that the recurrence
lets it reach and no others: o and dq from its token on, dk and dv up to it
(M_t sums over s >= t), in a value its own column alone.  Everything else has
the bits of a run with a finite value there."""
import pytest
import torch

import selective_state_space_30_amd as ssm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
L = 300


def inputs(dtype, heads, qk_heads, dk, dv):
    gen = torch.Generator().manual_seed(70 + dk)
    r = lambda *s: torch.randn(1, L, *s, generator=gen).to(dtype).to(DEV)  # noqa: E731
    return {"q": r(qk_heads, dk), "k": r(qk_heads, dk), "v": r(heads, dv), "do": r(heads, dv),
            "g": -0.5 * torch.rand(1, L, heads, generator=gen).to(DEV)}


def run(t, want_dg=True):
    o, h = ssm.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["g"])
    d = ssm.ssm_linattn_bwd(t["q"], t["k"], t["v"], t["g"], do=t["do"], want_dg=want_dg)
    return {"o": o, "h": h, **d}


def with_value(t, name, at, value):
    t = dict(t)
    t[name] = t[name].clone()
    t[name][0, at, 0, 3] = value  # head 0, element 3
    return t


SHAPES = [(2, 1, 64, 64), (3, 3, 64, 40), (2, 2, 128, 128), (2, 1, 40, 160), (1, 1, 200, 64)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "h%d_%d_k%d_v%d" % s)
@pytest.mark.parametrize("value", [NAN, INF, -INF], ids=["nan", "inf", "minf"])
def test_reaches_no_other_token(dtype, shape, value):
    heads, qk_heads, dk, dv = shape
    rep = heads // qk_heads
    clean = inputs(dtype, *shape)
    for at in (0, 7, 31, 32, 63, 64, 130, 299):
        for want_dg in (True, False):
            want = run(clean, want_dg)
            for name in ("q", "k", "v", "do"):
                got = run(with_value(clean, name, at, value), want_dg)
                what = "%s at %d" % (name, at)
                before, behind = slice(0, at), slice(at + 1, L)
                for n in ("o", "dq"):
                    assert torch.equal(got[n][:, before], want[n][:, before]), (what, n)
                for n in ("dk", "dv"):
                    assert torch.equal(got[n][:, behind], want[n][:, behind]), (what, n)
                if name == "q":      # read by its own token alone
                    assert torch.equal(got["o"][:, behind], want["o"][:, behind]), what
                    assert not torch.isfinite(got["o"][0, at, :rep]).any(), what
                    assert torch.equal(got["o"][0, at, rep:], want["o"][0, at, rep:]), what
                    assert torch.equal(got["h"], want["h"]), what
                elif name == "v":    # one column of the state
                    keep = torch.ones(dv, dtype=torch.bool)
                    keep[3] = False
                    assert not torch.isfinite(got["o"][0, at:, 0, 3]).any(), what
                    assert torch.equal(got["o"][:, :, 0, keep], want["o"][:, :, 0, keep]), what
                    assert torch.equal(got["o"][:, :, 1:], want["o"][:, :, 1:]), what
                    assert not torch.isfinite(got["h"][0, 0, :, 3]).any(), what
                    assert torch.equal(got["h"][..., 0, :, keep], want["h"][..., 0, :, keep]), what
                elif name == "k":    # one row of the state, read by every column
                    assert not torch.isfinite(got["o"][0, at:, :rep]).any(), what
                    assert torch.equal(got["o"][:, :, rep:], want["o"][:, :, rep:]), what
                else:                # one column of the adjoint
                    keep = torch.ones(dv, dtype=torch.bool)
                    keep[3] = False
                    assert torch.equal(got["o"], want["o"]), what
                    assert not torch.isfinite(got["dv"][0, :at + 1, 0, 3]).any(), what
                    assert torch.equal(got["dv"][:, :, 0, keep], want["dv"][:, :, 0, keep]), what


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nan_decay_reaches_no_token_before_it(dtype):
    clean = inputs(dtype, 2, 1, 64, 64)
    want = run(clean)
    for at in (0, 20, 64, 200):
        t = dict(clean, g=clean["g"].clone())
        t["g"][0, at, 1] = NAN
        got = run(t)
        assert torch.equal(got["o"][:, :at], want["o"][:, :at])
        assert torch.equal(got["o"][:, :, 0], want["o"][:, :, 0])
        assert torch.isnan(got["o"][0, at:, 1]).all()
        assert torch.equal(got["dv"][:, :, 0], want["dv"][:, :, 0])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_padding_of_nan_behind_each_sequence(dtype):
    """Sequences padded to one length with rows of NaN: the rows before the
    padding are those of zeros there."""
    clean = inputs(dtype, 2, 1, 64, 64)
    lens = (300, 37, 1, 200)
    pad = {n: torch.cat([clean[n]] * 4) for n in ("q", "k", "v", "g")}
    zero = {n: x.clone() for n, x in pad.items()}
    for i, n in enumerate(lens):
        for name in pad:
            pad[name][i, n:] = NAN
            zero[name][i, n:] = 0
    o, _ = ssm.ssm_linattn_fwd(pad["q"], pad["k"], pad["v"], pad["g"])
    o0, _ = ssm.ssm_linattn_fwd(zero["q"], zero["k"], zero["v"], zero["g"])
    for i, n in enumerate(lens):
        assert torch.equal(o[i, :n], o0[i, :n])
