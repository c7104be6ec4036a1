"""The gradients' global norm and clipping (ssm_grad_norm, ssm_grad_clip)
against their formula in 64 bits.

Tolerances: squares of fp32 values are exact in 64 bits and their sums are off
by less than 2^-40, so the norm is off by the rounding to fp32: 2^-24, with
some room 2^-23.  A clipped element has the factor's rounding (2^-24) and the
product's (2^-24, or 2^-8 to bf16), and below fp32's normal range half of its
smallest step.
"""
import math

import pytest
import torch

import model_reference as ref
import selective_state_space_30_amd as ssm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
CODES = {"f": F32, "b": BF16}


def make(sizes, seed=0, mul=1.0):
    """sizes: (shape or size, "f" or "b") of each tensor."""
    gen = torch.Generator().manual_seed(seed)
    return [(mul * torch.randn(n, generator=gen)).to(CODES[t]) for n, t in sizes]


def close_norm(got, want):
    assert got.dtype == F32 and got.shape == ()
    assert abs(float(got) - want) <= 2.0 ** -23 * want, (float(got), want)


def close(got, want):
    step = 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -24
    bound = (step + 2.0 ** -23) * want.abs() + 2.0 ** -150
    assert ((got.double().cpu() - want).abs() <= bound).all()


SETS = {
    "one element": [(1, "f")],
    "one of each": [(1, "f"), (1, "b")],
    "odd sizes": [(7, "f"), (8, "b"), (9, "b"), (1023, "f"), (2049, "b"), (8191, "f"), (8200, "b")],
    "chunk borders": [(16383, "f"), (16384, "b"), (16385, "f"), (32768, "b"), (32777, "f")],
    "with empty ones": [(0, "f"), (5, "b"), (0, "b"), (0, "f"), (33, "f"), (0, "b")],
    "matrices": [((300, 70), "b"), ((5, 6, 7), "f"), ((1000, 999), "f")],
    # 160 tensors fit a launch's arguments, 65536 elements one workgroup
    "a table": [(3 + i % 40, "fb"[i % 2]) for i in range(160)],
    "a table and one": [(3 + i % 40, "fb"[i % 2]) for i in range(161)],
    "two tables and one": [(30000 + i % 40, "fb"[i % 2]) for i in range(321)],
    "one workgroup": [(65529, "f"), (7, "b")],
    "over one workgroup": [(65529, "f"), (8, "f"), (1, "b")],
    "many": [(1 + (i * 37) % 500, "fb"[i % 3 == 0]) for i in range(700)],
    "many chunks": [(40_000_003, "b"), (5, "f"), (20_000_001, "f")],
}


@pytest.mark.parametrize("name", SETS)
def test_norm_and_clip(name):
    grads = make(SETS[name], seed=len(name))
    dev = [g.to(DEV) for g in grads]
    norm = ref.grad_norm(grads)
    close_norm(ssm.ssm_grad_norm(dev), norm)
    keep = [g.clone() for g in dev]
    for share in (0.37, 1.5):
        # into tensors of the same and of the other type
        for other in (False, True):
            out = [torch.full(g.shape, float("nan"), device=DEV,
                              dtype=(F32 if g.dtype == BF16 else BF16) if other else g.dtype)
                   for g in dev]
            close_norm(ssm.ssm_grad_clip(dev, share * norm, out=out), norm)
            for o, w, g in zip(out, ref.grad_clip(grads, share * norm)[1], dev):
                close(o, w)
                if share > 1:
                    assert torch.equal(o, g.to(o.dtype))
        assert all(torch.equal(a, b) for a, b in zip(dev, keep))
    close_norm(ssm.ssm_grad_clip(dev, 2 * norm), norm)
    assert all(torch.equal(a, b) for a, b in zip(dev, keep))
    close_norm(ssm.ssm_grad_clip(dev, 0.01 * norm), norm)
    for g, w in zip(dev, ref.grad_clip(grads, 0.01 * norm)[1]):
        close(g, w)


def test_norm_that_is_given():
    grads = make([(1000, "f"), (77, "b")], seed=2)
    dev = [g.to(DEV) for g in grads]
    given = torch.tensor(50.0, device=DEV)
    assert ssm.ssm_grad_clip(dev, 5.0, norm=given) is given and float(given) == 50.0
    for g, w in zip(dev, ref.grad_clip(grads, 5.0, norm=50.0)[1]):
        close(g, w)
    keep = [g.clone() for g in dev]
    for still in (4.0, 5.0, float("inf"), float("nan")):
        ssm.ssm_grad_clip(dev, 5.0, norm=torch.tensor(still, device=DEV))
        assert all(torch.equal(a, b) for a, b in zip(dev, keep))


def test_views_of_a_bucket_at_any_element():
    flat = torch.randn(50000).to(BF16)
    cuts = [0, 1, 4, 11, 1000, 17385, 17386, 40001, 49999]
    grads = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
    dev = flat.to(DEV)
    dgrads = [dev[a:b] for a, b in zip(cuts, cuts[1:])]
    wide = torch.full((50003,), float("nan"), device=DEV)
    out = [wide[a + 2:b + 2] for a, b in zip(cuts, cuts[1:])]
    norm, want = ref.grad_clip(grads, 3.0)
    close_norm(ssm.ssm_grad_clip(dgrads, 3.0, out=out), norm)
    for o, w in zip(out, want):
        close(o, w)
    assert wide[:2].isnan().all() and wide[50001:].isnan().all()
    assert torch.isfinite(wide[2:50001]).all()
    ssm.ssm_grad_clip(dgrads, 3.0)
    for o, w in zip(dgrads, want):
        close(o, w)
    assert dev[49999] == flat[49999]


def test_transposed_and_some_in_place():
    a, b, c = (torch.randn(40, 30) for _ in range(3))
    grads = [a.to(DEV).t(), b.to(DEV), c.to(DEV)]
    out = [torch.empty(40, 30, device=DEV).t(), grads[1], torch.empty(40, 30, device=DEV)]
    norm, want = ref.grad_clip([a.t(), b, c], 1.0)
    close_norm(ssm.ssm_grad_clip(grads, 1.0, out=out), norm)
    for o, w in zip(out, want):
        close(o, w)
    assert torch.equal(grads[0].cpu(), a.t()) and torch.equal(grads[2].cpu(), c)


def test_zeros_no_tensors_and_no_limit():
    z = [torch.zeros(10, device=DEV), torch.zeros(5, dtype=BF16, device=DEV)]
    assert float(ssm.ssm_grad_clip(z, 1.0)) == 0 and not any(t.any() for t in z)
    assert float(ssm.ssm_grad_norm([])) == 0 and float(ssm.ssm_grad_clip([], 1.0)) == 0
    assert float(ssm.ssm_grad_norm([torch.zeros(0, device=DEV)])) == 0
    g = [torch.randn(100, device=DEV)]
    keep = g[0].clone()
    ssm.ssm_grad_clip(g, float("inf"))
    assert torch.equal(g[0], keep)
    ssm.ssm_grad_clip(g, 0.0)
    assert not g[0].any()


def test_large_and_small_elements():
    """Squares outside fp32's range."""
    for mul in (1e25, 1e-30):
        grads = make([(1000, "f"), (50, "f")], seed=4, mul=mul)
        dev = [g.to(DEV) for g in grads]
        norm, want = ref.grad_clip(grads, 0.125 * mul)
        close_norm(ssm.ssm_grad_clip(dev, 0.125 * mul), norm)
        for g, w in zip(dev, want):
            close(g, w)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_not_finite_leaves_the_gradients(value):
    grads = make([(5000, "f"), (300, "b")], seed=5)
    grads[1][77] = value
    dev = [g.to(DEV) for g in grads]
    out = [torch.zeros_like(g) for g in dev]
    for norm in (ssm.ssm_grad_norm(dev), ssm.ssm_grad_clip(dev, 1.0),
                 ssm.ssm_grad_clip(dev, 1.0, out=out)):
        assert math.isnan(float(norm)) if math.isnan(value) else float(norm) == math.inf
    for g, d, o in zip(grads, dev, out):
        assert torch.equal(d.cpu().nan_to_num(7), g.nan_to_num(7))
        assert torch.equal(o.cpu().nan_to_num(7), g.nan_to_num(7))


def test_norm_over_fp32_is_infinite_and_leaves_the_gradients():
    dev = [torch.full((1000,), 3e38, device=DEV)]
    assert float(ssm.ssm_grad_clip(dev, 1.0)) == math.inf
    assert (dev[0] == 3e38).all()


def test_deterministic_whatever_the_workspace_holds():
    dev = [g.to(DEV) for g in make(SETS["many"], seed=9)] + [torch.randn(10_000_001, device=DEV)]
    a = ssm.ssm_grad_norm(dev)
    for fill in (0, 255):
        ws = torch.full((ssm.ssm_grad_workspace_size(),), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(ssm.ssm_grad_norm(dev, workspace=ws), a)


@pytest.mark.slow
def test_offsets_past_32_bits():
    n = 2 ** 31 + 5000
    g = torch.ones(n, dtype=BF16, device=DEV)
    g[-1] = 1000.0
    want = math.sqrt(n - 1 + 1e6)
    close_norm(ssm.ssm_grad_norm([g]), want)
    ssm.ssm_grad_clip([g], want / 2)
    assert (g[-5000:-1] == 0.5).all() and g[-1] == 500.0 and (g[:5000] == 0.5).all()
