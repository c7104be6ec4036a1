"""The plain implementations that the linear-attention and block-norm tests
compare with: hand-worked values, the masked quadratic form, and gradients
against central differences."""
import math

import pytest
import torch

import linattn_reference as ref

F64 = torch.float64


def test_two_tokens_by_hand():
    # one head, 1 x 1 state: S_0 = 2 -> S_1 = 2 e^-1 + 3 * 5, S_2 = S_1 e^-2 + 7 * 11
    q = torch.tensor([[[[1.0]], [[2.0]]]], dtype=F64)
    k = torch.tensor([[[[3.0]], [[7.0]]]], dtype=F64)
    v = torch.tensor([[[[5.0]], [[11.0]]]], dtype=F64)
    g = torch.tensor([[[-1.0], [-2.0]]], dtype=F64)
    o, h = ref.batch(q, k, v, g, 0.5, torch.full((1, 1, 1, 1), 2.0, dtype=F64))
    s1 = 2 * math.exp(-1) + 15
    s2 = s1 * math.exp(-2) + 77
    assert torch.allclose(o.flatten(), torch.tensor([0.5 * s1, s2], dtype=F64))
    assert abs(h.item() - s2) < 1e-12


def test_matches_the_masked_quadratic_form():
    gen = torch.Generator().manual_seed(0)
    L, H, Hk, dk, dv = 9, 4, 2, 3, 5
    r = lambda *s: torch.randn(*s, generator=gen, dtype=F64)  # noqa: E731
    q, k, v, g = r(1, L, Hk, dk), r(1, L, Hk, dk), r(1, L, H, dv), -torch.rand(1, L, H, dtype=F64)
    o, _ = ref.batch(q, k, v, g, 0.7)
    a = g.cumsum(1)[0].T                                     # (H, L)
    m = torch.exp(a[:, :, None] - a[:, None, :]).tril()
    qk = torch.einsum("thd,shd->hts", ref.heads_of(q[0], H), ref.heads_of(k[0], H))
    want = 0.7 * torch.einsum("hts,shd->thd", qk * m, v[0])
    assert torch.allclose(o[0], want)


@pytest.mark.parametrize("offsets", [None, [0, 1, 1, 4, 6]])
def test_gradients_against_differences(offsets):
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=F64)  # noqa: E731
    lead = (2, 4) if offsets is None else (7,)
    n = 2 if offsets is None else 4
    q, k, v = r(*lead, 1, 2), r(*lead, 1, 2), r(*lead, 2, 3)
    g, h0 = -torch.rand(*lead, 2, dtype=F64), r(n, 2, 2, 3)
    do, dh = r(*lead, 2, 3), r(n, 2, 2, 3)
    got = ref.gradients(q, k, v, g, 0.6, h0, do, dh, offsets)
    args = {"q": q, "k": k, "v": v, "g": g, "h0": h0}

    def loss():
        o, h = ref.batch(args["q"], args["k"], args["v"], args["g"], 0.6, args["h0"], offsets)
        return ((o * do).sum() + (h * dh).sum()).item()

    for name, t in args.items():
        flat = t.view(-1)
        for i in range(0, flat.numel(), 3):
            keep = flat[i].item()
            flat[i] = keep + 1e-5
            up = loss()
            flat[i] = keep - 1e-5
            down = loss()
            flat[i] = keep
            # central differences of step 1e-5: 1e-10 of the third
            # derivative, 1e-16 / 1e-5 of the loss
            assert abs((up - down) / 2e-5 - got["d" + name].view(-1)[i].item()) < 1e-7, (name, i)


def test_block_norm_gradients_against_differences():
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=F64)  # noqa: E731
    inp = {"x": r(3, 6), "w_post": r(6), "z": r(3, 6), "scale": r(6), "residual": r(3, 6),
           "w_pre": r(6)}
    dr, dy = r(3, 6), r(3, 6)
    got = ref.block_norm_gradients(inp, 2, 1e-3, dr, dy)

    def loss():
        a, b = ref.block_norm(**inp, groups=2, eps=1e-3)
        return ((a * dr).sum() + (b * dy).sum()).item()

    for name, t in inp.items():
        flat = t.view(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + 1e-5
            up = loss()
            flat[i] = keep - 1e-5
            down = loss()
            flat[i] = keep
            assert abs((up - down) / 2e-5 - got["d" + name].view(-1)[i].item()) < 1e-6, (name, i)
