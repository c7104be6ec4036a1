"""The 64-bit references of the embedding, layer norm and clipping tests, held
against differences and by hand."""
import torch

import model_reference as ref


def _difference(f, t, at, h=1e-6):
    a, b = t.clone(), t.clone()
    a.view(-1)[at] += h
    b.view(-1)[at] -= h
    return (f(a) - f(b)) / (2 * h)


def test_layer_norm_gradients_are_differences():
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    inp = dict(x=r(3, 7), weight=1 + 0.3 * r(7), bias=r(7), residual=r(3, 7))
    dr, dy = r(3, 7), r(3, 7)

    def loss(**over):
        a, b = ref.layer_norm(**{**inp, **over})
        return float((a * dr).sum() + (b * dy).sum())
    got = ref.layer_norm_gradients(**inp, dr=dr, dy=dy)
    for name in ("x", "weight", "bias", "residual"):
        g = got["d" + name].reshape(-1)
        for at in range(g.numel()):
            want = _difference(lambda t: loss(**{name: t}), inp[name], at)
            assert abs(float(g[at]) - want) < 1e-7, (name, at)


def test_embed_gradient_is_differences():
    gen = torch.Generator().manual_seed(2)
    w = torch.randn(5, 3, generator=gen, dtype=torch.float64)
    ids = torch.tensor([[4, 1, -1], [1, 5, 1]])
    dy = torch.randn(2, 3, 3, generator=gen, dtype=torch.float64)
    dw, mag, count = ref.embed_gradient(ids, dy, 5, 0.7)
    for at in range(15):
        want = _difference(lambda t: float((ref.embed(ids, t, 0.7) * dy.reshape(6, 3)).sum()), w, at)
        assert abs(float(dw.view(-1)[at]) - want) < 1e-7
    assert count.tolist() == [0, 3, 0, 0, 1] and (mag >= dw.abs()).all()


def test_clip_by_hand():
    norm, g = ref.grad_clip([torch.tensor([3.0]), torch.tensor([[4.0]])], 1.0)
    assert norm == 5.0 and abs(float(g[0]) - 0.6) < 1e-15 and abs(float(g[1]) - 0.8) < 1e-15
    norm, g = ref.grad_clip([torch.tensor([3.0])], 4.0)
    assert norm == 3.0 and float(g[0]) == 3.0
