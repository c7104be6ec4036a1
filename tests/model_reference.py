"""The embedding, the layer norm and the gradients' norm in 64 bits on the CPU,
from their formulas; inputs are tensors of any type."""
import math

import torch

F64 = torch.float64


def embed(ids, weight, scale):
    ids = ids.reshape(-1).long()
    there = (ids >= 0) & (ids < weight.shape[0])
    out = weight.double()[torch.where(there, ids, 0)] * scale
    return out * there.unsqueeze(1)


def embed_gradient(ids, dy, vocab, scale, old=None):
    """The gradient, the sums of the absolute values of what is added, and how
    many terms each row has."""
    ids = ids.reshape(-1).long()
    dy = dy.double().reshape(ids.shape[0], -1)
    there = (ids >= 0) & (ids < vocab)
    dw, mag = (torch.zeros(vocab, dy.shape[1], dtype=F64) for _ in range(2))
    dw.index_add_(0, ids[there], dy[there] * scale)
    mag.index_add_(0, ids[there], dy[there].abs() * abs(scale))
    if old is not None:
        dw, mag = dw + old.double(), mag + old.double().abs()
    return dw, mag, torch.bincount(ids[there], minlength=vocab)


def layer_norm(x, weight=None, bias=None, residual=None, eps=1e-5):
    r = x.double() if residual is None else x.double() + residual.double()
    d = r - r.mean(-1, keepdim=True)
    y = d / (d.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * weight.double()
    return r, y if bias is None else y + bias.double()


def layer_norm_gradients(x, weight=None, bias=None, residual=None, eps=1e-5, dr=None, dy=None):
    """By the formula, which test_model_reference.py holds against differences."""
    r = x.double() if residual is None else x.double() + residual.double()
    d = r - r.mean(-1, keepdim=True)
    s = 1.0 / (d.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    h, dy = d * s, dy.double()
    g = dy if weight is None else dy * weight.double()
    D = s * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
    if dr is not None:
        D = D + dr.double()
    out = {"dx": D}
    if residual is not None:
        out["dresidual"] = D
    rows = tuple(range(dy.dim() - 1))
    if weight is not None:
        out["dweight"] = (dy * h).sum(rows)
    if bias is not None:
        out["dbias"] = dy.sum(rows)
    return out


def grad_norm(grads):
    return math.sqrt(math.fsum(float(g.double().pow(2).sum()) for g in grads))


def grad_clip(grads, max_norm, norm=None):
    norm = grad_norm(grads) if norm is None else norm
    c = max_norm / norm if norm > max_norm and math.isfinite(norm) else 1.0
    return norm, [g.double() * c for g in grads]
