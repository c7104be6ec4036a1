"""Plain 64-bit implementations of linear attention with a decay for each
head, its gradients, and the block norm, on the CPU.  One token after the
other, straight from the recurrence; gradients by torch's autograd through
it (held to differences in test_linattn_reference.py)."""
import torch

F64 = torch.float64


def heads_of(x, heads):
    return x.repeat_interleave(heads // x.shape[-2], dim=-2)


def linattn(q, k, v, g, scale, h0):
    """One sequence: q, k (L, Hk, dk), v (L, H, dv), g (L, H) or None, h0
    (H, dk, dv) or None, all float64.  Returns o (L, H, dv), state."""
    L, H, dv = v.shape
    dk = q.shape[-1]
    S = torch.zeros(H, dk, dv, dtype=F64) if h0 is None else h0
    o = []
    for t in range(L):
        if g is not None:
            S = S * torch.exp(g[t])[:, None, None]
        S = S + heads_of(k[t], H)[:, :, None] * v[t][:, None, :]
        o.append(scale * (heads_of(q[t], H)[:, :, None] * S).sum(1))
    return (torch.stack(o) if o else torch.zeros(0, H, dv, dtype=F64)), S


def batch(q, k, v, g, scale, h0=None, offsets=None):
    """As ssm_linattn_fwd, on float64 CPU tensors; ``offsets``: list of
    packed sequences' row offsets."""
    H = v.shape[-2]
    if offsets is None:
        n, L = v.shape[:2]
        rows = [(i * L, (i + 1) * L) for i in range(n)]
    else:
        rows = list(zip(offsets, offsets[1:]))
    fq, fk, fv = (x.reshape((-1,) + x.shape[-2:]) for x in (q, k, v))
    fg = None
    if g is not None:
        fg = g.expand(fv.shape[0], H) if g.dim() == 1 else g.reshape(-1, H)
    outs, states = [], []
    o = torch.zeros_like(fv)
    pieces = []
    for i, (a, b) in enumerate(rows):
        oi, Si = linattn(fq[a:b], fk[a:b], fv[a:b], None if fg is None else fg[a:b], scale,
                         None if h0 is None else h0[i])
        pieces.append((a, b, oi))
        states.append(Si)
    at = 0
    for a, b, oi in pieces:
        outs += [o[at:a], oi]
        at = b
    outs.append(o[at:])
    return torch.cat(outs).reshape(v.shape), torch.stack(states)


def gradients(q, k, v, g, scale, h0, do, dh, offsets=None):
    """Gradients of sum(o * do) + sum(state * dh) for every input."""
    leaf = {n: x.clone().requires_grad_() for n, x in
            (("q", q), ("k", k), ("v", v), ("g", g), ("h0", h0)) if x is not None}
    o, h = batch(leaf["q"], leaf["k"], leaf["v"], leaf.get("g"), scale, leaf.get("h0"), offsets)
    loss = (o * do).sum()
    if dh is not None:
        loss = loss + (h * dh).sum()
    got = torch.autograd.grad(loss, list(leaf.values()), allow_unused=True)
    return {"d" + n: (torch.zeros_like(leaf[n]) if x is None else x)
            for n, x in zip(leaf, got)}


def block_norm(x, w_post=None, z=None, scale=None, residual=None, w_pre=None, groups=1,
               eps=1e-5):
    n = x
    if w_post is not None:
        part = x.reshape(x.shape[0], groups, -1)
        n = (part / torch.sqrt((part * part).mean(-1, keepdim=True) + eps)).reshape(x.shape)
        n = n * w_post
    if z is not None:
        n = n * z / (1 + torch.exp(-z))
    if scale is not None:
        n = n * scale
    r = n if residual is None else residual + n
    y = None
    if w_pre is not None:
        y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * w_pre
    return r, y


def block_norm_gradients(inputs, groups, eps, dr, dy):
    """``inputs``: dict of float64 tensors (x, w_post, z, scale, residual, w_pre)."""
    leaf = {n: t.clone().requires_grad_() for n, t in inputs.items() if t is not None}
    r, y = block_norm(**leaf, groups=groups, eps=eps)
    loss = torch.zeros((), dtype=F64)
    if dr is not None:
        loss = loss + (r * dr).sum()
    if y is not None:
        loss = loss + (y * dy).sum()
    return {"d" + n: g for n, g in zip(leaf, torch.autograd.grad(loss, list(leaf.values())))}
