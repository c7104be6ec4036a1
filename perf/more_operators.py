"""Measured cases of the operators around a model's blocks: the embedding, the
layer norm, and the global norm of the gradients with their clipping.

``own = False``: each operator from elementary torch operations in 32 bits.
``own = True``: the library's calls of ``selective_state_space_30_amd``.

The embedding, with rows of zeros for ids outside 0..vocab-1 (padding):

    out_t = scale * weight[ids_t]
    dweight_v = scale * sum over t with ids_t = v of dy_t     (+ dweight_v)

"embed": out.  "embed_train": out, and the dense gradient of the weight for a
given gradient of out.  "embed_add": that gradient added to one that is there
(an output projection that shares the weight, or earlier micro-batches).

The layer norm, with the residual sum before it:

    r = x + residual
    y = (r - mean(r)) / sqrt(var(r) + eps) * weight + bias

"norm": r and y.  "norm_train": also the gradients of x, the residual, weight
and bias for given gradients of r and y.

The gradients' global norm, over all elements of all tensors, and clipping:

    norm = sqrt(sum g^2),   g' = g * min(1, max_norm / norm)

"clip": norm and g'.  "grad_norm": norm alone.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the next token of 8 sequences: latency
        _embed("embed_decode", "embed", 8, 50000, 2560, "bf16", "bf16", "bf16"),
        # prompts into a residual stream of 32 bits, rows scaled by sqrt(width)
        _embed("embed_prompt", "embed", 16384, 50000, 2560, "bf16", "f32", "bf16", scale=True),
        # a training step of 2 x 4096 tokens: the rows, and the weight's whole
        # gradient in 32 bits
        _embed("embed_train", "embed_train", 8192, 50000, 2560, "f32", "bf16", "f32"),
        # a padded batch of a narrower model, added to the gradient that the
        # output projection left in the shared weight
        _embed("embed_add", "embed_add", 65536, 32003, 768, "bf16", "bf16", "f32", pad=True),
        # residual sum and norm for 8 decoding rows: latency
        _norm("norm_decode", "norm", 8, 2560, "bf16", "bf16", "bf16", True),
        # prompts, residual stream in 32 bits
        _norm("norm_prompt", "norm", 16384, 2560, "bf16", "f32", "bf16", True),
        # training, residual stream in 32 bits
        _norm("norm_train", "norm_train", 8192, 2560, "bf16", "f32", "bf16", True),
        # training of a narrower model: many short rows, everything in 16 bits
        _norm("norm_train_short", "norm_train", 65536, 768, "bf16", "bf16", "bf16", True),
        # training in 32 bits with a width that no vector load divides
        _norm("norm_train_odd", "norm_train", 2003, 1537, "f32", "f32", "f32", False),
        # one block's gradients: latency
        _clip("clip_block", "clip", 1, 64, 0, "f32", "f32", 0.5),
        # 24 layers of width 1024 with their embedding, everything in 32 bits
        _clip("clip_f32", "clip", 24, 1024, 32000, "f32", "f32", 0.5),
        # 16 layers of width 2560, matrices in 16 bits
        _clip("clip_bf16", "clip", 16, 2560, 50000, "bf16", "bf16", 0.3),
    ]


def _named(name, c):
    return dict(name=name, **c) if name else c


def _embed(name, op, tokens, vocab, dim, wdtype, dtype, gdtype, scale=False, pad=False, wide_ids=True):
    """wdtype: the weight's type; dtype: that of out and dy; gdtype: dweight's."""
    return _named(name, dict(op=op, tokens=tokens, vocab=vocab, dim=dim, wdtype=wdtype, dtype=dtype,
                             gdtype=gdtype, scale=scale, pad=pad, wide_ids=wide_ids))


def _norm(name, op, rows, dim, xdtype, rdtype, ydtype, residual, affine=True):
    """Types of x, of the residual and r, and of y."""
    return _named(name, dict(op=op, rows=rows, dim=dim, xdtype=xdtype, rdtype=rdtype, ydtype=ydtype,
                             residual=residual, affine=affine))


def _clip(name, op, layers, width, vocab, dtype, odtype, clip):
    """dtype: the matrices' gradients (vectors are fp32); odtype: the clipped
    matrices'; clip: max_norm as a share of the norm to be expected."""
    return _named(name, dict(op=op, layers=layers, width=width, vocab=vocab, dtype=dtype,
                             odtype=odtype, clip=clip))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_train", "embed_add", "norm", "norm_train", "norm_train", "clip",
                     "clip", "grad_norm"])
    t = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("embed"):
        dim = _log(rng, 64, 8192)
        dim = dim if rng.random() < 0.3 else max(8, dim // 8 * 8)
        vocab = _log(rng, 500, max(600, min(200000, (1 << 27) // dim)))
        tokens = _log(rng, 1, max(2, min(200000, (1 << 26) // dim)))
        return _embed("", op, tokens, vocab, dim, rng.choice(["bf16", "f32"]), t,
                      rng.choice(["f32", "f32", "bf16"]) if op == "embed_train" else "f32",
                      rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.6)
    if op.startswith("norm"):
        dim = _log(rng, 16, 16384)
        dim = dim if rng.random() < 0.4 else max(8, dim // 8 * 8)
        rows = _log(rng, 1, max(2, min(400000, (1 << 25) // dim)))
        residual = rng.random() < 0.7
        r = "f32" if t == "f32" or rng.random() < 0.5 else "bf16"
        y = "bf16" if t == "f32" and rng.random() < 0.4 else t
        return _norm("", op, rows, dim, t, r if residual else t, y, residual, rng.random() < 0.8)
    width = 8 * _log(rng, 4, 256)
    layers = _log(rng, 1, max(2, min(64, (1 << 27) // (7 * width * width))))
    vocab = rng.choice([0, _log(rng, 100, max(200, min(50000, (1 << 27) // width)))])
    return _clip("", op, layers, width, vocab, t, rng.choice([t, "f32"]),
                 round(rng.choice([rng.uniform(0.05, 0.9), rng.uniform(1.1, 3.0)]), 3))


def _shapes(c):
    """(elements, matrix or vector) of the gradients of a model's parameters:
    a block's projections in and out, its convolution, the projections to the
    step and the two state vectors, the rates, the skip and the norm."""
    w, inner, n = c["width"], 2 * c["width"], 16
    rank = max(1, w // 16)
    block = [(2 * inner * w, True), (4 * inner, True), (inner, False), ((rank + 2 * n) * inner, True),
             (inner * rank, True), (inner, False), (inner * n, False), (inner, False),
             (w * inner, True), (w, False), (w, False)]
    ends = [(c["vocab"] * w, True), (w, False), (w, False)] if c["vocab"] else []
    return ends + block * c["layers"]


# ----------------------------------------------------------------- inputs --
def _frequencies(vocab):
    """How often an id comes: ids by falling frequency, as tokenizers have
    them, the frequency near the reciprocal of the rank."""
    p = 1.0 / (np.arange(vocab) + 2.7)
    return p / p.sum()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, dtype, mul=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * mul).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    if c["op"].startswith("embed"):
        n, vocab, dim = c["tokens"], c["vocab"], c["dim"]
        edges = torch.from_numpy(np.cumsum(_frequencies(vocab))).cuda()
        ids = torch.searchsorted(edges, rand(n).double()).clamp_(max=vocab - 1)
        if c["pad"]:  # sequences of different lengths, padded at their ends
            ids = torch.where(torch.arange(n, device="cuda") % 1024 < 940, ids, -1)
        s = dict(c, ids=ids if c["wide_ids"] else ids.to(torch.int32),
                 factor=math.sqrt(dim) if c["scale"] else 1.0)
        if c["op"] != "embed_add":
            s["weight"] = randn(vocab, dim, dtype=DT[c["wdtype"]], mul=0.02)
        if c["op"] != "embed":
            s["dy"] = randn(n, dim, dtype=DT[c["dtype"]], mul=0.1)
        if c["op"] == "embed_add":
            s["grad"] = randn(vocab, dim, dtype=DT[c["gdtype"]], mul=0.01)
        return s
    if c["op"].startswith("norm"):
        rows, dim = c["rows"], c["dim"]
        s = dict(c, x=randn(rows, dim, dtype=DT[c["xdtype"]], mul=1.5), w=None, b=None, res=None)
        if c["affine"]:
            s["w"] = 1.0 + randn(dim, dtype=torch.float32, mul=0.2)
            s["b"] = randn(dim, dtype=torch.float32, mul=0.2)
        if c["residual"]:
            # columns of the stream that have drifted away from 0
            s["res"] = (randn(rows, dim, dtype=torch.float32, mul=2.0) + 0.5 +
                        randn(dim, dtype=torch.float32)).to(DT[c["rdtype"]])
        if c["op"] == "norm_train":
            s["dr"] = randn(rows, dim, dtype=DT[c["rdtype"]])
            s["dy"] = randn(rows, dim, dtype=DT[c["ydtype"]])
        return s
    # gradients as autograd leaves them, tensor by tensor; the clipped ones lie
    # one after another in a buffer of each type, as an optimizer keeps them
    shapes = _shapes(c)
    grads = [randn(n, dtype=DT[c["dtype"]] if m else torch.float32, mul=0.01 * (1 + i % 5))
             for i, (n, m) in enumerate(shapes)]
    likely = math.sqrt(sum(n * (0.01 * (1 + i % 5)) ** 2 for i, (n, _) in enumerate(shapes)))
    s = dict(c, grads=grads, matrix=[m for _, m in shapes], max_norm=c["clip"] * likely)
    if c["op"] == "clip":
        total = {m: sum(n for n, k in shapes if k == m) for m in (True, False)}
        s["flat"] = {m: torch.zeros(total[m], dtype=DT[c["odtype"]] if m else torch.float32,
                                    device="cuda") for m in total}
        at = {True: 0, False: 0}
        s["out"] = []
        for n, m in shapes:
            s["out"].append(s["flat"][m][at[m]:at[m] + n])
            at[m] += n
    return s


# --------------------------------------------------------------- plain form --
def _plain_embed(s):
    ids = s["ids"].long()
    there = (ids >= 0) & (ids < s["vocab"])
    out = {}
    if s["op"] != "embed_add":
        rows = s["weight"][torch.where(there, ids, 0)].float() * s["factor"]
        out["out"] = torch.where(there.unsqueeze(1), rows, 0.0).to(DT[s["dtype"]])
    if s["op"] != "embed":
        # rows of ids outside go to one row more, which is left out
        sums = torch.zeros(s["vocab"] + 1, s["dim"], device=ids.device)
        sums.index_add_(0, torch.where(there, ids, s["vocab"]), s["dy"].float())
        sums = sums[:-1] * s["factor"]
        if s["op"] == "embed_add":
            s["grad"].copy_(s["grad"].float() + sums)
            out["dweight"] = s["grad"]
        else:
            out["dweight"] = sums.to(DT[s["gdtype"]])
    return out


def _plain_layer_norm(x, res, w, b):
    r = x.float() if res is None else x.float() + res.float()
    mean = r.mean(-1, keepdim=True)
    d = r - mean
    y = d * torch.rsqrt(d.square().mean(-1, keepdim=True) + EPS)
    return r, y if w is None else y * w + b


def _plain_norm(s):
    names = [n for n in ("x", "res", "w", "b") if s[n] is not None]
    train = s["op"] == "norm_train"
    leaf = {n: s[n].detach().requires_grad_(train) for n in names}
    r, y = _plain_layer_norm(*[leaf.get(n) for n in ("x", "res", "w", "b")])
    out = {"y": y.detach().to(DT[s["ydtype"]])}
    if s["res"] is not None:
        out["r"] = r.detach().to(DT[s["rdtype"]])
    if train:
        got = torch.autograd.grad([r, y], [leaf[n] for n in names], [s["dr"].float(), s["dy"].float()])
        out.update({"d" + n: g for n, g in zip(names, got)})
    return out


def _plain_clip(s):
    parts = {m: [g for g, k in zip(s["grads"], s["matrix"]) if k == m] for m in (True, False)}
    flat = {m: torch.cat(p).float() for m, p in parts.items()}
    # sums of up to a thousand million squares: 64 bits
    norm = (flat[True].square().sum(dtype=torch.float64) +
            flat[False].square().sum(dtype=torch.float64)).sqrt()
    out = {"norm": norm.float()}
    if s["op"] == "clip":
        c = (s["max_norm"] / norm).clamp(max=1.0).float()
        for m, name in ((True, "matrices"), (False, "vectors")):
            out[name] = (flat[m] * c).to(s["flat"][m].dtype)
    return out


# -------------------------------------------------------------------- run --
def run(state):
    s = state
    op = s["op"]
    if not own:
        plain = _plain_embed if op.startswith("embed") else _plain_norm if op.startswith("norm") else _plain_clip
        return plain(s)
    import selective_state_space_30_amd as ssm
    if op.startswith("embed"):
        out = {}
        if op != "embed_add":
            out["out"] = ssm.ssm_embed_fwd(s["ids"], s["weight"], s["factor"], dtype=DT[s["dtype"]])
        if op == "embed_train":
            out["dweight"] = ssm.ssm_embed_bwd(s["ids"], s["dy"], s["vocab"], s["factor"],
                                               dtype=DT[s["gdtype"]])
        elif op == "embed_add":
            out["dweight"] = ssm.ssm_embed_bwd(s["ids"], s["dy"], s["vocab"], s["factor"],
                                               dweight=s["grad"], accumulate=True)
        return out
    if op.startswith("norm"):
        r, y = ssm.ssm_layer_norm_fwd(s["x"], s["w"], s["b"], residual=s["res"], eps=EPS,
                                      dtype=DT[s["ydtype"]])
        out = {"y": y}
        if s["res"] is not None:
            out["r"] = r
        if op == "norm_train":
            d = ssm.ssm_layer_norm_bwd(s["x"], s["w"], s["b"], residual=s["res"], eps=EPS,
                                       dr=s["dr"], dy=s["dy"])
            out["dx"] = d["dx"]
            if s["res"] is not None:
                out["dres"] = d["dresidual"]
            if s["w"] is not None:
                out["dw"], out["db"] = d["dweight"], d["dbias"]
        return out
    if op == "grad_norm":
        return {"norm": ssm.ssm_grad_norm(s["grads"])}
    norm = ssm.ssm_grad_clip(s["grads"], s["max_norm"], out=s["out"])
    return {"norm": norm, "matrices": s["flat"][True], "vectors": s["flat"][False]}


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    """What run() gives for these inputs, in 64 bits: gathered and summed id by
    id, the layer norm's gradient by its formula, the norm tensor by tensor."""

    def embed(s):
        ids, factor, out = s["ids"].long(), s["factor"], {}
        if s["op"] != "embed_add":
            table = torch.cat([s["weight"].double(), s["weight"].new_zeros(1, s["dim"]).double()])
            row = ids.masked_fill((ids < 0) | (ids >= s["vocab"]), s["vocab"])
            out["out"] = table.index_select(0, row) * factor
        if s["op"] != "embed":
            keep = torch.nonzero((ids >= 0) & (ids < s["vocab"])).flatten()
            order = keep[torch.argsort(ids[keep], stable=True)]
            dw = torch.zeros(s["vocab"], s["dim"], dtype=torch.float64, device="cuda")
            if s["op"] == "embed_add":
                dw += s["grad"]
            which, count = torch.unique_consecutive(ids[order], return_counts=True)
            for part in torch.arange(s["dim"], device="cuda").split(512):
                # differences of a running sum over the sorted tokens
                run_ = s["dy"][:, part].double()[order].cumsum(0)
                last = run_[count.cumsum(0) - 1]
                dw[which[:, None], part] += factor * torch.diff(last, dim=0, prepend=torch.zeros_like(last[:1]))
            out["dweight"] = dw
        return out

    def norm(s):
        n = s["dim"]
        r = s["x"].double()
        if s["res"] is not None:
            r = r + s["res"]
        mean = r.sum(1, keepdim=True) / n
        inv = ((r - mean).pow(2).sum(1, keepdim=True) / n + EPS).pow(-0.5)
        hat = (r - mean) * inv
        out = {"y": hat}
        if s["w"] is not None:
            out["y"] = hat * s["w"].double() + s["b"].double()
        if s["res"] is not None:
            out["r"] = r
        if s["op"] == "norm_train":
            dy = s["dy"].double()
            g = dy if s["w"] is None else dy * s["w"].double()
            d = s["dr"].double() + inv * (g - g.sum(1, keepdim=True) / n -
                                          hat * ((g * hat).sum(1, keepdim=True) / n))
            out["dx"] = d
            if s["res"] is not None:
                out["dres"] = d
            if s["w"] is not None:
                out["dw"], out["db"] = (dy * hat).sum(0), dy.sum(0)
        return out

    def clip(s):
        total = math.sqrt(math.fsum(float(g.double().norm()) ** 2 for g in s["grads"]))
        out = {"norm": torch.tensor(total, dtype=torch.float64)}
        if s["op"] == "clip":
            c = min(1.0, s["max_norm"] / total)
            for m, name in ((True, "matrices"), (False, "vectors")):
                out[name] = torch.cat([g.double() * c for g, k in zip(s["grads"], s["matrix"]) if k == m])
        return out

    s = prepare(case, seed)
    return (embed if s["op"].startswith("embed") else norm if s["op"].startswith("norm") else clip)(s)


# -------------------------------------------------------------------- work --
def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"].startswith("embed"):
        T, V, D = c["tokens"], c["vocab"], c["dim"]
        real = T * 940 // 1024 if c["pad"] else T
        # rows of the weight that come at all
        rows = float((1.0 - (1.0 - _frequencies(V)) ** real).sum())
        bytes_, flops = 0.0, 0.0
        ids = T * (8 if c["wide_ids"] else 4)
        if c["op"] != "embed_add":
            bytes_ += ids + rows * D * size[c["wdtype"]] + T * D * size[c["dtype"]]
            flops += real * D
        if c["op"] != "embed":
            bytes_ += ids + real * D * size[c["dtype"]]
            bytes_ += 2 * rows * D * size[c["gdtype"]] if c["op"] == "embed_add" else V * D * size[c["gdtype"]]
            flops += 2 * real * D
        return {"bytes": bytes_, "flops": flops}
    if c["op"].startswith("norm"):
        n, x, r, y = c["rows"] * c["dim"], size[c["xdtype"]], size[c["rdtype"]], size[c["ydtype"]]
        r1 = r if c["residual"] else 0
        bytes_, flops = n * (x + 2 * r1 + y), 9.0 * n
        if c["op"] == "norm_train":
            # x and the residual again, the two gradients; those of x and of the
            # residual, which are one tensor where their types are the same
            bytes_ += n * (x + r1 + r + y) + n * (x + (r1 if r != x else 0))
            flops += 16.0 * n
        return {"bytes": float(bytes_), "flops": flops}
    shapes = _shapes(c)
    read = sum(n * (size[c["dtype"]] if m else 4) for n, m in shapes)
    wrote = sum(n * (size[c["odtype"]] if m else 4) for n, m in shapes) if c["op"] == "clip" else 0
    return {"bytes": float(read + wrote), "flops": 3.0 * sum(n for n, _ in shapes)}
