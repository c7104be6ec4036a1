"""The embedding, the layer norm and clipping as a model's training step and its
decoding use them, with linear attention between: against 64-bit arithmetic on
the CPU, captured in HIP graphs, on other streams, and two at once.

Tolerances: the step runs in fp32 (but for its last test), so a result is off by
its own sums' roundings (2e-5 of |r| + rms(r) for each operator, as in the
operators' own tests) and by what the operators before it leave; five stand in
a row, each passing errors on with a factor near 1: 5 * 2e-5, doubled for the
attention's gradients, which multiply two such results.
"""
import math

import pytest
import torch

import linattn_reference
import model_reference as ref
import selective_state_space_30_amd as ssm
from parity_metrics import report, scaled_max_err

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
B, L, H, D, V = 2, 40, 4, 16, 50
W = H * D
TOL = 2e-4


def check(got, want, what, tol=TOL):
    assert scaled_max_err(got, want) <= tol, "%s: %s" % (what, report(got, want))


def make(seed=0, dtype=F32):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    ids = torch.randint(0, V, (B, L), generator=gen)
    ids[0, L - 5:] = -1  # the shorter sequence's padding
    return {"ids": ids, "weight": r(V, W), "w1": 1 + 0.2 * r(W), "b1": 0.2 * r(W),
            "w2": 1 + 0.2 * r(W), "b2": 0.2 * r(W), "g": -torch.rand(B, L, H, generator=gen),
            "dy": r(B, L, W).to(dtype)}


def step(p, max_norm, dtype=F32):
    """Embedding, norm, linear attention, sum and norm; the gradients of the
    weights for a gradient dy of the last norm's result, clipped."""
    x = ssm.ssm_embed_fwd(p["ids"], p["weight"], 2.0)
    _, a = ssm.ssm_layer_norm_fwd(x, p["w1"], p["b1"], dtype=dtype)
    heads = a.view(B, L, H, D)
    o, _ = ssm.ssm_linattn_fwd(heads, heads, heads, p["g"])
    o = o.reshape(B, L, W)
    r, y = ssm.ssm_layer_norm_fwd(o, p["w2"], p["b2"], residual=x)
    d2 = ssm.ssm_layer_norm_bwd(o, p["w2"], p["b2"], residual=x, dy=p["dy"])
    da = ssm.ssm_linattn_bwd(heads, heads, heads, p["g"], do=d2["dx"].view(B, L, H, D),
                             want_dh0=False)
    da = (da["dq"].float() + da["dk"].float() + da["dv"].float()).to(dtype).view(B, L, W)
    d1 = ssm.ssm_layer_norm_bwd(x, p["w1"], p["b1"], dr=d2["dresidual"], dy=da)
    dw = ssm.ssm_embed_bwd(p["ids"], d1["dx"], V, 2.0)
    grads = [dw, d1["dweight"], d1["dbias"], d2["dweight"], d2["dbias"]]
    norm = ssm.ssm_grad_clip(grads, max_norm)
    return [y, r, norm] + grads


def reference(p, max_norm):
    leaf = {n: p[n].double().requires_grad_() for n in ("weight", "w1", "b1", "w2", "b2")}
    there = (p["ids"] >= 0).unsqueeze(-1)
    x = leaf["weight"][p["ids"].clamp(min=0)] * 2.0 * there
    _, a = ref.layer_norm(x, leaf["w1"], leaf["b1"])
    heads = a.view(B, L, H, D)
    o, _ = linattn_reference.batch(heads, heads, heads, p["g"].double(), D ** -0.5)
    r, y = ref.layer_norm(o.reshape(B, L, W), leaf["w2"], leaf["b2"], residual=x)
    got = torch.autograd.grad((y * p["dy"].double()).sum(), list(leaf.values()))
    norm, grads = ref.grad_clip(got, max_norm)
    return [y.detach(), r.detach(), torch.tensor(norm, dtype=torch.float64)] + grads


def test_training_step():
    p = make()
    got = step({n: t.to(DEV) for n, t in p.items()}, 3.0)
    want = reference(p, 3.0)
    assert float(want[2]) > 3.0
    for name, g, w in zip(("y", "r", "norm", "dweight", "dw1", "db1", "dw2", "db2"), got, want):
        check(g, w, name)
    assert not got[3][~torch.isin(torch.arange(V), p["ids"]).to(DEV)].any()


def test_training_step_in_bf16_runs_and_is_clipped():
    p = {n: t.to(DEV) for n, t in make(dtype=BF16).items()}
    x = p["weight"].to(BF16)
    got = step(dict(p, weight=x), 3.0, BF16)
    assert got[0].dtype == BF16 and all(torch.isfinite(t).all() for t in got)
    assert abs(float(ssm.ssm_grad_norm(got[3:])) - 3.0) < 1e-5


def test_micro_batches_add_up():
    """Two halves of a batch, the second added to the first's gradient, with the
    norm over both halves' processes given."""
    p = make(3)
    dy = torch.randn(B, L, W, generator=torch.Generator().manual_seed(4))
    ids = p["ids"].to(DEV)
    whole = ssm.ssm_embed_bwd(ids, dy.to(DEV), V)
    part = ssm.ssm_embed_bwd(ids[:1], dy[:1].to(DEV), V)
    ssm.ssm_embed_bwd(ids[1:], dy[1:].to(DEV), V, dweight=part, accumulate=True)
    check(part, whole, "dweight", 2e-5)
    squares = sum(ssm.ssm_grad_norm([t]).double() ** 2 for t in (whole, part))
    norm = squares.sqrt().float()
    ssm.ssm_grad_clip([whole], 1.0, norm=norm)
    ssm.ssm_grad_clip([part], 1.0, norm=norm)
    total = float(ssm.ssm_grad_norm([whole, part]))
    assert abs(total - 1.0) < 1e-5


def test_decoding():
    """A token at a time from an embedding in bf16 into an fp32 stream."""
    p = make(5)
    d = {n: t.to(DEV) for n, t in p.items()}
    weight = p["weight"].to(BF16)
    state = torch.zeros(B, H, D, D, device=DEV)
    want_state = torch.zeros(B, H, D, D, dtype=torch.float64)
    for t in range(6):
        ids = d["ids"][:, t].to(torch.int32)
        x = ssm.ssm_embed_fwd(ids, weight.to(DEV), dtype=F32)
        _, a = ssm.ssm_layer_norm_fwd(x, d["w1"], d["b1"])
        heads = a.view(B, H, D)
        o = ssm.ssm_linattn_step(state, heads, heads, heads, d["g"][:, t].contiguous())
        r, y = ssm.ssm_layer_norm_fwd(o.view(B, W), d["w2"], d["b2"], residual=x, r=x)
        assert r is x
        wx = ref.embed(p["ids"][:, t], weight, 1.0)
        wh = ref.layer_norm(wx, p["w1"], p["b1"])[1].view(B, H, D)
        want_state = want_state * p["g"][:, t].double().exp()[..., None, None] + (
            wh.unsqueeze(-1) * wh.unsqueeze(-2))
        wo = (wh.unsqueeze(-2) @ want_state).squeeze(-2) * D ** -0.5
        wr, wy = ref.layer_norm(wo.view(B, W), p["w2"], p["b2"], residual=wx)
        check(r, wr, "r of token %d" % t)
        check(y, wy, "y of token %d" % t)


def test_step_captured_and_replayed_over_other_inputs():
    """Every replay gives the eager call's bits, with eager work between and the
    workspaces and outputs of the graph overwritten."""
    p = {n: t.to(DEV) for n, t in make(6).items()}
    step(p, 3.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(p, 3.0)
    for seed in (7, 8, 9):
        for n, t in make(seed).items():
            p[n].copy_(t)
        for t in got:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = step(p, 3.0)
        for a, b in zip(kept, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n", [3000, 20000, 140000])
def test_embedding_gradient_captured(n):
    """The short sort and both long ones, whole and added."""
    gen = torch.Generator().manual_seed(n)
    ids = torch.randint(-1, 900, (n,), generator=gen).to(DEV)
    dy = torch.randn(n, 24, generator=gen).to(DEV)
    old = torch.randn(900, 24, generator=gen).to(DEV)
    grad = old.clone()

    def run():
        grad.copy_(old)
        ssm.ssm_embed_bwd(ids, dy, 900, dweight=grad, accumulate=True)
        return ssm.ssm_embed_bwd(ids, dy, 900)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for k in range(3):
        ids.copy_(torch.randint(-1, 900, (n,), generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        a, b = got.clone(), grad.clone()
        want = run()
        assert torch.equal(a, want) and torch.equal(b, grad)
        got.fill_(float("nan"))


def _calls():
    gen = torch.Generator().manual_seed(31)
    r = lambda *s, dtype=F32: torch.randn(*s, generator=gen).to(dtype).to(DEV)  # noqa: E731
    ids = torch.randint(0, 500, (20000,), generator=gen).to(DEV)
    w, dy = r(500, 96), r(20000, 96, dtype=BF16)
    x, res, dx = (r(3000, 600, dtype=BF16) for _ in range(3))
    nw, nb = r(600), r(600)
    grads = [r(100000), r(333, dtype=BF16), r(1)]
    return [
        (ssm.ssm_embed_fwd, lambda: dict(ids=ids, weight=w)),
        (ssm.ssm_embed_bwd, lambda: dict(ids=ids, dy=dy, vocab=500)),
        (ssm.ssm_layer_norm_fwd, lambda: dict(x=x, weight=nw, bias=nb, residual=res)),
        (ssm.ssm_layer_norm_bwd, lambda: dict(x=x, weight=nw, bias=nb, residual=res, dr=dx, dy=dx)),
        (ssm.ssm_grad_norm, lambda: dict(grads=grads)),
        (ssm.ssm_grad_clip, lambda: dict(grads=grads, max_norm=1.0,
                                         out=[torch.empty_like(g) for g in grads])),
    ]


def _tensors(result):
    if isinstance(result, dict):
        return [result[n] for n in sorted(result)]
    return list(result) if isinstance(result, tuple) else [result]


@pytest.mark.parametrize("which", range(6))
@pytest.mark.parametrize("positional", [True, False])
def test_outputs_and_workspace_belong_to_the_stream(monkeypatch, which, positional):
    import inspect
    call, make_args = _calls()[which]
    want = _tensors(call(**make_args()))
    side = torch.cuda.Stream()
    args = make_args()
    torch.cuda.synchronize()
    seen = []

    def spy(real):
        def made(*a, **kw):
            t = real(*a, **kw)
            if t.is_cuda:
                seen.append(torch.cuda.current_stream(t.device).cuda_stream)
            return t
        return made
    monkeypatch.setattr(torch, "empty", spy(torch.empty))
    monkeypatch.setattr(torch, "empty_like", spy(torch.empty_like))
    if positional:
        names = list(inspect.signature(call).parameters)
        defaults = {n: p.default for n, p in inspect.signature(call).parameters.items()}
        got = call(*[args.get(n, defaults[n]) for n in names[:names.index("stream")]], side)
    else:
        got = call(stream=side, **args)
    torch.cuda.synchronize()
    assert seen and all(s == side.cuda_stream for s in seen), seen
    assert all(torch.equal(a, b) for a, b in zip(_tensors(got), want))


def test_two_streams_at_once():
    """Calls with workspaces of their own run side by side."""
    calls = _calls()
    want = [_tensors(c(**a())) for c, a in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            got.append([_tensors(c(stream=s, **a())) for c, a in calls])
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_norm_of_gradients_by_name_is_that_of_torch():
    """Without clipping, against torch's own."""
    gen = torch.Generator().manual_seed(2)
    params = [torch.nn.Parameter(torch.randn(n, generator=gen)) for n in (10, 1000, 77777)]
    for q in params:
        q.grad = torch.randn(q.shape, generator=gen)
    want = torch.nn.utils.clip_grad_norm_(params, math.inf)
    got = ssm.ssm_grad_norm([q.grad.to(DEV) for q in params])
    assert abs(float(got) - float(want)) < 1e-5 * float(want)

