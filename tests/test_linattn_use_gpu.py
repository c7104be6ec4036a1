"""Linear attention and the block norm as a layer uses them together, and the
calls around them: a training step through a layer against autograd in 64
bits, prompts then decoding, HIP graphs, streams, empty inputs.

Tolerances: where the whole layer runs in fp32, the library's fp32 bar, 1e-4
on the scaled error; replays and other streams give the same bits."""
import pytest
import torch

import linattn_reference as ref
import selective_state_space_30_amd as ssm
from parity_metrics import report, scaled_max_err

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


def check(got, want, what, tol=1e-4):
    assert scaled_max_err(got, want) <= tol, "%s: %s" % (what, report(got, want))


class Layer:
    """x -> norm -> q, k, v, z, g -> linear attention -> norm of each head,
    gated -> projection -> residual sum and next norm."""

    def __init__(self, dim, H, Hk, dk, dv, seed):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
        self.H, self.Hk, self.dk, self.dv = H, Hk, dk, dv
        self.w = {n: r(dim, c) / dim ** 0.5 for n, c in
                  (("q", Hk * dk), ("k", Hk * dk), ("v", H * dv), ("z", H * dv), ("g", H))}
        self.w["o"] = r(H * dv, dim) / (H * dv) ** 0.5
        self.n1, self.nh, self.n2 = 1 + 0.2 * r(dim), 1 + 0.2 * r(H * dv), 1 + 0.2 * r(dim)

    def reference(self, x, h0):
        """x (B, L, dim) float64 with gradient; the residual and the next norm."""
        B, L, dim = x.shape
        flat = x.reshape(B * L, dim)
        _, a = ref.block_norm(flat, w_pre=self.n1)
        part = {n: a @ self.w[n] for n in ("q", "k", "v", "z", "g")}
        g = -torch.nn.functional.softplus(part["g"]).reshape(B, L, self.H)
        o, h = ref.batch(part["q"].reshape(B, L, self.Hk, self.dk),
                         part["k"].reshape(B, L, self.Hk, self.dk),
                         part["v"].reshape(B, L, self.H, self.dv), g, self.dk ** -0.5, h0)
        n, _ = ref.block_norm(o.reshape(B * L, -1), w_post=self.nh, z=part["z"], groups=self.H)
        r, y = ref.block_norm(n @ self.w["o"], residual=flat, w_pre=self.n2)
        return r, y, h


def test_a_layer_trained_and_served():
    B, L, dim, H, Hk, dk, dv = 2, 150, 96, 4, 2, 32, 24
    layer = Layer(dim, H, Hk, dk, dv, 1)
    gen = torch.Generator().manual_seed(2)
    r64 = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x64, h64 = r64(B, L, dim).requires_grad_(), r64(B, H, dk, dv).requires_grad_()
    dr64, dy64, dh64 = r64(B * L, dim), r64(B * L, dim), r64(B, H, dk, dv)
    rr, yy, hh = layer.reference(x64, h64)
    loss = (rr * dr64).sum() + (yy * dy64).sum() + (hh * dh64).sum()
    want_dx, want_dh0 = torch.autograd.grad(loss, (x64, h64))

    dev = lambda t: t.detach().to(F32).to(DEV).contiguous()  # noqa: E731
    w = {n: dev(t) for n, t in layer.w.items()}
    n1, nh, n2 = dev(layer.n1), dev(layer.nh), dev(layer.n2)
    x, h0, dr, dy, dh = (dev(t) for t in (x64, h64, dr64, dy64, dh64))
    flat = x.view(B * L, dim)
    # forward; one projection, its parts used in place
    names = ("q", "k", "v", "z", "g")
    W = torch.cat([w[n] for n in names], dim=1)
    sizes = [w[n].shape[1] for n in names]

    def project(rows):
        _, a = ssm.ssm_block_norm_fwd(rows, w_pre=n1)
        return dict(zip(names, (a @ W).split(sizes, dim=1)))

    part = project(flat)
    q, k = (part[n].view(B, L, -1).unflatten(-1, (Hk, dk)) for n in ("q", "k"))
    v, z = part["v"].view(B, L, -1).unflatten(-1, (H, dv)), part["z"]
    raw = part["g"].contiguous()
    g = -torch.nn.functional.softplus(raw).view(B, L, H)
    o, h = ssm.ssm_linattn_fwd(q, k, v, g, h0=h0)
    of = o.view(B * L, H * dv)
    n, _ = ssm.ssm_block_norm_fwd(of, w_post=nh, z=z, groups=H)
    out = n @ w["o"]
    r, y = ssm.ssm_block_norm_fwd(out, residual=flat, w_pre=n2)
    check(r, rr.detach(), "r")
    check(y, yy.detach(), "y")
    check(h, hh.detach(), "h")
    # backward
    b2 = ssm.ssm_block_norm_bwd(out, residual=flat, w_pre=n2, dr=dr, dy=dy)
    bn = ssm.ssm_block_norm_bwd(of, w_post=nh, z=z, groups=H, dr=b2["dx"] @ w["o"].T)
    ba = ssm.ssm_linattn_bwd(q, k, v, g, h0=h0, do=bn["dx"].view(B, L, H, dv), dh_final=dh)
    draw = -ba["dg"].view(B * L, H) * torch.sigmoid(raw)
    da = torch.cat([ba["dq"].view(B * L, -1), ba["dk"].view(B * L, -1), ba["dv"].view(B * L, -1),
                    bn["dz"], draw], dim=1) @ W.T
    b1 = ssm.ssm_block_norm_bwd(flat, w_pre=n1, dy=da)
    check((b1["dx"] + b2["dresidual"]).view(B, L, dim), want_dx, "dx")
    check(ba["dh0"], want_dh0, "dh0")
    # served: a prompt of 100 tokens in the slots of a cache, then token by token
    cache = torch.full((5, H, dk, dv), 3.0, device=DEV)
    slots = torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    _, cache[slots.long()] = ssm.ssm_linattn_fwd(
        q[:, :100].contiguous(), k[:, :100].contiguous(), v[:, :100].contiguous(),
        g[:, :100].contiguous(), h0=h0)
    for t in range(100, 110):
        p1 = project(x[:, t].contiguous())
        ot = ssm.ssm_linattn_step(cache, p1["q"].unflatten(-1, (Hk, dk)),
                                  p1["k"].unflatten(-1, (Hk, dk)), p1["v"].unflatten(-1, (H, dv)),
                                  -torch.nn.functional.softplus(p1["g"].contiguous()), slots=slots)
        nt, _ = ssm.ssm_block_norm_fwd(ot.view(B, H * dv), w_post=nh, z=p1["z"], groups=H)
        rt, yt = ssm.ssm_block_norm_fwd(nt @ w["o"], residual=x[:, t].contiguous(), w_pre=n2)
        check(rt, rr.detach().view(B, L, dim)[:, t], "r at %d" % t)
    assert (cache[[0, 2, 4]] == 3.0).all()


def inputs(L=700, dtype=BF16, seed=3):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k, v, do = (r(2, L, n, 64).to(dtype).to(DEV) for n in (2, 2, 4, 4))
    g, h0, dh = -torch.rand(2, L, 4, generator=gen).to(DEV), r(2, 4, 64, 64).to(DEV), r(
        2, 4, 64, 64).to(DEV)
    return q, k, v, g, h0, do, dh


def everything(t, out):
    """Each operator once, into the tensors of ``out``."""
    q, k, v, g, h0, do, dh = t
    ssm.ssm_linattn_fwd(q, k, v, g, h0=h0, o=out["o"], h_final=out["h"], workspace=out["ws"])
    ssm.ssm_linattn_bwd(q, k, v, g, h0=h0, do=do, dh_final=dh, out=out["grads"],
                        workspace=out["ws2"])
    ssm.ssm_linattn_step(out["state"], q[:, 0].contiguous(), k[:, 0].contiguous(),
                         v[:, 0].contiguous(), g[:, 0].contiguous(), o=out["step"])
    flat = out["o"].view(-1, 256)
    ssm.ssm_block_norm_fwd(flat, w_post=out["w"], z=do.view(-1, 256), residual=v.view(-1, 256),
                           w_pre=out["w"], groups=4, r=out["r"], y=out["y"])
    ssm.ssm_block_norm_bwd(flat, w_post=out["w"], z=do.view(-1, 256), residual=v.view(-1, 256),
                           w_pre=out["w"], groups=4, dr=do.view(-1, 256), dy=out["y"],
                           out=out["ngrads"], workspace=out["ws3"])


def buffers(L=700):
    e = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
    n = 2 * L
    out = {"o": e(2, L, 4, 64), "h": e(2, 4, 64, 64, dtype=F32), "step": e(2, 4, 64),
           "state": e(2, 4, 64, 64, dtype=F32), "r": e(n, 256), "y": e(n, 256),
           "w": torch.linspace(0.5, 1.5, 256, device=DEV),
           "grads": {"dq": e(2, L, 2, 64), "dk": e(2, L, 2, 64), "dv": e(2, L, 4, 64),
                     "dg": e(2, L, 4, dtype=F32), "dh0": e(2, 4, 64, 64, dtype=F32)},
           "ngrads": {"dx": e(n, 256), "dw_post": e(256, dtype=F32), "dz": e(n, 256),
                      "dresidual": e(n, 256), "dw_pre": e(256, dtype=F32)}}
    u8 = lambda b: torch.zeros(max(b, 256), dtype=torch.uint8, device=DEV)  # noqa: E731
    out["ws"] = u8(ssm.ssm_linattn_workspace_size(n, 2, 4, 2, 64, 64))
    out["ws2"] = u8(ssm.ssm_linattn_bwd_workspace_size(n, 2, 4, 2, 64, 64, want_dg=1))
    out["ws3"] = u8(ssm.ssm_block_norm_bwd_workspace_size(n, 256))
    return out


def results(out):
    return ([out[n].clone() for n in ("o", "h", "step", "state", "r", "y")] +
            [x.clone() for n in ("grads", "ngrads") for x in out[n].values()])


def test_captured_and_replayed():
    t = inputs()
    out = buffers()
    everything(t, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            everything(t, out)
    torch.cuda.current_stream().wait_stream(side)
    other = buffers()
    for replay in range(3):
        new = inputs(seed=20 + replay)
        for a, b in zip(t, new):
            a.copy_(b)
        out["state"].fill_(replay)
        for n in ("ws", "ws2", "ws3"):
            out[n].fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        other["state"].fill_(replay)
        everything(new, other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results(out), results(other))), replay


def test_another_stream():
    t = inputs(seed=5)
    out = buffers()
    everything(t, out)
    want = results(out)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q, k, v, g, h0, do, dh = t
    o, h = ssm.ssm_linattn_fwd(q, k, v, g, h0=h0, stream=s)
    d = ssm.ssm_linattn_bwd(q, k, v, g, h0=h0, do=do, dh_final=dh, stream=s)
    state = torch.zeros_like(h)
    s.wait_stream(torch.cuda.current_stream())
    st = ssm.ssm_linattn_step(state, q[:, 0], k[:, 0], v[:, 0], g[:, 0].contiguous(), stream=s)
    r, y = ssm.ssm_block_norm_fwd(o.view(-1, 256), w_post=out["w"], z=do.view(-1, 256),
                                  residual=v.view(-1, 256), w_pre=out["w"], groups=4, stream=s)
    s.synchronize()
    got = [o, h, st, state, r, y] + [d[n] for n in ("dq", "dk", "dv", "dg", "dh0")]
    for i, (a, b) in enumerate(zip(got, want[:11])):
        assert torch.equal(a, b), i


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_tokens(dtype):
    e = lambda *s: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
    h0 = torch.randn(2, 3, 16, 24, device=DEV)
    q, k, v = e(2, 0, 1, 16), e(2, 0, 1, 16), e(2, 0, 3, 24)
    g = torch.zeros(2, 0, 3, device=DEV)
    o, h = ssm.ssm_linattn_fwd(q, k, v, g, h0=h0)
    assert o.shape == v.shape and torch.equal(h, h0)
    d = ssm.ssm_linattn_bwd(q, k, v, g, h0=h0, do=v, dh_final=h0)
    assert torch.equal(d["dh0"], h0) and d["dg"].shape == g.shape
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    o, h = ssm.ssm_linattn_fwd(e(7, 1, 16), e(7, 1, 16), e(7, 3, 24), None, h0=h0, cu_seqlens=cu)
    assert torch.equal(h, h0)
    out = ssm.ssm_linattn_step(h0.clone(), e(0, 1, 16), e(0, 1, 16), e(0, 3, 24))
    assert out.shape == (0, 3, 24)


def test_offsets_outside_the_rows_touch_nothing_else():
    """Offsets beyond the rows, negative or falling are brought into range."""
    t, H, d = 40, 2, 16
    buf = torch.full((3 * t, H, d), 5.0, dtype=BF16, device=DEV)
    o = buf[t:2 * t]
    q = torch.randn(t, H, d, device=DEV).to(BF16)
    for cu in ([0, 30, 1000], [-50, 20, 40], [0, 30, 10], [100, 200, 300]):
        ssm.ssm_linattn_fwd(q, q, q, None, cu_seqlens=torch.tensor(cu, dtype=torch.int32,
                                                                    device=DEV), o=o)
        torch.cuda.synchronize()
        assert (buf[:t] == 5.0).all() and (buf[2 * t:] == 5.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nan_stays_in_its_sequence(dtype):
    """NaN in one packed sequence and in the rows outside all of them, and in
    idle rows and foreign slots of a step, reaches nothing else: the same bits
    as with finite values there."""
    cu = [5, 75, 140, 471]
    t, H, dk, dv = 480, 4, 64, 64
    gen = torch.Generator().manual_seed(21)
    r = lambda *s: torch.randn(*s, generator=gen).to(DEV)  # noqa: E731
    q, k = r(t, 2, dk).to(dtype), r(t, 2, dk).to(dtype)
    v, do, g = r(t, H, dv).to(dtype), r(t, H, dv).to(dtype), -torch.rand(t, H, generator=gen).to(DEV)
    h0, dh = r(3, H, dk, dv), r(3, H, dk, dv)
    off = torch.tensor(cu, dtype=torch.int32, device=DEV)

    def run(*a):
        q, k, v, do, g, h0, dh = a
        o, h = ssm.ssm_linattn_fwd(q, k, v, g, h0=h0, cu_seqlens=off)
        d = ssm.ssm_linattn_bwd(q, k, v, g, h0=h0, cu_seqlens=off, do=do, dh_final=dh)
        return [o] + [d[n] for n in ("dq", "dk", "dv", "dg")], [h, d["dh0"]]

    clean = (q, k, v, do, g, h0, dh)
    dirty = [x.clone() for x in clean]
    for x in dirty[:5]:
        x[:cu[0]] = x[cu[1]:cu[2]] = x[cu[3]:] = float("nan")
    for x in dirty[5:]:
        x[1] = float("nan")
    want, got = run(*clean), run(*dirty)
    for a, b in zip(want[0], got[0]):
        for rows in (slice(cu[0], cu[1]), slice(cu[2], cu[3])):
            assert torch.equal(a[rows], b[rows])
    for a, b in zip(want[1], got[1]):
        assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.isnan(b[1]).any()

    slots = torch.tensor([2, -1, 0], dtype=torch.int32, device=DEV)
    first = [x[:3].clone() for x in (q, k, v, g)]
    ref_state = h0.clone()
    ref_o = ssm.ssm_linattn_step(ref_state, *first, slots=slots)
    state = h0.clone()
    for x in first:
        x[1] = float("nan")
    state[1] = float("nan")
    o = ssm.ssm_linattn_step(state, *first, slots=slots)
    assert torch.equal(o, ref_o) and (o[1] == 0).all()
    assert torch.equal(state[[0, 2]], ref_state[[0, 2]]) and torch.isnan(state[1]).all()


def test_offsets_past_32_bits():
    """The last of three packed sequences lies more than 2^31 elements into v,
    o and their gradients, the last slot as far into the states."""
    t, H, dk, dv = 530000, 32, 16, 128
    cu = [100, 264000, 529000, 529900]
    gen = torch.Generator(device=DEV).manual_seed(22)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV, dtype=BF16)  # noqa: E731
    q, k, v, do = r(t, 1, dk), r(t, 1, dk), r(t, H, dv), r(t, H, dv)
    g = -torch.rand(t, H, generator=gen, device=DEV)
    off = torch.tensor(cu, dtype=torch.int32, device=DEV)
    own = slice(cu[2], cu[3])
    alone = [x[own][None] for x in (q, k, v, g)]
    o, h = ssm.ssm_linattn_fwd(q, k, v, g, cu_seqlens=off)
    o1, h1 = ssm.ssm_linattn_fwd(*alone)
    check(o[own].cpu(), o1[0].cpu().double(), "o", 2e-2)
    check(h[2:].cpu(), h1.cpu().double(), "h_final")
    del o
    d = ssm.ssm_linattn_bwd(q, k, v, g, cu_seqlens=off, do=do)
    d1 = ssm.ssm_linattn_bwd(*alone, do=do[own][None])
    for n in ("dq", "dk", "dv"):
        check(d[n][own].cpu(), d1[n][0].cpu().double(), n, 2e-2)
    check(d["dg"][own].cpu(), d1["dg"][0].cpu().double(), "dg")
    del d, v, do

    nslots, H, dk, dv = 8200, 16, 128, 128
    state = torch.zeros(nslots, H, dk, dv, device=DEV)
    state[nslots - 1].normal_(generator=gen)
    few = state[nslots - 2:].clone()
    a = (r(2, H, dk), r(2, H, dk), r(2, H, dv), -torch.rand(2, H, generator=gen, device=DEV))
    slots = torch.tensor([nslots - 1, nslots - 2], dtype=torch.int32, device=DEV)
    o = ssm.ssm_linattn_step(state, *a, slots=slots)
    o1 = ssm.ssm_linattn_step(few, *a, slots=slots - (nslots - 2))
    assert torch.equal(o, o1) and torch.equal(state[nslots - 2:], few)
    assert not state[:nslots - 2].any()
