"""Linear attention and the block norm on a stream other than torch's current
one, with ``stream`` given by position and by keyword: what a call allocates
belongs to that stream, and its results are those of the current stream."""
import inspect

import pytest
import torch

import selective_state_space_30_amd as ssm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def _calls():
    gen = torch.Generator().manual_seed(31)
    r = lambda *s, dtype=BF16: torch.randn(*s, generator=gen).to(dtype).to(DEV)  # noqa: E731
    L, H, d, n = 3000, 2, 64, 256
    q, k, v, do = (r(1, L, H, d) for _ in range(4))
    g = -torch.rand(1, L, H, generator=gen).to(DEV)
    state = r(3, H, d, d, dtype=torch.float32)
    x, z, res, dr, dy = (r(700, n) for _ in range(5))
    w = torch.linspace(0.5, 1.5, n, device=DEV)
    norm = dict(w_post=w, z=z, residual=res, w_pre=w, groups=4)
    one = lambda t: t[0, :3].contiguous()  # noqa: E731
    return [
        (ssm.ssm_linattn_fwd, lambda: dict(q=q, k=k, v=v, g=g)),
        (ssm.ssm_linattn_bwd, lambda: dict(q=q, k=k, v=v, g=g, do=do)),
        (ssm.ssm_linattn_step, lambda: dict(state=state.clone(), q=one(q), k=one(k), v=one(v),
                                            g=one(g))),
        (ssm.ssm_block_norm_fwd, lambda: dict(x=x, **norm)),
        (ssm.ssm_block_norm_bwd, lambda: dict(x=x, dr=dr, dy=dy, **norm)),
    ]


def _tensors(result):
    if isinstance(result, dict):
        return [result[n] for n in sorted(result)]
    return list(result) if isinstance(result, tuple) else [result]


@pytest.mark.parametrize("which", range(5))
@pytest.mark.parametrize("positional", [True, False])
def test_outputs_and_workspace_belong_to_the_stream(monkeypatch, which, positional):
    call, make = _calls()[which]
    want = _tensors(call(**make()))
    side = torch.cuda.Stream()
    args = make()
    torch.cuda.synchronize()
    seen = []
    real = torch.empty

    def empty(*a, **kw):
        t = real(*a, **kw)
        if t.is_cuda:
            seen.append(torch.cuda.current_stream(t.device).cuda_stream)
        return t
    monkeypatch.setattr(torch, "empty", empty)
    if positional:
        names = list(inspect.signature(call).parameters)
        defaults = {n: p.default for n, p in inspect.signature(call).parameters.items()}
        got = call(*[args.get(n, defaults[n]) for n in names[:names.index("stream")]], side)
    else:
        got = call(stream=side, **args)
    torch.cuda.synchronize()
    assert seen and all(s == side.cuda_stream for s in seen), seen
    assert all(torch.equal(a, b) for a, b in zip(_tensors(got), want))
