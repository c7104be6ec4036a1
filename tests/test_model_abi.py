"""Refusals of the embedding, layer-norm and gradient-norm entry points, and of
their binding, without a GPU: each call below fails a check before the first
HIP call."""
import ctypes

import pytest
import torch

import selective_state_space_30_amd as ssm
from test_linattn_binding import current  # noqa: F401  (a fixture)

FAKE = 0x7F0000000000  # never dereferenced
STEP = 0x10000000
BF16, F32 = ssm.SSM_DTYPE_BF16, ssm.SSM_DTYPE_F32
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return ssm.load_library()


def at(i, off=0):
    return FAKE + i * STEP + off


EFWD = dict(ids=at(1), w=at(2), ws=256, out=at(3), tokens=100, vocab=50, dim=256, scale=1.0,
            index=1, wdtype=F32, dtype=BF16, stream=None)
EBWD = dict(ids=at(1), dy=at(2), dys=256, dw=at(3), tokens=1000, vocab=50, dim=256, scale=1.0,
            flags=0, index=1, dtype=BF16, wdtype=F32, ws=at(4), wsb=1 << 24, stream=None)
NFWD = dict(x=at(1), xs=256, res=at(2), rs=256, w=at(3), b=at(4), r=at(5), y=at(6), rows=8,
            dim=256, eps=1e-5, xdtype=BF16, rdtype=F32, dtype=BF16, stream=None)
NBWD = dict(x=at(1), xs=256, res=at(2), rs=256, w=at(3), dr=at(5), dy=at(6), dx=at(7), dres=at(8),
            dw=at(9), db=at(10), rows=8, dim=256, eps=1e-5, xdtype=BF16, rdtype=F32, dtype=BF16,
            ws=at(11), wsb=1 << 24, stream=None)

EMBED = [
    (dict(ids=None), INVALID), (dict(ids=at(1, 4)), INVALID), (dict(tokens=-1), INVALID),
    (dict(vocab=0), INVALID), (dict(dim=0), INVALID), (dict(tokens=1 << 28), UNSUPPORTED),
    (dict(vocab=1 << 30), UNSUPPORTED), (dict(tokens=(1 << 28) - 1, dim=1025), UNSUPPORTED), (dict(index=2), INVALID), (dict(index=-1), INVALID),
    (dict(dtype=2), INVALID), (dict(wdtype=7), INVALID), (dict(scale=NAN), INVALID),
    (dict(scale=INF), INVALID), (dict(ids=at(1, 2), index=0), INVALID),
]
EFWD_BAD = EMBED + [
    (dict(w=None), INVALID), (dict(out=None), INVALID), (dict(ws=255), INVALID),
    (dict(ws=(1 << 22) + 1), UNSUPPORTED), (dict(dim=65537, ws=70000), UNSUPPORTED),
    (dict(w=at(2, 2)), INVALID), (dict(out=at(3, 1)), INVALID), (dict(out=at(2)), INVALID),
    (dict(out=at(1)), INVALID), (dict(out=at(2, 256 * 50 * 4 - 2)), INVALID),
]
EBWD_BAD = EMBED + [
    (dict(dy=None), INVALID), (dict(dw=None), INVALID), (dict(dys=255), INVALID),
    (dict(dys=(1 << 22) + 1), UNSUPPORTED), (dict(dim=65537, dys=70000), UNSUPPORTED),
    (dict(flags=1), INVALID), (dict(flags=128), INVALID), (dict(dy=at(2, 1)), INVALID),
    (dict(dw=at(3, 2)), INVALID), (dict(dw=at(2)), INVALID), (dict(dw=at(1)), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE), (dict(ws=at(4, 128)), INVALID),
    (dict(ws=at(3)), INVALID), (dict(ws=at(2)), INVALID), (dict(ws=at(1)), INVALID),
]
NORM = [
    (dict(x=None), INVALID), (dict(rows=-1), INVALID), (dict(dim=0), INVALID),
    (dict(dim=16385, xs=20000, rs=20000), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(xdtype=2), INVALID), (dict(rdtype=2), INVALID), (dict(dtype=3), INVALID),
    (dict(dtype=F32), INVALID), (dict(xdtype=F32, rdtype=BF16), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(eps=INF), INVALID), (dict(xs=255), INVALID), (dict(rs=255), INVALID),
    (dict(xs=(1 << 22) + 1), UNSUPPORTED), (dict(rs=(1 << 22) + 1), UNSUPPORTED),
    (dict(x=at(1, 1)), INVALID), (dict(res=at(2, 2)), INVALID), (dict(w=at(3, 2)), INVALID),
    (dict(res=None), INVALID),
]
NFWD_BAD = NORM + [
    (dict(y=None), INVALID), (dict(b=at(4, 1)), INVALID), (dict(r=at(5, 2)), INVALID),
    (dict(y=at(6, 1)), INVALID), (dict(res=None, rdtype=BF16), INVALID), (dict(y=at(1)), INVALID),
    (dict(y=at(2)), INVALID), (dict(y=at(5)), INVALID), (dict(r=at(1)), INVALID),
    (dict(r=at(2, 4)), INVALID), (dict(r=at(2), rs=300), INVALID), (dict(y=at(3)), INVALID),
    (dict(r=at(4)), INVALID),
]
NBWD_BAD = NORM + [
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(res=None, rdtype=BF16), INVALID),
    (dict(dr=at(5, 2)), INVALID), (dict(dres=at(8, 2)), INVALID), (dict(dy=at(6, 1)), INVALID),
    (dict(dx=at(7, 1)), INVALID), (dict(dw=at(9, 2)), INVALID), (dict(db=at(10, 1)), INVALID),
    (dict(dx=at(1)), INVALID), (dict(dx=at(6)), INVALID), (dict(dres=at(2)), INVALID),
    (dict(dres=at(5)), INVALID), (dict(dx=at(8)), INVALID), (dict(dw=at(3)), INVALID),
    (dict(db=at(9)), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=64), WORKSPACE),
    (dict(ws=at(11, 64)), INVALID), (dict(ws=at(6)), INVALID), (dict(ws=at(7)), INVALID),
]
ALL = ([("ssm_embed_fwd", EFWD, b) for b in EFWD_BAD] +
       [("ssm_embed_bwd", EBWD, b) for b in EBWD_BAD] +
       [("ssm_layer_norm_fwd", NFWD, b) for b in NFWD_BAD] +
       [("ssm_layer_norm_bwd", NBWD, b) for b in NBWD_BAD])


@pytest.mark.parametrize("case", ALL, ids=lambda c: "%s %s" % (c[0], sorted(c[2][0].items(), key=str)))
def test_refused_before_any_hip_call(lib, case):
    name, base, (bad, status) = case
    assert set(bad) <= set(base), "no such argument"
    got = getattr(lib, name)(*{**base, **bad}.values())
    assert got == status, ssm.ssm_last_error()
    assert ssm.ssm_last_error()


def grads(**over):
    """Arguments of ssm_grad_clip for three tensors of 100, 0 and 7 elements."""
    a = dict(grads=[at(1), None, at(2)], sizes=[100, 0, 7], dtypes=[F32, BF16, BF16], outs=None,
             out_dtypes=None, n=3, max_norm=1.0, have=0, norm=at(5), ws=at(6), wsb=1 << 20,
             stream=None)
    a.update(over)

    def array(kind, v):
        return None if v is None else (kind * len(v))(*v)
    a["grads"] = array(ctypes.c_void_p, a["grads"])
    a["outs"] = array(ctypes.c_void_p, a["outs"])
    a["sizes"] = array(ctypes.c_int64, a["sizes"])
    a["dtypes"] = array(ctypes.c_int, a["dtypes"])
    a["out_dtypes"] = array(ctypes.c_int, a["out_dtypes"])
    return a


GRADS_BAD = [
    (dict(n=-1), INVALID), (dict(n=(1 << 24) + 1), UNSUPPORTED), (dict(grads=None), INVALID),
    (dict(sizes=None), INVALID), (dict(dtypes=None), INVALID),
    (dict(sizes=[100, -1, 7]), INVALID), (dict(sizes=[100, 0, 1 << 40]), UNSUPPORTED),
    (dict(dtypes=[F32, 2, F32]), INVALID), (dict(grads=[at(1), None, None]), INVALID),
    (dict(grads=[at(1, 2), None, at(2)]), INVALID), (dict(grads=[at(1), None, at(2, 1)]), INVALID),
    (dict(norm=None), INVALID), (dict(norm=at(5, 2)), INVALID), (dict(norm=at(1, 8)), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=8), WORKSPACE), (dict(ws=at(6, 8)), INVALID),
    (dict(ws=at(1)), INVALID), (dict(norm=at(6, 16)), INVALID),
]
OUT = dict(outs=[at(3), None, at(4)], out_dtypes=[BF16, BF16, F32])
CLIP_BAD = GRADS_BAD + [
    (dict(max_norm=-1.0), INVALID), (dict(max_norm=NAN), INVALID),
    # the same tensor twice, and parts of one
    (dict(grads=[at(1), None, at(1)], dtypes=[F32] * 3), INVALID),
    (dict(grads=[at(1), None, at(1, 396)], dtypes=[F32] * 3), INVALID),
    (dict(OUT, grads=[at(1), None, at(1, 396)]), INVALID),
    (dict(outs=[at(3), None, at(4)]), INVALID), (dict(out_dtypes=[F32] * 3), INVALID),
    (dict(OUT, outs=[at(3), None, None]), INVALID), (dict(OUT, outs=[at(3), None, at(4, 2)]), INVALID),
    (dict(OUT, out_dtypes=[BF16, F32, 5]), INVALID), (dict(OUT, outs=[at(3), None, at(3)]), INVALID),
    (dict(OUT, outs=[at(1), None, at(4)]), INVALID),      # in place, but of another type
    (dict(OUT, outs=[at(1, 4), None, at(4)]), INVALID),
    (dict(OUT, outs=[at(2), None, at(4)]), INVALID), (dict(OUT, outs=[at(3), None, at(6)]), INVALID),
    (dict(OUT, outs=[at(3), None, at(5)]), INVALID),
    (dict(norm=None, have=1), INVALID), (dict(norm=at(1), have=1), INVALID),
]


@pytest.mark.parametrize("bad", CLIP_BAD, ids=lambda c: str(sorted(c[0].items())))
def test_clip_refused_before_any_hip_call(lib, bad):
    assert lib.ssm_grad_clip(*grads(**bad[0]).values()) == bad[1], ssm.ssm_last_error()
    assert ssm.ssm_last_error()


@pytest.mark.parametrize("bad", GRADS_BAD, ids=lambda c: str(sorted(c[0].items())))
def test_norm_refused_before_any_hip_call(lib, bad):
    a = grads(**bad[0])
    assert lib.ssm_grad_norm(*[a[k] for k in ("grads", "sizes", "dtypes", "n", "norm", "ws", "wsb",
                                              "stream")]) == bad[1], ssm.ssm_last_error()


def test_sizes(lib):
    size = ctypes.c_size_t(0)
    assert lib.ssm_embed_bwd_workspace_size(1, 1, 1, None) == INVALID
    assert lib.ssm_embed_bwd_workspace_size(-1, 1, 1, ctypes.byref(size)) == INVALID
    assert lib.ssm_embed_bwd_workspace_size(1, 1, 70000, ctypes.byref(size)) == UNSUPPORTED
    assert lib.ssm_layer_norm_bwd_workspace_size(8, 64, None) == INVALID
    assert lib.ssm_layer_norm_bwd_workspace_size(8, 16385, ctypes.byref(size)) == UNSUPPORTED
    assert lib.ssm_grad_workspace_size(None) == INVALID
    assert ssm.ssm_embed_bwd_workspace_size(0, 10, 64) == 0
    assert ssm.ssm_embed_bwd_workspace_size(256, 10, 64) == 0  # no sort
    assert ssm.ssm_embed_bwd_workspace_size(257, 10, 64) > 0
    assert ssm.ssm_layer_norm_bwd_workspace_size(0, 64) == 0
    assert ssm.ssm_grad_workspace_size() % 256 == 0
    # the partial sums stay a fraction of what is summed
    assert ssm.ssm_embed_bwd_workspace_size(65536, 50000, 1024) < 65536 * 1024 * 2 // 2
    assert ssm.ssm_layer_norm_bwd_workspace_size(1 << 20, 1024) <= 1 << 23


CPU = torch.zeros(4, 8)
IDS = torch.zeros(4, dtype=torch.int64)


@pytest.mark.parametrize("call", [
    lambda: ssm.ssm_embed_fwd(IDS, CPU), lambda: ssm.ssm_embed_fwd([0, 1], CPU),
    lambda: ssm.ssm_embed_fwd(IDS.float(), CPU), lambda: ssm.ssm_embed_fwd(IDS, CPU[0]),
    lambda: ssm.ssm_embed_bwd(IDS, CPU, 5), lambda: ssm.ssm_embed_bwd(IDS.short(), CPU, 5),
    lambda: ssm.ssm_layer_norm_fwd(CPU), lambda: ssm.ssm_layer_norm_fwd(CPU.half()),
    lambda: ssm.ssm_layer_norm_bwd(CPU, dy=CPU), lambda: ssm.ssm_layer_norm_bwd(CPU),
    lambda: ssm.ssm_grad_norm([CPU]), lambda: ssm.ssm_grad_norm(CPU),
    lambda: ssm.ssm_grad_norm([None]), lambda: ssm.ssm_grad_clip([CPU], 1.0),
    lambda: ssm.ssm_grad_clip(CPU, 1.0),
], ids=range(15))
def test_binding_refuses_without_a_device_tensor(call):
    with pytest.raises((TypeError, ValueError)):
        call()


def test_elements_without_gaps_in_any_order():
    t = torch.zeros(3, 4, 5)
    for good in (t, t.transpose(0, 2), t.permute(1, 0, 2), t[:1], t[1:, :, :], t[:, :1, :1][:1]):
        assert ssm._fills_its_memory(good)
    for bad in (t[:, ::2], t[:, :, 1:], t[::2], t[:1].expand(3, 4, 5), t[0, 0, :1].expand(2)):
        assert not ssm._fills_its_memory(bad)


def test_a_lists_first_tensor_and_stream(current):  # noqa: F811
    """The calls on lists run with their stream as torch's current one."""
    import inspect
    for call in (ssm.ssm_grad_norm, ssm.ssm_grad_clip):
        seen = []

        def body(*args, **kwargs):
            seen.append(list(current))
        body.__signature__ = inspect.signature(call)
        wrapped = ssm._on_device(body)
        n = list(inspect.signature(call).parameters).index("stream")
        side = object()
        wrapped([CPU], *[None] * (n - 1), side)
        wrapped([], stream=side)
        wrapped(grads=[None], stream=side)
        wrapped([CPU])
        assert seen == [[side]] * 3 + [[]]
