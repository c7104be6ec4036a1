"""Refusals of the linear-attention and block-norm entry points, without a
GPU: each call below fails a check before the first HIP call."""
import ctypes

import pytest
import torch

import selective_state_space_30_amd as ssm

FAKE = 0x7F0000000000  # never dereferenced
STEP = 0x10000000
BF16, F32 = ssm.SSM_DTYPE_BF16, ssm.SSM_DTYPE_F32


@pytest.fixture(scope="module")
def lib():
    return ssm.load_library()


def at(i, off=0):
    return FAKE + i * STEP + off


FWD = dict(q=at(1), qs=128, k=at(2), ks=128, v=at(3), vs=256, g=at(4), flags=0, scale=1.0, h0=at(5),
           cu=None, o=at(6), hf=at(7), tokens=128, nseq=2, heads=4, qk_heads=2, dk=64, dv=64,
           dtype=BF16, ws=None, wsb=0, stream=None)
BWD = dict(q=at(1), qs=128, k=at(2), ks=128, v=at(3), vs=256, g=at(4), flags=0, scale=1.0, h0=at(5),
           cu=None, do=at(6), dh=at(7), dq=at(8), dk_=at(9), dv_=at(10), dg=at(11), dh0=at(12),
           tokens=128, nseq=2, heads=4, qk_heads=2, dk=64, dv=64, dtype=BF16, ws=at(13),
           wsb=1 << 26, stream=None)
STEPS = dict(state=at(1), q=at(2), qs=128, k=at(3), ks=128, v=at(4), vs=256, g=at(5), flags=0,
             scale=1.0, slots=at(6), o=at(7), batch=4, nslots=4, heads=4, qk_heads=2, dk=64, dv=64,
             dtype=BF16, stream=None)
NFWD = dict(x=at(1), xs=256, w_post=at(2), z=at(3), zs=256, scale=at(4), res=at(5), rs=256,
            w_pre=at(6), r=at(7), y=at(8), rows=8, dim=256, groups=4, eps=1e-5, dtype=BF16,
            rdtype=F32, stream=None)
NBWD = dict(x=at(1), xs=256, w_post=at(2), z=at(3), zs=256, scale=at(4), res=at(5), rs=256,
            w_pre=at(6), dr=at(7), dy=at(8), dx=at(9), dw_post=at(10), dz=at(11), dscale=at(12),
            dres=at(13), dw_pre=at(14), rows=8, dim=256, groups=4, eps=1e-5, dtype=BF16, rdtype=F32,
            ws=at(15), wsb=1 << 26, stream=None)

SHARED = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(flags=1), 1), (dict(flags=16), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(heads=0), 1), (dict(qk_heads=0), 1), (dict(qk_heads=3), 1), (dict(dk=0), 1),
    (dict(dv=0), 1), (dict(dk=257, qs=600, ks=600), 2), (dict(dv=257, vs=2000), 2),
    (dict(qs=127), 1), (dict(ks=0), 1), (dict(vs=255), 1), (dict(vs=(1 << 22) + 1), 2),
    (dict(q=at(1, 1)), 1), (dict(v=at(3, 1)), 1), (dict(g=at(4, 2)), 1),
    (dict(heads=1 << 17, qk_heads=1 << 17), 2),
]
SEQS = SHARED + [
    (dict(tokens=-1), 1), (dict(nseq=0), 1), (dict(tokens=127), 1), (dict(tokens=1 << 31), 2),
    (dict(nseq=1 << 31, cu=at(20)), 2), (dict(cu=at(20, 2)), 1), (dict(h0=at(5, 2)), 1),
]
FWD_BAD = SEQS + [
    (dict(o=None), 1), (dict(o=at(6, 1)), 1), (dict(hf=at(7, 2)), 1),
    (dict(o=at(3)), 1), (dict(o=at(1, 128)), 1), (dict(hf=at(5)), 1), (dict(hf=at(6)), 1),
    (dict(o=at(4)), 1), (dict(cu=at(20), o=at(20)), 1),
    # few sequences, many tokens: segments, which need a workspace
    (dict(tokens=8192), 3), (dict(tokens=8192, ws=at(13), wsb=1000), 3),
    (dict(tokens=8192, ws=at(13, 16), wsb=1 << 27), 1),
    (dict(tokens=8192, ws=at(3), wsb=1 << 27), 1), (dict(tokens=8192, ws=at(6), wsb=1 << 27), 1),
]
BWD_BAD = SEQS + [
    (dict(do=None), 1), (dict(dq=None), 1), (dict(dk_=None), 1), (dict(dv_=None), 1),
    (dict(g=None), 1), (dict(do=at(6, 1)), 1), (dict(dg=at(11, 1)), 1), (dict(dh0=at(12, 2)), 1),
    (dict(dq=at(1)), 1), (dict(dk_=at(8)), 1), (dict(dv_=at(6)), 1), (dict(dg=at(4)), 1),
    (dict(dh0=at(7)), 1), (dict(ws=None), 3), (dict(wsb=100), 3), (dict(ws=at(13, 8)), 1),
    (dict(ws=at(6)), 1), (dict(ws=at(8)), 1),
]
STEP_BAD = SHARED + [
    (dict(state=None), 1), (dict(o=None), 1), (dict(state=at(1, 2)), 1), (dict(o=at(7, 1)), 1),
    (dict(batch=-1), 1), (dict(nslots=0), 1), (dict(slots=None, batch=5), 1),
    (dict(slots=at(6, 2)), 1), (dict(o=at(4)), 1), (dict(o=at(1, 64)), 1), (dict(state=at(2)), 1),
    (dict(state=at(6)), 1), (dict(batch=1 << 22), 2), (dict(nslots=1 << 31), 1),
]
NORM = [
    (dict(x=None), 1), (dict(rows=-1), 1), (dict(dim=0), 1), (dict(groups=0), 1),
    (dict(groups=3), 1), (dict(dim=16385, groups=1, xs=20000, zs=20000, rs=20000), 2),
    (dict(dim=8196, groups=4, xs=20000, zs=20000, rs=20000), 2), (dict(rows=1 << 22), 2),
    (dict(dtype=2), 1), (dict(rdtype=2), 1), (dict(dtype=F32, rdtype=BF16), 1),
    (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(w_post=None), 1), (dict(xs=255), 1), (dict(zs=255), 1), (dict(rs=255), 1),
    (dict(x=at(1, 1)), 1), (dict(z=at(3, 1)), 1), (dict(res=at(5, 2)), 1), (dict(w_post=at(2, 2)), 1),
]
NFWD_BAD = NORM + [
    (dict(y=None), 1), (dict(w_pre=None), 1), (dict(r=None, y=None, w_pre=None), 1),
    (dict(r=at(7, 1)), 1), (dict(y=at(8, 1)), 1), (dict(r=at(1)), 1), (dict(y=at(3)), 1),
    (dict(y=at(7)), 1), (dict(r=at(5, 4)), 1), (dict(r=at(5), rs=300), 1), (dict(y=at(5)), 1),
]
NBWD_BAD = NORM + [
    (dict(dx=None), 1), (dict(dy=None), 1), (dict(z=None), 1), (dict(scale=None), 1),
    (dict(res=None), 1), (dict(w_pre=None), 1), (dict(w_pre=None, dy=None), 1),
    (dict(w_post=None, groups=1), 1), (dict(dx=at(9, 1)), 1), (dict(dr=at(7, 2)), 1),
    (dict(dw_post=at(10, 2)), 1), (dict(dx=at(1)), 1), (dict(dz=at(9)), 1), (dict(dres=at(7)), 1),
    (dict(dw_pre=at(10)), 1), (dict(ws=None), 3), (dict(wsb=64), 3), (dict(ws=at(15, 4)), 1),
    (dict(ws=at(8)), 1), (dict(ws=at(9)), 1),
]
ALL = ([("ssm_linattn_fwd", FWD, b) for b in FWD_BAD] +
       [("ssm_linattn_bwd", BWD, b) for b in BWD_BAD] +
       [("ssm_linattn_step", STEPS, b) for b in STEP_BAD] +
       [("ssm_block_norm_fwd", NFWD, b) for b in NFWD_BAD] +
       [("ssm_block_norm_bwd", NBWD, b) for b in NBWD_BAD])


@pytest.mark.parametrize("case", ALL, ids=lambda c: "%s %s" % (c[0], sorted(c[2][0].items(), key=str)))
def test_refused_before_any_hip_call(lib, case):
    name, base, (bad, status) = case
    assert set(bad) <= set(base), "no such argument"
    got = getattr(lib, name)(*{**base, **bad}.values())
    assert got == status, ssm.ssm_last_error()
    assert ssm.ssm_last_error()


def test_sizes_and_plans(lib):
    size = ctypes.c_size_t(0)
    assert lib.ssm_linattn_workspace_size(64, 1, 0, 4, 4, 64, 64, BF16, None) == 1
    assert lib.ssm_linattn_workspace_size(64, 1, 0, 4, 4, 300, 64, BF16, ctypes.byref(size)) == 2
    assert lib.ssm_linattn_bwd_workspace_size(64, 1, 0, 4, 3, 64, 64, BF16, 0,
                                              ctypes.byref(size)) == 1
    assert lib.ssm_linattn_bwd_workspace_size(64, 1, 0, 4, 4, 64, 64, BF16, 3,
                                              ctypes.byref(size)) == 1
    assert lib.ssm_linattn_plan(64, 1, 0, 4, 4, 64, 64, BF16, 0, None) == 1
    assert lib.ssm_block_norm_bwd_workspace_size(8, 64, None) == 1
    # one short sequence, or many: nothing to cut, no workspace
    assert ssm.ssm_linattn_workspace_size(64, 1, 4, 4, 64, 64) == 0
    assert ssm.ssm_linattn_workspace_size(4096 * 64, 64, 16, 16, 128, 128) == 0
    assert ssm.ssm_linattn_workspace_size(8192, 1, 2, 2, 64, 64) > 0
    for packed in (False, True):
        for tokens, nseq in ((0, 1), (1, 1), (5000, 1), (5000, 4), (65536, 1)):
            for back in (0, 1, 2):
                p = ssm.ssm_linattn_plan(tokens, nseq, 8, 4, 128, 128, packed=packed, backward=back)
                assert p["segment"] % p["chunk"] == 0 and p["segments"] >= nseq
                assert back < 2 or p["segment"] <= 1024
                if packed:
                    # first slot of sequence i, whatever the lengths
                    assert p["segments"] >= tokens // p["segment"] + nseq


def test_binding_checks_its_arguments():
    q = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError):  # host tensors
        ssm.ssm_linattn_fwd(q, q, q)
    with pytest.raises(TypeError):
        ssm.ssm_linattn_fwd(q.double(), q.double(), q.double())
    with pytest.raises(ValueError):
        ssm.ssm_linattn_fwd(q[0], q[0], q[0])
    with pytest.raises(ValueError):
        ssm.ssm_linattn_bwd(q, q, q)
    with pytest.raises(TypeError):
        ssm.ssm_block_norm_fwd(torch.zeros(4, 8, dtype=torch.float16))
    with pytest.raises(ValueError):
        ssm.ssm_block_norm_fwd(torch.zeros(4, 8))
