"""Many packed prompts at once, of lengths from 0 to thousands of tokens:
three of them, first, longest and last, against the plain 64-bit recurrence.
Tolerances as in test_linattn_gpu.py."""
import random

import pytest
import torch

import linattn_reference as ref
import selective_state_space_30_amd as ssm
from test_linattn_gpu import check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def test_many_packed_prompts():
    nseq, H, dk, dv = 512, 80, 16, 16
    rng = random.Random(5)
    lens = [300] + [int(2 ** rng.uniform(0, 10)) for _ in range(nseq - 3)] + [0, 333]
    lens[100] = 1500
    offsets = [11]
    for n in lens:
        offsets.append(offsets[-1] + n)
    tokens = 262144
    assert offsets[-1] < tokens
    assert ssm.ssm_linattn_plan(tokens, nseq, H, 1, dk, dv, packed=True)["segments"] >= nseq
    gen = torch.Generator(device=DEV).manual_seed(17)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    q, k = r(tokens, 1, dk).bfloat16(), r(tokens, 1, dk).bfloat16()
    v, do = r(tokens, H, dv).bfloat16(), r(tokens, H, dv).bfloat16()
    g = -torch.rand(tokens, H, generator=gen, device=DEV)
    h0, dh = r(nseq, H, dk, dv), r(nseq, H, dk, dv)
    cu = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    o, h = ssm.ssm_linattn_fwd(q, k, v, g, 0.25, h0=h0, cu_seqlens=cu)
    d = ssm.ssm_linattn_bwd(q, k, v, g, 0.25, h0=h0, cu_seqlens=cu, do=do, dh_final=dh)
    assert torch.equal(h[nseq - 2], h0[nseq - 2]) and torch.equal(d["dh0"][nseq - 2], dh[nseq - 2])
    for i in (0, 100, nseq - 1):
        rows = slice(offsets[i], offsets[i + 1])
        a = [x[rows].cpu().double()[None] for x in (q, k, v, g, do)]
        s = [x[i:i + 1].cpu().double() for x in (h0, dh)]
        m = [x.abs() for x in a]
        sm = [x.abs() for x in s]
        want_o, want_h = ref.batch(*a[:4], 0.25, s[0])
        size_o, size_h = ref.batch(*m[:3], a[3], 0.25, sm[0])
        check(o[rows], want_o[0], "o of %d" % i, size_o[0])
        check(h[i], want_h[0], "h_final of %d" % i, size_h[0])
        want = ref.gradients(*a[:4], 0.25, s[0], a[4], s[1])
        size = ref.gradients(*m[:3], a[3], 0.25, sm[0], m[4], sm[1])
        size["dg"] = 2 * size["dg"].flip(-2).cumsum(-2).flip(-2)
        for n in ("dq", "dk", "dv", "dg"):
            check(d[n][rows], want[n][0], "%s of %d" % (n, i), size[n][0])
        check(d["dh0"][i], want["dh0"][0], "dh0 of %d" % i, size["dh0"][0])
