"""The block norm's gradients where a workgroup of the backward pass takes
three rows or more (it takes every 1024th): the next row's loads, its sums of
squares formed beside this row's sums, and the buffers that alternate, in
each form that the sums of the parts take.  Tolerances as in
test_block_norm_gpu.py."""
import pytest
import torch

import linattn_reference as ref
import selective_state_space_30_amd as ssm
from test_block_norm_gpu import ALL, BF16, DEV, F32, check, make

pytestmark = pytest.mark.gpu

CASES = [
    # dtype, rows, dim, groups, parts, wide
    (BF16, 3100, 64, 1, ALL, False),       # one wave a workgroup
    (BF16, 2100, 768, 1, ALL, True),
    (BF16, 3100, 512, 8, ALL, True),       # parts of a power of two of pieces
    (BF16, 3100, 1000, 5, ALL, False),     # parts of 25 pieces
    (BF16, 3100, 960, 80, ALL, True),      # parts of 12 elements: single ones
    (BF16, 3100, 130, 130, ALL, False),    # parts of one element
    (BF16, 3100, 384, 1, ("w_post", "z", "scale", "residual"), False),  # no dy
    (BF16, 3100, 640, 10, ("w_post", "z"), False),
    (BF16, 3100, 1000, 5, ("w_post", "scale", "residual"), True),
    (BF16, 3100, 320, 1, ("residual", "w_pre"), False),
    (BF16, 3100, 321, 1, ("z", "residual", "w_pre"), True),
    (BF16, 3100, 333, 3, ALL, False),      # odd width in parts of 111
    (BF16, 2051, 4096, 1, ALL, False),
    (F32, 3100, 256, 1, ALL, False),
    (F32, 3100, 256, 4, ALL, False),
    (F32, 3100, 96, 32, ALL, False),       # parts of 3
    (F32, 3100, 193, 1, ALL, False),
    (F32, 2100, 900, 9, ALL, False),       # parts of 25 pieces
    (F32, 3100, 192, 1, ("residual", "w_pre"), False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s_%dx%d_g%d_%s_%d" % (
    "bf16" if c[0] == BF16 else "f32", c[1], c[2], c[3], "".join(p[0] + p[-1] for p in c[4]), c[5]))
def test_three_rows_a_workgroup(case):
    dtype, rows, dim, groups, parts, wide = case
    inp, dr, dy = make(dtype, rows, dim, parts, wide, seed=rows + dim + groups)
    # rows of different sizes, so that one row's sums do not pass for another's
    factor = torch.exp2(torch.arange(rows).remainder(7) - 3.0)[:, None]
    for n in ("x", "residual"):
        if inp[n] is not None:
            inp[n] = (inp[n].float() * factor).to(inp[n].dtype)
    d = {n: None if t is None else t.to(DEV) for n, t in inp.items()}
    h = {n: None if t is None else t.double() for n, t in inp.items()}
    got = ssm.ssm_block_norm_bwd(**d, groups=groups, dr=dr.to(DEV),
                                 dy=None if dy is None else dy.to(DEV))
    want = ref.block_norm_gradients(h, groups, 1e-5, dr.double(),
                                    None if dy is None else dy.double())
    assert set(got) == set(want)
    for n in want:
        check(got[n], want[n], n)
        # row by row, so that large rows hide no small one's error; but where a
        # part is one element, dx = s h w_post (1 - s^2 x^2) cancels to eps s^2
        # of its terms in the rows of large x, which 32 bits do not hold
        if want[n].dim() == 2 and (n != "dx" or groups < dim):
            for k in range(7):
                check(got[n][k::7], want[n][k::7], "%s of rows %d mod 7" % (n, k))


@pytest.mark.parametrize("groups", [1, 4, 5])
def test_three_rows_a_workgroup_without_gradient_of_r(groups):
    inp, _, dy = make(BF16, 3100, 320, ALL, seed=groups)
    d = {n: t.to(DEV) for n, t in inp.items()}
    got = ssm.ssm_block_norm_bwd(**d, groups=groups, dy=dy.to(DEV))
    want = ref.block_norm_gradients({n: t.double() for n, t in inp.items()}, groups, 1e-5, None,
                                    dy.double())
    for n in want:
        check(got[n], want[n], n)
