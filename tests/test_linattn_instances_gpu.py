"""Every kernel that linear attention's dispatch reaches, by the classes of
the two head sizes (up to 64, 128 and 256), by whether heads of at most 64
columns share q and k in pairs, in 16-byte pieces and by elements, in several
segments, forward and gradients; resets and growth in the gradients.
Tolerances as in test_linattn_gpu.py."""
import pytest
import torch

from test_linattn_gpu import BF16, F32, Inputs, run_both

pytestmark = pytest.mark.gpu

SIZES = [(64, 40, 45), (128, 72, 97), (256, 160, 201)]  # class, whole pieces, odd
CASES = [(dtype, dk[0] if i == 0 else dk[i], dv[0] if i == 0 else dv[i], heads, qk_heads)
         for dtype in (BF16, F32) for dk in SIZES for dv in SIZES for i in (0, 1, 2)
         for heads, qk_heads in (((4, 2), (3, 3)) if dv[0] == 64 else ((2, 1),))
         if (dk[0], dv[0]) != (256, 256) or i < 2]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s_k%d_v%d_h%d_%d" % (
    ("bf16" if c[0] == BF16 else "f32",) + c[1:]))
def test_head_sizes(case):
    dtype, dk, dv, heads, qk_heads = case
    run_both(Inputs(dtype, (1, 300), 1, heads, qk_heads, dk, dv, "token", True, seed=dk + dv))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("at", [[0], [100], [64, 128], [299], [5, 6, 7, 150]])
def test_gradients_through_resets(dtype, at):
    """g = -inf: nothing passes, forward or backward, and dg is 0 there."""
    inp = Inputs(dtype, (1, 300), 1, 2, 1, 64, 64, "token", True, seed=40 + at[0])
    inp.g[0, at] = float("-inf")
    run_both(inp)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_through_packed_resets(dtype):
    inp = Inputs(dtype, (400,), 3, 2, 2, 64, 32, "token", True, seed=50)
    inp.g[[0, 130, 131, 399]] = float("-inf")
    run_both(inp, [0, 130, 270, 400])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_growth(dtype):
    """Positive g, between decays, of heads that grow and heads that decay."""
    inp = Inputs(dtype, (1, 300), 1, 2, 1, 64, 64, "token", True, seed=60)
    gen = torch.Generator().manual_seed(61)
    inp.g = 0.2 * torch.randn(1, 300, 2, generator=gen)
    inp.g[0, 150] = torch.tensor([3.0, -4.0])
    run_both(inp)
