"""The embedding and its gradient (ssm_embed_fwd, _bwd) against their formula in
64 bits.

Tolerances, element by element.  Forward: the product's rounding (2^-24 of it)
and the output's (half a step: 2^-8 in bf16).  Gradient: a term passes at most
as many additions as its id has terms (less where runs of 32 are joined), one
product with the scale and one addition to what was there, each off by at most
2^-24 of what has been added so far, which the sum of absolute values bounds:
(n + 2) 2^-24 of that sum, and the output's half step.
"""
import pytest
import torch

import model_reference as ref
import selective_state_space_30_amd as ssm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24


def within(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    assert over.max() <= 0 if over.numel() else True, "%s: %g over the bound at %d" % (
        what, over.max(), over.argmax())


def check_rows(got, want):
    within(got.reshape(want.shape), want, (STEP[got.dtype] + 2 * U) * want.abs() + 1e-44, "out")


def check_gradient(got, want):
    dw, mag, count = want
    bound = (count.unsqueeze(1) + 2) * U * mag
    within(got, dw, bound + STEP[got.dtype] * (dw.abs() + bound), "dweight")


def make(n, vocab, kind, seed=0, index=torch.int64):
    gen = torch.Generator().manual_seed(seed)
    if kind == "even":
        ids = torch.randint(0, vocab, (n,), generator=gen)
    elif kind == "skewed":  # few ids have most tokens
        ids = (vocab * torch.rand(n, generator=gen) ** 12).long().clamp_(max=vocab - 1)
    elif kind == "one":
        ids = torch.full((n,), vocab // 2)
    elif kind == "padded":
        ids = torch.randint(0, vocab, (n,), generator=gen)
        ids[torch.rand(n, generator=gen) < 0.3] = -1
        ids[torch.rand(n, generator=gen) < 0.05] = vocab
    else:
        ids = torch.full((n,), -1)
    return ids.to(index)


CASES = [
    # tokens, vocab, dim, ids, weight's type, activations' type
    (1, 1, 1, "even", F32, F32),
    (1, 10, 64, "even", BF16, BF16),
    (8, 1000, 2560, "even", BF16, BF16),
    (31, 7, 100, "even", F32, BF16),
    (32, 7, 100, "one", F32, F32),
    (33, 7, 72, "one", BF16, F32),
    (64, 3, 8, "skewed", BF16, BF16),
    (65, 300, 513, "padded", BF16, BF16),      # a piece over 64 pieces
    (100, 300, 257, "padded", F32, F32),
    (255, 50, 7, "skewed", F32, BF16),         # rows shorter than a piece
    (256, 3, 300, "skewed", BF16, F32),        # the most tokens that are not sorted
    (256, 9, 90, "one", F32, BF16),
    (257, 50, 7, "skewed", F32, BF16),
    (257, 3, 300, "padded", F32, F32),
    (1000, 255, 129, "skewed", BF16, BF16),
    (1000, 256, 130, "even", BF16, BF16),      # the last id over one pass's 8 bits
    (4095, 257, 40, "even", F32, BF16),
    (4096, 5000, 33, "skewed", BF16, BF16),    # a whole tile of the sort
    (4097, 5000, 24, "padded", F32, F32),
    (5000, 65536, 16, "even", F32, BF16),      # three passes
    (9000, 70000, 12, "skewed", F32, BF16),
    (8192, 300, 1030, "skewed", BF16, BF16),   # the short sort beside the clearing
    (8193, 300, 1030, "even", F32, F32),
    (4100, 40, 4000, "skewed", F32, BF16),     # runs of 16 and of 32
    (6000, 40, 4000, "one", F32, BF16),
    (16384, 600, 20, "skewed", F32, BF16),
    (16385, 600, 20, "skewed", F32, BF16),
    (40000, 20, 16, "one", F32, BF16),         # a thousand runs of one id
    (70000, 3000, 24, "skewed", BF16, BF16),
    (262145, 3000, 9, "skewed", F32, BF16),    # 4 keys a thread of the long sort
    (1048577, 70000, 8, "padded", F32, BF16),  # places in a launch of their own
    (300, 40, 96, "none", BF16, BF16),         # padding alone
    (20, 5, 9001, "even", BF16, BF16),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%dx%d_%s_%s_%s" % (
    c[:4] + tuple("bf16" if t == BF16 else "f32" for t in c[4:])))
@pytest.mark.parametrize("index", [torch.int64, torch.int32], ids=["i64", "i32"])
def test_embed(case, index):
    n, vocab, dim, kind, wt, at = case
    ids = make(n, vocab, kind, seed=n + vocab, index=index)
    gen = torch.Generator().manual_seed(dim)
    w = torch.randn(vocab, dim, generator=gen).to(wt)
    dy = torch.randn(n, dim, generator=gen).to(at)
    scale = 1.0 if n % 2 else dim ** 0.5
    d_ids = ids.to(DEV)
    out = ssm.ssm_embed_fwd(d_ids, w.to(DEV), scale, dtype=at)
    assert out.dtype == at and out.shape == (n, dim)
    check_rows(out, ref.embed(ids, w, scale))
    got = ssm.ssm_embed_bwd(d_ids, dy.to(DEV), vocab, scale, dtype=wt)
    assert got.dtype == wt
    check_gradient(got, ref.embed_gradient(ids, dy, vocab, scale))
    old = torch.randn(vocab, dim, generator=gen).to(wt)
    grad = old.to(DEV)
    same = ssm.ssm_embed_bwd(d_ids, dy.to(DEV), vocab, scale, dweight=grad, accumulate=True)
    assert same is grad
    want = ref.embed_gradient(ids, dy, vocab, scale, old)
    check_gradient(grad, want)
    untouched = want[2] == 0
    assert torch.equal(grad.cpu()[untouched], old[untouched])


def test_no_tokens():
    ids = torch.zeros(0, dtype=torch.int64, device=DEV)
    w = torch.randn(9, 20, device=DEV)
    assert ssm.ssm_embed_fwd(ids, w).shape == (0, 20)
    dy = torch.zeros(0, 20, device=DEV)
    dw = torch.full((9, 20), float("nan"), device=DEV)
    ssm.ssm_embed_bwd(ids, dy, 9, dweight=dw)
    assert (dw == 0).all()
    keep = w.clone()
    ssm.ssm_embed_bwd(ids, dy, 9, dweight=w, accumulate=True)
    assert torch.equal(w, keep)


def test_shapes_slices_and_given_outputs():
    gen = torch.Generator().manual_seed(4)
    ids = make(42, 30, "padded", seed=4).view(2, 3, 7)
    wide = torch.randn(30, 50, generator=gen).to(DEV)
    for lo in (0, 3):
        w = wide[:, lo:lo + 41]
        out = torch.full((2, 3, 7, 41), float("nan"), dtype=BF16, device=DEV)
        assert ssm.ssm_embed_fwd(ids.to(DEV), w, 2.0, out=out) is out
        check_rows(out, ref.embed(ids, w.cpu(), 2.0))
        dy = torch.randn(2, 3, 7, 50, generator=gen).to(BF16).to(DEV)[..., lo:lo + 41]
        dw = torch.full((30, 41), float("nan"), device=DEV)
        assert ssm.ssm_embed_bwd(ids.to(DEV), dy, 30, dweight=dw) is dw
        check_gradient(dw, ref.embed_gradient(ids, dy.cpu(), 30, 1.0))


def test_extreme_ids():
    """Ids whose low 32 bits would be a row."""
    w = torch.arange(1.0, 5.0, device=DEV).unsqueeze(1)
    ids = torch.tensor([2 ** 32 + 1, -2 ** 32, 2 ** 63 - 1, -2 ** 63, 3, 4], device=DEV)
    out = ssm.ssm_embed_fwd(ids, w)
    assert out.flatten().tolist() == [0, 0, 0, 0, 4, 0]
    dw = ssm.ssm_embed_bwd(ids, torch.ones(6, 1, device=DEV), 4)
    assert dw.flatten().tolist() == [0, 0, 0, 1]


def test_not_finite_stays_in_its_row_and_column():
    ids = make(500, 20, "even", seed=9)
    dy = torch.randn(500, 40)
    dy[7, 3], dy[8, 4] = float("nan"), float("inf")
    dw = ssm.ssm_embed_bwd(ids.to(DEV), dy.to(DEV), 20).cpu()
    bad = ~torch.isfinite(dw)
    assert bad.sum() == 2 and dw[ids[7], 3].isnan() and dw[ids[8], 4] == float("inf")
    # NaN in rows that no token has, and under padding, goes nowhere
    w = torch.full((20, 40), float("nan"))
    w[3] = 1.0
    out = ssm.ssm_embed_fwd(torch.tensor([3, -1, 20], device=DEV), w.to(DEV)).cpu()
    assert (out[0] == 1).all() and (out[1:] == 0).all()
    dy = torch.full((3, 40), float("nan"))
    dy[0] = 1.0
    dw = ssm.ssm_embed_bwd(torch.tensor([3, -1, 20], device=DEV), dy.to(DEV), 20).cpu()
    assert (dw[3] == 1).all() and dw.sum() == 40


@pytest.mark.parametrize("n", [5000, 30000])
def test_deterministic_whatever_the_workspace_holds(n):
    ids = make(n, 400, "skewed", seed=3).to(DEV)
    dy = torch.randn(n, 136, device=DEV).to(BF16)
    a = ssm.ssm_embed_bwd(ids, dy, 400)
    size = ssm.ssm_embed_bwd_workspace_size(n, 400, 136)
    for fill in (0, 255):
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(ssm.ssm_embed_bwd(ids, dy, 400, workspace=ws), a)


def test_short_sort_beside_a_large_weight():
    """16384 tokens and a weight of 256 MB, as one workgroup sorts them."""
    ids = make(16384, 66000, "skewed", seed=8)
    dy = torch.randn(16384, 1024, generator=torch.Generator().manual_seed(8))
    got = ssm.ssm_embed_bwd(ids.to(DEV), dy.to(DEV), 66000)
    rows = torch.unique(ids)
    want = ref.embed_gradient(torch.searchsorted(rows, ids), dy, rows.numel(), 1.0)
    check_gradient(got[rows.to(DEV)], want)
    got[rows.to(DEV)] = 0
    assert not got.any()


@pytest.mark.slow
def test_offsets_past_32_bits():
    """A weight of over 2^32 bytes and 2^31 elements."""
    vocab, dim = 540000, 4096
    ids = torch.tensor([vocab - 1, 0, vocab - 1, 17, 524288], device=DEV)
    dy = torch.randn(5, dim, device=DEV).to(BF16)
    dw = torch.full((vocab, dim), float("nan"), dtype=BF16, device=DEV)
    ssm.ssm_embed_bwd(ids, dy, vocab, dweight=dw)
    want = torch.stack([dy[1], dy[3], dy[4], (dy[0].float() + dy[2].float()).to(BF16)])
    rows = torch.tensor([0, 17, 524288, vocab - 1], device=DEV)
    assert torch.equal(dw[rows], want)
    assert torch.equal(ssm.ssm_embed_fwd(ids, dw)[[1, 3, 4, 0]], want)
    dw[rows] = 0
    for part in dw.split(100000):
        assert not part.any()
