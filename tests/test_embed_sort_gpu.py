"""The gradient of the embedding at every number of passes of its sorts, whose
keys are 0..vocab (vocab: padding) in digits of up to 9 bits: one pass up to 511
ids, two up to 262143, three from 262144 on.  Each with the sort by one workgroup
(up to 4096 tokens, or up to 8192 as a new gradient), with the long sort of one
key a thread (up to 131072 tokens) and of four, and, over 256 tiles of it, with
the places in a launch of their own.

Bounds as in test_embed_gpu.py: half a step of the output and 2^-24 an addition
of what has been added so far.
"""
import pytest
import torch

import model_reference as ref
import selective_state_space_30_amd as ssm
from test_embed_gpu import BF16, DEV, F32, check_gradient, check_rows

pytestmark = pytest.mark.gpu

PASSES = {511: 1, 512: 2, 262143: 2, 262144: 3, 300007: 3}
CASES = ([(n, vocab) for vocab in PASSES for n in (257, 1500, 5000, 20000, 131072, 140001)] +
         [(1050000, 511), (1050000, 262144), (1050000, 300007)])


def make(n, vocab, seed):
    """A third of the tokens anywhere, a third among the last ids, a tenth of one
    id, padding."""
    gen = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, vocab, (n,), generator=gen)
    kind = torch.rand(n, generator=gen)
    last = vocab - 1 - torch.randint(0, min(vocab, 40), (n,), generator=gen)
    ids = torch.where(kind < 0.33, last, ids)
    ids[(0.33 <= kind) & (kind < 0.43)] = vocab // 2
    ids[(0.43 <= kind) & (kind < 0.5)] = -1
    ids[(0.5 <= kind) & (kind < 0.55)] = vocab
    ids[0], ids[-1] = vocab - 1, 0
    return ids


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%d" % c)
def test_passes(case):
    n, vocab = case
    dim = 7 if n % 2 else 4
    at, wt = (BF16, F32) if vocab % 2 else (F32, BF16)
    index = torch.int32 if n % 5 else torch.int64
    ids = make(n, vocab, seed=n + vocab).to(index)
    gen = torch.Generator().manual_seed(vocab)
    dy = torch.randn(n, dim, generator=gen).to(at)
    old = torch.randn(vocab, dim, generator=gen).to(wt)
    d_ids, d_dy = ids.to(DEV), dy.to(DEV)
    got = ssm.ssm_embed_bwd(d_ids, d_dy, vocab, 0.5, dtype=wt)
    want = ref.embed_gradient(ids, dy, vocab, 0.5)
    check_gradient(got, want)
    assert not got.cpu()[want[2] == 0].any()
    grad = old.to(DEV)
    ssm.ssm_embed_bwd(d_ids, d_dy, vocab, 0.5, dweight=grad, accumulate=True)
    want = ref.embed_gradient(ids, dy, vocab, 0.5, old)
    check_gradient(grad, want)
    untouched = want[2] == 0
    assert torch.equal(grad.cpu()[untouched], old[untouched])
    check_rows(ssm.ssm_embed_fwd(d_ids, old.to(DEV), dtype=at), ref.embed(ids, old, 1.0))
