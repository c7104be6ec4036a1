"""The type of the embedding's gradient where both it and the tensor are given."""
import pytest
import torch

import selective_state_space_30_amd as ssm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("have, want", [(BF16, F32), (F32, BF16), (F32, torch.float16)])
def test_a_type_that_the_given_gradient_has_not(have, want, accumulate):
    ids = torch.tensor([1, 2, 1], device=DEV)
    dy = torch.ones(3, 8, device=DEV)
    dw = torch.full((4, 8), 3.0, dtype=have, device=DEV)
    with pytest.raises(TypeError, match="dweight"):
        ssm.ssm_embed_bwd(ids, dy, 4, dweight=dw, accumulate=accumulate, dtype=want)
    assert (dw == 3).all()


@pytest.mark.parametrize("kind", [BF16, F32])
def test_types_that_are_taken(kind):
    ids = torch.tensor([1, 2, 1], device=DEV)
    dy = torch.ones(3, 8, device=DEV)
    want = torch.tensor([0, 2, 1, 0], device=DEV).unsqueeze(1).expand(4, 8)
    for given in ({}, {"dtype": kind}):
        dw = torch.full((4, 8), 3.0, dtype=kind, device=DEV)
        assert ssm.ssm_embed_bwd(ids, dy, 4, dweight=dw, **given) is dw
        assert torch.equal(dw, want.to(kind))
        ssm.ssm_embed_bwd(ids, dy, 4, dweight=dw, accumulate=True, **given)
        assert torch.equal(dw, (2 * want).to(kind))
    assert ssm.ssm_embed_bwd(ids, dy, 4).dtype == F32
    assert ssm.ssm_embed_bwd(ids, dy, 4, dtype=kind).dtype == kind
