"""Flags and sizes that the linear-attention entry points take and refuse,
without a GPU: every refusal comes before the first HIP call."""
import pytest

import selective_state_space_30_amd as ssm
import test_linattn_abi as abi

OUTSIDE = ssm.SSM_FLAG_ZERO_OUTSIDE


@pytest.fixture(scope="module")
def lib():
    return ssm.load_library()


def refused(lib, name, base, **bad):
    return getattr(lib, name)(*{**base, **bad}.values())


def test_flags(lib):
    """A null q is refused after the flags are: SSM_FLAG_ZERO_OUTSIDE passes
    that check in the calls over sequences and not in the step."""
    for name, base in (("ssm_linattn_fwd", abi.FWD), ("ssm_linattn_bwd", abi.BWD)):
        for flags in (OUTSIDE, OUTSIDE | ssm.SSM_FLAG_HEAD_DECAY):
            assert refused(lib, name, base, flags=flags, q=None) == 1
            assert "q=" in ssm.ssm_last_error()
        assert refused(lib, name, base, flags=64) == 1
        assert "flag" in ssm.ssm_last_error()
    assert refused(lib, "ssm_linattn_step", abi.STEPS, flags=OUTSIDE) == 1
    assert "flag" in ssm.ssm_last_error()
