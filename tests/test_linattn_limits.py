"""Flags and sizes that the linear-attention entry points take and refuse,
without a GPU: every refusal comes before the first HIP call."""
import pytest
import torch

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


# tokens, packed prompts, heads, qk_heads, qk_dim, v_dim, dtype, calls (0
# forward, 1 backward, 2 with dg)
MANY = [
    (262144, 512, 80, 1, 128, 64, torch.bfloat16, (0, 1, 2)),
    (524288, 256, 80, 1, 128, 64, torch.bfloat16, (0, 1, 2)),
    (1 << 20, 1024, 16, 16, 128, 128, torch.bfloat16, (0, 1, 2)),
    (65536, 512, 80, 1, 128, 64, torch.float32, (0, 1, 2)),
    (65536, 65536, 16, 16, 128, 128, torch.float32, (0, 1, 2)),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "t%d_n%d_h%d_%s" % (
    c[0], c[1], c[2], "bf16" if c[6] == torch.bfloat16 else "f32"))
def test_many_packed_prompts_are_taken(case):
    """Sizes of ordinary batches: the launches grow with the tokens and the
    sequences, not with the sequences times the longest segment."""
    tokens, nseq, heads, qk_heads, dk, dv, dtype, calls = case
    for back in calls:
        p = ssm.ssm_linattn_plan(tokens, nseq, heads, qk_heads, dk, dv, dtype, packed=True,
                                 backward=back)
        assert p["segments"] >= tokens // p["segment"] + nseq
        size = (ssm.ssm_linattn_bwd_workspace_size(tokens, nseq, heads, qk_heads, dk, dv, dtype,
                                                   packed=True, want_dg=1) if back else
                ssm.ssm_linattn_workspace_size(tokens, nseq, heads, qk_heads, dk, dv, dtype,
                                               packed=True))
        assert size >= 0


def test_one_long_sequence_of_many_heads_is_taken():
    for back in (0, 1):
        ssm.ssm_linattn_plan(1 << 20, 1, 512, 512, 64, 64, backward=back)


@pytest.mark.parametrize("back", [0, 1, 2])
def test_launches_past_2_to_32_threads_are_refused(back):
    """Workgroups (of 512 threads) of the widest launch: segments times heads
    times output slices, with dg the chunks of 64 tokens times heads as well."""
    def groups(tokens, nseq, heads, d, plan):
        slices = 2 if d > 128 else 1
        n = plan["segments"] * heads * slices * (3 if back else 1)
        if back == 2:
            n += (tokens // 64 + nseq) * heads
        return n

    for heads, d in ((64, 128), (64, 256)):
        lo, hi = 1, 1 << 20  # sequences of one token each: the most that are taken
        while hi - lo > 1:
            mid = (lo + hi) // 2
            try:
                ssm.ssm_linattn_plan(mid, mid, heads, heads, d, d, packed=True, backward=back)
                lo = mid
            except RuntimeError as e:
                assert "UNSUPPORTED" in str(e) and "workgroups" in str(e)
                hi = mid
        plan = ssm.ssm_linattn_plan(lo, lo, heads, heads, d, d, packed=True, backward=back)
        n = groups(lo, lo, heads, d, plan)
        assert (1 << 23) - 8 * heads * 8 < n < 1 << 23
