"""The binding of the linear-attention and block-norm calls, without a GPU:
a call runs with its ``stream`` as torch's current stream, whichever way the
argument is given, so that what it allocates belongs to that stream."""
import contextlib
import inspect

import pytest
import torch

import selective_state_space_30_amd as ssm

CALLS = (ssm.ssm_linattn_fwd, ssm.ssm_linattn_bwd, ssm.ssm_linattn_step,
         ssm.ssm_block_norm_fwd, ssm.ssm_block_norm_bwd)


@pytest.fixture
def current(monkeypatch):
    """The streams entered by ``with torch.cuda.stream``, innermost last."""
    entered = []

    @contextlib.contextmanager
    def stream(s):
        entered.append(s)
        yield
        entered.pop()
    monkeypatch.setattr(torch.cuda, "stream", stream)
    return entered


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_stream_is_current_however_it_is_given(current, call):
    signature = inspect.signature(call)
    seen = []

    def body(*args, **kwargs):
        seen.append(list(current))
    body.__signature__ = signature
    wrapped = ssm._on_device(body)
    at = list(signature.parameters).index("stream")
    side = object()
    wrapped(*[None] * at, side)
    wrapped(*[None] * (at - 1), stream=side)
    wrapped(stream=side)
    wrapped(*[None] * at, None)
    wrapped(*[None] * at)
    wrapped(stream=None)
    wrapped()
    assert seen == [[side]] * 3 + [[]] * 4
