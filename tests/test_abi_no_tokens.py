"""Calls without tokens: an empty torch tensor has no address, so the rotary
and training calls take NULL tensors then, and still refuse a bad descriptor.
Every call here returns on the host before anything is queued."""

import pytest
import torch

from tests.test_abi_rotary_capped import ALPHA, STATUS, _desc, _refused, _state


def _empty(*shape):
    x = torch.empty(*shape)
    assert x.data_ptr() == 0
    return x


def test_rotation_of_no_tokens(duo):
    d, rope = _desc(duo), duo.rope_init(128, 256)
    q, k = _empty(2, 0, 8, 128), _empty(2, 0, 4, 128)
    duo.rope_qk(d, rope, q, k, q, k, 0, stream=0)
    duo.rope_qk(d, rope, q, None, q, None, 0, inverse=True, stream=0)
    duo.append_kv_rope(d, _state(duo), rope, q, k, k, q, 0, stream=0)
    rope.factor = float("nan")
    _refused(duo, "ERR_INVALID_ARG", duo.rope_qk, d, rope, q, k, q, k, 0)


def test_training_step_of_no_tokens(duo):
    d, x = _desc(duo), _empty(2, 0, 8, 128)
    duo.gated_mix_train(d, ALPHA, 30.0, x, x, x, 0, x, x, duo.gated_mix_saved_bytes(d, 0), STATUS, stream=0)
    _refused(duo, "ERR_INVALID_ARG", duo.gated_mix_train, d, ALPHA, -1.0, x, x, x, 0, x, x, 0, STATUS)
    # the backward pass of no tokens still zeroes dalpha, so it needs that one
    _refused(duo, "ERR_INVALID_ARG", duo.gated_mix_grad, d, ALPHA, 30.0, x, x, x, 0, x, 0, x, x, x, x, None, x, 0, STATUS)


@pytest.mark.gpu
def test_gradient_of_no_tokens(duo):
    d, x, da = _desc(duo), _empty(2, 0, 8, 128), torch.full((4,), 7.0, device="cuda")
    duo.gated_mix_grad(d, da.clone(), 30.0, x, x, x, 0, x, 0, x, x, x, x, da, x, 0, STATUS)
    assert not bool(da.any())
