"""Overlaps that would let a kernel read what it has just written: gates and
their gradient in one buffer, and outputs over the angles' arrays.  Every call
here returns on the host before anything is queued."""

import pytest

from tests.test_abi_rotary_capped import (ALPHA, DA, DK, DO, DQ, DV, K, KO, OUT, Q, QO, SAVED, STATUS, V, WS, _desc, _mix_sizes,
                                          _refused, _state)


def test_training_outputs_over_gates_and_status(duo):
    d, N = _desc(duo), 10
    saved, ws = _mix_sizes(duo, d, N)
    train = dict(alpha=ALPHA, cap=30.0, q=Q, k=K, v=V, N=N, out=OUT, saved=SAVED, saved_bytes=saved, status=STATUS)
    for kw in (dict(alpha=OUT), dict(alpha=SAVED + 16), dict(out=ALPHA), dict(status=OUT + 64), dict(status=SAVED), dict(status=Q),
               dict(status=ALPHA + 4)):
        _refused(duo, "ERR_INVALID_ARG", duo.gated_mix_train, d, *{**train, **kw}.values())
    grad = dict(alpha=ALPHA, cap=0.0, q=Q, k=K, v=V, N=N, saved=SAVED, saved_bytes=saved, dout=DO, dq=DQ, dk=DK, dv=DV, dalpha=DA,
                workspace=WS, ws_bytes=ws, status=STATUS)
    for kw in (dict(dalpha=ALPHA), dict(dalpha=ALPHA + 12), dict(dalpha=DQ + 32), dict(dalpha=WS), dict(dalpha=Q), dict(alpha=DK),
               dict(dalpha=SAVED), dict(status=DA + 4), dict(status=ALPHA), dict(status=WS + 4)):
        _refused(duo, "ERR_INVALID_ARG", duo.gated_mix_grad, d, *{**grad, **kw}.values())


@pytest.mark.parametrize("axes", [1, 3])
def test_rotation_outputs_over_the_angles(duo, axes):
    d, T = _desc(duo), 3
    nq, nk = 2 * T * 8 * 256, 2 * T * 4 * 256
    inv, pos, lengths = 1 << 28, 2 << 28, 3 << 28
    sections = [64] if axes == 1 else [16, 24, 24]
    for at in (inv, inv + 252, pos, pos + axes * 2 * T * 4 - 4, lengths + 4):
        rope = duo.rope_init(128, inv, sections=sections, pos=pos)
        for end in (0, 1):
            q_out, k_out = at // 16 * 16 - (nq - 16) * end, at // 16 * 16 - (nk - 16) * end
            _refused(duo, "ERR_INVALID_ARG", duo.rope_qk, d, rope, Q, K, q_out, KO, T, seq_len=lengths)
            _refused(duo, "ERR_INVALID_ARG", duo.rope_qk, d, rope, Q, K, QO, k_out, T, seq_len=lengths)
            st = _state(duo)
            st.seq_len = lengths
            _refused(duo, "ERR_INVALID_ARG", duo.append_kv_rope, d, st, rope, Q, K, V, q_out, T)
