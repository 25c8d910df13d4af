"""Refusals and no-ops of the rotary and capped entry points: every call here
returns on the host before anything is queued."""

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _desc(duo, **kw):
    args = dict(batch=2, n_q_heads=8, n_kv_heads=4, head_dim=128, dtype=duo.BF16, kv_perm=[0, 1, 2, 3], n_retrieval=2)
    args.update(kw)
    return duo.desc_init(**args)


def _state(duo, **kw):
    st = duo.KVState()
    for k, v in dict(k_full=16, v_full=32, capacity=1024, k_ring=48, v_ring=64, ring_pos=80, seq_len=96, counters=112,
                     status=128, **kw).items():
        setattr(st, k, v)
    return st


Q, K, V, QO, KO = (i << 24 for i in range(1, 6))


def _refused(duo, status, call, *args, **kw):
    with pytest.raises(duo.DuoError) as e:
        call(*args, **kw, stream=0)
    assert e.value.status == getattr(duo, status), str(e.value)
    assert duo.last_error()


def test_rope_struct_matches_the_c_compiler(duo, tmp_path):
    src = tmp_path / "rope.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "duo.h"\n'
                   'int main(void) { printf("%zu %zu %zu %zu %zu\\n", sizeof(duo_rope), offsetof(duo_rope, sections), '
                   'offsetof(duo_rope, factor), offsetof(duo_rope, inv_freq), offsetof(duo_rope, pos)); return 0; }\n')
    exe = tmp_path / "rope"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    R = duo.Rope
    assert got == [ctypes.sizeof(R), R.sections.offset, R.factor.offset, R.inv_freq.offset, R.pos.offset]


BAD_ROPES = [
    (dict(rot_dim=127), "ERR_SHAPE"), (dict(rot_dim=0), "ERR_SHAPE"), (dict(rot_dim=130), "ERR_SHAPE"),
    (dict(layout=2), "ERR_INVALID_ARG"), (dict(inv_freq=0), "ERR_INVALID_ARG"), (dict(inv_freq=6), "ERR_INVALID_ARG"),
    (dict(factor=float("nan")), "ERR_INVALID_ARG"), (dict(factor=float("inf")), "ERR_INVALID_ARG"),
    (dict(n_axes=0), "ERR_SHAPE"), (dict(n_axes=4), "ERR_SHAPE"), (dict(sections=[63]), "ERR_SHAPE"),
    (dict(sections=[-1, 65], pos=4096), "ERR_SHAPE"), (dict(sections=[32, 32]), "ERR_INVALID_ARG"),   # no positions
    (dict(sections=[2 ** 31 - 1, 2 ** 31 - 1, 64], pos=4096), "ERR_SHAPE"), (dict(pos=4098), "ERR_INVALID_ARG"),
]


@pytest.mark.parametrize("kw,status", BAD_ROPES)
def test_bad_rope_descriptors(duo, kw, status):
    kw = dict(kw)
    n_axes = kw.pop("n_axes", None)
    rope = duo.rope_init(kw.pop("rot_dim", 128), kw.pop("inv_freq", 256), **{**dict(layout=0), **kw}) if \
        "sections" in kw or "rot_dim" not in kw else duo.rope_init(kw["rot_dim"], 256)
    if n_axes is not None:
        rope.n_axes = n_axes
    _refused(duo, status, duo.rope_qk, _desc(duo), rope, Q, K, QO, KO, 3)
    _refused(duo, status, duo.append_kv_rope, _desc(duo), _state(duo), rope, Q, K, V, QO, 3)


def test_rope_takes_one_to_three_sections(duo):
    for sections in ([], [16] * 4):
        with pytest.raises(ValueError):
            duo.rope_init(128, 256, sections=sections)


def test_rope_tensors(duo):
    rope, d = duo.rope_init(128, 256), _desc(duo)
    nq, nk = 2 * 3 * 8 * 256, 2 * 3 * 4 * 256
    _refused(duo, "ERR_SHAPE", duo.rope_qk, d, rope, Q, K, QO, KO, -1)
    for args in ((None, None, None, None), (Q, K, None, KO), (Q, None, QO, KO), (Q + 8, K, QO, KO), (Q, K, QO, KO + 2),
                 (Q, K, Q + 16, KO), (Q, K, Q + nq - 16, KO), (Q, K, K, KO), (Q, K, K + nk - 16, KO), (Q, K, QO, Q),
                 (Q, K, QO, QO)):
        _refused(duo, "ERR_INVALID_ARG", duo.rope_qk, d, rope, *args, 3)
    duo.rope_qk(d, rope, Q, K, QO, KO, 0, stream=0)                     # no tokens: nothing to do
    with pytest.raises(duo.DuoError):
        duo.rope_qk(_desc(duo, head_dim=96), rope, Q, K, QO, KO, 0, stream=0)


def test_append_rope_tensors(duo):
    rope, d, st = duo.rope_init(128, 256), _desc(duo), _state(duo)
    nq, nk = 2 * 3 * 8 * 256, 2 * 3 * 4 * 256
    _refused(duo, "ERR_SHAPE", duo.append_kv_rope, d, st, rope, Q, K, V, QO, -1)
    for q, k, v, qo in ((Q, None, V, QO), (Q, K, None, QO), (Q, K, V, None), (None, K, V, QO), (Q, K + 8, V, QO),
                        (Q, K, V, Q + 16), (Q, K, V, K), (Q, K, V, V + nk - 16), (Q, K, V, Q - nq + 16)):
        _refused(duo, "ERR_INVALID_ARG", duo.append_kv_rope, d, st, rope, q, k, v, qo, 3)
    st.seq_len = None
    _refused(duo, "ERR_INVALID_ARG", duo.append_kv_rope, d, st, rope, Q, K, V, QO, 3)
    duo.append_kv_rope(d, _state(duo), rope, Q, K, V, QO, 0, stream=0)


@pytest.mark.parametrize("cap", [-1.0, float("nan"), float("inf"), -float("inf"), 1e-7, 3e38])
def test_bad_caps(duo, cap):
    d, st = _desc(duo), _state(duo)
    need = duo.workspace_bytes(d, duo.OP_DECODE, 1024)
    _refused(duo, "ERR_INVALID_ARG", duo.decode_attn_capped, d, st, cap, Q, QO, V, need)
    _refused(duo, "ERR_INVALID_ARG", duo.decode_step_capped, d, st, cap, Q, K, V, QO, KO, need)
    _refused(duo, "ERR_INVALID_ARG", duo.prefill_chunk_capped, d, st, cap, Q, K, V, 3, QO)


def test_capped_calls_refuse_what_the_plain_calls_refuse(duo):
    d, st = _desc(duo), _state(duo)
    need = duo.workspace_bytes(d, duo.OP_DECODE, 1024)
    _refused(duo, "ERR_CAPACITY", duo.decode_attn_capped, d, st, 30.0, Q, QO, V, need - 16)
    _refused(duo, "ERR_INVALID_ARG", duo.decode_attn_capped, d, st, 30.0, None, QO, V, need)
    _refused(duo, "ERR_INVALID_ARG", duo.decode_step_capped, d, st, 30.0, Q, K, V + 8, QO, KO, need)
    _refused(duo, "ERR_SHAPE", duo.prefill_chunk_capped, d, st, 30.0, Q, K, V, 0, QO)
    paged = duo.desc_init(2, 8, 4, 128, duo.BF16, [0, 1, 2, 3], 2, page_size=64)
    _refused(duo, "ERR_UNSUPPORTED", duo.prefill_chunk_capped, paged,
             _state(duo, page_table=144, max_pages=16, n_pages=16), 30.0, Q, K, V, 3, QO)
    assert "duo_prefill_chunk_capped" in duo.last_error()


# ---------------------------------------------------------------------------
# The gated mix's training step
# ---------------------------------------------------------------------------

ALPHA, OUT, SAVED, DO, DQ, DK, DV, DA, WS, STATUS = (i << 28 for i in range(1, 11))


def _mix_sizes(duo, d, N):
    return duo.gated_mix_saved_bytes(d, N), duo.gated_mix_grad_workspace_bytes(d, N)


def test_mix_buffer_sizes(duo):
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    for dtype, hd in ((duo.BF16, 64), (duo.FP32, 64), (duo.BF16, 128)):
        d = duo.desc_init(3, 8, 4, hd, dtype, [0, 1, 2, 3], 4)
        saved, ws = _mix_sizes(duo, d, 130)
        # both log-sums; one attention in bf16 beside them (tensor cores) or both in fp32
        rows = 3 * 130 * 8
        assert saved == up(2 * rows * 4) + (up(rows * 128 * 2) if hd == 128 else 2 * up(rows * 64 * 4))
        assert ws == up(3 * 8 * 4 * 256 * 4) + up(3 * 2 * 16 * 4)      # rows padded to 256; a share per KV head and 32 rows
    assert _mix_sizes(duo, d, -1) == (0, 0)
    d.head_dim = 96
    assert _mix_sizes(duo, d, 130) == (0, 0)


def test_mix_train_rejects(duo):
    d, N = _desc(duo), 10
    saved, _ = _mix_sizes(duo, d, N)
    good = dict(alpha=ALPHA, cap=30.0, q=Q, k=K, v=V, N=N, out=OUT, saved=SAVED, saved_bytes=saved, status=STATUS)

    def refused(expected, **kw):
        _refused(duo, expected, duo.gated_mix_train, d, *{**good, **kw}.values())

    for name in ("alpha", "q", "k", "v", "out", "saved", "status"):
        refused("ERR_INVALID_ARG", **{name: None})
    for name in ("q", "k", "v", "out", "saved"):
        refused("ERR_INVALID_ARG", **{name: good[name] + 8})
    for cap in (-1.0, float("nan"), float("inf"), 1e-7):
        refused("ERR_INVALID_ARG", cap=cap)
    refused("ERR_SHAPE", N=-1)
    refused("ERR_CAPACITY", saved_bytes=saved - 1)
    for kw in (dict(out=Q), dict(out=K - 16), dict(saved=V - 16), dict(saved=Q + 16), dict(out=SAVED), dict(out=SAVED + saved - 16)):
        refused("ERR_INVALID_ARG", **kw)
    duo.gated_mix_train(d, *{**good, "N": 0, "saved_bytes": 0}.values(), stream=0)


def test_mix_grad_rejects(duo):
    d, N = _desc(duo), 10
    saved, ws = _mix_sizes(duo, d, N)
    good = dict(alpha=ALPHA, cap=0.0, q=Q, k=K, v=V, N=N, saved=SAVED, saved_bytes=saved, dout=DO, dq=DQ, dk=DK, dv=DV, dalpha=DA,
                workspace=WS, ws_bytes=ws, status=STATUS)

    def refused(expected, **kw):
        _refused(duo, expected, duo.gated_mix_grad, d, *{**good, **kw}.values())

    for name in ("alpha", "q", "k", "v", "saved", "dout", "dq", "dk", "dv", "dalpha", "workspace", "status"):
        refused("ERR_INVALID_ARG", **{name: None})
    for name in ("q", "k", "v", "saved", "dout", "dq", "dk", "dv", "workspace"):
        refused("ERR_INVALID_ARG", **{name: good[name] + 8})
    refused("ERR_SHAPE", N=-3)
    refused("ERR_CAPACITY", saved_bytes=saved - 1)
    refused("ERR_CAPACITY", ws_bytes=ws - 1)
    refused("ERR_INVALID_ARG", cap=-2.0)
    for kw in (dict(dq=Q), dict(dq=DO), dict(dk=K), dict(dv=V - 16), dict(dk=SAVED + 256), dict(workspace=SAVED), dict(dk=DQ),
               dict(dv=DK), dict(workspace=DV + 16), dict(workspace=DO - 16)):
        refused("ERR_INVALID_ARG", **kw)
