"""The debug build's index checks over the rotary, capped and training entry
points: no check fires, and the results that do not depend on the order of
drawn tiles are the release build's bit for bit."""

import numpy as np
import pytest

from head_split_kv_b200 import synthetic as S
from tests.gpu_helpers import Layer, bits, f64, torch
from tests.test_gpu_debug_bounds import duo_debug  # noqa: F401  (a fixture)
from tests.test_gpu_mix_train import _case, _step

pytestmark = pytest.mark.gpu

LAYERS = [   # hq, hkv, d, dtype, retrieval, quant, paged, chunks
    (8, 2, 128, "bf16", [1], "none", False, [300, 77]),
    (8, 4, 128, "bf16", [0, 2], "none", True, [130, 1]),
    (8, 4, 128, "bf16", [3], "int8", False, [130, 40]),
    (8, 4, 128, "bf16", [3], "int4", False, [130, 40]),
    (8, 4, 64, "fp32", [1, 2], "none", False, [90, 33]),
    (4, 4, 64, "bf16", [0], "none", False, [70, 1]),
]


def _serve(duo, case):
    """Rotation, capped pre-fill and rotated append of the chunks, then two
    decode steps; (pre-fill outputs and caches, decode outputs, status)."""
    hq, hkv, d, dtype, ret, quant, paged, chunks = case
    t = torch()
    sh = S.LayerShape(hq, hkv, d, dtype)
    kvq = {"none": duo.KV_PLAIN, "int8": duo.KV_INT8, "int4": duo.KV_INT4}[quant]
    table = np.arange(8, dtype=np.int32)[None] if paged else None
    lay = Layer(duo, sh, ret, 1, capacity=512, page_size=64 if paged else 0, page_table=table, n_pages=8 if paged else 0,
                kv_quant=kvq)
    st = lay.caches.state
    inv = t.linspace(1.0, 1e-4, d // 2, device="cuda")
    rope = duo.rope_init(d, inv)
    seq = t.zeros(1, dtype=t.int32, device="cuda")
    t.manual_seed(11)
    dt = t.bfloat16 if dtype == "bf16" else t.float32
    fixed, decoded = [], []
    ws = None if paged else duo.Workspace(lay.desc, duo.OP_PREFILL, max(chunks), state=st)
    for C in chunks + [1, 1]:
        q, k, v = (t.randn(1, C, h, d, device="cuda").to(dt) for h in (hq, hkv, hkv))
        qr, kr = t.empty_like(q), t.empty_like(k)
        duo.rope_qk(lay.desc, rope, q, k, qr, kr, C, seq_len=seq)
        fixed += [bits(qr), bits(kr)]
        if not paged and C > 1:
            out = t.empty_like(q)
            duo.prefill_chunk_capped(lay.desc, st, 30.0, qr, kr, v, C, out, ws.ptr, ws.nbytes)
            fixed.append(bits(out))
        qo = t.empty_like(q)
        duo.append_kv_rope(lay.desc, st, rope, q, k, v, qo, C)
        fixed.append(bits(qo))
        seq += C
        if C == 1:
            out = t.empty_like(qo)
            duo.decode_attn_capped(lay.desc, st, 30.0, qo, out, lay.ws.ptr, lay.ws.nbytes)
            decoded.append(f64(out))
            step = t.empty_like(qo)
            duo.decode_step_capped(lay.desc, st, 30.0, qo, kr, v, step, lay.ws.ptr, lay.ws.nbytes)
            decoded.append(f64(step))
            seq += 1
    t.cuda.synchronize()
    return fixed, decoded, lay.status()


@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_serving_calls(duo, duo_debug, case):  # noqa: F811
    fixed, decoded, status = _serve(duo, case)
    fixed_d, decoded_d, status_d = _serve(duo_debug, case)
    assert status == 0 and status_d == 0
    for a, b in zip(fixed, fixed_d):
        assert np.array_equal(a, b)
    for a, b in zip(decoded, decoded_d):
        # each within half a step of its weights, twice, and of the store (8 bits; fp32: sums of 200 terms)
        eps = 2.0 ** -8 if case[3] == "bf16" else 64 * 2.0 ** -24
        assert np.abs(a - b).max() <= 2 * 3 * eps * 5.0     # |v| of a few hundred normal draws stays below 5


@pytest.mark.parametrize("case", [(8, 2, 128, "bf16", 2, 300, 30.0), (4, 2, 128, "bf16", 1, 140, 0.0),
                                  (4, 2, 128, "bf16", 1, 140, 200.0), (4, 2, 64, "fp32", 2, 90, 20.0)],
                         ids=lambda c: "-".join(str(x) for x in c))
def test_training_step(duo, duo_debug, case):  # noqa: F811
    hq, hkv, d, dtype, B, N, cap = case
    desc, q, k, v, do, al = _case(duo, hq, hkv, d, dtype, B, N, cap, 2.0)
    desc_d = _case(duo_debug, hq, hkv, d, dtype, B, N, cap, 2.0)[0]
    for a, b in zip(_step(duo, desc, cap, q, k, v, do, al), _step(duo_debug, desc_d, cap, q, k, v, do, al)):
        assert np.array_equal(bits(a), bits(b))
