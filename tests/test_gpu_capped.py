"""Capped decode and pre-fill against the formula in fp64, over every kind of
cache, at scores far below, near and far above the cap."""

import numpy as np
import pytest

import oracle as O
from head_split_kv_b200 import synthetic as S
from tests.gpu_helpers import Layer, bits, f64, to_dev, torch
from tests.rotary_and_cap import attend_ref, attend_tolerance

pytestmark = pytest.mark.gpu


def _rows(lay, b, h):
    pos, k, v = lay.oracle.rows(b, h)
    return np.asarray(pos), O.as_f64(k) if len(pos) else np.zeros((0, lay.shape.head_dim)), \
        O.as_f64(v) if len(pos) else np.zeros((0, lay.shape.head_dim))


def _check_decode(lay, q, got, cap):
    sh, g = lay.shape, lay.shape.group
    scale = 1.0 / np.sqrt(sh.head_dim)
    for b in range(lay.B):
        for h in range(sh.n_kv_heads):
            _, k, v = _rows(lay, b, h)
            qq = O.as_f64(q[b, h * g:(h + 1) * g])
            want = attend_ref(qq, k, v, np.ones((g, len(k)), bool), cap, scale)
            tol = attend_tolerance(qq, k, v, cap, scale, sh.dtype)
            err = np.abs(got[b, h * g:(h + 1) * g] - want).max()
            assert err <= tol, f"b={b} h={h} n={len(k)}: {err:.3e} > {tol:.3e}"


DECODES = [   # hq, hkv, d, dtype, retrieval, quant, paged, lengths, gain, cap
    (32, 8, 128, "bf16", [1, 3, 4, 6], "none", False, [4097], 3.0, 50.0),
    (32, 8, 128, "bf16", [0, 7], "none", True, [1, 64, 65, 700], 3.0, 20.0),
    (8, 8, 128, "bf16", [5], "none", False, [0, 16, 81], 30.0, 5.0),      # scores far past the cap
    (16, 2, 128, "bf16", [0], "none", False, [333, 5], 1.0, 1000.0),      # far below
    (8, 4, 64, "bf16", [1], "none", True, [200, 79], 3.0, 30.0),
    (8, 4, 64, "fp32", [1, 2], "none", False, [200, 17], 10.0, 7.0),
    (8, 1, 128, "fp32", [0], "none", True, [130], 3.0, 30.0),
    (4, 4, 128, "fp32", [], "none", False, [130, 3], 3.0, 30.0),
    (8, 4, 128, "bf16", [0, 2], "int8", False, [513, 1], 3.0, 30.0),
    (8, 8, 128, "bf16", [0, 2], "int4", False, [300, 64], 30.0, 10.0),
    (32, 4, 128, "bf16", [3], "int4", False, [1000], 3.0, 50.0),
    (16, 4, 128, "bf16", [1, 2], "none", True, [513, 2], 3.0, 1e6),       # so far below that tanh's own
    (8, 4, 128, "bf16", [0, 2], "int8", False, [300, 9], 3.0, 1e38),      # absolute error would show
    (8, 4, 64, "fp32", [1, 2], "none", False, [200, 17], 10.0, 1e30),
]


@pytest.mark.parametrize("case", DECODES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
@pytest.mark.parametrize("fused", [False, True])
def test_capped_decode(duo, case, fused):
    hq, hkv, d, dtype, ret, quant, paged, lengths, gain, cap = case
    t = torch()
    sh = S.LayerShape(hq, hkv, d, dtype)
    kvq = {"none": duo.KV_PLAIN, "int8": duo.KV_INT8, "int4": duo.KV_INT4}[quant]
    B, per = len(lengths), (max(lengths) + 64) // 64 + 1
    table = np.random.default_rng(2).permutation(B * per).reshape(B, per) if paged else None
    lay = Layer(duo, sh, ret, B, capacity=per * 64, page_size=64 if paged else 0, page_table=table,
                n_pages=B * per if paged else 0, kv_quant=kvq)
    if quant == "none":
        lay.load_state(S.decode_state(sh, ret, lengths, seed=4))
    else:   # a quantized layer takes its rows through the library
        n = min(lengths)
        _, k, v = S.prompt(sh, n, seed=4, batch=B)
        lay.append(k, v)
    qs, ks, vs = S.decode_steps(sh, B, 2, seed=6)
    for i in range(2):
        q = O.as_f64(qs[i]) * gain
        q = bits(t.from_numpy(q).to(t.bfloat16)) if dtype == "bf16" else q.astype(np.float32)
        qd, out = to_dev(q), t.full(q.shape, float("nan"), device="cuda", dtype=t.bfloat16 if dtype == "bf16" else t.float32)
        kd, vd = to_dev(ks[i]), to_dev(vs[i])
        if fused:
            duo.decode_step_capped(lay.desc, lay.caches.state, cap, qd, kd, vd, out, lay.ws.ptr, lay.ws.nbytes)
        else:
            duo.append_kv(lay.desc, lay.caches.state, kd, vd, 1)
            duo.decode_attn_capped(lay.desc, lay.caches.state, cap, qd, out, lay.ws.ptr, lay.ws.nbytes)
        lay.oracle.append(ks[i][:, None], vs[i][:, None])
        _check_decode(lay, q, f64(out), cap)
    lay.assert_caches_match()
    assert lay.status() == 0


def test_capped_decode_of_empty_sequences_is_zero(duo):
    t = torch()
    for dtype, d in (("bf16", 128), ("fp32", 64)):
        sh = S.LayerShape(8, 4, d, dtype)
        lay = Layer(duo, sh, [0, 2], 2, capacity=128)
        q = t.randn(2, 8, d, device="cuda").to(t.bfloat16 if dtype == "bf16" else t.float32)
        out = t.full_like(q, float("nan"))
        duo.decode_attn_capped(lay.desc, lay.caches.state, 30.0, q, out, lay.ws.ptr, lay.ws.nbytes)
        assert not bits(out).any()


def test_cap_of_zero_is_the_plain_call(duo):
    t = torch()
    sh = S.LayerShape(8, 4, 128, "bf16")
    lay = Layer(duo, sh, [0, 2], 1, capacity=128)
    lay.load_state(S.decode_state(sh, [0, 2], [100], seed=4))
    q = t.randn(1, 8, 128, device="cuda").bfloat16()
    a, b = t.empty_like(q), t.empty_like(q)
    duo.decode_attn(lay.desc, lay.caches.state, q, a, lay.ws.ptr, lay.ws.nbytes)
    duo.decode_attn_capped(lay.desc, lay.caches.state, 0.0, q, b, lay.ws.ptr, lay.ws.nbytes)
    assert np.array_equal(bits(a), bits(b))


def test_rows_past_the_length_do_not_reach_a_capped_decode(duo):
    """NaN, infinities and stale rows behind each sequence's last token."""
    t = torch()
    sh = S.LayerShape(8, 4, 128, "bf16")
    for paged in (False, True):
        lay = Layer(duo, sh, [0, 2], 2, capacity=256, page_size=64 if paged else 0,
                    page_table=np.arange(8).reshape(2, 4) if paged else None, n_pages=8)
        lay.load_state(S.decode_state(sh, [0, 2], [70, 130], seed=4))
        for b, L in enumerate((70, 130)):
            for x, bad in ((lay.caches.k_full, float("inf")), (lay.caches.v_full, float("nan"))):
                for p in range(L, 256):
                    if paged:
                        x[4 * b + p // 64, :, p % 64] = bad
                    else:
                        x[b, :, p] = bad
        q = S.decode_steps(sh, 2, 1, seed=6)[0][0]
        out = t.empty(2, 8, 128, device="cuda", dtype=t.bfloat16)
        duo.decode_attn_capped(lay.desc, lay.caches.state, 30.0, to_dev(q), out, lay.ws.ptr, lay.ws.nbytes)
        _check_decode(lay, q, f64(out), 30.0)


PREFILLS = [   # hq, hkv, d, dtype, retrieval, quant, mode, B, chunks, gain, cap
    (8, 4, 128, "bf16", [0, 3], "none", "lambda", 1, [300, 1, 129, 70], 3.0, 30.0),
    (8, 2, 128, "bf16", [1], "none", "chunk", 2, [256, 77], 3.0, 20.0),
    (8, 8, 128, "bf16", [1, 2], "none", "lambda", 1, [1, 5, 200], 30.0, 5.0),
    (4, 4, 128, "bf16", [], "none", "lambda", 1, [90, 140], 1.0, 1000.0),
    (8, 4, 128, "bf16", [0, 3], "int8", "lambda", 1, [130, 200], 3.0, 30.0),
    (8, 4, 128, "bf16", [0, 3], "int4", "chunk", 2, [64, 150], 30.0, 20.0),
    (8, 4, 64, "bf16", [1], "none", "lambda", 2, [33, 90], 3.0, 30.0),
    (8, 4, 64, "fp32", [1, 2], "none", "chunk", 1, [33, 1, 90], 10.0, 7.0),
    (4, 4, 128, "fp32", [0, 1, 2, 3], "none", "lambda", 1, [100, 31], 3.0, 30.0),
    (8, 4, 128, "bf16", [0, 3], "none", "lambda", 1, [130, 200], 3.0, 1e6),
    (8, 4, 128, "bf16", [0, 3], "int8", "lambda", 1, [130, 200], 3.0, 1e38),
    (8, 4, 64, "fp32", [1, 2], "none", "chunk", 1, [33, 90], 10.0, 1e30),
]


@pytest.mark.parametrize("case", PREFILLS, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_capped_prefill(duo, case):
    hq, hkv, d, dtype, ret, quant, mode, B, chunks, gain, cap = case
    t = torch()
    sh = S.LayerShape(hq, hkv, d, dtype)
    kvq = {"none": duo.KV_PLAIN, "int8": duo.KV_INT8, "int4": duo.KV_INT4}[quant]
    lay = Layer(duo, sh, ret, B, capacity=sum(chunks) + 8, kv_quant=kvq,
                stream_prefill=duo.STREAM_CHUNK if mode == "chunk" else duo.STREAM_LAMBDA)
    n, g, scale = sum(chunks), sh.group, 1.0 / np.sqrt(d)
    q, k, v = S.prompt(sh, n, seed=12, batch=B)
    q = O.as_f64(q) * gain
    q = bits(t.from_numpy(q).to(t.bfloat16)) if dtype == "bf16" else q.astype(np.float32)
    ws = duo.Workspace(lay.desc, duo.OP_PREFILL, max(chunks), state=lay.caches.state)
    c0 = 0
    for C in chunks:
        sl = slice(c0, c0 + C)
        qd, kd, vd = (to_dev(np.ascontiguousarray(x[:, sl])) for x in (q, k, v))
        out = t.full_like(qd, float("nan"))
        duo.prefill_chunk_capped(lay.desc, lay.caches.state, cap, qd, kd, vd, C, out, ws.ptr, ws.nbytes)
        got = f64(out)
        P = np.arange(c0, c0 + C)[:, None]
        for b in range(B):
            for h in range(hkv):
                pos, kh, vh = _rows(lay, b, h)
                key = np.concatenate([pos, P[:, 0]]).astype(np.int64)[None]
                kk, vv = np.concatenate([kh, O.as_f64(k[b, sl, h])]), np.concatenate([vh, O.as_f64(v[b, sl, h])])
                seen = key <= P
                if h not in ret:
                    near = key >= c0 - sh.recent if mode == "chunk" else P - key < sh.recent
                    seen = seen & ((key < sh.sink) | near)
                for qh in range(h * g, (h + 1) * g):
                    qq = O.as_f64(q[b, sl, qh])
                    err = np.abs(got[b, :, qh] - attend_ref(qq, kk, vv, seen, cap, scale)).max()
                    tol = attend_tolerance(qq, kk, vv, cap, scale, dtype)
                    assert err <= tol, f"c0={c0} b={b} h={qh}: {err:.3e} > {tol:.3e}"
        duo.append_kv(lay.desc, lay.caches.state, kd, vd, C)
        lay.oracle.append(k[:, sl], v[:, sl])
        c0 += C
    assert lay.status() == 0


def test_capped_prefill_with_key_splits(duo):
    """Long enough for the key-range splits, scores on both sides of the
    polynomial's range."""
    t = torch()
    sh = S.LayerShape(8, 2, 128, "bf16")
    lay = Layer(duo, sh, [0], 1, capacity=13000)
    n, C, cap, scale = 12800, 512, 10.0, 1.0 / np.sqrt(128)
    q, k, v = S.prompt(sh, n + C, seed=13)
    q = bits(t.from_numpy(O.as_f64(q) * 2.5).to(t.bfloat16))
    kd, vd = to_dev(k[:, :n]), to_dev(v[:, :n])
    duo.append_kv(lay.desc, lay.caches.state, kd, vd, n)
    ws = duo.Workspace(lay.desc, duo.OP_PREFILL, C, state=lay.caches.state)
    assert ws.nbytes > 256
    qd, kc, vc = (to_dev(np.ascontiguousarray(x[:, n:])) for x in (q, k, v))
    out = t.empty_like(qd)
    duo.prefill_chunk_capped(lay.desc, lay.caches.state, cap, qd, kc, vc, C, out, ws.ptr, ws.nbytes)
    got, rows = f64(out), np.array([0, 1, 127, 128, 300, 511])
    kk, vv = O.as_f64(k[0, :, 0]), O.as_f64(v[0, :, 0])
    seen = np.arange(n + C)[None] <= (n + rows)[:, None]
    for qh in range(4):
        qq = O.as_f64(q[0, n + rows, qh])
        err = np.abs(got[0, rows, qh] - attend_ref(qq, kk, vv, seen, cap, scale)).max()
        assert err <= attend_tolerance(qq, kk, vv, cap, scale, "bf16")
    assert lay.status() == 0


def test_rotary_capped_model_end_to_end(duo):
    """Two pre-fill chunks (rotation, capped attention, append), then decode
    steps (rotated append, capped decode), against fp64 over the rotated rows
    as the caches hold them."""
    t = torch()
    sh = S.LayerShape(8, 4, 128, "bf16")
    ret, cap, scale = [0, 3], 30.0, 1.0 / np.sqrt(128)
    lay = Layer(duo, sh, ret, 1, capacity=512)
    inv = t.from_numpy(np.power(10000.0, -2.0 * np.arange(64) / 128).astype(np.float32)).cuda()
    rope = duo.rope_init(128, inv)
    ws = duo.Workspace(lay.desc, duo.OP_PREFILL, 150, state=lay.caches.state)
    keys, values = [], []
    t.manual_seed(3)
    for C in (150, 70, 1, 1, 1):
        q, k, v = (t.randn(1, C, h, 128, device="cuda").mul(s).bfloat16() for h, s in ((8, 3.0), (4, 1.0), (4, 1.0)))
        c0 = sum(x.shape[1] for x in keys)
        qr, kr = t.empty_like(q), t.empty_like(k)
        duo.rope_qk(lay.desc, rope, q, k, qr, kr, C, seq_len=lay.caches.seq_len)
        out = t.empty_like(q)
        if C > 1:
            duo.prefill_chunk_capped(lay.desc, lay.caches.state, cap, qr, kr, v, C, out, ws.ptr, ws.nbytes)
            duo.append_kv(lay.desc, lay.caches.state, kr, v, C)
        else:
            qo = t.empty_like(q)
            duo.append_kv_rope(lay.desc, lay.caches.state, rope, q, k, v, qo, 1)
            assert np.array_equal(bits(qo), bits(qr))
            duo.decode_attn_capped(lay.desc, lay.caches.state, cap, qo, out, lay.ws.ptr, lay.ws.nbytes)
        keys.append(f64(kr))
        values.append(f64(v))
        kk, vv = np.concatenate(keys, 1)[0], np.concatenate(values, 1)[0]
        P, j = np.arange(c0, c0 + C)[:, None], np.arange(c0 + C)[None]
        got, qq = f64(out)[0], f64(qr)[0]
        for h in range(4):
            seen = j <= P if h in ret else (j <= P) & ((j < 16) | (P - j < 64))
            for qh in (2 * h, 2 * h + 1):
                err = np.abs(got[:, qh] - attend_ref(qq[:, qh], kk[:, h], vv[:, h], seen, cap, scale)).max()
                assert err <= attend_tolerance(qq[:, qh], kk[:, h], vv[:, h], cap, scale, "bf16")
    assert lay.status() == 0
