"""duo_rope_qk and duo_append_kv_rope against the rotation's formula in fp64,
and the rotated append against a rotation followed by the plain append, bit
for bit, over every kind of cache."""

import numpy as np
import pytest

from head_split_kv_b200 import synthetic as S
from tests.gpu_helpers import Layer, bits, f64, torch
from tests.rotary_and_cap import rope_ref, rope_tolerance

pytestmark = pytest.mark.gpu


def _inv_freq(rot, base=500000.0):
    return np.power(base, -2.0 * np.arange(rot // 2) / rot).astype(np.float32)


def _setup(duo, shape, B, T, rot, sections, layout, factor, seed, pos=None):
    t = torch()
    t.manual_seed(seed)
    dt = t.bfloat16 if shape.dtype == "bf16" else t.float32
    x = [t.randn(B, T, h, shape.head_dim, device="cuda").to(dt) for h in (shape.n_q_heads, shape.n_kv_heads, shape.n_kv_heads)]
    inv = t.from_numpy(_inv_freq(rot)).cuda()
    pos_d = None if pos is None else t.from_numpy(np.ascontiguousarray(pos, dtype=np.int32)).cuda()
    rope = duo.rope_init(rot, inv, layout=duo.ROPE_HALVES if layout == "halves" else duo.ROPE_PAIRS, sections=sections,
                         factor=factor, pos=pos_d)
    return x, inv, pos_d, rope


def _check(got, x, pos, rot, sections, layout, factor, dtype, sign=1.0):
    want = rope_ref(f64(x), pos, _inv_freq(rot), rot, sections, layout, factor, sign)
    err = np.abs(f64(got) - want)
    tol = rope_tolerance(f64(x), rot, layout, factor, dtype)
    assert np.all(err <= tol), f"max excess {np.max(err - tol):.3e}"


CASES = [   # hq, hkv, d, dtype, B, T, rot, sections, layout, factor, start
    (32, 8, 128, "bf16", 1, 300, 128, [64], "halves", 1.0, 126976),
    (32, 8, 128, "bf16", 2, 5, 128, [64], "pairs", 1.2, 1_000_000_000),
    (8, 8, 64, "bf16", 3, 1, 32, [16], "halves", 1.0, 0),
    (8, 4, 128, "bf16", 1, 7, 20, [10], "halves", 1.0, 77),        # half a rotation is not whole 16-byte pieces
    (8, 1, 64, "fp32", 2, 33, 64, [32], "halves", 1.0, 1_048_575),
    (4, 4, 128, "fp32", 1, 17, 96, [48], "pairs", 0.7, 12345),
    (4, 2, 64, "fp32", 1, 9, 6, [3], "halves", 1.0, 31),
    (4, 2, 64, "fp32", 1, 9, 6, [3], "pairs", 1.0, 31),
    (16, 4, 128, "bf16", 2, 67, 128, [16, 24, 24], "halves", 1.0, None),
    (16, 4, 128, "fp32", 1, 67, 96, [12, 18, 18], "pairs", 1.0, None),
    (16, 4, 64, "bf16", 1, 3, 64, [0, 32], "halves", 1.0, None),   # an axis without pairs
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_matches_the_formula(duo, case, inverse):
    hq, hkv, d, dtype, B, T, rot, sections, layout, factor, start = case
    t = torch()
    sh = S.LayerShape(hq, hkv, d, dtype)
    rng = np.random.default_rng(5)
    pos, seq_len = None, None
    if start is None:
        pos = rng.integers(-1000, 70000, (len(sections), B, T))
        at = pos
    else:
        starts = start + np.arange(B)
        seq_len = t.from_numpy(starts.astype(np.int32)).cuda()
        at = (starts[:, None] + np.arange(T))[None]
    (q, k, _), inv, pos_d, rope = _setup(duo, sh, B, T, rot, sections, layout, factor, 3, pos)
    desc = duo.desc_init(B, hq, hkv, d, duo.BF16 if dtype == "bf16" else duo.FP32, list(range(hkv)), hkv)
    qo, ko = t.full_like(q, float("nan")), t.full_like(k, float("nan"))
    duo.rope_qk(desc, rope, q, k, qo, ko, T, seq_len=seq_len, inverse=inverse)
    sign = -1.0 if inverse else 1.0
    _check(qo, q, at, rot, sections, layout, factor, dtype, sign)
    _check(ko, k, at, rot, sections, layout, factor, dtype, sign)
    # channels past rot_dim pass through, in place gives the same, and each tensor alone too
    assert np.array_equal(bits(qo)[..., rot:], bits(q)[..., rot:])
    q2, k2 = q.clone(), k.clone()
    duo.rope_qk(desc, rope, q2, None, q2, None, T, seq_len=seq_len, inverse=inverse)
    duo.rope_qk(desc, rope, None, k2, None, k2, T, seq_len=seq_len, inverse=inverse)
    assert np.array_equal(bits(q2), bits(qo)) and np.array_equal(bits(k2), bits(ko))


@pytest.mark.parametrize("layout,rot", [("pairs", 6), ("pairs", 20), ("halves", 6), ("halves", 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_channels_past_the_rotation_are_kept(duo, layout, rot, dtype):
    """Infinities, NaN and -0 behind rot_dim come out as they went in, and reach no other channel."""
    t = torch()
    sh = S.LayerShape(4, 2, 128, dtype)
    (q, k, _), inv, _, rope = _setup(duo, sh, 1, 5, rot, [rot // 2], layout, 1.0, 2)
    for x in (q, k):
        x[..., rot::4], x[..., rot + 1::4], x[..., rot + 2::4] = float("inf"), -0.0, float("nan")
    desc = duo.desc_init(1, 4, 2, 128, duo.BF16 if dtype == "bf16" else duo.FP32, [0, 1], 2)
    qo, ko = t.zeros_like(q), t.zeros_like(k)
    duo.rope_qk(desc, rope, q, k, qo, ko, 5, seq_len=t.tensor([70], dtype=t.int32, device="cuda"))
    for x, y in ((q, qo), (k, ko)):
        x, y = f64(x), f64(y)
        assert np.array_equal(y[..., rot:], x[..., rot:], equal_nan=True)
        assert np.all(np.signbit(y[..., rot + 1::4]))
        assert np.all(np.isfinite(y[..., :rot]))


def test_rope_gradient_is_the_transpose(duo):
    """<rope(x), g> = <x, rope_inverse(g)>, and a difference quotient of a loss
    agrees with the gradient (the map is linear, so up to rounding)."""
    t = torch()
    sh = S.LayerShape(4, 4, 64, "fp32")
    (q, k, g), inv, _, rope = _setup(duo, sh, 2, 19, 48, [24], "halves", 1.3, 8)
    desc = duo.desc_init(2, 4, 4, 64, duo.FP32, list(range(4)), 4)
    seq = t.tensor([5, 900], dtype=t.int32, device="cuda")
    y, dx, step = t.empty_like(k), t.empty_like(k), t.empty_like(k)
    duo.rope_qk(desc, rope, None, k, None, y, 19, seq_len=seq)
    duo.rope_qk(desc, rope, None, g, None, dx, 19, seq_len=seq, inverse=True)
    n = k.numel()
    # sums of n products, each within 12 half-steps of sizes about 1.3
    tol = 12 * 2.0 ** -24 * float((y.double().abs() * g.double().abs()).sum() + (k.double().abs() * dx.double().abs()).sum())
    assert abs(float((y.double() * g.double()).sum() - (k.double() * dx.double()).sum())) <= tol
    h = 2.0 ** -3
    moved = k.clone()
    moved[1, 7, 2, 11] += h
    duo.rope_qk(desc, rope, None, moved, None, step, 19, seq_len=seq)
    diff = float(((step.double() - y.double()) * g.double()).sum()) / h
    assert abs(diff - float(dx[1, 7, 2, 11])) <= 64 * 2.0 ** -24 * (4.0 / h) * float(g.abs().max())
    assert n


def test_rope_of_no_tokens_does_nothing(duo):
    t = torch()
    sh = S.LayerShape(4, 4, 64, "fp32")
    (q, k, _), inv, _, rope = _setup(duo, sh, 1, 2, 64, [32], "halves", 1.0, 8)
    desc = duo.desc_init(1, 4, 4, 64, duo.FP32, list(range(4)), 4)
    out = t.full_like(q, 7.0)
    duo.rope_qk(desc, rope, q, None, out, None, 0)
    assert bool((out == 7.0).all())


APPENDS = [   # hq, hkv, d, dtype, retrieval, quant, paged, B, Ts, layout, rot, io
    (32, 8, 128, "bf16", [1, 4, 6], "none", False, 2, [300, 1, 1, 70], "halves", 128, "model"),
    (8, 8, 128, "bf16", [0, 3], "none", True, 3, [65, 1, 2], "pairs", 64, "block"),
    (8, 4, 64, "fp32", [2], "none", False, 2, [16, 1, 100, 1], "halves", 64, "model"),
    (8, 4, 64, "bf16", [], "none", False, 1, [3, 90, 1], "halves", 20, "model"),
    (8, 4, 128, "fp32", [0, 1, 2, 3], "none", True, 2, [130, 1], "pairs", 128, "model"),
    (8, 4, 128, "bf16", [1, 2], "int8", False, 2, [100, 1, 64], "halves", 128, "model"),
    (8, 4, 128, "bf16", [1, 2], "int4", False, 2, [100, 1, 64], "pairs", 96, "block"),
    (8, 2, 128, "bf16", [1], "int4", False, 1, [1, 1, 33], "halves", 20, "model"),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_rotated_append_is_rotation_then_append(duo, case):
    hq, hkv, d, dtype, ret, quant, paged, B, Ts, layout, rot, io = case
    t = torch()
    sh = S.LayerShape(hq, hkv, d, dtype)
    kvq = {"none": duo.KV_PLAIN, "int8": duo.KV_INT8, "int4": duo.KV_INT4}[quant]
    cap = (sum(Ts) + 63) // 64 * 64
    table = np.random.default_rng(2).permutation(B * (cap // 64)).reshape(B, -1) if paged else None
    one, two = (Layer(duo, sh, ret, B, capacity=cap, page_size=64 if paged else 0, page_table=table,
                      n_pages=B * (cap // 64) if paged else 0, kv_quant=kvq,
                      io_order=duo.ORDER_BLOCK if io == "block" else duo.ORDER_MODEL) for _ in range(2))
    names = ("k_full", "v_full", "k_ring", "v_ring", "ring_pos", "seq_len", "counters", "k_scale", "v_scale")
    for i, T in enumerate(Ts):
        (q, k, v), inv, _, rope = _setup(duo, sh, B, T, rot, [rot // 2], layout, 1.1, 40 + i)
        qr, kr, qo = t.empty_like(q), t.empty_like(k), t.empty_like(q)
        duo.rope_qk(two.desc, rope, q, k, qr, kr, T, seq_len=two.caches.seq_len)
        duo.append_kv(two.desc, two.caches.state, kr, v, T)
        duo.append_kv_rope(one.desc, one.caches.state, rope, q, k, v, qo, T)
        assert np.array_equal(bits(qo), bits(qr))
        for n in names:
            a, b = getattr(one.caches, n), getattr(two.caches, n)
            if a is not None:
                assert np.array_equal(bits(a), bits(b)), (n, i)
    assert one.status() == 0 and two.status() == 0
    # without queries, and with the queries in place
    (q, k, v), inv, _, rope = _setup(duo, sh, B, 0 + 1, rot, [rot // 2], layout, 1.0, 77)
    one.caches.seq_len.sub_(1)
    before = q.clone()
    duo.append_kv_rope(one.desc, one.caches.state, rope, None, k, v, None, 1)
    assert np.array_equal(bits(q), bits(before))
    one.caches.seq_len.sub_(1)
    qo = t.empty_like(q)
    duo.append_kv_rope(one.desc, one.caches.state, rope, q, k, v, qo, 1)
    one.caches.seq_len.sub_(1)
    duo.append_kv_rope(one.desc, one.caches.state, rope, q, k, v, q, 1)
    assert np.array_equal(bits(q), bits(qo))


def test_rotated_append_takes_positions_on_several_axes(duo):
    t = torch()
    sh = S.LayerShape(8, 4, 128, "bf16")
    B, T, sections = 2, 37, [16, 24, 24]
    pos = np.random.default_rng(9).integers(0, 5000, (3, B, T))
    (q, k, v), inv, pos_d, rope = _setup(duo, sh, B, T, 128, sections, "halves", 1.0, 4, pos)
    lay = Layer(duo, sh, [0, 2], B, capacity=64)
    qo = t.empty_like(q)
    duo.append_kv_rope(lay.desc, lay.caches.state, rope, q, k, v, qo, T)
    _check(qo, q, pos, 128, sections, "halves", 1.0, "bf16")
    want, tol = rope_ref(f64(k), pos, _inv_freq(128), 128, sections, "halves", 1.0), rope_tolerance(f64(k), 128, "halves", 1.0, "bf16")
    got = f64(lay.caches.k_full)
    for s, h in enumerate(lay.perm[:2]):
        assert np.all(np.abs(got[:, s, :T] - want[:, :, h]) <= tol[:, :, h])
    assert list(bits(lay.caches.seq_len)) == [T, T] and np.array_equal(bits(lay.caches.ring_pos)[0, :T], np.arange(T))


def test_rotated_append_reports_what_the_plain_append_reports(duo):
    """A page table entry of -1, a full cache and a negative length: the rows
    are skipped, everything else is written, the bit is set."""
    t = torch()
    sh = S.LayerShape(8, 4, 128, "bf16")
    lay = Layer(duo, sh, [0, 2], 2, page_size=64, page_table=[[0, -1], [1, 2]], n_pages=3)
    (q, k, v), inv, _, rope = _setup(duo, sh, 2, 70, 128, [64], "halves", 1.0, 4)
    qo = t.empty_like(q)
    duo.append_kv_rope(lay.desc, lay.caches.state, rope, q, k, v, qo, 70)
    assert lay.status() == duo.DEV_BAD_PAGE
    assert np.array_equal(bits(lay.caches.v_full)[1, 0], bits(v)[1, :64, lay.perm[0]])
    assert np.array_equal(bits(lay.caches.v_full)[2, 0, :6], bits(v)[1, 64:, lay.perm[0]])
    assert not bits(lay.caches.v_full)[2, 0, 6:].any()
    small = Layer(duo, sh, [0, 2], 1, capacity=8)
    (q, k, v), inv, _, rope = _setup(duo, sh, 1, 10, 128, [64], "halves", 1.0, 5)
    qo = t.empty_like(q)
    duo.append_kv_rope(small.desc, small.caches.state, rope, q, k, v, qo, 10)
    assert small.status() == duo.DEV_FULL_CACHE_OVERFLOW
    assert np.array_equal(bits(small.caches.v_full)[0, 1], bits(v)[0, :8, small.perm[1]])
    for quant in (duo.KV_INT8, duo.KV_PLAIN):
        bad = Layer(duo, sh, [0, 2], 1, capacity=64, kv_quant=quant)
        bad.caches.seq_len.fill_(-3)
        duo.append_kv_rope(bad.desc, bad.caches.state, rope, q[:, :1].contiguous(), k[:, :1].contiguous(), v[:, :1].contiguous(),
                           t.empty_like(q[:, :1]), 1)
        assert bad.status() == duo.DEV_FULL_CACHE_OVERFLOW | duo.DEV_BAD_LENGTH
        assert not bits(bad.caches.k_full).any() and not bits(bad.caches.k_ring).any()


def test_rotated_append_captured_and_replayed(duo):
    """A graph that holds one rotated append, replayed: every replay appends
    the next token."""
    t = torch()
    sh = S.LayerShape(8, 4, 128, "bf16")
    (q, k, v), inv, _, rope = _setup(duo, sh, 2, 1, 128, [64], "halves", 1.0, 6)
    a, b = (Layer(duo, sh, [0, 2], 2, capacity=64) for _ in range(2))
    qo, qr = t.empty_like(q), t.empty_like(q)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=side):
        duo.append_kv_rope(a.desc, a.caches.state, rope, q, k, v, qo, 1)
    for _ in range(5):
        graph.replay()
        duo.append_kv_rope(b.desc, b.caches.state, rope, q, k, v, qr, 1)
    t.cuda.synchronize()
    assert np.array_equal(bits(qo), bits(qr)) and list(bits(a.caches.seq_len)) == [5, 5]
    for n in ("k_full", "v_full", "k_ring", "v_ring", "ring_pos"):
        assert np.array_equal(bits(getattr(a.caches, n)), bits(getattr(b.caches, n)))
