"""The rotated append reports what the plain append reports, whatever the
lengths hold."""

import numpy as np
import pytest

from head_split_kv_b200 import synthetic as S
from tests.gpu_helpers import Layer, bits, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,rot", [("fp32", 64, 64), ("bf16", 128, 128), ("bf16", 128, 20)])
@pytest.mark.parametrize("sink", [0, 4])
@pytest.mark.parametrize("length,T", [(-5, 40), (-5, 9), (-1, 1), (-100, 40), (0, 40), (3, 40), (250, 40)])
@pytest.mark.parametrize("ret", [(), (1,)])
def test_status_bits_are_the_plain_appends(duo, dtype, d, rot, sink, length, T, ret):
    """Negative lengths (reported, their rows skipped), ordinary ones, and rows past the capacity."""
    t = torch()
    sh = S.LayerShape(8, 4, d, dtype, sink=sink, recent=8)
    dt = t.bfloat16 if dtype == "bf16" else t.float32
    t.manual_seed(2)
    k, v = (t.randn(2, T, 4, d, device="cuda").to(dt) for _ in range(2))
    inv = t.linspace(1.0, 1e-3, rot // 2, device="cuda")
    rope = duo.rope_init(rot, inv)
    one, two = (Layer(duo, sh, list(ret), 2, capacity=256) for _ in range(2))
    for lay in (one, two):
        lay.caches.seq_len.copy_(t.tensor([length, 20], dtype=t.int32))
    kr = t.empty_like(k)
    duo.rope_qk(two.desc, rope, None, k, None, kr, T, seq_len=two.caches.seq_len)
    duo.append_kv(two.desc, two.caches.state, kr, v, T)
    duo.append_kv_rope(one.desc, one.caches.state, rope, None, k, v, None, T)
    assert one.status() == two.status()
    assert (one.status() != 0) == (length < 0 or (length + T > 256 and len(ret) > 0))
    for n in ("k_full", "v_full", "k_ring", "v_ring", "ring_pos", "seq_len"):
        a, b = getattr(one.caches, n), getattr(two.caches, n)
        assert np.array_equal(bits(a), bits(b)), n
