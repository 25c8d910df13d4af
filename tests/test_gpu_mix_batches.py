"""The training step over batches of any size: more sequences than a grid's
second and third dimension hold, of one token each, where the mix is the
identity on v."""

import pytest

from tests.gpu_helpers import torch
from tests.test_gpu_mix_train import _case, _step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dtype", [(64, "fp32"), (128, "bf16")])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_more_sequences_than_65535(duo, d, dtype, cap):
    t = torch()
    B = 66_000
    desc, q, k, v, do, al = _case(duo, 2, 1, d, dtype, B, 1, cap, 1.0, alpha=[0.25])
    out, dq, dk, dv, da = _step(duo, desc, cap, q, k, v, do, al)
    half = 2.0 ** -24 if dtype == "fp32" else 2.0 ** -8
    # one key: both weights are 1, so out = v for either query head, dv = the sum of both dout, the score has no
    # gradient but the rounding of dP - D (half a step of a sum of d products, 8 sigma of it) times one key or query
    assert float((out.float() - v.float()).abs().max()) <= 4 * half * float(v.float().abs().max())
    want = do.float().sum(2, keepdim=True)
    assert float((dv.float() - want).abs().max()) <= 4 * half * 2 * float(do.float().abs().max())
    noise = 64 * 2.0 ** -24 * d ** 0.5 * float(v.float().abs().max()) * float(do.float().abs().max())
    for g, x in ((dq, k), (dk, q)):
        assert float(g.float().abs().max()) <= 2 * noise * float(x.float().abs().max())
    assert float(da.abs().max()) == 0.0        # inside the window both attentions are one
