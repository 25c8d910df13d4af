"""Capped calls of layers with one class of heads only, and with one KV head."""

import pytest

from tests.test_gpu_capped import test_capped_decode as _decode, test_capped_prefill as _prefill

pytestmark = pytest.mark.gpu

ALL4 = [0, 1, 2, 3]


@pytest.mark.parametrize("case", [   # hq, hkv, d, dtype, retrieval, quant, mode, B, chunks, gain, cap
    (8, 4, 128, "bf16", ALL4, "none", "lambda", 2, [140, 1, 200], 3.0, 30.0),
    (8, 4, 128, "bf16", ALL4, "int8", "lambda", 1, [130, 70], 3.0, 30.0),
    (8, 4, 128, "bf16", ALL4, "int4", "chunk", 1, [130, 70], 3.0, 100.0),
    (8, 4, 128, "bf16", ALL4, "none", "lambda", 1, [140, 60], 3.0, 100.0),
    (8, 4, 128, "bf16", [], "none", "chunk", 1, [140, 60], 3.0, 50.0),
    (8, 4, 128, "bf16", [], "int4", "lambda", 1, [90, 60], 3.0, 50.0),
    (8, 1, 128, "bf16", [0], "none", "lambda", 1, [200, 129], 3.0, 60.0),
    (8, 1, 128, "bf16", [], "none", "lambda", 1, [200, 129], 3.0, 20.0),
    (8, 1, 64, "fp32", [0], "none", "lambda", 1, [70, 65], 3.0, 20.0),
    (8, 4, 64, "bf16", [], "none", "chunk", 1, [70, 65], 3.0, 20.0),
], ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_prefill_of_one_class(duo, case):
    _prefill(duo, case)


@pytest.mark.parametrize("case", [   # hq, hkv, d, dtype, retrieval, quant, paged, lengths, gain, cap
    (8, 4, 128, "bf16", ALL4, "none", True, [300, 1], 3.0, 30.0),
    (8, 4, 128, "bf16", ALL4, "int8", False, [300, 70], 3.0, 30.0),
    (8, 4, 128, "bf16", [], "int8", False, [300, 70], 3.0, 30.0),
    (8, 4, 128, "bf16", [], "none", False, [0, 500], 3.0, 100.0),
    (8, 1, 128, "bf16", [0], "none", False, [700], 3.0, 50.0),
    (8, 1, 128, "bf16", [], "none", False, [700], 3.0, 50.0),
    (8, 4, 64, "fp32", ALL4, "none", True, [90, 5], 3.0, 20.0),
], ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
@pytest.mark.parametrize("fused", [False, True])
def test_decode_of_one_class(duo, case, fused):
    _decode(duo, case, fused)
