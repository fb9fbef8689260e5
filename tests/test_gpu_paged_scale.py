"""Paged attention with scales other than 1 / sqrt(D), and with infinite scores
at the start of a row, where a running maximum has nothing finite to go by yet.
Tolerances: tests/paged_cases.py, whose score terms take the scale."""
import numpy as np
import pytest
import torch

import w8a8_activation_quantized_b200 as cider
from tests.paged_cases import Batch, check

pytestmark = pytest.mark.gpu
SCALES = [0.05, 0.5, 0.7, 1.0, 3.0]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cider.cider_device_status()
    yield
    cider.cider_device_status()


@pytest.fixture(params=[0, 1, 2])
def kernel(request):
    cider.cider_test_set_paged_kernel(request.param)
    yield request.param
    cider.cider_test_set_paged_kernel(0)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("scale", SCALES)
def test_scales(kernel, scale, dt):
    for D, page, lens, w, s in ((128, 16, [(1, 1), (65, 1), (1025, 1)], 0, 0), (64, 64, [(700, 4), (129, 3)], 50, 3),
                                (128, 64, [(130, 70), (260, 129)], 0, 0), (64, 16, [(900, 515)], 60, 5)):
        b = Batch(lens, 8, 2, D=D, page=page, dt=dt, seed=D + len(lens), window=w, sinks=s)
        b.q *= 0.25  # scores of a few units at the largest scale, too
        b.scale = scale
        check(b, b.run(cider, scale=scale))


def _minus_infinity(b, r, keys):
    """Keys of request r whose score is -inf for every query (all queries are positive)."""
    for j in keys:
        b.k[int(b.table[r, j // b.page]), :, j % b.page, 0] = float("-inf")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [None, 1e-38, 0.5, 1.0, 3.0])
@pytest.mark.parametrize("lens,keys", [
    ([(1, 1), (40, 1)], {1: range(16)}),               # the first step of one warp
    ([(300, 1), (200, 60)], {0: range(64), 1: range(128)}),  # a whole block of keys
    ([(300, 100)], {0: range(299)}),                   # all but the last key
    ([(5000, 1)], {0: range(4900)}),                   # whole pieces of a row that several CTAs share
    ([(3000, 20)], {0: list(range(2000)) + [2990]}),
    ([(900, 300)], {0: range(0, 900, 2)}),
])
def test_keys_of_score_minus_infinity_have_no_weight(kernel, lens, keys, scale, D, dt):
    """Also where a query has seen no other key yet, and where it sees no other
    at all: there the formula is 0 / 0."""
    b = Batch(lens, 8, 2, D=D, page=32, dt=dt, seed=len(lens) + D)
    b.q = b.q.abs() * 0.25
    if scale is not None:
        b.scale = scale
    for r, js in keys.items():
        _minus_infinity(b, r, js)
    out = b.run(cider, scale=b.scale)
    want, mag, _, cnt = b.oracle()
    nan = np.isnan(want) & (cnt > 0)[:, None, None]
    np.testing.assert_array_equal(np.isnan(out.double().cpu().numpy()), nan)
    b.k[b.k.isinf()] = 0.0
    smax = b.oracle()[2]  # of the finite products
    check(b, out, (want, np.where(np.isfinite(mag), mag, 0), smax, cnt))
    assert (~nan[cnt > 0]).any()
