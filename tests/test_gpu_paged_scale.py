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


@pytest.mark.parametrize("lens,window", [([(1, 1), (700, 1)], 0), ([(9000, 1)], 0), ([(300, 5), (129, 3)], 0),
                                         ([(260, 129), (33, 33)], 0), ([(5000, 40)], 0), ([(900, 200)], 100)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dt,power", [("f16", 0), ("f16", 4), ("f16", 8), ("f16", 15), ("bf16", 0), ("bf16", 16), ("bf16", 60),
                                      ("bf16", 110)])
def test_large_scores(kernel, dt, power, sign, D, lens, window):
    """All dims of a query are 2^power and all dims of a key one small integer,
    so scores are exact in fp32 and differ by D 2^power at least: a query's
    weight is shared evenly by the seen keys of the largest integer, however
    large the scores are.

    Off by: the weights of those keys 4 e each (ex2.approx; the same for all) and
    e per rescale or join (R = N / 16 + 8), twice; their sums 2 N e, twice; P once
    u; the division and its product 3 e; the result u, in fp16 half of the smallest
    subnormal.  Where the scores lie below 2^16 in base two, the product of the
    maximum and the scale is off by 2^-9 at most: 2^-9 ln 2 per weight, twice.  The
    others' weights are below 2^-60 (D 2^power scale log2 e >= 64 x 1.44)."""
    b = Batch(lens, 8, 2, D=D, page=32, dt=dt, seed=D + power + len(lens), window=window)
    t = b.q.dtype
    g = torch.Generator(device="cuda").manual_seed(power)
    b.q = torch.full_like(b.q, 2.0 ** power)
    own = ~b.k.isnan()
    lo, hi = (1000, 1008) if dt == "f16" else (200, 208)
    k = torch.randint(lo, hi, b.k.shape[:3] + (1,), generator=g, device="cuda") * sign
    b.k = torch.where(own, k.to(t), b.k)
    if dt == "bf16" and power == 110:  # D 2^110 200 stays below 2^127
        b.k = b.k / 4
    b.scale = 1.0
    got = b.run(cider, scale=1.0).double().cpu().numpy()
    want, mag, _, cnt = b.oracle()
    u, e = (2.0 ** -11, 2.0 ** -24) if dt == "f16" else (2.0 ** -8, 2.0 ** -24)
    n = cnt[:, None, None]
    rel = u + 2 * (4 * e + (n / 16 + 8) * 5 * e + 2 * n * e) + 3 * e + 2 * 2.0 ** -9 * np.log(2)
    tol = rel * mag * (1 + u) + u * np.abs(want) + (2.0 ** -25 if dt == "f16" else 0.0)
    err = np.abs(got - want)
    assert (err <= tol).all(), f"{(~(err <= tol)).sum()} of {err.size} off, worst {np.nanmax(err / tol)} of the tolerance"
