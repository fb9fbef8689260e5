"""The device status word: every condition is reported once, also when two of
them came between two reads."""
import pytest
import torch

import w8a8_activation_quantized_b200 as cider

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    for _ in range(2):  # start clean
        try:
            cider.cider_device_status()
        except cider.CiderError:
            pass


def _skipped_slot(stream=None):
    k, v = (torch.zeros((2, 2, 16, 64), dtype=torch.float16, device="cuda") for _ in range(2))
    x = torch.ones((1, 2, 64), dtype=torch.float16, device="cuda")
    y, slots = x.clone(), torch.tensor([32], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    cider.cider_paged_append(x, y, k, v, slots, stream=stream)
    torch.cuda.synchronize()


def _status():
    try:
        cider.cider_device_status()
    except cider.CiderError as e:
        return e.status
    return 0


def test_a_timeout_and_a_slot_outside_the_cache_are_both_reported():
    for first in (True, False):
        if first:
            cider.cider_test_bounded_wait(1_000_000)
        _skipped_slot()
        if not first:
            cider.cider_test_bounded_wait(1_000_000)
        torch.cuda.synchronize()
        assert [_status() for _ in range(3)] == [4, 1, 0]


def test_the_same_condition_twice_is_one_report():
    _skipped_slot()
    _skipped_slot(torch.cuda.Stream())
    torch.cuda.synchronize()
    assert [_status() for _ in range(2)] == [1, 0]
