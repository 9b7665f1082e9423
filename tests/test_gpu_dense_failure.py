"""Failure detection of the dense kernels without a fault: their bounded wait, on a phase
that nothing completes, gives up, is reported once, and leaves the context usable."""
import pytest
import torch

from bit_ptq_looped_b200 import lq

pytestmark = pytest.mark.gpu


def products_work():
    x = torch.eye(32, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.arange(24 * 64, device="cuda").view(24, 64).remainder(101).to(torch.bfloat16)
    y, _ = lq.lq_dense_linear(x, w)
    assert torch.equal(y, w[:, :32].t())
    lq.lq_check_device()


def test_dense_wait_times_out_and_reports_once():
    lq.lq_check_device()  # clean state
    lq.lq_selftest_dense_wait(2000)  # 2 ms limit
    with pytest.raises(lq.LQError) as e:
        lq.lq_check_device()
    assert e.value.status == lq.LQ_ERR_DEVICE_TIMEOUT and "dense" in str(e.value)
    lq.lq_check_device()  # the status word was cleared
    products_work()


def test_both_status_words_are_one_report():
    lq.lq_check_device()
    lq.lq_selftest_bounded_wait(2000)
    lq.lq_selftest_dense_wait(2000)
    with pytest.raises(lq.LQError) as e:
        lq.lq_check_device()
    assert e.value.status == lq.LQ_ERR_DEVICE_TIMEOUT
    lq.lq_check_device()
    products_work()


def test_dense_wait_on_another_stream():
    lq.lq_check_device()
    s = torch.cuda.Stream()
    lq.lq_selftest_dense_wait(2000, stream=s)
    with pytest.raises(lq.LQError) as e:
        lq.lq_check_device(s)
    assert e.value.status == lq.LQ_ERR_DEVICE_TIMEOUT
    lq.lq_check_device()
