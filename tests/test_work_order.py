"""The order of a work handle's calls where one of them fails (CPU, a fake runtime): what a
call has queued before it failed still uses the shared workspace, so that the next call on
another stream, and a wait for the handle, have to wait for it."""
import pytest

import server_side_fedavg_gb300 as fa
from tests.work_shim import Work

A, B, OUT, D, PRE, DA, DB = (i << 36 for i in range(1, 8))
M, N, K = 300, 260, 516


def failed_product(w):
    w.fail("product")
    return w.product(M, N, K, A, B, OUT, stream=1), ["split:1", "product:1"]


def failed_backward(w):
    w.fail("product", 1)
    return (w.backward(M, N, K, A, B, D, DA, DB, act="gelu", pre=PRE, ldp=N, stream=1),
            ["act_grad:1", "split:1", "product:1", "split:1", "product:1"])


def failed_bias(w):
    w.fail("col_sum")
    return (w.backward(M, N, K, A, B, D, None, None, d_bias=DA, stream=1), ["act_grad:1", "col_sum:1"])


@pytest.mark.parametrize("failing", [failed_product, failed_backward, failed_bias])
def test_a_call_after_a_failed_one_waits_for_what_that_had_queued(failing):
    w = Work(workspace_bytes=1 << 28)
    status, launches = failing(w)
    assert status == fa.FA_ERR_CUDA and "name" in w.error()
    assert [c for c in w.log() if c.split(":")[0] not in ("record", "malloc")] == launches
    w.L.ws_clear_log()
    assert w.product(M, N, K, A, B, OUT, stream=2) == fa.FA_OK
    log = w.log()
    assert log.index("wait:2") < log.index("split:2")
    assert w.close() == fa.FA_OK


@pytest.mark.parametrize("failing", [failed_product, failed_backward, failed_bias])
def test_a_wait_for_the_handle_covers_a_failed_call(failing):
    w = Work(timeout_ms=20, workspace_bytes=1 << 28)
    assert failing(w)[0] == fa.FA_ERR_CUDA
    w.L.ws_pending(1)                 # the kernels that it queued do not end
    assert w.sync() == fa.FA_ERR_TIMEOUT
    assert w.close() == fa.FA_ERR_TIMEOUT
    w.L.ws_pending(0)
    assert w.sync() == fa.FA_OK and w.close() == fa.FA_OK


def test_the_first_error_is_the_one_reported():
    w = Work()
    w.fail("product")
    assert w.product(M, N, K, A, B, OUT, stream=1) == fa.FA_ERR_CUDA
    assert w.error().startswith("product:")
    assert w.close() == fa.FA_OK


def test_calls_that_succeed_are_ordered_across_streams():
    w = Work()
    assert w.product(M, N, K, A, B, OUT, stream=1) == fa.FA_OK
    assert w.product(M, N, K, A, B, OUT, stream=1) == fa.FA_OK
    assert not any(c.startswith("wait") for c in w.log())
    assert w.product(M, N, K, A, B, OUT, stream=2) == fa.FA_OK
    assert "wait:2" in w.log()
    assert w.close() == fa.FA_OK
