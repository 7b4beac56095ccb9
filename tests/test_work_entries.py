"""A work handle's entry points where the host or the runtime fails (CPU, a fake runtime): no
exception leaves a C function, the handle stays usable, its numbers are true."""
import pytest

import server_side_fedavg_gb300 as fa
from tests.work_shim import Work

A, B, OUT, D, PRE, DA, DB = (i << 36 for i in range(1, 8))


@pytest.mark.parametrize("entry", ["sync", "close"])
def test_no_exception_leaves_a_wait(entry):
    """Memory for an error's text may run out: here a call of the runtime throws in its place."""
    w = Work()
    assert w.product(300, 260, 516, A, B, OUT, stream=1) == fa.FA_OK
    w.fail("query", throwing=True)
    assert getattr(w, entry)() == fa.FA_ERR_NOMEM
    assert w.sync() == fa.FA_OK            # the handle is still open
    assert w.product(300, 260, 516, A, B, OUT, stream=1) == fa.FA_OK
    assert w.close() == fa.FA_OK


def test_the_error_word_is_zero_before_the_handle_is_handed_out():
    """Kernels on the caller's streams may set it at once, and fa_work_sync reads it on a stream of
    its own: neither waits for a memset that is still queued."""
    w = Work()
    log = w.opened
    memset = next(i for i, c in enumerate(log) if c.startswith("memset"))
    stream = log[memset].split(":")[1]
    assert f"synchronize:{stream}" in log[memset:]
    assert w.close() == fa.FA_OK


@pytest.mark.parametrize("name", ["malloc", "memset", "event", "stream", "host_alloc", "synchronize"])
def test_a_failed_open_says_so(name):
    import ctypes
    w = Work()
    w.close()
    w.L.ws_reset()
    w.fail(name)
    h = ctypes.c_void_p()
    status = w.L.fa_work_open(None, ctypes.byref(h))
    assert status in (fa.FA_ERR_NOMEM, fa.FA_ERR_CUDA) and h.value is None


def test_the_workspace_is_as_large_as_the_handle_says():
    w = Work()
    assert w.product(300, 260, 516, A, B, OUT) == fa.FA_OK
    before = w.stats().workspace_bytes
    assert before > 0
    w.fail("malloc")
    assert w.product(3000, 2600, 5160, A, B, OUT) == fa.FA_ERR_NOMEM
    assert w.stats().workspace_bytes == 0          # the old one had been given up for the larger
    w.L.ws_clear_log()
    assert w.product(300, 260, 516, A, B, OUT) == fa.FA_OK
    assert "malloc" in w.log() and w.stats().workspace_bytes == before
    assert w.close() == fa.FA_OK
