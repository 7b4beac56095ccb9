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
