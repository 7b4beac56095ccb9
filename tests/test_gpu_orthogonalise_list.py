"""Products of a batch as one list in a cooperative launch: a wait that gives up ends all of it."""
import ctypes

import pytest
import torch

import server_side_fedavg_gb300 as fa
from tests.test_gpu_orthogonalise import QUINTIC, iterate, make, near

pytestmark = pytest.mark.gpu


def launches(work):
    st = fa.fa_work_stats()
    assert fa.lib().fa_work_get_stats(work, ctypes.byref(st)) == fa.FA_OK
    return st.kernel_launches


@pytest.mark.parametrize("count,rows,cols", [(24, 512, 512), (24, 1024, 1024)])
def test_an_expired_wait_is_reported_and_ends(count, rows, cols):
    u = make(count, rows, cols, "f32", 71)
    out = torch.empty_like(u)
    bad, good = fa.fa_work_open(flags=fa.FA_TEST_WAIT_EXPIRES), fa.fa_work_open()
    try:
        for _ in range(2):
            before = launches(bad)
            fa.fa_orthogonalise(bad, count, rows, cols, u, out, "f32", "f32")
            assert launches(bad) - before == 4                # norm, scale, the list, the result
            with pytest.raises(fa.FedAvgError) as e:
                fa.fa_work_sync(bad)
            assert e.value.status == fa.FA_ERR_INTERNAL and "device-side wait" in e.value.detail
        fa.fa_orthogonalise(good, count, rows, cols, u, out, "f32", "f32")
        fa.fa_work_sync(good)
        near(out, iterate(u, 5, QUINTIC, 1e-7), 1.0, None, "f32", 5)
    finally:
        fa.fa_work_close(bad)
        fa.fa_work_close(good)
