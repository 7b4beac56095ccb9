"""The sizes of tests/product_forms.py reach the forms that they name, every form with each kind
of result, and those that walk over tiles more tiles than run at one time (CPU)."""
import pytest

import server_side_fedavg_gb300 as fa
from tests import product_forms as F
from tests.work_shim import Work


@pytest.fixture(scope="module")
def work():
    w = Work()
    yield w
    w.close()


@pytest.mark.parametrize("m,n,k,din,dout,form", F.FORMS)
def test_a_size_takes_its_form(work, m, n, k, din, dout, form):
    work.L.ws_clear_log()
    assert work.product(m, n, k, 1 << 40, 2 << 40, 3 << 40, din, dout) == fa.FA_OK
    assert any(c.startswith("product") for c in work.log())
    assert work.choice()[0] == form and work.choice()[2] == (dout == "f32")


def test_every_form_is_there():
    assert {(f[5], f[4]) for f in F.FORMS} >= {(form, out) for form in F.TILE for out in ("bf16", "f32")}
    for form in (F.PAIR256, F.PAIR128, F.SINGLE128, F.SWAP64, F.SWAP32, F.SWAP16):
        assert any(f[5] == form and F.tiles(f[0], f[1], form) > F.TILE[form][2] for f in F.FORMS), form
