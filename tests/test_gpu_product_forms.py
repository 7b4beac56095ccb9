"""Every form of the tensor-core product against fp64, element by element, at sizes with ragged
edges and with more tiles than run at one time; its gradients at ragged sizes in all storage
orders; waits that run out.  Tolerances and checks as in test_gpu_product.py."""
import pytest
import torch

import server_side_fedavg_gb300 as fa
from tests.product_forms import FORMS
from tests.test_gpu_product import TORCH, _backward, _forward, work  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k,din,dout,form", FORMS)
def test_epilogue(work, m, n, k, din, dout, form):  # noqa: F811
    _forward(work, m, n, k, din, dout, bias=True, act="gelu", res="other", pre=True, alpha=0.5, beta=-0.75, seed=m)
    _forward(work, m, n, k, din, dout, bias=True, act="silu", pre=True, seed=m + 1)
    _forward(work, m, n, k, din, dout, res="out", beta=0.5, seed=m + 2)
    _forward(work, m, n, k, din, dout, bias=True, res="other", seed=m + 3)
    _forward(work, m, n, k, din, dout, seed=m + 4)


@pytest.mark.parametrize("ta,tb", [(False, False), (True, True), (True, False)])
@pytest.mark.parametrize("m,n,k,din,dout,form", FORMS)
def test_storage_orders(work, m, n, k, din, dout, form, ta, tb):  # noqa: F811
    _forward(work, m, n, k, din, dout, ta, tb, bias=True, act="relu", res="out", seed=n)


@pytest.mark.parametrize("pad", [(0, 0, 1, 3), (8, 8, 2, 2), (3, 5, 8, 8)])
@pytest.mark.parametrize("m,n,k,din,dout,form", [f for f in FORMS if f[0] * f[1] < 6_000_000])
def test_strides(work, m, n, k, din, dout, form, pad):  # noqa: F811
    """Outputs that TMA cannot write (and that two or four elements of a store can be aligned for),
    operands that have to be laid out first."""
    _forward(work, m, n, k, din, dout, bias=True, act="silu", res="other", pre=True, pad=pad, seed=k)
    _forward(work, m, n, k, din, dout, res="out", pad=pad, seed=k)


@pytest.mark.parametrize("ta", [False, True])
@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("din,ddout,dgrad", [("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"), ("bf16", "f32", "f32"),
                                             ("f32", "f32", "f32")])
@pytest.mark.parametrize("m,n,k", [(1300, 2100, 700), (2600, 1304, 1500)])
def test_gradients(work, m, n, k, din, ddout, dgrad, ta, tb):  # noqa: F811
    _backward(work, m, n, k, din, ddout, dgrad, ta, tb, "gelu", seed=m)
    _backward(work, m, n, k, din, ddout, dgrad, ta, tb, "none", bias=False, seed=m + 1)


@pytest.mark.parametrize("m,n,k,din,dout,form", [f for f in FORMS if f[0] * f[1] < 3_000_000])
def test_same_bits_every_time(work, m, n, k, din, dout, form):  # noqa: F811
    a = _forward(work, m, n, k, din, dout, bias=True, act="gelu", res="other", pre=True, seed=1).clone()
    for _ in range(3):
        assert torch.equal(a, _forward(work, m, n, k, din, dout, bias=True, act="gelu", res="other", pre=True, seed=1))


@pytest.mark.parametrize("m,n,k,din,dout,form", FORMS)
def test_an_expired_wait_is_reported_and_ends(m, n, k, din, dout, form):
    """With and without residuals loaded ahead: the product ends, and the handle says so once."""
    a, b = (torch.zeros(s, device="cuda", dtype=TORCH[din]) for s in ((m, k), (n, k)))
    res, out = (torch.zeros((m, n), device="cuda", dtype=TORCH[dout]) for _ in range(2))
    w = fa.fa_work_open(flags=fa.FA_TEST_WAIT_EXPIRES)
    try:
        for r in (None, res):
            fa.fa_product(w, m, n, k, a, k, b, k, out, n, din, dout, False, True, residual=r, ldr=n)
            with pytest.raises(fa.FedAvgError) as e:
                fa.fa_work_sync(w)
            assert e.value.status == fa.FA_ERR_INTERNAL and "device-side wait" in e.value.detail
        fa.fa_work_sync(w)
    finally:
        fa.fa_work_close(w)
