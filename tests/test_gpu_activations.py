"""gelu and silu and their derivatives in fp32 against fp64: a product of zeros with the values as
its bias gives the activation alone, the bias gradient of one row the derivative alone.

fp32 results are as good as the formula's own in fp32 (z Phi(z) with Phi from erf, z / (1 + exp(-z)))
to within a factor of two of its root-mean-square error over normally distributed values.  For z
below -1 the result is relatively exact: z Phi(z) is a product of z, a polynomial and exp(-z^2 / 2),
off by 2^-23 (z^2 / 2 for the exponential's argument, and 8 for the other roundings)."""
import pytest
import torch

import server_side_fedavg_gb300 as fa

pytestmark = pytest.mark.gpu

FN = {"gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu}
N = 1 << 20


@pytest.fixture(scope="module")
def work():
    w = fa.fa_work_open()
    yield w
    fa.fa_work_close(w)


def _act(work, act, z, rows):
    """act(z), by the kernels for one row or for `rows` of the tensor cores."""
    n = z.numel()
    a, b = torch.zeros((rows, 64), device="cuda"), torch.zeros((n, 64), device="cuda")
    out = torch.empty((rows, n), device="cuda")
    fa.fa_product(work, rows, n, 64, a, 64, b, 64, out, n, "f32", "f32", trans_b=True, bias=z, act=act)
    torch.cuda.synchronize()
    assert torch.equal(out[0].expand_as(out).view(torch.int32), out.view(torch.int32))
    return out[0]


def _derivative(work, act, z):
    n = z.numel()
    a, b, ones, d = (torch.zeros((1, 64), device="cuda"), torch.zeros((n, 64), device="cuda"), torch.ones((1, n), device="cuda"),
                     torch.empty((n,), device="cuda"))
    fa.fa_product_backward(work, 1, n, 64, a, 64, b, 64, ones, n, None, 64, None, 64, "f32", "f32", "f32", trans_b=True,
                           act=act, pre=z, ldp=n, d_bias=d)
    torch.cuda.synchronize()
    return d


def _slope(act, z):
    z = z.clone().requires_grad_()
    return torch.autograd.grad(FN[act](z).sum(), z)[0]


def _rms(x, exact):
    return (x.double() - exact).square().mean().sqrt().item()


def _normal():
    g = torch.Generator(device="cuda").manual_seed(0)
    return torch.randn((N,), generator=g, device="cuda")


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_activations_are_fp32_results(work, act, rows):
    z = _normal()[: N // rows]
    exact = FN[act](z.double())
    assert _rms(_act(work, act, z, rows), exact) <= 2 * _rms(FN[act](z), exact)


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_derivatives_are_fp32_results(work, act):
    z = _normal()
    exact = _slope(act, z.double())
    assert _rms(_derivative(work, act, z), exact) <= 2 * _rms(_slope(act, z), exact)


@pytest.mark.parametrize("rows", [1, 40])
def test_the_lower_tail_of_gelu(work, rows):
    z = torch.linspace(-12.5, -1, N // rows, device="cuda")
    z64 = z.double()
    exact = z64 * 0.5 * torch.erfc(-z64 * 0.5 ** 0.5)
    got = _act(work, "gelu", z, rows).double()
    assert ((got - exact).abs() <= exact.abs() * 2.0 ** -23 * (8 + z64 * z64 / 2)).all()


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_far_values(work, act):
    z = torch.tensor([-3.0e38, -1e30, -1e10, -200.0, -90.0, -0.0, 0.0, 20.0, 90.0, 1e10, 1e30, 3.0e38, float("nan")], device="cuda")
    out, d = _act(work, act, z, 1), _derivative(work, act, z)
    assert (out[:4].abs() <= 1e-30).all() and torch.equal(out[7:12], z[7:12]) and torch.isnan(out[12])
    assert (d[:4].abs() <= 1e-30).all() and (d[5:7] - 0.5).abs().max() <= 2.0 ** -22
    assert (d[7:12] - 1).abs().max() <= 1e-6 and torch.isnan(d[12])
