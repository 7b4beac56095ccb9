"""A first round of fa_orthogonalise: no momentum yet, one to be written.  x is the update itself, with
or without FA_ORTHO_NESTEROV, whatever mu is."""
import pytest
import torch

import server_side_fedavg_gb300 as fa
from tests.test_gpu_orthogonalise import make, work  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(30, 50), (60, 500), (200, 130), (300, 1500)])
@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("mu", [0.9, -1.0, 1e30])
@pytest.mark.parametrize("din", ["f32", "bf16"])
def test_x_is_the_update(work, rows, cols, nesterov, mu, din):  # noqa: F811
    """eps is of the update's size, so that a factor of x shows.  Steps of 0 scale alone: the norm is a sum
    of rows x cols terms, in runs of at most 2^11 to a thread (2^-13 at worst, halved by the root; far
    less where roundings are random), X is held to 2^-22 of its largest element or better."""
    u = make(2, rows, cols, din, 51)
    eps = u[0].double().norm().item()
    mom, out, other = (torch.full((2, rows, cols), 7.0, device="cuda") for _ in range(3))
    fa.fa_orthogonalise(work, 2, rows, cols, u, out, din, "f32", steps=0, eps=eps, momentum_out=mom, mu=mu, nesterov=nesterov)
    assert torch.equal(mom, u.float())
    x = u.double()
    want = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    assert ((out.double() - want).abs() <= 2.0 ** -14 * want.abs() + 2.0 ** -22 * want.abs().max()).all()
    # and the iteration's result is the one without any momentum, to the bit
    fa.fa_orthogonalise(work, 2, rows, cols, u, out, din, "f32", eps=eps, momentum_out=mom, mu=mu, nesterov=nesterov)
    fa.fa_orthogonalise(work, 2, rows, cols, u, other, din, "f32", eps=eps)
    assert torch.equal(out, other)
