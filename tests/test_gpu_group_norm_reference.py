"""Group norm statistics where single positions, or the first ones, are far from the rest: a background
voxel in the corner, the edge of a padded convolution, an outlier.  In both forms of the forward call."""
import pytest
import torch

import server_side_fedavg_gb300 as fa
from tests.test_gpu_group_norm import HALF_STEP, NEAR, T, forward64, work  # noqa: F401

pytestmark = pytest.mark.gpu

# positions, channels, groups: two passes, in vectors of several lengths; one kernel (4 MB and more)
SIZES = [(5000, 8, 8), (5000, 32, 4), (4999, 6, 3), (70, 3, 1), (30000, 1, 1), (900, 2048, 32), (300000, 16, 16), (131073, 32, 8), (20000, 256, 4)]


def unlike(x, kind, far):
    """x with some positions `far` away from the others."""
    P = x.shape[1]
    if kind == "first zero":                 # the others have the mean `far`
        x += far
        x[:, 0] = 0
    elif kind == "first":
        x[:, 0] += far
    elif kind == "last":
        x[:, P - 1] -= far
    elif kind == "first quarter":
        x[:, :P // 4] += far
    elif kind == "edges":                    # the first of each row of 128
        x += far
        x[:, ::128] = 0
    return x


@pytest.mark.parametrize("P,C,G", SIZES)
@pytest.mark.parametrize("kind", ["first zero", "first", "last", "first quarter", "edges"])
@pytest.mark.parametrize("far", [30.0, 1e2, 1e3])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_positions_unlike_the_others(work, P, C, G, kind, far, dtype):  # noqa: F811
    """Bounds as for ordinary data, in units of the group's own spread: what a reference that is off
    costs is at most the ratio by which the run grows until it is moved, a small factor of the sums'
    rounding that NEAR allows 128 + 32 of."""
    n = 2
    g = torch.Generator(device="cuda").manual_seed(21)
    x = unlike(torch.randn((n, P, C), generator=g, device="cuda"), kind, far).to(T[dtype])
    gamma = 1 + 0.3 * torch.randn(C, generator=g, device="cuda")
    beta = 0.3 * torch.randn(C, generator=g, device="cuda")
    y, mean, rstd = torch.full_like(x, 7), torch.empty((n, G), device="cuda"), torch.empty((n, G), device="cuda")
    fa.fa_group_norm(work, n, P, C, G, x, y, dtype, gamma, beta, "f32", mean=mean, rstd=rstd)
    want, xhat, m64, r64 = forward64(x, G, gamma, beta, "none", 1e-5)
    spread = (x.double().view(n, P, G, -1) - m64[:, None, :, None]).abs().mean((1, 3))
    assert ((rstd.double() / r64 - 1).abs() <= NEAR).all(), (rstd.double() / r64 - 1).abs().max()
    assert ((mean.double() - m64).abs() <= NEAR * spread + 2.0 ** -23 * m64.abs()).all()
    size = NEAR * (xhat.abs() + 1) * gamma.double().abs() + NEAR * beta.double().abs() + (HALF_STEP[dtype] + 2.0 ** -22) * want.abs()
    assert ((y.double() - want).abs() <= size).all()


@pytest.mark.parametrize("P,C,G", [(216, 256, 8), (40000, 32, 8)])
def test_the_kept_mean_is_rounded_to_its_own_size(work, P, C, G):  # noqa: F811
    """Over many groups the mean's error is that of its own rounding, at most 2^-25 of it in the root
    mean square, and of sums of P C / G terms of random error, here below 2^-27 of the spread: not
    that of a value of x, which is 2^-24 / 3^(1/2) at the sizes from 1 to 2."""
    n = 32
    g = torch.Generator(device="cuda").manual_seed(22)
    x = torch.randn((n, P, C), generator=g, device="cuda") * 1.5 + torch.randn((n, 1, C), generator=g, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty((n, G), device="cuda"), torch.empty((n, G), device="cuda")
    fa.fa_group_norm(work, n, P, C, G, x, y, "f32", None, None, "f32", mean=mean, rstd=rstd)
    m64 = x.double().view(n, P, G, -1).mean((1, 3))
    rms = lambda t: t.square().mean().sqrt().item()  # noqa: E731
    assert rms(mean.double() - m64) <= 2.0 ** -25 * rms(m64) + 2.0 ** -27 * 1.8
