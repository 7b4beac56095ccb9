"""The one-kernel form of the group norm on samples of 25 to 77 MB, whose stages are fetched twice where
shared memory does not hold them: outputs over inputs, wider rows and gaps between samples, what is not
finite."""
import ctypes

import pytest
import torch

import server_side_fedavg_gb300 as fa
from tests.test_gpu_group_norm import HALF_STEP, NEAR, T, forward64, gradients64, make, stats, work  # noqa: F401

pytestmark = pytest.mark.gpu

G = 8
SIZES = [(2, 700001, 16, "f32"), (2, 300001, 64, "bf16"), (3, 12001, 1024, "bf16")]


def launches(work):  # noqa: F811
    st = fa.fa_work_stats()
    assert fa.lib().fa_work_get_stats(work, ctypes.byref(st)) == fa.FA_OK
    return st.kernel_launches


def one(work, call, most):  # noqa: F811
    """The call, which takes the one kernel (and `most` - 1 others)."""
    before = launches(work)
    call()
    assert launches(work) - before == most


def forward(work, x, y, n, P, C, dtype, gamma, beta, mean=None, rstd=None, **kw):  # noqa: F811
    one(work, lambda: fa.fa_group_norm(work, n, P, C, G, x, y, dtype, gamma, beta, "f32", act="silu", mean=mean, rstd=rstd, **kw), 1)


def near(y, x, gamma, beta, dtype):
    want, xhat, *_ = forward64(x, G, gamma, beta, "silu", 1e-5)
    size = 1.13 * (NEAR * (xhat.abs() + 1) * gamma.double().abs() + NEAR * beta.double().abs()) + (HALF_STEP[dtype] + 2.0 ** -22) * want.abs()
    assert ((y.double() - want).abs() <= size).all()


@pytest.mark.parametrize("n,P,C,dtype", SIZES)
def test_in_place(work, n, P, C, dtype):  # noqa: F811
    x, gamma, beta, dout = make(n, P, C, dtype, "f32", 61)
    y, mean, rstd = torch.empty_like(x), torch.empty((n, G), device="cuda"), torch.empty((n, G), device="cuda")
    forward(work, x, y, n, P, C, dtype, gamma, beta, mean, rstd)
    near(y, x, gamma, beta, dtype)
    over = x.clone()
    forward(work, over, over, n, P, C, dtype, gamma, beta)
    assert torch.equal(over, y)
    dx, d_gamma, d_beta = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)

    def backward(a, b, to, dg, db):
        one(work, lambda: fa.fa_group_norm_backward(work, n, P, C, G, a, b, to, dtype, gamma, beta, "f32", mean, rstd, act="silu",
                                                    d_gamma=dg, d_beta=db), 2)
    backward(x, dout, dx, d_gamma, d_beta)
    for which in (0, 1):
        pair, dg, db = [x.clone(), dout.clone()], torch.empty_like(gamma), torch.empty_like(beta)
        backward(*pair, pair[which], dg, db)
        assert torch.equal(pair[which], dx) and torch.equal(dg, d_gamma) and torch.equal(db, d_beta)
        assert torch.equal(pair[1 - which], (dout, x)[which])


@pytest.mark.parametrize("n,P,C,dtype", SIZES)
def test_wider_rows_of_the_result_and_gaps_between_samples(work, n, P, C, dtype):  # noqa: F811
    """x and dout dense with a gap behind each sample, y and dx a slice of wider rows; what is beside them stays."""
    x, gamma, beta, dout = make(n, P, C, dtype, "f32", 62)
    gap, wide, at = 3 * C, C + 24, 8
    apart = P * C + gap
    xs, ds = (torch.full((n, apart), 9.0, device="cuda", dtype=T[dtype]) for _ in range(2))
    xs[:, :P * C], ds[:, :P * C] = x.view(n, -1), dout.view(n, -1)
    out = torch.full((n, P + 5, wide), 5.0, device="cuda", dtype=T[dtype])
    y = out[:, :P, at:at + C]
    mean, rstd = torch.empty((n, G), device="cuda"), torch.empty((n, G), device="cuda")
    forward(work, xs, y, n, P, C, dtype, gamma, beta, mean, rstd, step_x=apart, ldy=wide, step_y=(P + 5) * wide)
    dense = torch.empty_like(x)
    forward(work, x, dense, n, P, C, dtype, gamma, beta)
    assert torch.equal(y, dense)
    near(dense, x, gamma, beta, dtype)
    y[:] = 5.0
    assert (out == 5).all()
    one(work, lambda: fa.fa_group_norm_backward(work, n, P, C, G, xs, ds, y, dtype, gamma, beta, "f32", mean, rstd, act="silu",
                                                step_x=apart, step_d=apart, lddx=wide, step_dx=(P + 5) * wide), 1)
    one(work, lambda: fa.fa_group_norm_backward(work, n, P, C, G, x, dout, dense, dtype, gamma, beta, "f32", mean, rstd, act="silu"), 1)
    assert torch.equal(y, dense)
    y[:] = 5.0
    assert (out == 5).all() and (xs[:, P * C:] == 9).all() and (ds[:, P * C:] == 9).all()


@pytest.mark.parametrize("n,P,C,dtype", SIZES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("place", [0, 12000])
def test_what_is_not_finite_spoils_its_group_alone(work, n, P, C, dtype, bad, place):  # noqa: F811
    x, gamma, beta, dout = make(n, P, C, dtype, "f32", 63)
    per = C // G
    x[1, place, 2 * per] = bad
    y, mean, rstd, dx = torch.empty_like(x), torch.empty((n, G), device="cuda"), torch.empty((n, G), device="cuda"), torch.empty_like(x)
    forward(work, x, y, n, P, C, dtype, gamma, beta, mean, rstd)
    one(work, lambda: fa.fa_group_norm_backward(work, n, P, C, G, x, dout, dx, dtype, gamma, beta, "f32", mean, rstd, act="silu"), 1)
    spoilt = torch.zeros((n, 1, C), device="cuda", dtype=torch.bool)
    spoilt[1, :, 2 * per:3 * per] = True
    for t in (y, dx):
        assert torch.equal(torch.isfinite(t), ~spoilt.expand_as(t))
    assert not torch.isfinite(mean[1, 2]) and torch.isfinite(mean).sum() == n * G - 1


@pytest.mark.parametrize("n,P,C,dtype", SIZES)
def test_gradients(work, n, P, C, dtype):  # noqa: F811
    """Against the formula in fp64, by the 2-norm: sums of up to 700001 terms over some 200 a thread, and z
    formed anew in fp32, are each off by less than NEAR of their terms' sizes."""
    x, gamma, beta, dout = make(n, P, C, dtype, "f32", 64)
    m64, r64 = stats(x, G, 1e-5)
    mean, rstd = m64.float(), r64.float()
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
    fa.fa_group_norm_backward(work, n, P, C, G, x, dout, dx, dtype, gamma, beta, "f32", mean, rstd, act="silu", d_gamma=dg, d_beta=db)
    w_dx, w_g, w_b, size, sg, sb, *_ = gradients64(x, G, gamma, beta, mean, rstd, "silu", dout)
    assert (dx.double() - w_dx).norm() <= NEAR * size.norm() + HALF_STEP[dtype] * w_dx.norm()
    assert ((dg.double() - w_g).abs() <= 2 * NEAR * sg).all() and ((db.double() - w_b).abs() <= 2 * NEAR * sb).all()
