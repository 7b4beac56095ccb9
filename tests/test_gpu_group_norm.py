"""fa_group_norm and its gradients against fp64: sizes, odd channels, strides, offsets far larger
than the spread, activations, exchanged buffers, graphs."""
import pytest
import torch

import server_side_fedavg_gb300 as fa

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
FN = {"none": lambda z: z, "relu": torch.nn.functional.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu}
# Sums run over up to 128 terms in a thread (the rows of its run), then over trees: an error below
# (128 + 32) x 2^-24 of the sum of the terms' sizes, in the mean, the variance and the gradients'
# sums alike, and a few roundings beside these.
NEAR = 256 * 2.0 ** -24


@pytest.fixture(scope="module")
def work():
    w = fa.fa_work_open()
    yield w
    fa.fa_work_close(w)


def make(n, P, C, dtype, param, seed, offset=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((n, P, C), generator=g, device="cuda") * 1.5 + offset * torch.randn((n, 1, C), generator=g, device="cuda")).to(T[dtype])
    gamma = (1 + 0.3 * torch.randn(C, generator=g, device="cuda")).to(T[param])
    beta = (0.3 * torch.randn(C, generator=g, device="cuda")).to(T[param])
    dout = torch.randn((n, P, C), generator=g, device="cuda").to(T[dtype])
    return x, gamma, beta, dout


def stats(x, G, eps):
    n, P, C = x.shape
    v = x.double().view(n, P, G, C // G)
    mean = v.mean((1, 3))
    var = (v - mean[:, None, :, None]).square().mean((1, 3))
    return mean, 1 / torch.sqrt(var + eps)


def forward64(x, G, gamma, beta, act, eps):
    n, P, C = x.shape
    mean, rstd = stats(x, G, eps)
    xhat = ((x.double().view(n, P, G, C // G) - mean[:, None, :, None]) * rstd[:, None, :, None]).view(n, P, C)
    return FN[act](xhat * gamma.double() + beta.double()), xhat, mean, rstd


def check_forward(work, n, P, C, G, dtype, param, act, seed, offset=1.0, eps=1e-5):
    x, gamma, beta, _ = make(n, P, C, dtype, param, seed, offset)
    y, mean, rstd = torch.full_like(x, 7), torch.empty((n, G), device="cuda"), torch.empty((n, G), device="cuda")
    fa.fa_group_norm(work, n, P, C, G, x, y, dtype, gamma, beta, param, act=act, eps=eps, mean=mean, rstd=rstd)
    want, xhat, m64, r64 = forward64(x, G, gamma, beta, act, eps)
    spread = (x.double().view(n, P, G, -1) - m64[:, None, :, None]).abs().mean((1, 3))
    assert ((mean.double() - m64).abs() <= NEAR * spread + 2.0 ** -23 * m64.abs()).all()
    assert ((rstd.double() / r64 - 1).abs() <= NEAR).all()
    # z is off by what mean and rstd are, in units of the spread, whatever the offset; the activations'
    # slope is below 1.13
    size = 1.13 * (NEAR * (xhat.abs() + 1) * gamma.double().abs() + NEAR * beta.double().abs()) + HALF_STEP[dtype] * want.abs() + 2.0 ** -22 * want.abs()
    assert ((y.double() - want).abs() <= size).all()


@pytest.mark.parametrize("n,P,C,G,dtype,param,act", [
    (1, 216, 256, 8, "f32", "f32", "silu"), (2, 1, 64, 8, "f32", "f32", "gelu"), (3, 1, 8, 8, "bf16", "f32", "none"),
    (4, 64, 256, 32, "bf16", "bf16", "relu"), (2, 4097, 32, 8, "bf16", "f32", "silu"), (1, 30000, 16, 4, "f32", "f32", "gelu"),
    (5, 77, 33, 3, "f32", "f32", "silu"), (5, 77, 33, 33, "bf16", "bf16", "silu"), (2, 999, 6, 1, "bf16", "f32", "gelu"),
    (1, 50, 8192, 1, "bf16", "f32", "silu"), (1, 33, 5001, 3, "f32", "bf16", "none"), (700, 3, 24, 4, "f32", "f32", "relu"),
    (1, 100000, 48, 8, "bf16", "f32", "silu"), (1, 1, 1, 1, "f32", "f32", "none"), (64, 512, 64, 8, "bf16", "f32", "none"),
    (3, 300000, 32, 8, "bf16", "f32", "silu"), (2, 700001, 16, 16, "f32", "f32", "relu"), (5, 40000, 64, 8, "f32", "bf16", "gelu"),
    (200, 16, 1024, 32, "bf16", "f32", "silu"), (1, 2000, 1024, 1024, "f32", "f32", "none"), (33, 3000, 24, 3, "bf16", "f32", "silu")])
def test_forward(work, n, P, C, G, dtype, param, act):
    check_forward(work, n, P, C, G, dtype, param, act, 1)


@pytest.mark.parametrize("offset", [1e3, 1e5])
def test_an_offset_costs_no_digits(work, offset):
    """Channels whose mean is far larger than their spread, alone in their group."""
    check_forward(work, 2, 5000, 8, 8, "f32", "f32", "none", 2, offset=offset)


def gradients64(x, G, gamma, beta, mean, rstd, act, dout):
    n, P, C = x.shape
    m, r = mean.double()[:, None, :, None], rstd.double()[:, None, :, None]
    xhat = ((x.double().view(n, P, G, -1) - m) * r).view(n, P, C)
    z = (xhat * gamma.double() + beta.double()).requires_grad_()
    (dz,) = torch.autograd.grad(FN[act](z), z, dout.double())
    dh = (dz * gamma.double()).view(n, P, G, -1)
    h = xhat.view(n, P, G, -1)
    dx = (r * (dh - dh.mean((1, 3), keepdim=True) - h * (dh * h).mean((1, 3), keepdim=True))).view(n, P, C)
    size = (r * (dh.abs() + dh.abs().mean((1, 3), keepdim=True) + h.abs() * (dh * h).abs().mean((1, 3), keepdim=True))).view(n, P, C)
    return dx, (dz * xhat).sum((0, 1)), dz.sum((0, 1)), size, (dz * xhat).abs().sum((0, 1)), dz.abs().sum((0, 1)), dz, xhat


def check_backward(work, n, P, C, G, dtype, param, act, seed, call=None):
    x, gamma, beta, dout = make(n, P, C, dtype, param, seed)
    m64, r64 = stats(x, G, 1e-5)
    mean, rstd = m64.float(), r64.float()
    dx, d_gamma, d_beta = torch.full_like(x, 7), torch.full_like(gamma, 7), torch.full_like(beta, 7)
    fa.fa_group_norm_backward(work, n, P, C, G, x, dout, dx, dtype, gamma, beta, param, mean, rstd, act=act, d_gamma=d_gamma,
                              d_beta=d_beta)
    w_dx, w_g, w_b, size, sg, sb, dz, xhat = gradients64(x, G, gamma, beta, mean, rstd, act, dout)
    # act' of the rounded z: its slope is below 1.6 (relu's step apart, where z would have to round
    # across 0), so dz is off by 2^-21 of |dout| (|z| + 1); with the sums' own error
    wobble = 2.0 ** -21 * (dout.double().abs() * (xhat.abs() * gamma.double().abs() + beta.double().abs() + 1))
    r = r64[:, None, :, None].expand(n, P, G, C // G).reshape(n, P, C)
    bound = NEAR * size + r * gamma.double().abs() * wobble * 2 + HALF_STEP[dtype] * w_dx.abs() + r * wobble.mean() * (1 + xhat.abs())
    assert ((dx.double() - w_dx).abs() <= bound).all()
    assert ((d_gamma.double() - w_g).abs() <= NEAR * sg + (wobble * xhat.abs()).sum((0, 1)) + HALF_STEP[param] * w_g.abs()).all()
    assert ((d_beta.double() - w_b).abs() <= NEAR * sb + wobble.sum((0, 1)) + HALF_STEP[param] * w_b.abs()).all()


@pytest.mark.parametrize("n,P,C,G,dtype,param,act", [
    (1, 216, 256, 8, "f32", "f32", "silu"), (2, 1, 64, 8, "f32", "f32", "gelu"), (4, 64, 256, 32, "bf16", "bf16", "none"),
    (2, 4097, 32, 8, "bf16", "f32", "silu"), (1, 30000, 16, 4, "f32", "f32", "gelu"), (5, 77, 33, 3, "f32", "f32", "silu"),
    (5, 77, 33, 33, "bf16", "bf16", "gelu"), (2, 999, 6, 1, "bf16", "f32", "silu"), (1, 50, 8192, 1, "bf16", "f32", "none"),
    (1, 33, 5001, 3, "f32", "bf16", "gelu"), (700, 3, 24, 4, "f32", "f32", "silu"), (1, 100000, 48, 8, "bf16", "f32", "silu"),
    (64, 512, 64, 8, "bf16", "f32", "none"), (3, 300000, 32, 8, "bf16", "f32", "silu"), (2, 400001, 16, 16, "f32", "f32", "gelu"),
    (5, 40000, 64, 8, "f32", "bf16", "none"), (200, 16, 1024, 32, "bf16", "f32", "silu"), (1, 2000, 1024, 1024, "f32", "f32", "none"),
    (33, 3000, 24, 3, "bf16", "f32", "silu")])
def test_backward(work, n, P, C, G, dtype, param, act):
    check_backward(work, n, P, C, G, dtype, param, act, 3)


def test_relu_gradient_away_from_zero(work):
    """z is kept away from 0, where rounding would decide the step."""
    n, P, C, G = 2, 300, 32, 4
    x, gamma, beta, dout = make(n, P, C, "f32", "f32", 4)
    m64, r64 = stats(x, G, 1e-5)
    z = ((x.double().view(n, P, G, -1) - m64[:, None, :, None]) * r64[:, None, :, None]).view(n, P, C) * gamma.double() + beta.double()
    dout = torch.where(z.abs() < 1e-3, 0.0, dout)
    mean, rstd, dx = m64.float(), r64.float(), torch.empty_like(x)
    fa.fa_group_norm_backward(work, n, P, C, G, x, dout, dx, "f32", gamma, beta, "f32", mean, rstd, act="relu")
    w_dx, *_, size = gradients64(x, G, gamma, beta, mean, rstd, "relu", dout)[:4]
    assert ((dx.double() - w_dx).abs() <= 2 * NEAR * size + 2.0 ** -20).all()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_gradients_against_differences(work, act):
    """Along a direction, the gradients are the change of the forward call's own fp64 formula."""
    n, P, C, G = 2, 12, 16, 4
    x, gamma, beta, dout = make(n, P, C, "f32", "f32", 5)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty((n, G), device="cuda"), torch.empty((n, G), device="cuda")
    d_gamma, d_beta = torch.empty_like(gamma), torch.empty_like(beta)
    fa.fa_group_norm(work, n, P, C, G, x, y, "f32", gamma, beta, "f32", act=act, mean=mean, rstd=rstd)
    fa.fa_group_norm_backward(work, n, P, C, G, x, dout, dx, "f32", gamma, beta, "f32", mean, rstd, act=act, d_gamma=d_gamma, d_beta=d_beta)
    g = torch.Generator(device="cuda").manual_seed(6)
    step, h = [torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64) for t in (x, gamma, beta)], 1e-6
    value = lambda s: (forward64(x.double() + s * step[0], G, gamma.double() + s * step[1], beta.double() + s * step[2], act, 1e-5)[0] * dout.double()).sum()  # noqa: E731
    slope = (value(h) - value(-h)) / (2 * h)
    parts = [(dx.double() * step[0]), (d_gamma.double() * step[1]), (d_beta.double() * step[2])]
    assert abs(slope - sum(p.sum() for p in parts)) <= 1e-5 * sum(p.abs().sum() for p in parts)


def test_column_slices_and_sample_strides(work):
    """Channels are a slice of a wider buffer (a skip connection's concatenation), samples apart by
    more than their positions; what is beside them stays."""
    n, P, C, G, wide, gap = 3, 50, 24, 4, 40, 7
    buf = torch.randn((n, P + gap, wide), device="cuda")
    out = torch.full((n, P + gap, wide), 5.0, device="cuda")
    x, y = buf[:, :, 8:8 + C], out[:, :, 16:16 + C]
    gamma, beta = torch.rand(C, device="cuda") + 0.5, torch.randn(C, device="cuda")
    fa.fa_group_norm(work, n, P, C, G, x, y, "f32", gamma, beta, "f32", act="silu", ldx=wide, step_x=(P + gap) * wide, ldy=wide,
                     step_y=(P + gap) * wide)
    want = forward64(x[:, :P].contiguous(), G, gamma, beta, "silu", 1e-5)[0]
    assert ((y[:, :P].double() - want).abs() <= NEAR * 8).all()
    out[:, :P, 16:16 + C] = 5.0
    assert (out == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(work, dtype):
    n, P, C, G = 2, 700, 32, 8
    x, gamma, beta, dout = make(n, P, C, dtype, "f32", 7)
    y, mean, rstd = torch.empty_like(x), torch.empty((n, G), device="cuda"), torch.empty((n, G), device="cuda")
    fa.fa_group_norm(work, n, P, C, G, x, y, dtype, gamma, beta, "f32", act="gelu", mean=mean, rstd=rstd)
    dx = torch.empty_like(x)
    fa.fa_group_norm_backward(work, n, P, C, G, x, dout, dx, dtype, gamma, beta, "f32", mean, rstd, act="gelu")
    for who in (x, dout):
        a, b = x.clone(), dout.clone()
        to = a if who is x else b
        fa.fa_group_norm_backward(work, n, P, C, G, a, b, to, dtype, gamma, beta, "f32", mean, rstd, act="gelu")
        assert torch.equal(to, dx)
    fa.fa_group_norm(work, n, P, C, G, x, x, dtype, gamma, beta, "f32", act="gelu")
    assert torch.equal(x, y)


def test_without_parameters_and_empty(work):
    x = torch.randn((2, 30, 8), device="cuda")
    y = torch.empty_like(x)
    fa.fa_group_norm(work, 2, 30, 8, 2, x, y, "f32")
    want = forward64(x, 2, torch.ones(8, device="cuda"), torch.zeros(8, device="cuda"), "none", 1e-5)[0]
    assert ((y.double() - want).abs() <= NEAR * 6).all()
    g, b = torch.full((8,), 3.0, device="cuda"), torch.full((8,), 3.0, device="cuda")
    fa.fa_group_norm(work, 0, 30, 8, 2, None, None, "f32")
    fa.fa_group_norm_backward(work, 2, 0, 8, 2, None, None, None, "f32", None, None, "f32", None, None, d_gamma=g, d_beta=b)
    assert (g == 0).all() and (b == 0).all()


def test_a_nan_spoils_its_group_alone(work):
    x = torch.randn((2, 500, 16), device="cuda")
    x[1, 321, 6] = float("nan")
    y = torch.empty_like(x)
    fa.fa_group_norm(work, 2, 500, 16, 4, x, y, "f32")
    bad = torch.isnan(y)
    assert bad[1, :, 4:8].all() and not bad[0].any() and not bad[1, :, :4].any() and not bad[1, :, 8:].any()


def test_the_same_bits_each_time_captured_or_not(work):
    n, P, C, G = 2, 9000, 32, 8
    x, gamma, beta, dout = make(n, P, C, "bf16", "f32", 8)
    out = [torch.empty_like(x) for _ in range(4)]
    st = [torch.empty((n, G), device="cuda") for _ in range(2)]
    d = [torch.empty_like(gamma) for _ in range(4)]

    def both(y, dx, dg, db, stream):
        fa.fa_group_norm(work, n, P, C, G, x, y, "bf16", gamma, beta, "f32", act="silu", mean=st[0], rstd=st[1], stream=stream)
        fa.fa_group_norm_backward(work, n, P, C, G, x, dout, dx, "bf16", gamma, beta, "f32", st[0], st[1], act="silu", d_gamma=dg,
                                  d_beta=db, stream=stream)

    both(out[0], out[1], d[0], d[1], torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(out[2], out[3], d[2], d[3], torch.cuda.current_stream())
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(out[i], out[i + 2]) and torch.equal(d[i], d[i + 2])
