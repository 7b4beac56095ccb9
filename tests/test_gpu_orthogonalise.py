"""fa_orthogonalise against the iteration in fp64: sizes of either orientation, batches, momentum,
weights, strides, aliases, what is not finite."""
import math

import pytest
import torch

import server_side_fedavg_gb300 as fa

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
QUINTIC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def work():
    w = fa.fa_work_open()
    yield w
    fa.fa_work_close(w)


def make(count, rows, cols, dtype, seed, rank=None):
    """An update of a few strong directions over noise; or of `rank` alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = rank or min(8, rows, cols)
    strong = torch.randn((count, rows, r), generator=g, device="cuda") @ torch.randn((count, r, cols), generator=g, device="cuda")
    noise = 0.0 if rank else torch.randn((count, rows, cols), generator=g, device="cuda")
    return ((noise + 0.3 * strong) * 1e-3).to(T[dtype])


def iterate(x, steps, coefficients, eps):
    """X and the norm's factor in fp64."""
    x = x.double()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    a, b, c = coefficients
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    for _ in range(steps):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.transpose(1, 2) if tall else x


def most_slope(coefficients, top=1.3):
    a, b, c = coefficients
    s = torch.linspace(0, top, 1001, dtype=torch.float64)
    return (a + 3 * b * s ** 2 + 5 * c * s ** 4).abs().max().item()


def near(got, x64, alpha, res, dtype, steps, coefficients=QUINTIC, full=True):
    """Each step holds some six matrices to 2^-22 of their size, and its sums to 2^-21: an error of
    2^-19 of |X|, which is at most (short side)^(1/2) x 1.3 and grows in the steps after by up to the
    iteration's slope each.  At the first step |X| is 1.  So in the root of the sum of squares:
    2^-19 x sum over steps of slope^(steps - i) x min(slope^i, 1.3 sqrt(m)), a bound that random
    errors stay well below; on top, the result's own rounding."""
    m, slope = min(x64.shape[1:]), most_slope(coefficients)
    size = 2.0 ** -19 * sum(slope ** (steps - i) * min(slope ** i, 1.3 * math.sqrt(m)) for i in range(steps + 1))
    want = alpha * x64 + (0 if res is None else res)
    off = (got.double() - want).square().sum((1, 2)).sqrt()
    assert (off <= abs(alpha) * size + HALF_STEP[dtype] * want.square().sum((1, 2)).sqrt() + 1e-12).all(), (off, size)
    # And, well inside that bound, the accuracy of fp32, measured against the norm of X, where the
    # update has many directions.  (Not where it has one: X is held to 2^-23 of its norm, 1, and that
    # grows by up to 3.4445^5 = 485 in the directions that the update does not have, to 5.8e-5 of a
    # result whose norm is 0.7: 8e-5, which the bound above allows for and 2e-5 would not.)
    if full and dtype == "f32" and res is None and steps <= 5:
        assert (off <= 2e-5 * want.square().sum((1, 2)).sqrt() + 1e-12).all(), off


SIZES = [(1, 1, 1), (1, 1, 300), (1, 300, 1), (1, 10, 256), (3, 16, 70), (2, 64, 64), (1, 65, 130), (2, 128, 128), (1, 129, 257),
         (1, 300, 200), (3, 256, 1000), (1, 1000, 256), (2, 513, 520), (5, 33, 4099), (1, 4099, 31), (1, 1024, 1024),
         (40, 16, 512), (40, 512, 16), (1, 600, 2100), (70, 100, 120), (9, 300, 700), (2, 8, 20000), (200, 30, 1100), (500, 700, 7), (80, 60, 2100), (3, 2060, 30), (1, 32, 7000), (1, 31, 9000)]


@pytest.mark.parametrize("count,rows,cols", SIZES)
@pytest.mark.parametrize("din,dout", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_sizes(work, count, rows, cols, din, dout):
    u = make(count, rows, cols, din, 1)
    out = torch.full((count, rows, cols), 7.0, device="cuda", dtype=T[dout])
    fa.fa_orthogonalise(work, count, rows, cols, u, out, din, dout)
    fa.fa_work_sync(work)
    near(out, iterate(u, 5, QUINTIC, 1e-7), 1.0, None, dout, 5)


@pytest.mark.parametrize("count,rows,cols", [(1, 100, 10007), (1, 9000, 40), (1, 130, 900), (1, 300, 1500), (3, 65, 2600), (5, 3333, 70),
                                             (1, 512, 512), (1, 700, 4100), (40, 64, 4096), (12, 130, 260)])
@pytest.mark.parametrize("din,dout", [("f32", "f32"), ("bf16", "bf16")])
def test_few_tiles(work, count, rows, cols, din, dout):
    """Products of few tiles, whose sums are shared out; momentum and weight beside them; the same bits twice."""
    u, mom = make(count, rows, cols, din, 31), make(count, rows, cols, "f32", 32)
    weight = (torch.randn((count, rows, cols), device="cuda") * 0.02).to(T[dout])
    outs = [torch.full((count, rows, cols), 7.0, device="cuda", dtype=T[dout]) for _ in range(2)]
    for out in outs:
        fa.fa_orthogonalise(work, count, rows, cols, u, out, din, dout, momentum=mom, mu=0.5, residual=weight, alpha=-0.1)
    fa.fa_work_sync(work)
    near(outs[0], iterate(0.5 * mom.double() + u.double(), 5, QUINTIC, 1e-7), -0.1, weight.double(), dout, 5)
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("rows,cols", [(96, 96), (96, 200), (200, 40)])
@pytest.mark.parametrize("steps", [0, 1, 2, 3, 4, 6, 7])
def test_steps(work, rows, cols, steps):
    u = make(2, rows, cols, "f32", 2)
    out = torch.empty_like(u)
    fa.fa_orthogonalise(work, 2, rows, cols, u, out, "f32", "f32", steps=steps, alpha=0.5)
    near(out, iterate(u, steps, QUINTIC, 1e-7), 0.5, None, "f32", steps)


@pytest.mark.parametrize("coefficients", [(1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (2.0, -1.5, 0.5), (1.0, 0.0, 0.0)])
def test_other_polynomials(work, coefficients):
    u = make(1, 150, 260, "f32", 3)
    out = torch.empty_like(u)
    fa.fa_orthogonalise(work, 1, 150, 260, u, out, "f32", "f32", steps=5, coefficients=coefficients)
    near(out, iterate(u, 5, coefficients, 1e-7), 1.0, None, "f32", 5, coefficients)


@pytest.mark.parametrize("rows,cols,dtype", [(40, 72, "f32"), (260, 140, "bf16"), (300, 300, "f32")])
@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_momentum_and_weight(work, rows, cols, dtype, nesterov, inplace):
    n, mu, lr, decay = 3, 0.9, 0.02, 0.99
    u = make(n, rows, cols, dtype, 4)
    mom = make(n, rows, cols, "f32", 5) * 3
    weight = (torch.randn((n, rows, cols), device="cuda") * 0.02).to(T[dtype])
    g = mu * mom.double() + u.double()
    x64 = iterate(u.double() + mu * g if nesterov else g, 5, QUINTIC, 1e-7)
    w64 = decay * weight.double()
    mom_out, out = (mom, weight) if inplace else (torch.empty_like(mom), torch.empty_like(weight))
    size = 2.0 ** -23 * (mu * mom.double().abs() + u.double().abs())
    fa.fa_orthogonalise(work, n, rows, cols, u, out, dtype, dtype, momentum=mom, momentum_out=mom_out, mu=mu, nesterov=nesterov,
                        residual=weight, alpha=-lr, beta=decay)
    assert ((mom_out.double() - g).abs() <= size).all()
    near(out, x64, -lr, w64, dtype, 5)


def test_a_first_round_starts_the_momentum(work):
    u = make(2, 30, 50, "bf16", 6)
    mom, out = torch.empty((2, 30, 50), device="cuda"), torch.empty((2, 30, 50), device="cuda")
    fa.fa_orthogonalise(work, 2, 30, 50, u, out, "bf16", "f32", momentum_out=mom, mu=0.9, nesterov=True)
    assert torch.equal(mom, u.float())
    near(out, iterate(1.9 * u.double(), 5, QUINTIC, 1e-7), 1.0, None, "f32", 5)


@pytest.mark.parametrize("rows,cols", [(24, 40), (200, 130)])
def test_strides(work, rows, cols):
    """Matrices in a wider buffer, other layers' keys between them; what is beside them stays."""
    n, wide, gap = 3, cols + 13, 5
    buf = torch.randn((n, rows + gap, wide), device="cuda")
    u = buf[:, :rows, 3:3 + cols]
    to = torch.full((n, rows + gap, wide), 4.0, device="cuda")
    out = to[:, :rows, 1:1 + cols]
    fa.fa_orthogonalise(work, n, rows, cols, u, out, "f32", "f32", ldu=wide, step_u=(rows + gap) * wide, ldo=wide,
                        step_o=(rows + gap) * wide)
    near(out, iterate(u, 5, QUINTIC, 1e-7), 1.0, None, "f32", 5)
    out[:] = 4.0
    assert (to == 4).all()


@pytest.mark.parametrize("rows,cols", [(20, 90), (150, 90)])
def test_over_the_update_itself(work, rows, cols):
    u = make(2, rows, cols, "f32", 8)
    x64 = iterate(u, 5, QUINTIC, 1e-7)
    fa.fa_orthogonalise(work, 2, rows, cols, u, u, "f32", "f32")
    near(u, x64, 1.0, None, "f32", 5)


@pytest.mark.parametrize("rows,cols", [(12, 40), (140, 260), (300, 100)])
def test_low_rank_zero_and_extreme_updates(work, rows, cols):
    u = torch.cat((make(1, rows, cols, "f32", 9, rank=1), torch.zeros((1, rows, cols), device="cuda"),
                   make(1, rows, cols, "f32", 10) * 1e22, make(1, rows, cols, "f32", 11) * 1e-22))
    u[3, 0, 0] = 1e-12
    out = torch.empty_like(u)
    fa.fa_orthogonalise(work, 4, rows, cols, u, out, "f32", "f32", eps=1e-30)
    assert (out[1] == 0).all()
    near(out, iterate(u, 5, QUINTIC, 1e-30), 1.0, None, "f32", 5, full=False)


@pytest.mark.parametrize("rows,cols", [(12, 40), (140, 260)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_what_is_not_finite_spoils_its_matrix_alone(work, rows, cols, bad):
    u = make(3, rows, cols, "f32", 12)
    x64 = iterate(u, 5, QUINTIC, 1e-7)
    u[1, 3, 5] = bad
    out = torch.empty_like(u)
    fa.fa_orthogonalise(work, 3, rows, cols, u, out, "f32", "f32")
    assert not torch.isfinite(out[1]).any()
    near(out[[0, 2]], x64[[0, 2]], 1.0, None, "f32", 5)


@pytest.mark.parametrize("rows,cols", [(16, 300), (64, 64), (200, 200), (180, 600)])
def test_singular_values_end_near_one(work, rows, cols):
    u = make(1, rows, cols, "f32", 13)
    out = torch.empty_like(u)
    fa.fa_orthogonalise(work, 1, rows, cols, u, out, "f32", "f32")
    s = torch.linalg.svdvals(out[0].double())
    start = torch.linalg.svdvals(u[0].double())
    assert (s[start / start.norm() > 5e-3] > 0.6).all() and s.max() < 1.25


def test_the_same_bits_each_time_captured_or_not(work):
    t = [make(2, 200, 328, "bf16", 14), make(6, 16, 256, "bf16", 15)]
    one = [torch.empty_like(u) for u in t]
    two = [torch.empty_like(u) for u in t]

    def call(outs, stream=None):
        for u, o in zip(t, outs):
            fa.fa_orthogonalise(work, *u.shape, u, o, "bf16", "bf16", stream=stream)

    call(one, torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(two, torch.cuda.current_stream())
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one, two))


@pytest.mark.parametrize("rows,cols", [(130, 200), (520, 2000)])
def test_an_expired_wait_is_reported_and_ends(rows, cols):
    u = make(1, rows, cols, "f32", 16)
    out = torch.empty_like(u)
    bad, good = fa.fa_work_open(flags=fa.FA_TEST_WAIT_EXPIRES), fa.fa_work_open()
    try:
        fa.fa_orthogonalise(bad, 1, rows, cols, u, out, "f32", "f32")
        with pytest.raises(fa.FedAvgError) as e:
            fa.fa_work_sync(bad)
        assert e.value.status == fa.FA_ERR_INTERNAL and "device-side wait" in e.value.detail
        fa.fa_orthogonalise(good, 1, rows, cols, u, out, "f32", "f32")
        fa.fa_work_sync(good)
        near(out, iterate(u, 5, QUINTIC, 1e-7), 1.0, None, "f32", 5)
    finally:
        fa.fa_work_close(bad)
        fa.fa_work_close(good)
