"""fa_product and fa_product_backward against fp64: types, storage orders, strides, odd and
empty sizes, every part of the epilogue, gradients by formula and by differences, refusals.

Tolerances, from the arithmetic.  S2 is the root of the sum of the squared terms of one
output, the size its partial sums have.  fp32 results: about K roundings of partial sums of
up to 4 S2, random: 16 sqrt(K + 16) 2^-24 S2 at four sigma, and the result's own rounding.
bf16 results: sums may be truncated once per 16 terms, K / 16 steps of up to 2^-23 of 4 S2
each, and half a bf16 ulp (up to 2^-8) of the result.  Activations have slopes up to 1.13 and are
evaluated to 2^-20."""
import math

import pytest
import torch

import server_side_fedavg_gb300 as fa

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
FN = {"none": lambda z: z, "relu": torch.nn.functional.relu, "gelu": torch.nn.functional.gelu,
      "silu": torch.nn.functional.silu}


@pytest.fixture(scope="module")
def work():
    w = fa.fa_work_open()
    yield w
    fa.fa_work_sync(w)
    fa.fa_work_close(w)


def _mat(g, rows, cols, dtype, scale=1.0, pad=0, offset=0):
    """A [rows, cols] matrix with `pad` spare elements a row, starting `offset` elements into
    its buffer; the spare places hold NaN, so that reading one shows."""
    ld = cols + pad
    buf = torch.full((rows * ld + offset,), float("nan"), device="cuda", dtype=TORCH[dtype])
    v = buf[offset:].view(rows, ld)[:, :cols]
    v.copy_(torch.randn((rows, cols), generator=g, device="cuda") * scale)
    return v, ld, buf


def _tol(exact, s2, k, out, act):
    t = 16 * math.sqrt(k + 16) * 2 ** -24 * s2
    if out == "bf16":
        t = t + (k / 16 + 1) * 2 ** -21 * s2 + exact.abs() * 2 ** -7.99
    if act != "none":
        t = 1.13 * t + 2 ** -20 * (exact.abs() + s2)
    return t + exact.abs() * 2 ** -22 + 1e-30


def _check(got, exact, tol, what):
    bad = ~((got.double() - exact).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{((got.double() - exact).abs() / tol).nan_to_num(9e9).max().item():.3g} x tolerance")


def _forward(work, m, n, k, din, dout, ta=False, tb=True, bias=False, act="none", res=None, pre=False,
             alpha=1.0, beta=1.0, pad=(0, 0, 0, 0), offset=(0, 0, 0), seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, lda, _ = _mat(g, *((k, m) if ta else (m, k)), din, scale, pad[0], offset[0])
    b, ldb, _ = _mat(g, *((n, k) if tb else (k, n)), din, scale, pad[1], offset[1])
    out, ldo, buf = _mat(g, m, n, dout, 1.0, pad[2], offset[2])
    bi = torch.randn((n,), generator=g, device="cuda").to(TORCH[din]) if bias else None
    r, ldr = None, 0
    if res == "other":
        r, ldr, _ = _mat(g, m, n, dout, 1.0, pad[3])
    elif res == "out":
        r, ldr = out, ldo
    p = torch.full((m * ldo + 1,), float("nan"), device="cuda", dtype=TORCH[dout]) if pre else None
    A = (a.t() if ta else a).double()
    B = (b.t() if tb else b).double()
    z = alpha * (A @ B)
    s2 = abs(alpha) * ((A * A) @ (B * B)).sqrt()
    if bias:
        z = z + bi.double()
    y = FN[act](z)
    if r is not None:
        y = y + beta * r.double()
    spare = buf.clone()
    fa.fa_product(work, m, n, k, a, lda, b, ldb, out, ldo, din, dout, ta, tb, alpha, bi, act, r, ldr, beta, p)
    torch.cuda.synchronize()
    what = f"{m}x{n}x{k} {din}->{dout} ta={ta} tb={tb} {act}"
    mag = s2 + (bi.double().abs() if bias else 0) + (abs(beta) * r.double().abs() if res == "other" else 0)
    _check(out, y, _tol(y, mag, k, dout, act), what)
    if pre:
        _check(p[:m * ldo].view(m, ldo)[:, :n], z, _tol(z, mag, k, dout, "none"), what + " pre")
        assert torch.isnan(p[:m * ldo].view(m, ldo)[:, n:]).all() and torch.isnan(p[m * ldo:]).all()
    if pad[2]:
        full, was = buf[offset[2]:].view(m, ldo), spare[offset[2]:].view(m, ldo)
        assert torch.isnan(full[:, n:]).all() and torch.isnan(was[:, n:]).all(), "written past a row's end"
    if dout == "f32" and m * n >= 64:
        rel = ((out.double() - y).norm() / y.norm()).item()
        assert rel <= 1.5e-6, f"{what}: relative error {rel:.3g}"
    return out


SIZES = [(1, 1, 1), (1, 10, 256), (1, 4096, 4096), (4, 1000, 777), (7, 129, 65), (8, 256, 64), (16, 16, 16),
         (33, 72, 1000), (64, 640, 512), (65, 1, 130), (127, 255, 63), (128, 128, 128), (129, 257, 191),
         (200, 1000, 8), (256, 256, 2048), (300, 520, 1032), (515, 2056, 264), (1030, 776, 520)]


@pytest.mark.parametrize("din,dout", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_sizes(work, m, n, k, din, dout):
    _forward(work, m, n, k, din, dout, bias=True, act="gelu", res="other", seed=m + n + k)
    _forward(work, m, n, k, din, dout, tb=False, seed=m + n + k + 1)


@pytest.mark.parametrize("ta", [False, True])
@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("din", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(3, 40, 24), (24, 200, 136), (136, 264, 328), (257, 131, 99), (640, 384, 512)])
def test_product_storage_orders(work, m, n, k, din, ta, tb):
    _forward(work, m, n, k, din, din, ta, tb, bias=True, act="silu", res="out", pre=True, alpha=0.5, beta=-0.75)


@pytest.mark.parametrize("pad,offset", [((3, 5, 7, 1), (0, 0, 0)), ((8, 16, 8, 24), (8, 8, 8)),
                                        ((0, 0, 0, 0), (1, 3, 5)), ((1, 0, 0, 0), (0, 1, 0))])
@pytest.mark.parametrize("din", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(2, 264, 320), (40, 264, 320), (264, 136, 160), (300, 300, 300)])
def test_product_strides_and_alignment(work, m, n, k, din, pad, offset):
    _forward(work, m, n, k, din, din, bias=True, act="relu", res="other", pre=True, pad=pad, offset=offset)
    _forward(work, m, n, k, din, din, True, False, pad=pad, offset=offset)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("res", [None, "other", "out"])
@pytest.mark.parametrize("m", [5, 200])
def test_product_epilogue(work, m, act, bias, res):
    for din, dout in (("bf16", "bf16"), ("f32", "f32")):
        _forward(work, m, 328, 264, din, dout, bias=bias, act=act, res=res, pre=bias, alpha=1.5, beta=0.5)


@pytest.mark.parametrize("k", [4096, 11008])
def test_product_long_sums(work, k):
    for m in (1, 48, 260):
        _forward(work, m, 384, k, "bf16", "bf16", scale=0.3)
        _forward(work, m, 384, k, "bf16", "f32", scale=0.3)
        _forward(work, m, 384, k, "f32", "f32", scale=0.3)


def test_product_rank_of_an_adapter(work):
    for r in (1, 4, 8, 16, 64):
        _forward(work, 1000, 520, r, "bf16", "bf16", False, False, res="out", alpha=2.0)


def test_product_empty(work):
    out = torch.full((4, 8), 3.0, device="cuda")
    bias = torch.arange(8, device="cuda", dtype=torch.float32) - 3
    for m, n in ((0, 8), (4, 0)):
        fa.fa_product(work, m, n, 5, None, 5, None, 5, None, 8, "f32", "f32")
    fa.fa_product(work, 4, 8, 0, None, 1, None, 8, out, 8, "f32", "f32", bias=bias, act="relu", residual=out, ldr=8,
                  beta=2.0)
    torch.cuda.synchronize()
    assert torch.equal(out, torch.relu(bias).expand(4, 8) + 6.0)


def test_product_beta_zero_does_not_read_the_residual(work):
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = (torch.randn((64, 64), generator=g, device="cuda") for _ in range(2))
    r = torch.full((64, 64), float("nan"), device="cuda")
    out = torch.empty((64, 64), device="cuda")
    fa.fa_product(work, 64, 64, 64, a, 64, b, 64, out, 64, "f32", "f32", residual=r, ldr=64, beta=0.0)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("m", [2, 150])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_product_nonfinite_stays_in_its_row(work, m, dtype):
    """A NaN or infinity in one row of a, or past the summed range of a padded row, shows in
    that row alone."""
    g = torch.Generator(device="cuda").manual_seed(2)
    n, k = 136, 72
    a, lda, _ = _mat(g, m, k, dtype, 1.0, 8)
    b, ldb, _ = _mat(g, n, k, dtype, 1.0, 8)
    a[1, 3] = float("nan")
    out = torch.empty((m, n), device="cuda", dtype=TORCH[dtype])
    fa.fa_product(work, m, n, k, a, lda, b, ldb, out, n, dtype, dtype, False, True)
    torch.cuda.synchronize()
    assert torch.isnan(out[1]).all() and torch.isfinite(out[0]).all() and torch.isfinite(out[2:]).all()
    a[1, 3] = float("inf")
    fa.fa_product(work, m, n, k, a, lda, b, ldb, out, n, dtype, dtype, False, True)
    torch.cuda.synchronize()
    assert (~torch.isfinite(out[1])).all() and torch.isfinite(out[0]).all() and torch.isfinite(out[2:]).all()


def test_product_fp32_range(work):
    """fp32 operands near the ends of their range: no overflow in the operands' split."""
    for scale in (3.0e38, 1e-30):
        a = torch.full((130, 64), 0.0, device="cuda")
        a[:, 5] = scale
        b = torch.zeros((136, 64), device="cuda")
        b[:, 5] = 1.0
        out = torch.empty((130, 136), device="cuda")
        fa.fa_product(work, 130, 136, 64, a, 64, b, 64, out, 136, "f32", "f32", False, True)
        torch.cuda.synchronize()
        want = torch.tensor(scale, dtype=torch.float32).item()
        assert ((out.double() - want).abs() <= 2 ** -22 * want).all()


def test_product_same_bits_every_time(work):
    g = torch.Generator(device="cuda").manual_seed(3)
    for m, n, k, dt in ((1, 4096, 4096, "bf16"), (16, 1024, 4096, "bf16"), (300, 512, 4096, "f32"), (8, 64, 8192, "f32")):
        a, b = (torch.randn(s, generator=g, device="cuda").to(TORCH[dt]) for s in ((m, k), (n, k)))
        outs = []
        for _ in range(3):
            out = torch.empty((m, n), device="cuda", dtype=TORCH[dt])
            fa.fa_product(work, m, n, k, a, k, b, k, out, n, dt, dt, False, True)
            outs.append(out)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_product_streams_share_the_workspace_in_order(work):
    """Calls of one handle on alternating streams: each waits for the one before (they share
    the workspace); the caller orders its own tensors."""
    g = torch.Generator(device="cuda").manual_seed(4)
    m, n, k = 300, 260, 516
    s = [torch.cuda.Stream() for _ in range(2)]
    ops = []
    for i in range(6):
        a = torch.randn((m, k), generator=g, device="cuda")
        b = torch.randn((n, k), generator=g, device="cuda")
        ops.append((a, b, torch.empty((m, n), device="cuda")))
    torch.cuda.synchronize()
    for i, (a, b, out) in enumerate(ops):
        fa.fa_product(work, m, n, k, a, k, b, k, out, n, "f32", "f32", False, True, stream=s[i % 2])
    fa.fa_work_sync(work)
    for a, b, out in ops:
        y = a.double() @ b.double().t()
        assert ((out.double() - y).norm() / y.norm()).item() < 1.5e-6


def _backward(work, m, n, k, din, ddout, dgrad, ta=False, tb=True, act="gelu", bias=True, want=(True, True),
              pad=0, alpha=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, lda, _ = _mat(g, *((k, m) if ta else (m, k)), din, 1.0, pad)
    b, ldb, _ = _mat(g, *((n, k) if tb else (k, n)), din, 1.0, pad)
    dout, ldd, _ = _mat(g, m, n, ddout, 1.0, pad)
    pre, ldp, _ = _mat(g, m, n, ddout, 1.0, pad)
    if act == "none":
        pre, ldp = None, 0
    da, ldda, dabuf = _mat(g, *a.shape, dgrad, 1.0, pad)
    db, lddb, dbbuf = _mat(g, *b.shape, dgrad, 1.0, pad)
    dbias = torch.empty((n,), device="cuda", dtype=TORCH[dgrad]) if bias else None
    fa.fa_product_backward(work, m, n, k, a, lda, b, ldb, dout, ldd, da if want[0] else None, ldda,
                           db if want[1] else None, lddb, din, ddout, dgrad, ta, tb, alpha, act, pre, ldp, dbias)
    torch.cuda.synchronize()
    dz = dout.double()
    if act != "none":
        z = pre.double().requires_grad_()
        (dz,) = torch.autograd.grad(FN[act](z), z, dz)
    A, B = (a.t() if ta else a).double(), (b.t() if tb else b).double()
    what = f"{m}x{n}x{k} {din},{ddout}->{dgrad} ta={ta} tb={tb} {act}"

    # act' is a sum of terms of up to 1 (gelu's crosses zero near -0.75): dZ is off by 2^-22 of
    # dout, whatever is left of it
    off = dout.double() * (2.0 ** -22 if act != "none" else 0.0)

    def held(x, y, summed, store_t, got, name, ox=None, oy=None):
        y64, s2 = alpha * (x @ y), abs(alpha) * ((x * x) @ (y * y)).sqrt()
        # a dZ held in bf16 adds a random 2^-8 of each term: six sigma of 2^-8 / sqrt(3) of S2
        tol = _tol(y64, s2, summed, dgrad, "none") + (2 ** -6.2 * s2 if dgrad == "bf16" else 2 ** -20 * s2)
        ox, oy = (x if ox is None else ox), (y if oy is None else oy)
        tol = tol + 4 * abs(alpha) * ((ox * ox) @ (oy * oy)).sqrt()
        _check(got.t() if store_t else got, y64, tol, f"{what} {name}")
        # ... which over a whole gradient is 2^-8 / sqrt(3) of its norm, as its own rounding
        rel = ((got.double() - (y64.t() if store_t else y64)).norm() / y64.norm().clamp(min=1e-30)).item()
        assert rel <= (3.2e-3 if dgrad == "bf16" else 1.5e-6) or y64.numel() < 64, f"{what} {name}: rel {rel:.3g}"

    if want[0]:
        held(dz, B.t(), n, ta, da, "d_a", ox=off)
        assert not pad or torch.isnan(dabuf.view(a.shape[0], ldda)[:, a.shape[1]:]).all()
    if want[1]:
        held(A.t(), dz, m, tb, db, "d_b", oy=off)
        assert not pad or torch.isnan(dbbuf.view(b.shape[0], lddb)[:, b.shape[1]:]).all()
    if bias:
        y64, s2 = dz.sum(0), dz.square().sum(0).sqrt()
        _check(dbias, y64, _tol(y64, s2, m, "f32", act) + 4 * off.square().sum(0).sqrt() + (y64.abs() * 2 ** -7.99 if dgrad == "bf16" else 0), what + " d_bias")


@pytest.mark.parametrize("din,ddout,dgrad", [("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"), ("f32", "f32", "f32"),
                                             ("bf16", "f32", "f32"), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 264, 72), (5, 10, 256), (17, 129, 63), (64, 72, 136), (200, 136, 264),
                                   (257, 515, 131), (1031, 264, 520)])
def test_backward_sizes(work, m, n, k, din, ddout, dgrad):
    _backward(work, m, n, k, din, ddout, dgrad, act="gelu", seed=m + n + k)
    _backward(work, m, n, k, din, ddout, dgrad, act="none", seed=m + n + k + 1)


@pytest.mark.parametrize("ta", [False, True])
@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("din", ["bf16", "f32"])
def test_backward_storage_orders_and_strides(work, din, ta, tb):
    for pad in (0, 3, 8):
        _backward(work, 136, 264, 72, din, din, din, ta, tb, "silu", pad=pad, alpha=0.5)
        _backward(work, 131, 75, 203, din, din, din, ta, tb, "relu", pad=pad)


def test_backward_parts(work):
    for want in ((True, False), (False, True), (False, False)):
        for act in ("none", "gelu"):
            _backward(work, 150, 136, 72, "bf16", "bf16", "bf16", act=act, want=want)
    _backward(work, 150, 136, 72, "bf16", "bf16", "f32", bias=False)


def test_backward_without_rows_is_zero(work):
    db = torch.full((8, 5), 7.0, device="cuda")
    dbias = torch.full((8,), 7.0, device="cuda")
    fa.fa_product_backward(work, 0, 8, 5, None, 5, None, 5, None, 8, None, 5, db, 5, "f32", "f32", "f32", False, True,
                           1.0, "none", None, 0, dbias)
    da = torch.full((6, 5), 7.0, device="cuda")
    fa.fa_product_backward(work, 6, 0, 5, None, 5, None, 5, None, 8, da, 5, None, 5, "f32", "f32", "f32", False, True)
    torch.cuda.synchronize()
    assert not db.any() and not dbias.any() and not da.any()


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_backward_against_differences(work, act):
    """Directional central differences of sum(out * v) in fp32: with steps of 2^-6 the
    third-order term is about 2^-12 of the derivative's scale and the forward's fp32
    rounding 2^-24 sqrt(m n) / 2^-6; 1 % of the scale covers both."""
    g = torch.Generator(device="cuda").manual_seed(11)
    m, n, k = 70, 40, 130
    r = lambda *s, c=1.0: torch.randn(s, generator=g, device="cuda") * c  # noqa: E731
    a, b, bias, v = r(m, k), r(n, k, c=k ** -0.5), r(n), r(m, n)
    out, pre = torch.empty((m, n), device="cuda"), torch.empty((m, n), device="cuda")

    def f(a, b, bias):
        fa.fa_product(work, m, n, k, a, k, b, k, out, n, "f32", "f32", False, True, 1.0, bias, act, None, 0, 1.0, pre)
        return (out.double() * v.double()).sum().item()

    f(a, b, bias)
    da, db, dbias = torch.empty_like(a), torch.empty_like(b), torch.empty_like(bias)
    fa.fa_product_backward(work, m, n, k, a, k, b, k, v, n, da, k, db, k, "f32", "f32", "f32", False, True, 1.0, act,
                           pre, n, dbias)
    torch.cuda.synchronize()
    h = 2.0 ** -6
    for i, (x, d) in enumerate(((a, da), (b, db), (bias, dbias))):
        u = r(*x.shape)
        u /= u.norm()
        args = [a, b, bias]
        hi, lo = list(args), list(args)
        hi[i], lo[i] = x + h * u, x - h * u
        slope = (f(*hi) - f(*lo)) / (2 * h)
        assert abs(slope - (d.double() * u.double()).sum().item()) <= 0.01 * d.double().norm().item()


def test_product_in_a_graph(work):
    g = torch.Generator(device="cuda").manual_seed(12)
    m, n, k = 200, 264, 136
    a, b = (torch.randn(s, generator=g, device="cuda") for s in ((m, k), (n, k)))
    out = torch.empty((m, n), device="cuda")
    call = lambda s=None: fa.fa_product(work, m, n, k, a, k, b, k, out, n, "f32", "f32", False, True, stream=s)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(torch.cuda.current_stream())
    for _ in range(2):
        a.copy_(torch.randn((m, k), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        y = a.double() @ b.double().t()
        assert ((out.double() - y).norm() / y.norm()).item() < 1.5e-6


def test_growth_is_refused_while_capturing():
    w = fa.fa_work_open()
    m, n, k = 200, 264, 136
    a, b, d, pre = (torch.zeros(s, device="cuda") for s in ((m, k), (n, k), (m, n), (m, n)))
    da = torch.empty_like(a)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    try:
        with torch.cuda.graph(graph):
            with pytest.raises(fa.FedAvgError) as e:
                fa.fa_product_backward(w, m, n, k, a, k, b, k, d, n, da, k, None, k, "f32", "f32", "f32", False, True,
                                       1.0, "gelu", pre, n, None, torch.cuda.current_stream())
            assert e.value.status == fa.FA_ERR_STATE
            d.add_(1.0)      # the capture itself goes on
    finally:
        fa.fa_work_close(w)


def test_product_refusals(work):
    a, b, out = (torch.zeros((64, 64), device="cuda") for _ in range(3))
    host = torch.zeros((64, 64))
    ok = dict(m=64, n=64, k=64, a=a, lda=64, b=b, ldb=64, out=out, ldo=64, dtype_in="f32", dtype_out="f32")

    def refused(status, **kw):
        with pytest.raises(fa.FedAvgError) as e:
            fa.fa_product(work, **{**ok, **kw})
        assert e.value.status == status and e.value.detail

    refused(fa.FA_ERR_ARG, a=None)
    refused(fa.FA_ERR_ARG, b=None)
    refused(fa.FA_ERR_ARG, out=None)
    refused(fa.FA_ERR_ARG, a=host)
    refused(fa.FA_ERR_ARG, out=host)
    refused(fa.FA_ERR_ARG, out=a)
    refused(fa.FA_ERR_ARG, out=b)
    refused(fa.FA_ERR_ARG, pre=out)
    refused(fa.FA_ERR_ARG, bias=host)
    refused(fa.FA_ERR_ARG, a=a.data_ptr() + 2)
    refused(fa.FA_ERR_ARG, alpha=float("nan"))
    refused(fa.FA_ERR_ARG, beta=float("inf"), residual=out, ldr=64)
    refused(fa.FA_ERR_ARG, residual=out.data_ptr() + 256, ldr=64)
    refused(fa.FA_ERR_RANGE, lda=63)
    refused(fa.FA_ERR_RANGE, ldb=63)
    refused(fa.FA_ERR_RANGE, ldo=63)
    refused(fa.FA_ERR_RANGE, residual=b, ldr=63)
    refused(fa.FA_ERR_RANGE, m=1 << 31)
    for kw in ({"dtype_in": "f64"}, {"act": "tanh"}):
        with pytest.raises(KeyError):
            fa.fa_product(work, **{**ok, **kw})
    fa.fa_product(work, **ok)
    fa.fa_work_sync(work)


def test_backward_refusals(work):
    t = [torch.zeros((64, 64), device="cuda") for _ in range(6)]
    a, b, d, pre, da, db = t

    def refused(status, **kw):
        args = dict(m=64, n=64, k=64, a=a, lda=64, b=b, ldb=64, dout=d, ldd=64, d_a=da, ldda=64, d_b=db, lddb=64,
                    dtype_in="f32", dtype_dout="f32", dtype_grad="f32", act="gelu", pre=pre, ldp=64)
        with pytest.raises(fa.FedAvgError) as e:
            fa.fa_product_backward(work, **{**args, **kw})
        assert e.value.status == status and e.value.detail

    refused(fa.FA_ERR_ARG, dout=None)
    refused(fa.FA_ERR_ARG, pre=None)
    refused(fa.FA_ERR_ARG, a=None)
    refused(fa.FA_ERR_ARG, b=None)
    refused(fa.FA_ERR_ARG, d_a=d)
    refused(fa.FA_ERR_ARG, d_b=a)
    refused(fa.FA_ERR_ARG, d_b=da)
    refused(fa.FA_ERR_ARG, d_bias=pre)
    refused(fa.FA_ERR_RANGE, ldd=63)
    refused(fa.FA_ERR_RANGE, lddb=3)
    refused(fa.FA_ERR_ARG, alpha=float("inf"))
