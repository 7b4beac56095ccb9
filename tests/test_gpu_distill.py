"""fa_distill_loss and fa_distill_grad against fp64: types, vocabularies from one entry to
more than any SM's shared memory holds, lists with unused places, shared and repeated
entries, absent clients, masked rows, closed vocabulary entries, refusals.

Tolerances, from the arithmetic.  A probability comes from an exponential evaluated to
2^-22 at an argument of up to A = max |z - top| / T whose rounding is A 2^-23, divided by a
sum of like errors: relative 2^-20 (1 + A / 4).  A gradient is w T times the difference of
two such numbers.  A loss sums p (log p - log q), whose terms' logarithms are off by 2^-22 of
their size.  Results in bf16 add half an ulp, up to 2^-8."""
import pytest
import torch

import server_side_fedavg_gb300 as fa

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
INF = float("inf")


@pytest.fixture(scope="module")
def work():
    w = fa.fa_work_open()
    yield w
    fa.fa_work_close(w)


def oracle(z, index, value, weight, T, row_weight, lse=None):
    """The definition in fp64, dense targets.  Returns loss, lse, grad, the size of the
    loss's terms and the dense target."""
    rows, vocab = z.shape
    z = z.double() / T
    own = torch.logsumexp(z, 1)
    use = own if lse is None else lse.double()
    logq = z - use[:, None]
    target = torch.zeros_like(z)
    entropy, size, total = (torch.zeros(rows, dtype=torch.float64, device=z.device) for _ in range(3))
    for idx, val, n in zip(index, value, weight):
        ok = (idx >= 0) & (idx < vocab)
        u = torch.where(ok, val.double() / T, -INF)
        on = u.amax(1) > -INF
        u = torch.where(on[:, None], u, 0.0)
        lp = u - torch.logsumexp(u, 1)[:, None]
        p = torch.where(on[:, None] & ok, torch.exp(lp), 0.0)
        target.scatter_add_(1, idx.clamp(0, vocab - 1).long(), n * p)
        entropy += n * torch.where(p > 0, p * lp, 0.0).sum(1)
        size += n * torch.where(p > 0, p * lp.abs(), 0.0).sum(1)
        total += n * on
    some = torch.where(total > 0, total, 1.0)
    w = torch.where((total > 0) & (row_weight > 0), row_weight.double(), 0.0)
    target /= some[:, None]
    cross = torch.where(target > 0, target * logq, 0.0)
    loss = w * T * T * (entropy / some - cross.sum(1))
    loss = torch.where(w > 0, loss, 0.0)
    size = w * T * T * (size / some + cross.abs().sum(1) + use.abs())
    grad = torch.where((w > 0)[:, None], (w * T)[:, None] * (torch.exp(logq) - target), 0.0)
    return loss, torch.where(row_weight > 0, own, 0.0), grad, size, (w * T)[:, None] * (torch.exp(logq) + target)


def make(rows, vocab, J, topk, dtype, vdtype="f32", seed=0, spread=2.5, distinct=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = (torch.randn((rows, vocab), generator=g, device="cuda") * spread).to(TORCH[dtype])
    index, value = [], []
    for j in range(J):
        k = topk if isinstance(topk, int) else topk[j]
        if distinct and rows * vocab <= 1 << 24:
            idx = torch.rand((rows, vocab), generator=g, device="cuda").argsort(1)[:, :k]
        else:
            idx = torch.randint(0, vocab, (rows, k), generator=g, device="cuda")
        index.append(idx.to(torch.int32).contiguous())
        value.append((torch.randn((rows, k), generator=g, device="cuda") * 2).to(TORCH[vdtype]))
    weight = [float(100 + 37 * j) for j in range(J)]
    row_weight = torch.rand((rows,), generator=g, device="cuda") + 0.25
    return z, index, value, weight, row_weight


def check(work, z, index, value, weight, row_weight, T, dtype, vdtype="f32", saved=False, inplace=False, ld=None,
          fused_loss=True):
    rows, vocab = z.shape
    lists = fa.distill_lists(index, value, [i.shape[1] for i in index], weight, vdtype)
    rw = torch.ones(rows, device="cuda") if row_weight is None else row_weight
    ld = ld or vocab
    buf = torch.full((rows, ld), 77.0, device="cuda", dtype=TORCH[dtype])
    buf[:, :vocab] = z
    loss, lse = (torch.full((rows,), -7.0, device="cuda") for _ in range(2))
    fa.fa_distill_loss(work, rows, vocab, buf, ld, dtype, lists, T, row_weight, loss, lse)
    torch.cuda.synchronize()
    e_loss, e_lse, e_grad, size, both = oracle(z, index, value, weight, T, rw)
    live = rw > 0
    spread = torch.where(torch.isfinite(z), z.float(), 0.0).abs().amax(1).double() * 2 / T
    rel = 2.0 ** -20 * (1 + spread / 4)

    def same(got, want, tol, what):
        d = (got.double() - want).abs()
        ok = (d <= tol) | (got.double() == want) | (torch.isnan(got) & torch.isnan(want))
        assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.numel()} off, worst {d[~ok].max().item():.3g}"

    same(lse, e_lse, torch.where(live, rel + 2.0 ** -22 * e_lse.abs(), 0.0), "lse")
    same(loss, e_loss, rel * torch.where(size == size, size, 0.0) + 1e-30, "loss")
    out = buf if inplace else torch.full((rows, ld), 55.0, device="cuda", dtype=TORCH[dtype])
    loss2 = torch.full((rows,), -7.0, device="cuda") if fused_loss else None
    use = lse.clone() if saved else None
    fa.fa_distill_grad(work, rows, vocab, buf, ld, dtype, lists, T, row_weight, use, loss2, out, ld)
    torch.cuda.synchronize()
    if saved:
        e_loss, _, e_grad, size, both = oracle(z, index, value, weight, T, rw, torch.where(live, lse, 0.0))
        rel = rel + 2.0 ** -22 * e_lse.abs()      # the kept statistic's rounding is given; z / T - lse rounds again
    tol = (rel + 2.0 ** -19)[:, None] * both + 1e-30
    if dtype == "bf16":
        tol = tol + e_grad.abs() * 2.0 ** -7.99
    same(out[:, :vocab], e_grad, tol, "grad")
    if fused_loss:
        same(loss2, e_loss, rel * torch.where(size == size, size, 0.0) + 1e-30, "loss of the gradient call")
    if ld > vocab:
        assert (out[:, vocab:] == (77.0 if inplace else 55.0)).all(), "written past a row's end"
    return out[:, :vocab], loss


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,J,topk,T", [
    (1, 1, 1, 1, 1.0), (3, 2, 2, 2, 2.0), (5, 10, 3, 4, 1.0), (7, 33, 4, 16, 4.0), (1, 1000, 1, 64, 1.0),
    (64, 257, 8, 20, 2.0), (129, 4096, 2, 32, 1.0), (300, 1003, 16, 5, 3.0), (40, 32000, 8, 32, 2.0),
    (11, 32003, 5, 100, 1.0), (4, 50001, 2, 256, 0.5), (33, 8191, 1, 2048, 1.0)])
def test_sizes(work, rows, vocab, J, topk, T, dtype):
    z, index, value, weight, rw = make(rows, vocab, J, topk, dtype, seed=rows + vocab)
    check(work, z, index, value, weight, rw, T, dtype)
    check(work, z, index, value, weight, None, T, dtype, saved=True, fused_loss=False)
    check(work, z, index, value, weight, rw, T, dtype, inplace=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [65536, 100003, 131075, 200000, 262144, 500009, 1000000])
def test_large_vocabularies(work, vocab, dtype):
    z, index, value, weight, rw = make(5, vocab, 3, 50, dtype, seed=vocab)
    check(work, z, index, value, weight, rw, 1.0, dtype)
    check(work, z, index, value, weight, rw, 2.0, dtype, saved=True, inplace=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab,ld", [(1000, 1003), (1000, 1008), (999, 1001), (32000, 32008), (131072, 131073)])
def test_strides(work, vocab, ld, dtype):
    z, index, value, weight, rw = make(9, vocab, 3, 12, dtype)
    for inplace in (False, True):
        check(work, z, index, value, weight, rw, 1.0, dtype, ld=ld, inplace=inplace)


@pytest.mark.parametrize("vdtype", ["f32", "bf16"])
def test_lists_of_different_lengths_and_value_types(work, vdtype):
    z, index, value, weight, rw = make(20, 777, 4, [1, 7, 33, 200], "bf16", vdtype)
    check(work, z, index, value, weight, rw, 2.0, "bf16", vdtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [500, 70001])
def test_absent_clients_masked_rows_unused_places(work, vocab, dtype):
    rows = 24
    z, index, value, weight, rw = make(rows, vocab, 4, 16, dtype)
    index[0][:, 5:] = -1                     # a short list
    index[1][::2] = -1                       # absent from every other row
    value[2][3] = -INF                       # present in name only
    value[2][4, ::2] = -INF
    for i in index:
        i[7] = -1                            # a row that nobody sent
    rw[::5] = 0.0
    z[10] = float("nan")                     # a masked row may hold anything
    z[15] = INF
    rw[10] = rw[15] = 0.0
    weight[3] = 0.0                          # a client of no weight
    for j in (0, 1, 2):
        index[j][9] = -1                     # a row that only the client of no weight sent
    grad, loss = check(work, z, index, value, weight, rw, 2.0, dtype)
    for r in (0, 7, 9, 10, 15):
        assert loss[r] == 0 and not grad[r].any()
    check(work, z, index, value, weight, rw, 2.0, dtype, saved=True, inplace=True)
    check(work, z, index, value, [0.0] * 4, rw, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_closed_vocabulary_entries_and_extreme_values(work, dtype):
    vocab = 1200
    z, index, value, weight, rw = make(8, vocab, 2, 10, dtype)
    low = torch.finfo(TORCH[dtype]).min
    z[:, 1000:] = -INF
    for i in index:
        i %= 1000
    z[1, :1000] = low                        # uniform over the open entries
    z[2, :500] = low                         # masked by the type's lowest value
    z[3] = -INF                              # nothing open: NaN by the definition
    z[4, 3] = INF                            # NaN
    z[5, 7] = float("nan")
    index[0][6, 0] = 1100                    # mass on a closed entry: infinite loss, finite gradient
    high = 3.0e38 if dtype == "f32" else torch.finfo(torch.bfloat16).max
    z[7, 1] = high
    z[7, 2] = -high
    lists = fa.distill_lists(index, value, [10, 10], weight)
    loss = torch.empty(8, device="cuda")
    grad = torch.empty_like(z)
    fa.fa_distill_grad(work, 8, vocab, z, vocab, dtype, lists, 1.0, rw, None, loss, grad, vocab)
    torch.cuda.synchronize()
    assert torch.isnan(grad[3]).any() and torch.isnan(grad[4]).any() and torch.isnan(grad[5]).any()
    assert torch.isnan(loss[[3, 4, 5]]).all()
    assert loss[6] == INF and torch.isfinite(grad[6]).all()
    keep = torch.tensor([0, 1, 2], device="cuda")
    check(work, z[keep], [i[keep].contiguous() for i in index], [v[keep].contiguous() for v in value], weight,
          rw[keep].contiguous(), 1.0, dtype)
    assert torch.isfinite(grad[7]).all()


def test_nan_in_a_list_reaches_its_entries(work):
    z, index, value, weight, rw = make(2, 300, 2, 8, "f32")
    value[1][0, 3] = float("nan")
    lists = fa.distill_lists(index, value, [8, 8], weight)
    loss, grad = torch.empty(2, device="cuda"), torch.empty_like(z)
    fa.fa_distill_grad(work, 2, 300, z, 300, "f32", lists, 1.0, rw, None, loss, grad, 300)
    torch.cuda.synchronize()
    assert torch.isnan(loss[0]) and torch.isfinite(loss[1])
    hit = torch.zeros(300, dtype=torch.bool, device="cuda")
    hit[index[1][0].long()] = True
    assert torch.isnan(grad[0][hit]).all() and torch.isfinite(grad[0][~hit]).all() and torch.isfinite(grad[1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeated_entries_add(work, dtype):
    """Every client names the same few entries, some twice: the shares add, and the sum does
    not depend on the run."""
    z, index, value, weight, rw = make(6, 400, 8, 64, dtype)
    index = [(i % 40).contiguous() for i in index]
    g0, _ = check(work, z, index, value, weight, rw, 1.0, dtype)
    for _ in range(4):
        g1, _ = check(work, z, index, value, weight, rw, 1.0, dtype)
        assert torch.equal(g0, g1)


def test_entries_out_of_range_are_left_out_and_reported(work):
    z, index, value, weight, rw = make(4, 100, 2, 6, "f32")
    bad = [index[0].clone(), index[1]]
    bad[0][1, 2] = 100
    bad[0][2, 0] = 2 ** 31 - 1
    check(work, z, bad, value, weight, rw, 1.0, "f32")
    with pytest.raises(fa.FedAvgError) as e:
        fa.fa_work_sync(work)
    assert e.value.status == fa.FA_ERR_RANGE
    fa.fa_work_sync(work)                    # reported once


def test_gradient_against_differences(work):
    """Central differences of the summed loss along random directions, fp32: with a step of
    2^-5 the third-order term is about 2^-11 of the curvature's scale, the losses' rounding
    2^-21 sqrt(rows) / 2^-5; 1 % of the gradient's norm covers both."""
    rows, vocab = 50, 300
    z, index, value, weight, rw = make(rows, vocab, 3, 12, "f32", spread=1.0)
    lists = fa.distill_lists(index, value, [12] * 3, weight)
    grad, loss = torch.empty_like(z), torch.empty(rows, device="cuda")
    fa.fa_distill_grad(work, rows, vocab, z, vocab, "f32", lists, 2.0, rw, None, loss, grad, vocab)
    g = torch.Generator(device="cuda").manual_seed(5)

    def total(x):
        fa.fa_distill_loss(work, rows, vocab, x, vocab, "f32", lists, 2.0, rw, loss)
        return loss.double().sum().item()

    for _ in range(3):
        u = torch.randn((rows, vocab), generator=g, device="cuda")
        u /= u.norm() / 4
        h = 2.0 ** -5
        slope = (total(z + h * u) - total(z - h * u)) / (2 * h)
        assert abs(slope - (grad.double() * u.double()).sum().item()) <= 0.01 * 4 * grad.double().norm().item()


def test_gradient_rows_sum_to_zero(work):
    z, index, value, weight, rw = make(30, 5000, 4, 20, "f32")
    grad, _ = check(work, z, index, value, weight, rw, 1.0, "f32")
    assert (grad.double().sum(1).abs() <= 1e-4 * rw.double()).all()


def test_rows_in_a_graph_and_on_a_stream(work):
    z, index, value, weight, rw = make(20, 3000, 3, 16, "bf16")
    lists = fa.distill_lists(index, value, [16] * 3, weight)
    grad, loss = torch.empty_like(z), torch.empty(20, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fa.fa_distill_grad(work, 20, 3000, z, 3000, "bf16", lists, 1.0, rw, None, loss, grad, 3000,
                           torch.cuda.current_stream())
    z.copy_(z.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    want = torch.empty_like(z)
    fa.fa_distill_grad(work, 20, 3000, z, 3000, "bf16", lists, 1.0, rw, None, loss, want, 3000, torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(grad, want)


def test_rows_past_32_bit_offsets(work):
    """The last rows of a matrix of more than 2^32 elements (a large row stride)."""
    vocab, ld, rows = 100, 1 << 29, 10
    buf = torch.empty(((rows - 1) * ld + vocab,), device="cuda", dtype=torch.bfloat16)
    z, index, value, weight, rw = make(rows, vocab, 2, 6, "bf16")
    for r in range(rows):
        buf[r * ld:r * ld + vocab] = z[r]
    lists = fa.distill_lists(index, value, [6, 6], weight)
    loss, grad = torch.empty(rows, device="cuda"), torch.empty_like(z)
    fa.fa_distill_grad(work, rows, vocab, buf, ld, "bf16", lists, 1.0, rw, None, loss, grad, vocab)
    want = torch.empty_like(z)
    fa.fa_distill_grad(work, rows, vocab, z, vocab, "bf16", lists, 1.0, rw, None, loss, want, vocab)
    torch.cuda.synchronize()
    assert torch.equal(grad, want)


def test_refusals(work):
    z, index, value, weight, rw = make(4, 100, 2, 6, "f32")
    loss, lse, grad = torch.empty(4, device="cuda"), torch.empty(4, device="cuda"), torch.empty_like(z)
    lists = fa.distill_lists(index, value, [6, 6], weight)
    ok = dict(rows=4, vocab=100, logits=z, ld=100, dtype="f32", lists=lists, temperature=1.0, row_weight=rw,
              lse=None, loss=loss, grad=grad, ldg=100)

    def refused(status, **kw):
        with pytest.raises(fa.FedAvgError) as e:
            fa.fa_distill_grad(work, **{**ok, **kw})
        assert e.value.status == status and e.value.detail

    mk = fa.distill_lists
    refused(fa.FA_ERR_ARG, logits=None)
    refused(fa.FA_ERR_ARG, logits=z.cpu())
    refused(fa.FA_ERR_ARG, grad=None)
    refused(fa.FA_ERR_ARG, loss=lse.cpu())
    refused(fa.FA_ERR_ARG, loss=rw)
    refused(fa.FA_ERR_ARG, grad=z.data_ptr() + 4)
    refused(fa.FA_ERR_ARG, lse=loss)
    refused(fa.FA_ERR_ARG, temperature=0.0)
    refused(fa.FA_ERR_ARG, temperature=-1.0)
    refused(fa.FA_ERR_ARG, temperature=float("nan"))
    refused(fa.FA_ERR_RANGE, ld=99)
    refused(fa.FA_ERR_RANGE, ldg=99)
    refused(fa.FA_ERR_RANGE, vocab=0)
    refused(fa.FA_ERR_RANGE, rows=1 << 31)
    refused(fa.FA_ERR_RANGE, lists=mk(index, value, [6, 0], weight))
    refused(fa.FA_ERR_RANGE, lists=mk(index, value, [2000, 2000], weight))
    refused(fa.FA_ERR_ARG, lists=mk([index[0], None], value, [6, 6], weight))
    refused(fa.FA_ERR_ARG, lists=mk(index, [value[0].cpu(), value[1]], [6, 6], weight))
    refused(fa.FA_ERR_ARG, lists=mk([], [], [], []))
    refused(fa.FA_ERR_ARG, lists=mk(index[:1] * 17, value[:1] * 17, [6] * 17, [1.0] * 17))
    refused(fa.FA_ERR_WEIGHT, lists=mk(index, value, [6, 6], [1.0, -1.0]))
    refused(fa.FA_ERR_WEIGHT, lists=mk(index, value, [6, 6], [1.0, float("inf")]))
    with pytest.raises(fa.FedAvgError):
        fa.fa_distill_loss(work, 4, 100, z, 100, "f32", lists, 1.0, rw, None)
    fa.fa_distill_grad(work, **{**ok, "rows": 0})
    fa.fa_distill_grad(work, **ok)
    fa.fa_work_sync(work)


@pytest.mark.parametrize("rows,vocab,dtype,topk", [
    (1, 5000, "f32", 16), (2, 33000, "bf16", 16), (9, 131075, "bf16", 64), (300, 131075, "bf16", 8), (40, 200003, "f32", 100),
    (3, 800001, "bf16", 16), (700, 40000, "f32", 4), (2000, 16500, "bf16", 3)])
def test_slices_of_rows_with_a_given_statistic(work, rows, vocab, dtype, topk):
    """With the statistic given a row may be divided in any number of slices: few rows, many
    rows, rows longer than a cluster holds, with and without the loss, in place or not."""
    z, index, value, weight, _ = make(rows, vocab, 3, topk, dtype, seed=5)
    rw = torch.ones(rows, device="cuda")
    rw[::7] = 0.0
    rw[0] = 0.5
    for inplace, fused_loss in ((False, True), (False, False), (True, False), (True, True)):
        check(work, z, index, value, weight, rw, 1.5, dtype, saved=True, inplace=inplace, fused_loss=fused_loss)


@pytest.mark.parametrize("dtype,vocab", [("f32", 20011), ("bf16", 70001), ("f32", 130000)])
def test_many_rows_over_clusters_take_turns(work, dtype, vocab):
    """More rows than run at one time, with masked rows and rows that need the plain form (and
    its further exchanges) between ordinary ones."""
    rows = 600
    z, index, value, weight, _ = make(rows, vocab, 2, 8, dtype, seed=6)
    z[3::5, :] += 3.0e6
    z[4::11, vocab // 3:] = -INF
    z[5::13, : vocab - 40] = torch.finfo(TORCH[dtype]).min
    rw = torch.ones(rows, device="cuda")
    rw[::3] = 0.0            # below: A <= 14 at these logits, 2^-20 (1 + A / 4) < 2^-17
    lists = fa.distill_lists(index, value, [8, 8], weight, "f32")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    grad = torch.empty_like(z)
    fa.fa_distill_loss(work, rows, vocab, z, vocab, dtype, lists, 2.0, rw, loss, lse)
    fa.fa_distill_grad(work, rows, vocab, z, vocab, dtype, lists, 2.0, rw, None, None, grad, vocab)
    fa.fa_work_sync(work)
    want = torch.where(rw > 0, torch.logsumexp(z.double() / 2.0, 1), 0.0)
    assert ((lse.double() - want).abs() <= 2.0 ** -20 + 2.0 ** -22 * want.abs()).all()
    # the gradient beside the lists' entries
    q = torch.softmax(z.double() / 2.0, 1) * rw[:, None].double() * 2.0
    d = (grad.double() - q)
    d.scatter_(1, index[0].long(), 0.0)
    d.scatter_(1, index[1].long(), 0.0)
    tol = q * ((2.0 ** -7.99 if dtype == "bf16" else 0.0) + 2.0 ** -17 + 2.0 ** -22 * want.abs()[:, None]) + 1e-30
    assert (d.abs() <= tol).all()


def test_an_expired_exchange_is_reported_and_ends():
    z, index, value, weight, _ = make(50, 70001, 2, 8, "f32", seed=7)
    lists = fa.distill_lists(index, value, [8, 8], weight, "f32")
    loss, lse = torch.empty(50, device="cuda"), torch.empty(50, device="cuda")
    bad = fa.fa_work_open(flags=fa.FA_TEST_WAIT_EXPIRES)
    try:
        fa.fa_distill_loss(bad, 50, 70001, z, 70001, "f32", lists, 1.0, None, loss, lse)
        with pytest.raises(fa.FedAvgError) as e:
            fa.fa_work_sync(bad)
        assert e.value.status == fa.FA_ERR_INTERNAL and "device-side wait" in e.value.detail
        fa.fa_work_sync(bad)
    finally:
        fa.fa_work_close(bad)
