"""Clients' weights of very different size: where the heavy clients have nothing for a row,
its target is that of the light ones alone, in full precision.  The gradient is the loss's
derivative whatever the ratio.

Against fp64 with the tolerances of test_gpu_distill.py.  Only the weights' ratios matter:
the oracle gets them divided by the largest (it holds a row's total in fp32)."""
import pytest
import torch

import server_side_fedavg_gb300 as fa
from tests.test_gpu_distill import make, oracle, work  # noqa: F401

pytestmark = pytest.mark.gpu


def compare(work, z, index, value, weight, rw, T, dtype, saved, inplace, with_loss):  # noqa: F811
    rows, vocab = z.shape
    lists = fa.distill_lists(index, value, [i.shape[1] for i in index], weight)
    lse = torch.logsumexp(z.double() / T, 1).float() if saved else None
    loss, out = torch.full((rows,), -7.0, device="cuda"), z.clone() if inplace else torch.empty_like(z)
    fa.fa_distill_grad(work, rows, vocab, out if inplace else z, vocab, dtype, lists, T, rw, lse,
                       loss if with_loss else None, out, vocab)
    torch.cuda.synchronize()
    want_loss, _, want, size, both = oracle(z, index, value, [v / max(weight) for v in weight], T, rw, lse)
    A = z.float().abs().amax(1).double() * 2 / T
    rel = 2.0 ** -20 * (1 + A / 4)
    if saved:
        rel = rel + 2.0 ** -22 * lse.double().abs()
    tol = (rel + 2.0 ** -19)[:, None] * both + 1e-30
    if dtype == "bf16":
        tol = tol + want.abs() * 2.0 ** -7.99
    d = (out.double() - want).abs()
    assert (d <= tol).all(), f"{int((~(d <= tol)).sum())} of {d.numel()} off, worst {(d / tol).max().item():.3g} x tolerance"
    if with_loss:
        assert ((loss.double() - want_loss).abs() <= rel * size + 1e-30).all()


# short lists, long lists, few slots; whole rows, clusters, streamed rows
@pytest.mark.parametrize("vocab,dtype,topk", [(500, "f32", 8), (500, "bf16", 200), (3000, "f32", 40), (20000, "f32", 16),
                                              (40000, "bf16", 64), (70001, "f32", 30), (131075, "bf16", 100),
                                              (200000, "f32", 16)])
@pytest.mark.parametrize("weight", [[1e6, 1.0, 3.0], [1e6, 1e-3, 2e-3], [1e6, 1e-7, 3e-7], [2.0 ** 24, 1e-10, 1e-12],
                                    [1e3, 1e-20, 3e-20], [1e6, 1e-30, 1e-31], [1e-9, 1e-30, 1e-44], [1e-40, 1e-43, 3e-43],
                                    [1e-200, 3e-200, 1e-201]])
def test_rows_that_only_light_clients_sent(work, vocab, dtype, topk, weight):  # noqa: F811
    rows = 30
    z, index, value, _, rw = make(rows, vocab, 3, topk, dtype, seed=vocab + topk)
    index[0][::2] = -1                # the heavy client is absent from every other row,
    index[1][::6] = -1                # the lightest alone in some,
    index[0][1] = index[2][1] = -1    # one row has the middle one alone
    index[2][3::4] = -1
    rw[::5] = 0.0
    for saved, inplace, with_loss in ((False, False, True), (False, True, True), (True, False, False), (True, True, True),
                                      (True, True, False)):
        compare(work, z, index, value, weight, rw, 1.5, dtype, saved, inplace, with_loss)


@pytest.mark.parametrize("ratio", [254.0, 256.0, 300.0, 4094.0, 4095.0, 4096.0, 4097.0, 5000.0])
def test_weights_about_the_ratio_at_which_shares_are_taken_again(work, ratio):  # noqa: F811
    z, index, value, _, rw = make(20, 4000, 2, 40, "f32", seed=9)
    index[0][::2] = -1
    compare(work, z, index, value, [ratio, 1.0], rw, 1.0, "f32", False, False, True)


def test_entries_that_light_clients_share(work):  # noqa: F811
    """Every light client names the same few entries; a NaN among their values reaches its
    entries, in the row that has it."""
    z, index, value, _, rw = make(8, 400, 8, 64, "f32")
    index = [(i % 40).contiguous() for i in index]
    index[0][::2] = -1
    weight = [1e9] + [1e-3 * j for j in range(1, 8)]
    weight[0] = 1e7
    compare(work, z, index, value, weight, rw, 1.0, "f32", False, False, True)
    value[3][2, 5] = float("nan")
    lists = fa.distill_lists(index, value, [64] * 8, weight)
    grad = torch.empty_like(z)
    fa.fa_distill_grad(work, 8, 400, z, 400, "f32", lists, 1.0, rw, None, None, grad, 400)
    torch.cuda.synchronize()
    assert torch.isnan(grad[2, :40]).any() and torch.isfinite(grad[2, 40:]).all()
    keep = [0, 1, 3, 4, 5, 6, 7]
    assert torch.isfinite(grad[keep]).all()


def test_a_weight_of_no_share_at_all_is_none(work):  # noqa: F811
    """Below 2^-225 of the largest weight a client counts as one of weight 0."""
    z, index, value, _, rw = make(6, 300, 2, 5, "f32")
    index[0][2] = -1
    got = []
    for light in (0.0, 1e-80):
        grad, loss = torch.empty_like(z), torch.empty(6, device="cuda")
        fa.fa_distill_grad(work, 6, 300, z, 300, "f32", fa.distill_lists(index, value, [5, 5], [1.0, light]), 1.0, rw, None,
                           loss, grad, 300)
        torch.cuda.synchronize()
        assert loss[2] == 0 and not grad[2].any()
        got.append((grad, loss))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("vocab,dtype,topk", [(500, "f32", 8), (500, "bf16", 200), (70001, "f32", 30), (200000, "f32", 16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_client_of_no_weight_has_no_part_in_a_row(work, vocab, dtype, topk, bad):  # noqa: F811
    """Whatever its values are: the loss leaves it out, and so does the loss's derivative."""
    z, index, value, _, rw = make(10, vocab, 3, topk, dtype, seed=4)
    value[1][::3, 1] = bad
    weight, without = [2.0, 0.0, 5.0], ([index[0], index[2]], [value[0], value[2]], [2.0, 5.0])
    for saved, inplace, with_loss in ((False, False, True), (False, True, True), (True, False, False)):
        lse = torch.logsumexp(z.double() / 1.5, 1).float() if saved else None
        got = []
        for i, v, w in ((index, value, weight), without):
            out = z.clone()
            loss = torch.zeros(10, device="cuda")
            fa.fa_distill_grad(work, 10, vocab, out if inplace else z, vocab, dtype,
                               fa.distill_lists(i, v, [topk] * len(i), w), 1.5, rw, lse, loss if with_loss else None, out, vocab)
            torch.cuda.synchronize()
            got.append((out, loss))
        assert torch.equal(got[0][0], got[1][0])
        assert ((got[0][1] - got[1][1]).abs() <= 2.0 ** -22 * got[1][1].abs()).all()      # (the clients' order in a sum)
