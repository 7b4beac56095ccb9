"""The softmax statistics of fa_distill_loss and fa_distill_grad where a row's logits are far
apart: the sums are over a reference that is seen at a few places of the row, and a part of
the row whose logits lie some 80 to 128 powers of two above its reference must neither be
lost when the parts are merged nor spoil the sum.

Against fp64, with the tolerances of test_gpu_distill.py (a probability is off by
2^-20 (1 + A / 4), A = max |z - top| / T) and the units that shares of list entries are held
in: 2^-51 of the row's weight, so that a gradient is off by half a unit for each place that
names the entry, however small its share."""
import pytest
import torch

import server_side_fedavg_gb300 as fa
from tests.test_gpu_distill import TORCH, make, oracle, work  # noqa: F401

pytestmark = pytest.mark.gpu

# whole rows (128 and 256 threads), rows over clusters of 2, 4 and 8, rows that are streamed
FORMS = [(8000, "bf16"), (4000, "f32"), (32000, "bf16"), (16000, "f32"), (70001, "bf16"), (32003, "f32"),
         (131075, "bf16"), (131075, "f32"), (300007, "bf16")]


def compare(work, z, index, value, weight, rw, T, dtype):  # noqa: F811
    rows, vocab = z.shape
    places = [i.shape[1] for i in index]
    lists = fa.distill_lists(index, value, places, weight)
    want_loss, want_lse, want, size, both = oracle(z, index, value, weight, T, rw)
    A = z.float().abs().amax(1).double() * 2 / T
    rel = 2.0 ** -20 * (1 + A / 4)
    tol = (rel + 2.0 ** -19)[:, None] * both + (rw.double() * T * sum(places) * 2.0 ** -52)[:, None] + 1e-30
    if dtype == "bf16":
        tol = tol + want.abs() * 2.0 ** -7.99
    loss, lse, loss2 = (torch.empty(rows, device="cuda") for _ in range(3))
    fa.fa_distill_loss(work, rows, vocab, z, vocab, dtype, lists, T, rw, loss, lse)
    apart, inplace = torch.empty_like(z), z.clone()
    fa.fa_distill_grad(work, rows, vocab, z, vocab, dtype, lists, T, rw, None, None, apart, vocab)
    fa.fa_distill_grad(work, rows, vocab, inplace, vocab, dtype, lists, T, rw, None, loss2, inplace, vocab)
    torch.cuda.synchronize()

    def same(got, exact, t, what):
        d = (got.double() - exact).abs()
        assert (d <= t).all(), f"{what}: {int((~(d <= t)).sum())} of {d.numel()} off, worst {(d / t).max().item():.3g} x tolerance"

    same(lse, want_lse, rel + 2.0 ** -22 * want_lse.abs(), "lse")
    same(loss, want_loss, rel * size, "loss")
    same(loss2, want_loss, rel * size, "loss of the gradient call")
    same(apart, want, tol, "grad")
    same(inplace, want, tol, "grad in place")


@pytest.mark.parametrize("T", [1.0, 0.5])
@pytest.mark.parametrize("vocab,dtype", FORMS)
def test_a_few_open_logits_over_a_distant_floor(work, vocab, dtype, T):  # noqa: F811
    """All logits at a floor 80 to 90 (times T) below zero, a few at random places above zero:
    warps that look at the floor hold sums of 2^115 to 2^130 times their reference's term."""
    rows = 512 if vocab < 60000 else 192
    z, index, value, weight, rw = make(rows, vocab, 2, 12, dtype, seed=vocab)
    g = torch.Generator(device="cuda").manual_seed(1)
    floor = torch.linspace(-80, -90, rows, device="cuda")[:, None] * T
    z.copy_((floor + 0.01 * torch.randn((rows, vocab), generator=g, device="cuda")).to(TORCH[dtype]))
    for _ in range(4):
        at = torch.randint(0, vocab, (rows, 1), generator=g, device="cuda")
        z.scatter_(1, at, (T * (1 + 3 * torch.rand((rows, 1), generator=g, device="cuda"))).to(TORCH[dtype]))
    compare(work, z, index, value, weight, rw, T, dtype)


@pytest.mark.parametrize("vocab,dtype", FORMS)
def test_the_largest_logit_is_where_no_reference_is_taken(work, vocab, dtype):  # noqa: F811
    """One logit of 3 at a hundred places along the row in turn and one of 2.5 in the row's first
    vector, over floors between which 2^126 and 2^128 lie."""
    v = 16 // torch.finfo(TORCH[dtype]).bits * 8
    at = torch.arange(v, vocab - v, max(1, vocab // 96), device="cuda")
    rows = at.numel()
    for low in (-84.0, -84.5, -85.0, -85.5, -86.0):
        z, index, value, weight, rw = make(rows, vocab, 1, 3, dtype, seed=3)
        z.fill_(low)
        z[:, 0] = 2.5
        z.scatter_(1, at[:, None], 3.0)
        compare(work, z, index, value, weight, rw, 1.0, dtype)


@pytest.mark.parametrize("T", [0.1, 0.05, 0.03, 0.02, 0.01, 2.0 ** -10])
@pytest.mark.parametrize("vocab,dtype", FORMS)
def test_low_temperatures(work, vocab, dtype, T):  # noqa: F811
    """Normally distributed logits at low temperatures: the warps' references are tens to
    hundreds of powers of two apart."""
    rows = 256 if vocab < 60000 else 64
    z, index, value, weight, rw = make(rows, vocab, 2, 20, dtype, seed=vocab + 1)
    compare(work, z, index, value, weight, rw, T, dtype)
