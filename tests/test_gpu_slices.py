"""The training operators on column slices of one buffer: outputs beside inputs, residuals and
one another give the bits that they give in buffers of their own, and nothing else of the
buffer changes."""
import pytest
import torch

import server_side_fedavg_gb300 as fa

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def work():
    w = fa.fa_work_open()
    yield w
    fa.fa_work_close(w)


def _buffer(rows, widths, dtype, gap, seed):
    """A buffer of `rows` rows with slices of the given widths, `gap` elements between them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = sum(widths) + gap * len(widths)
    buf = torch.randn((rows, ld), generator=g, device="cuda").to(TORCH[dtype])
    parts, at = [], 0
    for n in widths:
        parts.append(buf[:, at:at + n])
        at += n + gap
    return buf, ld, parts


def _kept(buf, was, written):
    """Only the slices in `written` differ from before."""
    for part in written:
        at = (part.data_ptr() - buf.data_ptr()) // buf.element_size()
        was[:, at:at + part.shape[1]] = part
    return torch.equal(buf.view(torch.uint8), was.view(torch.uint8))


@pytest.mark.parametrize("gap", [0, 1, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(3, 24, 40), (40, 136, 72), (300, 264, 200), (1000, 1032, 520)])
def test_product(work, m, n, k, dtype, gap):
    buf, ld, (a, out, pre, res) = _buffer(m, (k, n, n, n), dtype, gap, m + gap)
    g = torch.Generator(device="cuda").manual_seed(1)
    b = torch.randn((n, k), generator=g, device="cuda").to(TORCH[dtype])
    was, a2, res2 = buf.clone(), a.contiguous(), res.contiguous()
    out2, pre2 = torch.empty_like(res2), torch.empty_like(res2)
    fa.fa_product(work, m, n, k, a, ld, b, k, out, ld, dtype, dtype, False, True, 1.0, None, "silu", res, ld, 0.5, pre)
    fa.fa_product(work, m, n, k, a2, k, b, k, out2, n, dtype, dtype, False, True, 1.0, None, "silu", res2, n, 0.5, pre2)
    torch.cuda.synchronize()
    y = torch.nn.functional.silu(a2.double() @ b.double().t()) + 0.5 * res2.double()
    for got in (out, out2):
        assert ((got.double() - y).norm() / y.norm()).item() < (4e-3 if dtype == "bf16" else 1.5e-6)
    assert ((pre.double() - pre2.double()).norm() / pre2.double().norm()).item() < (4e-3 if dtype == "bf16" else 1.5e-6)
    assert _kept(buf, was, (out, pre))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(40, 24, 56), (264, 264, 200)])
def test_gradients(work, m, n, k, dtype):
    """d_a beside dout, d_b beside b."""
    buf, ld, (dout, da) = _buffer(m, (n, k), dtype, 0, 5)
    wide, ldw, (b, db) = _buffer(n, (k, k), dtype, 0, 6)
    g = torch.Generator(device="cuda").manual_seed(2)
    a = torch.randn((m, k), generator=g, device="cuda").to(TORCH[dtype])
    was, was_wide = buf.clone(), wide.clone()
    fa.fa_product_backward(work, m, n, k, a, k, b, ldw, dout, ld, da, ld, db, ldw, dtype, dtype, dtype, False, True)
    torch.cuda.synchronize()
    for got, want in ((da, dout.double() @ b.double()), (db, dout.double().t() @ a.double())):
        assert ((got.double() - want).norm() / want.norm()).item() < (4e-3 if dtype == "bf16" else 1.5e-6)
    assert _kept(buf, was, (da,)) and _kept(wide, was_wide, (db,))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [77, 5000, 70001])
def test_distillation(work, vocab, dtype):
    rows = 20
    buf, ld, (z, grad) = _buffer(rows, (vocab, vocab), dtype, 1, 7)
    g = torch.Generator(device="cuda").manual_seed(3)
    index = [torch.rand((rows, vocab), generator=g, device="cuda").argsort(1)[:, :9].int().contiguous() for _ in range(3)]
    value = [torch.randn((rows, 9), generator=g, device="cuda") for _ in range(3)]
    lists = fa.distill_lists(index, value, [9] * 3, [1.0, 2.0, 3.0])
    was, loss, loss2 = buf.clone(), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    # a copy whose rows lie at the same alignment: the same sums
    apart, grad2 = buf.clone(), torch.empty_like(buf)
    fa.fa_distill_grad(work, rows, vocab, z, ld, dtype, lists, 1.5, None, None, loss, grad, ld)
    fa.fa_distill_grad(work, rows, vocab, apart, ld, dtype, lists, 1.5, None, None, loss2, grad2, ld)
    torch.cuda.synchronize()
    assert torch.equal(grad, grad2[:, :vocab]) and torch.equal(loss, loss2) and torch.isfinite(grad).all()
    assert _kept(buf, was, (grad,))
