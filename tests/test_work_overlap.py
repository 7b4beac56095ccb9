"""Which overlaps of a call's tensors are refused (CPU, a fake runtime: nothing is read).
Matrices that share no element are taken, column slices of one buffer among them."""
import random

import pytest

import server_side_fedavg_gb300 as fa
from tests.work_shim import Work

BASE = 1 << 36
FAR = [i << 40 for i in range(1, 9)]


@pytest.fixture(scope="module")
def work():
    w = Work()
    yield w
    w.close()


def test_column_slices_of_one_buffer_are_taken(work):
    m, n, k, size = 64, 32, 48, 4
    ld = 200
    a, b, bias = FAR[:3]
    ok = lambda **kw: work.product(**{**dict(m=m, n=n, k=k, a=a, b=b, out=BASE, ldo=ld), **kw}) == fa.FA_OK  # noqa: E731
    assert ok(pre=BASE + n * size)                                  # out | pre
    assert ok(a=BASE + n * size, lda=ld)                            # out | a
    assert ok(a=BASE + (ld - k) * size, lda=ld)                     # out | ... | a
    assert ok(out=BASE + 8, a=BASE + 8 - k * size + ld * size, lda=ld)      # a's rows wrap to before out's next row
    assert ok(residual=BASE + 4 * n * size, ldr=ld, pre=BASE + 2 * n * size)
    assert ok(b=BASE + n * size, ldb=ld, m=8, k=48)                 # fewer rows of out than of b
    assert ok(bias=BASE + n * size)                                 # a row between out's rows
    assert ok(bias=BASE + (ld * 5 - n) * size)


def test_slices_that_share_an_element_are_refused(work):
    m, n, k, size, ld = 64, 32, 48, 4, 200
    a, b = FAR[:2]

    def refused(**kw):
        assert work.product(**{**dict(m=m, n=n, k=k, a=a, b=b, out=BASE, ldo=ld), **kw}) == fa.FA_ERR_ARG
        assert "overlap" in work.error()

    refused(pre=BASE + (n - 1) * size)
    refused(a=BASE + (n - 1) * size, lda=ld)
    refused(a=BASE + (ld - k + 1) * size, lda=ld)       # its last column is out's first, a row on
    refused(a=BASE + 3 * ld * size - (k - 1) * size, lda=ld)
    refused(residual=BASE + size, ldr=ld)
    refused(bias=BASE + (ld * 5 - n + 1) * size)
    refused(a=BASE, lda=ld)
    refused(b=BASE + 3 * ld * size, ldb=ld)
    # rows of different lengths: where their spans meet
    refused(a=BASE + n * size, lda=ld + 1)
    refused(pre=BASE + n * size, ldo=n + 1)
    # the same bytes apart in elements of another size
    refused(a=BASE + (n - 1) * size, lda=2 * ld, din="bf16", dout="f32")


def test_gradients_in_slices_of_one_buffer(work):
    m, n, k, size, ld = 40, 24, 56, 4, 128
    a, b, d = FAR[:3]
    call = lambda **kw: work.backward(**{**dict(m=m, n=n, k=k, a=a, b=b, dout=d, d_a=BASE, d_b=BASE + k * size, ldda=ld, lddb=ld), **kw})  # noqa: E731
    assert call() == fa.FA_OK
    assert call(d_bias=BASE + 2 * k * size if ld >= 2 * k + n else FAR[4]) == fa.FA_OK
    assert call(dout=BASE + (2 * k - 8) * size, ldd=ld, d_b=FAR[4]) == fa.FA_OK
    assert call(d_b=BASE + (k - 1) * size) == fa.FA_ERR_ARG
    assert call(dout=BASE + (k - 1) * size, ldd=ld, d_b=FAR[4]) == fa.FA_ERR_ARG


def test_distillation_in_slices_of_one_buffer(work):
    rows, vocab, ld, size = 30, 50, 128, 4
    index, value = FAR[:2]
    call = lambda **kw: work.distill_grad(**{**dict(rows=rows, vocab=vocab, logits=BASE, ld=ld, grad=BASE + vocab * size, ldg=ld,  # noqa: E731
                                                    index=index, value=value), **kw})
    assert call() == fa.FA_OK
    assert call(grad=BASE) == fa.FA_OK                  # in place
    assert call(grad=BASE + size) == fa.FA_ERR_ARG
    assert call(grad=BASE + (ld - vocab + 1) * size) == fa.FA_ERR_ARG
    assert call(grad=BASE, ldg=ld + 1) == fa.FA_ERR_ARG
    assert call(loss=BASE + 2 * vocab * size, rows=20) == fa.FA_OK       # 20 of the 28 spare places of the first row
    assert call(loss=BASE + 2 * vocab * size, rows=29) == fa.FA_ERR_ARG


def test_against_every_element():
    """Random pairs of an output and an input of equal row distance, against the sets of their bytes."""
    w, rng = Work(), random.Random(5)
    seen = [0, 0]
    for _ in range(4000):
        ld = rng.randint(1, 12)
        m, n, k = rng.randint(1, 6), rng.randint(1, ld), rng.randint(1, ld)
        at = rng.randint(-8 * ld, 8 * ld)
        out = {BASE + (i * ld + j) * 4 for i in range(m) for j in range(n)}
        a = {BASE + (at + i * ld + j) * 4 for i in range(m) for j in range(k)}
        r = w.product(m, n, k, BASE + at * 4, FAR[0], BASE, lda=ld, ldo=ld)
        assert r == (fa.FA_ERR_ARG if out & a else fa.FA_OK), (ld, m, n, k, at)
        seen[r == fa.FA_OK] += 1
    assert min(seen) > 500
    for _ in range(2000):          # a single row beside rows of any distance
        ldo, m, n, width = rng.randint(1, 12), rng.randint(1, 6), rng.randint(1, 6), rng.randint(1, 40)
        ldo = max(ldo, n)
        at = rng.randint(-40, 8 * ldo)
        out = {BASE + (i * ldo + j) * 4 for i in range(m) for j in range(n)}
        b = {BASE + (at + j) * 4 for j in range(n * width)}
        r = w.product(m, n, width, FAR[0], BASE + at * 4, BASE, ldb=width, ldo=ldo)       # b stored [n, width], whole rows
        if out & b:
            assert r == fa.FA_ERR_ARG
        elif n == 1:
            assert r == fa.FA_OK, (ldo, m, n, width, at)
    w.close()
