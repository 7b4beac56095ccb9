"""A bf16 result of fa_orthogonalise is the fp64 one rounded, and little else: no product of the
iteration takes fewer digits because the result has few."""
import pytest
import torch

import server_side_fedavg_gb300 as fa
from tests.test_gpu_orthogonalise import QUINTIC, iterate, make, work  # noqa: F401

pytestmark = pytest.mark.gpu

# The distance to the nearest bf16 number is a function of slope 1, so a result that is off by e before
# its rounding is off by at most |r(x) - x| + 2 |e| after it (2-norms).  Sums here are of up to 5 blocks of
# 64 terms, each of 12 additions that truncate to 2^-23 of the sum at worst: 7.2e-6 of a product.  The
# step's polynomial passes them on by |b| + 2 |c| = 8.8 at most, 6.3e-5; what the steps before have left
# is, at slopes of 0 to 4 around the singular values that they end at, about half of that again.  Twice
# 1e-4, then; a step of 11-bit products is off by 1.2e-3.
MORE = 2e-4


@pytest.mark.parametrize("count,rows,cols", [(2, 300, 320), (1, 320, 300), (3, 256, 256), (24, 256, 256), (1, 320, 320), (5, 130, 128),
                                             (1, 200, 320), (1, 70, 300), (4, 48, 300), (3, 16, 320)])
@pytest.mark.parametrize("steps", [1, 2, 4, 5])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_bf16_result_is_off_by_its_rounding(work, count, rows, cols, steps, dtype):  # noqa: F811
    u = make(count, rows, cols, dtype, 41)
    out = torch.empty((count, rows, cols), device="cuda", dtype=torch.bfloat16)
    fa.fa_orthogonalise(work, count, rows, cols, u, out, dtype, "bf16", steps=steps)
    x = iterate(u, steps, QUINTIC, 1e-7)
    norm = lambda t: t.square().sum((1, 2)).sqrt()  # noqa: E731
    assert (norm(out.double() - x) <= norm(x.bfloat16().double() - x) + MORE * norm(x)).all()
