"""The distillation example (tests/example_distill.py) runs as written, its operators work
together -- the loss falls -- and a device-side wait that gives up is reported."""
import math
import os
import runpy

import pytest
import torch

import server_side_fedavg_gb300 as fa

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_example_runs_and_learns():
    ns = runpy.run_path(os.path.join(HERE, "example_distill.py"), run_name="__example__")
    losses = ns["losses"]
    assert all(math.isfinite(v) for v in losses) and losses[2] < losses[1] < losses[0]


@pytest.mark.parametrize("m,n,k,din,dout", [(4096, 4096, 512, "bf16", "bf16"), (600, 520, 2048, "bf16", "f32"),
                                            (16, 512, 4096, "bf16", "bf16"), (300, 300, 1024, "f32", "f32")])
def test_an_expired_wait_is_reported_and_ends(m, n, k, din, dout):
    """Every form of the tensor-core product (pairs, splits over a cluster, few tokens, planes)
    leaves when a wait gives up: the status says so, on that handle alone, and the next
    handle's products are right."""
    t = {"bf16": torch.bfloat16, "f32": torch.float32}
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randn((m, k), generator=g, device="cuda").to(t[din])
    b = torch.randn((n, k), generator=g, device="cuda").to(t[din])
    res = torch.randn((m, n), generator=g, device="cuda").to(t[dout])
    out = torch.empty((m, n), device="cuda", dtype=t[dout])
    bad, good = fa.fa_work_open(flags=fa.FA_TEST_WAIT_EXPIRES), fa.fa_work_open()
    try:
        for r in (None, res):
            fa.fa_product(bad, m, n, k, a, k, b, k, out, n, din, dout, False, True, residual=r, ldr=n)
            with pytest.raises(fa.FedAvgError) as e:
                fa.fa_work_sync(bad)
            assert e.value.status == fa.FA_ERR_INTERNAL and "device-side wait" in e.value.detail
        fa.fa_work_sync(bad)                  # reported once
        fa.fa_product(good, m, n, k, a, k, b, k, out, n, din, dout, False, True, residual=res, ldr=n)
        fa.fa_work_sync(good)
        want = a.double() @ b.double().t() + res.double()
        assert ((out.double() - want).norm() / want.norm()).item() < (4e-3 if dout == "bf16" else 1.5e-6)
    finally:
        fa.fa_work_close(bad)
        fa.fa_work_close(good)


def test_a_workspace_that_grows_leaves_captured_graphs_valid():
    """A graph replays with the workspace it was captured with, after a larger call has
    replaced the handle's."""
    w = fa.fa_work_open()
    g = torch.Generator(device="cuda").manual_seed(2)

    def make(m, n, k):
        return (torch.randn((m, k), generator=g, device="cuda"), torch.randn((n, k), generator=g, device="cuda"),
                torch.empty((m, n), device="cuda"))

    def call(t, stream=None):
        a, b, out = t
        fa.fa_product(w, a.shape[0], b.shape[0], a.shape[1], a, a.shape[1], b, b.shape[1], out, out.shape[1], "f32", "f32",
                      False, True, stream=stream)

    small, large = make(200, 264, 136), make(2000, 3000, 1000)
    call(small)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(small, torch.cuda.current_stream())
    before = fa.fa_work_get_stats(w)["workspace_bytes"]
    call(large)
    assert fa.fa_work_get_stats(w)["workspace_bytes"] > before
    small[0].copy_(torch.randn_like(small[0]))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, out in (small, large):
        want = a.double() @ b.double().t()
        assert ((out.double() - want).norm() / want.norm()).item() < 1.5e-6
    fa.fa_work_close(w)
