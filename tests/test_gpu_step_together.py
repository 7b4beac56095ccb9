"""The layer and weight-step operators as a server may run them at one time: two handles on two
streams, whose kernels share the SMs, and calls of one handle on several streams.  Every result is the
bits that a call by itself gives."""
import pytest
import torch

import server_side_fedavg_gb300 as fa

pytestmark = pytest.mark.gpu


def tensors(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s, t=torch.bfloat16: torch.randn(s, generator=g, device="cuda").to(t)  # noqa: E731
    return dict(update=rand(10, 520, 520), one=rand(300, 4000), small=rand(12, 16, 2000), x=rand(3, 70000, 32), dout=rand(3, 70000, 32),
                q=rand(2, 1500, 16, 128), gamma=rand(32, t=torch.float32), beta=rand(32, t=torch.float32))


def calls(work, t, stream):
    """A run of them; its results."""
    out = {k: torch.empty_like(t[k]) for k in ("update", "one", "small", "x", "dout", "q")}
    out["mean"], out["rstd"] = torch.empty(3, 8, device="cuda"), torch.empty(3, 8, device="cuda")
    out["d_gamma"], out["d_beta"] = torch.empty(32, device="cuda"), torch.empty(32, device="cuda")
    turns = fa.rotary_turns(128)
    for _ in range(3):
        fa.fa_orthogonalise(work, 10, 520, 520, t["update"], out["update"], "bf16", "bf16", stream=stream)
        fa.fa_group_norm(work, 3, 70000, 32, 8, t["x"], out["x"], "bf16", t["gamma"], t["beta"], "f32", act="silu", mean=out["mean"],
                         rstd=out["rstd"], stream=stream)
        fa.fa_orthogonalise(work, 1, 300, 4000, t["one"], out["one"], "bf16", "bf16", stream=stream)
        fa.fa_group_norm_backward(work, 3, 70000, 32, 8, t["x"], t["dout"], out["dout"], "bf16", t["gamma"], t["beta"], "f32", out["mean"],
                                  out["rstd"], act="silu", d_gamma=out["d_gamma"], d_beta=out["d_beta"], stream=stream)
        fa.fa_rotary(work, 2, 1500, 128, turns, "bf16", t["q"], 16, out["q"], stream=stream)
        fa.fa_orthogonalise(work, 12, 16, 2000, t["small"], out["small"], "bf16", "bf16", stream=stream)
    return out


def same(a, b):
    return [k for k in a if not torch.equal(a[k], b[k])]


def test_two_handles_on_two_streams():
    works = [fa.fa_work_open(), fa.fa_work_open()]
    try:
        data = [tensors(1), tensors(2)]
        alone = []
        for w, t in zip(works, data):
            alone.append(calls(w, t, torch.cuda.current_stream()))
            torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        together = [calls(w, t, s) for w, t, s in zip(works, data, streams)]
        torch.cuda.synchronize()
        for w in works:
            fa.fa_work_sync(w)
        assert [same(a, b) for a, b in zip(alone, together)] == [[], []]
    finally:
        for w in works:
            fa.fa_work_close(w)


def test_one_handle_captured_and_replayed_between_direct_calls():
    work = fa.fa_work_open()
    try:
        t = tensors(3)
        alone = calls(work, t, torch.cuda.current_stream())
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            inside = calls(work, t, torch.cuda.current_stream())
        for _ in range(2):
            for k in inside.values():
                k.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert same(alone, inside) == []
            after = calls(work, t, stream)
            torch.cuda.synchronize()
            assert same(alone, after) == []
        fa.fa_work_sync(work)
    finally:
        fa.fa_work_close(work)
