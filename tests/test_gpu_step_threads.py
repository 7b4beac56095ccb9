"""Two handles in two host threads, whose calls take different amounts of shared memory: a call's
launch does not depend on what the other thread's call has just asked for."""
import threading

import pytest
import torch

import server_side_fedavg_gb300 as fa

pytestmark = pytest.mark.gpu


def norm(P, C, G, dtype):
    g = torch.Generator(device="cuda").manual_seed(C)
    x = torch.randn((1, P, C), generator=g, device="cuda").to({"bf16": torch.bfloat16, "f32": torch.float32}[dtype])
    y, mean, rstd = torch.empty_like(x), torch.empty((1, G), device="cuda"), torch.empty((1, G), device="cuda")
    dx = torch.empty_like(x)

    def call(work, stream):
        fa.fa_group_norm(work, 1, P, C, G, x, y, dtype, act="silu", mean=mean, rstd=rstd, stream=stream)
        fa.fa_group_norm_backward(work, 1, P, C, G, x, y, dx, dtype, None, None, "f32", mean, rstd, act="silu", stream=stream)
    return call, [y, mean, rstd, dx]


def rotary(tokens, heads, interleaved):
    g = torch.Generator(device="cuda").manual_seed(heads)
    q = torch.randn((1, tokens, heads, 128), generator=g, device="cuda").to(torch.bfloat16)
    out, turns = torch.empty_like(q), fa.rotary_turns(128)

    def call(work, stream):
        fa.fa_rotary(work, 1, tokens, 128, turns, "bf16", q, heads, out, layout="interleaved" if interleaved else "half", stream=stream)
    return call, [out]


def ortho(count, rows, cols):
    g = torch.Generator(device="cuda").manual_seed(cols)
    u = torch.randn((count, rows, cols), generator=g, device="cuda")
    out = torch.empty_like(u)

    def call(work, stream):
        fa.fa_orthogonalise(work, count, rows, cols, u, out, "f32", "f32", stream=stream)
    return call, [out]


@pytest.mark.parametrize("one,two", [
    (lambda: norm(20000, 64, 8, "f32"), lambda: norm(2000, 1024, 8, "f32")),           # one kernel
    (lambda: norm(40000, 64, 8, "bf16"), lambda: norm(4000, 1024, 8, "bf16")),
    (lambda: norm(20, 8192, 8192, "f32"), lambda: norm(20, 6144, 6144, "f32")),          # two passes, more than 48 KB
    (lambda: norm(20, 8192, 8, "bf16"), lambda: norm(20, 5000, 8, "bf16")),
    (lambda: rotary(2000, 16, False), lambda: rotary(2000, 128, False)),                  # ring
    (lambda: rotary(2000, 16, True), lambda: rotary(2000, 128, True)),
    (lambda: ortho(2, 16, 600), lambda: ortho(2, 16, 4000)),
    (lambda: ortho(2, 6, 600), lambda: ortho(2, 6, 4000)),
    (lambda: ortho(2, 60, 500), lambda: ortho(2, 60, 1000))])
def test_two_threads(one, two):
    calls = [one(), two()]
    works, streams = [fa.fa_work_open() for _ in calls], [torch.cuda.Stream() for _ in calls]
    try:
        alone = []
        for (call, outs), w, s in zip(calls, works, streams):
            call(w, s)
            torch.cuda.synchronize()
            alone.append([o.clone() for o in outs])
            for o in outs:
                o.zero_()
        torch.cuda.synchronize()
        failed = []

        def loop(call, w, s):
            try:
                for _ in range(4000):
                    call(w, s)
            except Exception as e:  # noqa: BLE001
                failed.append(e)

        threads = [threading.Thread(target=loop, args=(call, w, s)) for (call, _), w, s in zip(calls, works, streams)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not failed, failed
        for (_, outs), want, w in zip(calls, alone, works):
            fa.fa_work_sync(w)
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
    finally:
        for w in works:
            fa.fa_work_close(w)
