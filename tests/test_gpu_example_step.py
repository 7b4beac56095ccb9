"""The training-step example (tests/example_step.py) runs as written, and every tensor that its
operators hand to one another is what the whole chain gives in fp64: loss, gradients of weights and
inputs, weight steps."""
import math
import os
import runpy

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def ns():
    return runpy.run_path(os.path.join(HERE, "example_step.py"), run_name="__example__")


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def orthogonal(x, steps=5):
    a, b, c = 3.4445, -4.7750, 2.0315
    x = x / (x.norm(dim=(-2, -1), keepdim=True) + 1e-7)
    tall = x.shape[-2] > x.shape[-1]
    x = x.transpose(-1, -2) if tall else x
    for _ in range(steps):
        g = x @ x.transpose(-1, -2)
        x = a * x + (b * g + c * g @ g) @ x
    return x.transpose(-1, -2) if tall else x


# fp32 throughout: each call is good to 1e-6 of its result (2-norm), a chain of six to 1e-5
NEAR = 1e-5


def test_the_decoder_step(ns):
    batch, seq, heads, dim, hidden, tokens = (ns[k] for k in ("batch", "seq", "heads", "dim", "hidden", "tokens"))
    f = torch.tensor([10000.0 ** (-2 * i / dim) for i in range(dim // 2)], dtype=torch.float64, device="cuda")
    keep = ((32 * f / (2 * math.pi) - 1) / 3).clamp(0, 1)
    angle = ns["place"].double()[..., None, None] * (f * (keep + (1 - keep) / 4))
    live = ns["live"]
    w, head = ns["w_qkv"].double().requires_grad_(), ns["head"].double().requires_grad_()
    qkv = (ns["x"].double() @ w.t()).view(batch, seq, 3, heads, dim)

    def turned(t):
        u, v = t[..., :dim // 2], t[..., dim // 2:]
        r = torch.cat((u * angle.cos() - v * angle.sin(), v * angle.cos() + u * angle.sin()), -1)
        return torch.where(live[:, :, None, None], r, t)

    q, k, v = turned(qkv[:, :, 0]).transpose(1, 2), turned(qkv[:, :, 1]).transpose(1, 2), qkv[:, :, 2].transpose(1, 2)
    score = (q @ k.transpose(-1, -2) * dim ** -0.5).masked_fill(~live[:, None, None, :], -torch.inf)
    h = (torch.softmax(score, -1) @ v).transpose(1, 2).reshape(tokens, hidden)
    logq = torch.log_softmax(h @ head.t() / 2.0, 1)
    loss = torch.zeros(tokens, dtype=torch.float64, device="cuda")
    for i, val, n in zip(ns["index"], ns["value"], (100.0, 250.0, 400.0)):
        logp = torch.log_softmax(val.double() / 2.0, 1)
        loss = loss + n / 750.0 * (logp.exp() * (logp - logq.gather(1, i.long()))).sum(1)
    loss = loss * 4.0 * ns["weight"].double()
    d_w, d_head = torch.autograd.grad(loss.sum(), (w, head))
    assert off(ns["loss"], loss.detach()) < NEAR
    assert off(ns["d_head"], d_head) < NEAR and off(ns["d_w"], d_w) < NEAR
    assert torch.equal(ns["momentum"].view_as(ns["d_w"]), ns["d_w"])
    # from the gradient as it is: what the step adds
    o = orthogonal(ns["d_w"].double().view(3, hidden, hidden) * 1.95)
    want = 0.999 * ns["w_qkv"].double().view(3, hidden, hidden) - 0.02 * o
    assert off(ns["w_next"], want) < NEAR


def test_the_image_step(ns):
    n, P, G, C = ns["n"], ns["P"], ns["groups"], ns["c_out"]
    leaves = [ns[k].double().requires_grad_() for k in ("u", "w_conv", "gamma", "beta")]
    u, w, gamma, beta = leaves
    z = (u @ w.t()).view(n, P, G, C // G)
    d = z - z.mean((1, 3), keepdim=True)
    xhat = (d / torch.sqrt(d.square().mean((1, 3), keepdim=True) + 1e-5)).view(n, P, C)
    y = torch.nn.functional.silu(xhat * gamma + beta)
    grads = torch.autograd.grad((y * ns["d_y"].double()).sum(), leaves)
    assert off(ns["y"], y.detach()) < NEAR
    for got, want in zip(("d_u", "d_conv", "d_gamma", "d_beta"), grads):
        assert off(ns[got], want) < NEAR, got
    assert off(ns["conv_next"], w.detach() - 0.02 * orthogonal(ns["d_conv"].double())) < NEAR


def test_the_clients_mean_steps_the_weight(ns):
    mean = sum(n * d.double() for n, d in zip((100.0, 200.0, 300.0), ns["deltas"])) / 600.0
    size = ns["c_out"] * ns["c_in"]
    assert off(ns["outs"][0], mean[:size]) < 1e-6
    o = orthogonal(mean[:size].view(ns["c_out"], ns["c_in"]))
    assert off(ns["server_next"], ns["w_conv"].double() + 0.02 * o) < NEAR
