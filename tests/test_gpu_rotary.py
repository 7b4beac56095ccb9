"""fa_rotary against the rotation in fp64: layouts, parts of a head, scaled frequencies, far
positions, strides, padding, gradients."""
import math

import pytest
import torch

import server_side_fedavg_gb300 as fa

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def work():
    w = fa.fa_work_open()
    yield w
    fa.fa_work_close(w)


def frequencies(r, base=10000.0, scaling="none", factor=1.0, context=0.0, low=1.0, high=32.0):
    if scaling == "base" and r > 2:
        base = base * factor ** (r / (r - 2))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if scaling == "linear":
        f = [v / factor for v in f]
    if scaling == "banded":
        keep = [min(1.0, max(0.0, (context * v / (2 * math.pi) - low) / (high - low))) for v in f]
        f = [v * (k + (1 - k) / factor) for v, k in zip(f, keep)]
    return torch.tensor(f, dtype=torch.float64, device="cuda")


def expect(x, pos, freq, layout, inverse=False, scale=1.0):
    """The rotation in fp64 and a bound on its error in the library's arithmetic."""
    r = 2 * freq.numel()
    angle = pos.double()[..., None, None] * freq * (-1 if inverse else 1)
    c, s = torch.cos(angle) * scale, torch.sin(angle) * scale
    y, size = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    at = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    u, v = x[..., at[0]].double(), x[..., at[1]].double()
    y[..., at[0]], y[..., at[1]] = u * c - v * s, v * c + u * s
    # sine and cosine: the angle's rest up to pi / 4 rounded to fp32 (0.8 x 2^-24), the function
    # 2 ulp below 1 (2 x 2^-24), times scale, two products and their sum (3 x 2^-24): below
    # 8 x 2^-24 of |u| + |v|; and the frequency's own rounding, position x frequency x 2^-50
    near = 8 * 2.0 ** -24 + pos.double()[..., None, None].abs() * freq * 2.0 ** -50
    size[..., at[0]] = size[..., at[1]] = near * abs(scale) * (u.abs() + v.abs())
    return y, size + HALF_STEP["bf16" if x.dtype == torch.bfloat16 else "f32"] * y.abs()


def inputs(batch, seq, heads, dim, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((batch, seq, heads, dim), generator=g, device="cuda").to(T[dtype])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("batch,seq,qh,kh,dim,r,dtype", [
    (1, 1, 32, 32, 128, 128, "bf16"), (1, 1, 1, 0, 2, 2, "f32"), (2, 37, 8, 2, 64, 64, "bf16"), (3, 5, 3, 1, 80, 20, "f32"),
    (1, 300, 5, 5, 72, 72, "bf16"), (2, 19, 4, 4, 33, 22, "bf16"), (2, 19, 4, 2, 33, 6, "f32"), (1, 64, 2, 2, 512, 512, "f32"),
    (2, 1000, 20, 4, 128, 64, "bf16"), (1, 2, 64, 64, 600, 512, "bf16"), (2, 3, 2, 2, 1201, 10, "f32"), (1, 2, 1, 1, 5000, 512, "bf16"),
    (3000, 1, 3, 1, 64, 64, "bf16"), (4, 129, 12, 12, 96, 48, "f32")])
def test_queries_and_keys(work, layout, batch, seq, qh, kh, dim, r, dtype):
    q, k = inputs(batch, seq, qh, dim, dtype, 1), inputs(batch, seq, max(kh, 1), dim, dtype, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.randint(0, 4096, (batch, seq), generator=g, device="cuda", dtype=torch.int32)
    q_out, k_out = torch.full_like(q, 9), torch.full_like(k, 9)
    turns = fa.rotary_turns(r)
    for inverse, scale in ((False, 1.0), (True, 1.25)):
        fa.fa_rotary(work, batch, seq, dim, turns, dtype, q, qh, q_out, k, kh, k_out, position=pos, layout=layout,
                     inverse=inverse, scale=scale)
        for x, out, heads in ((q, q_out, qh), (k, k_out, kh)):
            if heads == 0:
                assert (out == 9).all()
                continue
            want, size = expect(x, pos, frequencies(r), layout, inverse, scale)
            assert ((out.double() - want).abs() <= size).all()


@pytest.mark.parametrize("scaling,kw", [("linear", {"factor": 4.0}), ("base", {"factor": 8.0}),
                                        ("banded", {"factor": 8.0, "context": 8192.0, "low": 1.0, "high": 4.0})])
def test_scaled_frequencies(work, scaling, kw):
    q = inputs(1, 50, 2, 64, "f32", 4)
    pos = (torch.arange(50, device="cuda", dtype=torch.int32) * 2617)[None]
    out = torch.empty_like(q)
    fa.fa_rotary(work, 1, 50, 64, fa.rotary_turns(64, 500000.0, scaling, **kw), "f32", q, 2, out, position=pos)
    want, size = expect(q, pos, frequencies(64, 500000.0, scaling, **kw), "half")
    assert ((out.double() - want).abs() <= size).all()


def test_far_positions_are_as_exact_as_near_ones(work):
    """The angle is the product of two whole numbers modulo 2^64; the expectation takes it so too."""
    pos = torch.tensor([[0, 1, 2 ** 20 - 1, 2 ** 24 + 1, 2 ** 31 - 1]], device="cuda", dtype=torch.int32)
    q = inputs(1, 5, 3, 64, "f32", 5)
    out, turns = torch.empty_like(q), fa.rotary_turns(64)
    fa.fa_rotary(work, 1, 5, 64, turns, "f32", q, 3, out, position=pos)
    angle = torch.tensor([[(p * t % 2 ** 64) / 2 ** 64 * 2 * math.pi for t in turns] for p in pos[0].tolist()],
                         dtype=torch.float64, device="cuda")[None, :, None]
    u, v = q[..., :32].double(), q[..., 32:].double()
    want = torch.cat((u * angle.cos() - v * angle.sin(), v * angle.cos() + u * angle.sin()), -1)
    size = 8 * 2.0 ** -24 * (u.abs() + v.abs()).repeat(1, 1, 1, 2) + 2.0 ** -24 * want.abs()
    assert ((out.double() - want).abs() <= size).all()


def test_positions_may_be_counted_from_first(work):
    q = inputs(3, 40, 2, 64, "f32", 6)
    a, b, turns = torch.empty_like(q), torch.empty_like(q), fa.rotary_turns(64)
    fa.fa_rotary(work, 3, 40, 64, turns, "f32", q, 2, a, first=1000)
    pos = torch.arange(1000, 1040, device="cuda", dtype=torch.int32).expand(3, 40).contiguous()
    fa.fa_rotary(work, 3, 40, 64, turns, "f32", q, 2, b, position=pos)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_is_left_as_it_is(work, dtype):
    q = inputs(2, 30, 4, 64, dtype, 7)
    pos = torch.arange(30, device="cuda", dtype=torch.int32).repeat(2, 1)
    pos[0, 11:] = -1
    pos[1, :] = -5
    out = torch.full_like(q, 3.0)
    fa.fa_rotary(work, 2, 30, 64, fa.rotary_turns(32), dtype, q, 4, out, position=pos)
    assert (out[0, 11:] == 3).all() and (out[1] == 3).all()
    want, size = expect(q[:1, :11], pos[:1, :11], frequencies(32), "half")
    assert ((out[:1, :11].double() - want).abs() <= size).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,dim,r", [("bf16", 64, 64), ("f32", 48, 32), ("bf16", 40, 18)])
def test_in_place_in_a_packed_buffer(work, layout, dtype, dim, r):
    """q and k are slices of one projection's output, turned where they are; v and the columns
    behind are not touched."""
    qh, kh, b, s = 6, 2, 2, 33
    width = (qh + 2 * kh) * dim + 8
    packed = inputs(b, s, 1, width, dtype, 8).view(b, s, width)
    before = packed.clone()
    q, k = packed[:, :, :qh * dim], packed[:, :, qh * dim:]
    st = (s * width, width, dim)
    pos = torch.arange(s, device="cuda", dtype=torch.int32).repeat(b, 1)
    fa.fa_rotary(work, b, s, dim, fa.rotary_turns(r), dtype, q, qh, q, k, kh, k, position=pos, layout=layout, q_strides=st,
                 q_out_strides=st, k_strides=st, k_out_strides=st)
    for at, heads in ((0, qh), (qh * dim, kh)):
        x = before[:, :, at:at + heads * dim].reshape(b, s, heads, dim)
        want, size = expect(x, pos, frequencies(r), layout)
        got = packed[:, :, at:at + heads * dim].reshape(b, s, heads, dim)
        assert ((got.double() - want).abs() <= size).all()
    assert torch.equal(packed[:, :, (qh + kh) * dim:], before[:, :, (qh + kh) * dim:])


def test_heads_first_out_and_a_shared_input(work):
    """Output as [batch, heads, seq, dim]; the input's one head read by every head (stride 0)."""
    b, s, h, d = 2, 21, 4, 32
    x = inputs(b, s, 1, d, "f32", 9)
    out = torch.empty((b, h, s, d), device="cuda")
    fa.fa_rotary(work, b, s, d, fa.rotary_turns(d), "f32", x, h, out, q_strides=(s * d, d, 0), q_out_strides=(h * s * d, d, s * d))
    pos = torch.arange(s, device="cuda").repeat(b, 1)
    want, size = expect(x.expand(b, s, h, d), pos, frequencies(d), "half")
    assert ((out.transpose(1, 2).double() - want).abs() <= size).all()


def test_the_inverse_is_the_gradient(work):
    """<R x, g> = <x, R' g> for the turned pairs and the copied rest, and R' is autograd's."""
    b, s, h, d, r = 2, 17, 3, 40, 24
    x, g = inputs(b, s, h, d, "f32", 10), inputs(b, s, h, d, "f32", 11)
    y, dx, turns = torch.empty_like(x), torch.empty_like(x), fa.rotary_turns(r)
    pos = torch.randint(0, 100000, (b, s), device="cuda", dtype=torch.int32)
    fa.fa_rotary(work, b, s, d, turns, "f32", x, h, y, position=pos, scale=0.75)
    fa.fa_rotary(work, b, s, d, turns, "f32", g, h, dx, position=pos, scale=0.75, inverse=True)
    leaf = x.double().requires_grad_()
    angle = pos.double()[..., None, None] * frequencies(r)
    u, v = leaf[..., :r // 2], leaf[..., r // 2:r]
    turned = 0.75 * torch.cat((u * angle.cos() - v * angle.sin(), v * angle.cos() + u * angle.sin()), -1)
    (want,) = torch.autograd.grad(torch.cat((turned, leaf[..., r:]), -1), leaf, g.double())
    assert (dx.double() - want).abs().max() <= 16 * 2.0 ** -24 * 2 * g.abs().max().double()
    left, right = (y.double() * g.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(left - right) <= 16 * 2.0 ** -24 * (y.double() * g.double()).abs().sum() * 4


def test_captured_and_on_another_stream(work):
    q = inputs(2, 50, 4, 64, "bf16", 12)
    out, turns = torch.empty_like(q), fa.rotary_turns(64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fa.fa_rotary(work, 2, 50, 64, turns, "bf16", q, 4, out, stream=torch.cuda.current_stream())
    q.copy_(inputs(2, 50, 4, 64, "bf16", 13))
    graph.replay()
    torch.cuda.synchronize()
    pos = torch.arange(50, device="cuda").repeat(2, 1)
    want, size = expect(q, pos, frequencies(64), "half")
    assert ((out.double() - want).abs() <= size).all()
    with torch.cuda.stream(side):
        again = torch.empty_like(q)
        fa.fa_rotary(work, 2, 50, 64, turns, "bf16", q, 4, again, stream=side)
    side.synchronize()
    assert torch.equal(again, out)


def test_infinities_and_nan_stay_in_their_pair(work):
    q = inputs(1, 4, 2, 16, "f32", 14)
    q[0, 1, 0, 3], q[0, 2, 1, 12] = math.inf, math.nan
    out = torch.empty_like(q)
    fa.fa_rotary(work, 1, 4, 16, fa.rotary_turns(16), "f32", q, 2, out)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 1, 0, 3] = want[0, 1, 0, 11] = want[0, 2, 1, 4] = want[0, 2, 1, 12] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("batch,seq,qh,kh,dim,r,dtype", [(3, 1900, 16, 16, 128, 128, "bf16"), (2, 2777, 24, 8, 96, 48, "bf16"),
                                                         (1, 9001, 32, 0, 72, 36, "bf16"), (5, 1500, 16, 2, 128, 26, "bf16")])
def test_many_tokens(work, layout, batch, seq, qh, kh, dim, r, dtype):
    """Large enough for the form that streams tokens through shared memory: out of place with padding,
    and in place in a packed buffer, both as the fp64 rotation has it."""
    width = (qh + kh) * dim + 8
    packed = inputs(batch, seq, 1, width, dtype, 21).view(batch, seq, width)
    before = packed.clone()
    q, k = packed[:, :, :qh * dim], packed[:, :, qh * dim:]
    pos = torch.randint(0, 100000, (batch, seq), device="cuda", dtype=torch.int32)
    pos[:, seq - 300:] = -1
    live = (pos >= 0)[:, :, None, None]
    st, turns = (seq * width, width, dim), fa.rotary_turns(r)
    outs = [torch.full((batch, seq, max(h, 1), dim), 3.0, device="cuda", dtype=T[dtype]) for h in (qh, kh)]
    fa.fa_rotary(work, batch, seq, dim, turns, dtype, q, qh, outs[0], k, kh, outs[1], position=pos, layout=layout, inverse=True,
                 q_strides=st, k_strides=st)
    fa.fa_rotary(work, batch, seq, dim, turns, dtype, q, qh, q, k, kh, k, position=pos, layout=layout, inverse=True, q_strides=st,
                 k_strides=st)
    fa.fa_work_sync(work)
    for at, heads, out in ((0, qh, outs[0]), (qh * dim, kh, outs[1])):
        if heads == 0:
            continue
        x = before[:, :, at:at + heads * dim].reshape(batch, seq, heads, dim)
        want, size = expect(x, pos, frequencies(r), layout, True)
        assert torch.where(live, (out.double() - want).abs() <= size, out == 3).all()
        got = packed[:, :, at:at + heads * dim].reshape(batch, seq, heads, dim)
        assert torch.equal(torch.where(live, out, x), got)
    assert torch.equal(packed[:, :, (qh + kh) * dim:], before[:, :, (qh + kh) * dim:])
