"""What the operators around the products and the loss of a server-side training step are
measured on.

  orthogonalise   a weight step from an aggregated update: momentum, then the update made
                  orthogonal by Newton-Schulz products, scaled and added to the weight
  group_norm      group norm with an activation, channels last, and its gradients: the
                  image students' normalisation
  rotary          rotary positions of a decoder's queries and keys, and their gradients

`listed` and `draw` give cases, `prepare` a case's inputs on the GPU, `run` one pass -- in
elementary fp32 torch operations, or with `own` through the package's calls -- `work` the
bytes and operations that a pass cannot do without, and `exact` its outputs in fp64.
"""
import math

import torch

own = False

ELEM = {"bf16": 2, "f32": 4}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
QUINTIC = (3.4445, -4.7750, 2.0315)
MU, LR, DECAY, EPS_ORTHO, EPS_NORM = 0.9, 0.02, 0.999, 1e-7, 1e-5

_handle = None
_turns = {}


def _work():
    """The library handle that a server process opens once and keeps."""
    global _handle
    if _handle is None:
        import server_side_fedavg_gb300 as fa
        _handle = fa.fa_work_open()
    return _handle


# ---------------------------------------------------------------- the cases
def _ortho(name, count, rows, cols, dtype, out, steps=5, momentum=False, residual=False):
    return {"name": name, "op": "orthogonalise", "count": count, "rows": rows, "cols": cols, "dtype": dtype,
            "out": out, "steps": steps, "momentum": momentum, "residual": residual}


def _norm(name, op, n, positions, channels, groups, dtype, act="silu"):
    return {"name": name, "op": op, "n": n, "positions": positions, "channels": channels, "groups": groups,
            "dtype": dtype, "act": act}


def _rot(name, batch, seq, q_heads, k_heads, head_dim, rotary_dim, dtype, layout="half", inverse=False,
         scaling="none", factor=1.0, far=False, padded=False):
    return {"name": name, "op": "rotary", "batch": batch, "seq": seq, "q_heads": q_heads, "k_heads": k_heads,
            "head_dim": head_dim, "rotary_dim": rotary_dim, "dtype": dtype, "layout": layout, "inverse": inverse,
            "scaling": scaling, "factor": factor, "far": far, "padded": padded}


def listed():
    return [
        # the classifier of the small CNN (fc 10 x 256), one update: latency alone
        _ortho("ortho_fc", 1, 10, 256, "f32", "f32"),
        # the rank-16 adapters' A matrices of the 128 projections of a 7B decoder, in one call
        _ortho("ortho_adapters", 128, 16, 4096, "bf16", "bf16", momentum=True),
        # the square projections of the vision tower's 24 layers, one kind at a time
        _ortho("ortho_vit", 24, 1024, 1024, "bf16", "bf16", momentum=True, residual=True),
        # one attention projection of the decoder, the server's fp32 master weight stepped
        _ortho("ortho_projection_f32", 1, 4096, 4096, "f32", "f32", momentum=True, residual=True),
        # the decoder's gate projection: the largest matrix of a layer, tall
        _ortho("ortho_gate", 1, 11008, 4096, "bf16", "bf16", residual=True),
        # the deepest U-Net block on one patch: a few positions, latency alone
        _norm("norm_deepest", "group_norm", 1, 216, 256, 8, "f32"),
        # the U-Net's widest level on two volumes of 128 x 128 x 128
        _norm("norm_widest", "group_norm", 2, 128 ** 3, 32, 8, "bf16"),
        # an odd crop in fp32 at the second level, forward kept
        _norm("norm_crop_backward_f32", "group_norm_backward", 3, 45 * 47 * 51, 64, 8, "f32"),
        # the first level's gradients on a volume of 96 x 96 x 96
        _norm("norm_backward", "group_norm_backward", 2, 96 ** 3, 32, 8, "bf16"),
        # one new token of the 7B decoder: latency alone
        _rot("rotary_one_token", 1, 1, 32, 32, 128, 128, "bf16", far=True),
        # a training batch's queries and keys
        _rot("rotary_batch", 4, 4096, 32, 32, 128, 128, "bf16", layout="half"),
        # gradients where a part of each head turns, interleaved pairs, positions of a long
        # context by bands, ragged rows padded
        _rot("rotary_long_backward_f32", 3, 2731, 32, 8, 96, 64, "f32", layout="interleaved", inverse=True,
             scaling="banded", factor=8.0, far=True, padded=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case: sizes log-uniform over the listed range, odd ones as they fall."""
    op = rng.choice(("orthogonalise", "group_norm", "group_norm_backward", "rotary"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "orthogonalise":
        while True:
            rows, cols = _log(rng, 8, 11008), _log(rng, 8, 11008)
            if rng.random() < 0.5:
                rows, cols = (rows + 7) // 8 * 8, (cols + 7) // 8 * 8
            count = 1 if rng.random() < 0.5 else _log(rng, 1, 128)
            steps = rng.choice((5, 5, 5, 3, 6))
            m, n = min(rows, cols), max(rows, cols)
            if count * steps * m * m * (m + 3 * n) <= 5 * 4096 ** 2 * (4096 + 3 * 11008) and count * m * n <= 4096 * 11008:
                break
        out = "f32" if dtype == "f32" else rng.choice(("bf16", "bf16", "f32"))
        c = _ortho("", count, rows, cols, dtype, out, steps, rng.random() < 0.5, rng.random() < 0.5)
    elif op.startswith("group_norm"):
        while True:
            n, positions = _log(rng, 1, 32), _log(rng, 1, 128 ** 3)
            groups = rng.choice((1, 2, 4, 8, 8, 16, 32))
            channels = groups * _log(rng, 1, 64)
            most = 2 * 128 ** 3 * 32 * 2 / (1 if op == "group_norm" else 2)
            if channels <= 512 and n * positions * channels * ELEM[dtype] <= most:
                break
        c = _norm("", op, n, positions, channels, groups, dtype, rng.choice(("none", "relu", "gelu", "silu")))
    else:
        while True:
            batch, seq = _log(rng, 1, 16), _log(rng, 1, 16384)
            k_heads = rng.choice((1, 2, 4, 8, 12, 32))
            q_heads = k_heads * rng.choice((1, 1, 2, 4, 5))
            head_dim = rng.choice((32, 64, 72, 80, 96, 128, 128, 256))
            if q_heads <= 64 and batch * seq * (q_heads + k_heads) * head_dim * ELEM[dtype] <= 4 * 4096 * 64 * 128 * 2:
                break
        rotary_dim = head_dim if rng.random() < 0.5 else 2 * rng.randint(1, head_dim // 2)
        scaling = rng.choice(("none", "none", "linear", "base", "banded"))
        c = _rot("", batch, seq, q_heads, k_heads, head_dim, rotary_dim, dtype, rng.choice(("half", "interleaved")),
                 rng.random() < 0.5, scaling, 1.0 if scaling == "none" else rng.choice((2.0, 4.0, 8.0)),
                 rng.random() < 0.5, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _normal(g, shape, scale, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _prepare_ortho(c, g, s):
    B, m, n = c["count"], c["rows"], c["cols"]
    t, o = TORCH[c["dtype"]], TORCH[c["out"]]
    # a mean of clients' updates: a few strong directions over noise
    r = min(8, m, n)
    strong = torch.matmul(torch.randn((B, m, r), generator=g, device="cuda"),
                          torch.randn((B, r, n), generator=g, device="cuda"))
    s["update"] = ((torch.randn((B, m, n), generator=g, device="cuda") + 0.3 * strong) * 1e-3).to(t)
    s["momentum"] = _normal(g, (B, m, n), 3e-3, torch.float32) if c["momentum"] else None
    s["momentum_out"] = torch.empty_like(s["momentum"]) if c["momentum"] else None
    s["residual"] = _normal(g, (B, m, n), 0.02, o) if c["residual"] else None
    s["out"] = torch.empty((B, m, n), device="cuda", dtype=o)


def _prepare_norm(c, g, s):
    n, P, C, G = c["n"], c["positions"], c["channels"], c["groups"]
    t = TORCH[c["dtype"]]
    offset = torch.randn((n, 1, C), generator=g, device="cuda")
    s["x"] = (torch.randn((n, P, C), generator=g, device="cuda") * 1.5 + offset).to(t)
    s["gamma"] = 1 + _normal(g, (C,), 0.2, torch.float32)
    s["beta"] = _normal(g, (C,), 0.2, torch.float32)
    if c["op"] == "group_norm":
        s["y"] = torch.empty_like(s["x"])
        s["mean"], s["rstd"] = (torch.empty((n, G), device="cuda") for _ in range(2))
        return
    s["dout"] = _normal(g, (n, P, C), 1.0, t)
    # kept by the forward call
    x = s["x"].view(n, P, G, C // G)
    mean = x.mean((1, 3), dtype=torch.float64)
    var = torch.stack([(x[i].double() - mean[i][None, :, None]).square().mean((0, 2)) for i in range(n)])
    s["mean"], s["rstd"] = mean.float(), torch.rsqrt(var + EPS_NORM).float()
    s["dx"] = torch.empty_like(s["x"])
    s["d_gamma"], s["d_beta"] = torch.empty_like(s["gamma"]), torch.empty_like(s["beta"])


def _prepare_rotary(c, g, s):
    B, S, D, t = c["batch"], c["seq"], c["head_dim"], TORCH[c["dtype"]]
    s["q"] = _normal(g, (B, S, c["q_heads"], D), 1.0, t)
    s["k"] = _normal(g, (B, S, c["k_heads"], D), 1.0, t)
    first = torch.randint(0, 1 << 17, (B, 1), generator=g, device="cuda") if c["far"] else \
        torch.zeros((B, 1), device="cuda", dtype=torch.long)
    pos = first + torch.arange(S, device="cuda")
    if c["padded"]:                      # a row's tokens behind its sequence: no position
        length = torch.randint(S // 2, S + 1, (B, 1), generator=g, device="cuda")
        pos = torch.where(torch.arange(S, device="cuda") < length, pos, -1)
    s["position"] = pos.to(torch.int32).contiguous()
    s["q_out"], s["k_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "orthogonalise":
        _prepare_ortho(case, g, s)
    elif case["op"] == "rotary":
        _prepare_rotary(case, g, s)
    else:
        _prepare_norm(case, g, s)
    return s


# ---------------------------------------------------------------- the plain form
def _plain_ortho(s):
    c = s["case"]
    x, mom = s["update"].float(), None
    if c["momentum"]:
        mom = MU * s["momentum"] + x
        x = x + MU * mom                 # Nesterov's form
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt().float()
    x = x / (norm + EPS_ORTHO)
    tall = c["rows"] > c["cols"]
    if tall:
        x = x.transpose(1, 2)
    a, b, q = QUINTIC
    for _ in range(c["steps"]):
        gram = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * gram + q * torch.matmul(gram, gram), x)
    if tall:
        x = x.transpose(1, 2)
    out = LR * x
    if c["residual"]:
        out = DECAY * s["residual"].float() - out
    return {"out": out.to(TORCH[c["out"]]).contiguous(), "momentum": mom}


def _act(act, z):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(act, z):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    return torch.ones_like(z)


def _grouped(t, c):
    return t.view(c["n"], c["positions"], c["groups"], c["channels"] // c["groups"])


def _plain_norm(s):
    c = s["case"]
    x = _grouped(s["x"].float(), c)
    mean = x.mean((1, 3), keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt(d.square().mean((1, 3), keepdim=True) + EPS_NORM)
    z = (d * rstd).view(s["x"].shape) * s["gamma"] + s["beta"]
    return {"y": _act(c["act"], z).to(s["x"].dtype), "mean": mean.reshape(c["n"], c["groups"]),
            "rstd": rstd.reshape(c["n"], c["groups"])}


def _plain_norm_backward(s):
    c = s["case"]
    mean, rstd = s["mean"][:, None, :, None], s["rstd"][:, None, :, None]
    xhat = (_grouped(s["x"].float(), c) - mean) * rstd
    flat = xhat.view(s["x"].shape)
    dz = s["dout"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(c["act"], flat * s["gamma"] + s["beta"])
    d_gamma, d_beta = (dz * flat).sum((0, 1)), dz.sum((0, 1))
    dh = _grouped(dz * s["gamma"], c)
    dx = rstd * (dh - dh.mean((1, 3), keepdim=True) - xhat * (dh * xhat).mean((1, 3), keepdim=True))
    return {"dx": dx.view(s["x"].shape).to(s["x"].dtype), "d_gamma": d_gamma, "d_beta": d_beta}


BASE, CONTEXT, LOW, HIGH = 10000.0, 8192, 1.0, 4.0


def _frequencies(c):
    """Angle per position of each pair, in fp64."""
    r, f = c["rotary_dim"], c["factor"]
    i = torch.arange(r // 2, device="cuda", dtype=torch.float64)
    base = BASE * f ** (r / (r - 2)) if c["scaling"] == "base" and r > 2 else BASE
    freq = base ** (-2 * i / r)
    if c["scaling"] == "linear":
        freq = freq / f
    elif c["scaling"] == "banded":       # by the turns that a pair makes over the first context
        keep = ((CONTEXT * freq / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        freq = freq * (keep + (1 - keep) / f)
    return freq


def _turned(x, cos, sin, c):
    r = c["rotary_dim"]
    part, rest = x[..., :r], x[..., r:]
    if c["layout"] == "half":
        u, v = part[..., :r // 2], part[..., r // 2:]
        part = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    else:
        u, v = part[..., 0::2], part[..., 1::2]
        part = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    return torch.cat((part, rest), -1)


def _plain_rotary(s):
    c = s["case"]
    angle = s["position"].double()[..., None] * _frequencies(c)
    if c["inverse"]:
        angle = -angle
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    live = (s["position"] >= 0)[:, :, None, None]
    return {"q": torch.where(live, _turned(s["q"].float(), cos, sin, c).to(s["q"].dtype), s["q_out"]),
            "k": torch.where(live, _turned(s["k"].float(), cos, sin, c).to(s["k"].dtype), s["k_out"])}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import server_side_fedavg_gb300 as fa
    c = s["case"]
    work, stream = _work(), torch.cuda.current_stream()
    if c["op"] == "orthogonalise":
        fa.fa_orthogonalise(work, c["count"], c["rows"], c["cols"], s["update"], s["out"], c["dtype"], c["out"],
                            steps=c["steps"], eps=EPS_ORTHO, momentum=s["momentum"], momentum_out=s["momentum_out"],
                            mu=MU, nesterov=True, residual=s["residual"], alpha=-LR if c["residual"] else LR,
                            beta=DECAY, stream=stream)
        return {"out": s["out"], "momentum": s["momentum_out"]}
    if c["op"] == "rotary":
        kind = (c["rotary_dim"], c["scaling"], c["factor"])
        if kind not in _turns:           # of a model: made once
            _turns[kind] = fa.rotary_turns(c["rotary_dim"], BASE, c["scaling"], c["factor"], CONTEXT, LOW, HIGH)
        fa.fa_rotary(work, c["batch"], c["seq"], c["head_dim"], _turns[kind], c["dtype"], s["q"], c["q_heads"], s["q_out"],
                     s["k"], c["k_heads"], s["k_out"], position=s["position"], layout=c["layout"],
                     inverse=c["inverse"], stream=stream)
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "group_norm":
        fa.fa_group_norm(work, c["n"], c["positions"], c["channels"], c["groups"], s["x"], s["y"], c["dtype"],
                         s["gamma"], s["beta"], "f32", act=c["act"], eps=EPS_NORM, mean=s["mean"], rstd=s["rstd"],
                         stream=stream)
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    fa.fa_group_norm_backward(work, c["n"], c["positions"], c["channels"], c["groups"], s["x"], s["dout"], s["dx"],
                              c["dtype"], s["gamma"], s["beta"], "f32", s["mean"], s["rstd"], act=c["act"],
                              d_gamma=s["d_gamma"], d_beta=s["d_beta"], stream=stream)
    return {"dx": s["dx"], "d_gamma": s["d_gamma"], "d_beta": s["d_beta"]}


_PLAIN = {"orthogonalise": _plain_ortho, "group_norm": _plain_norm, "group_norm_backward": _plain_norm_backward,
          "rotary": _plain_rotary}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- bytes, operations, fp64
def work(case):
    c, i = case, ELEM[case["dtype"]]
    if c["op"] == "orthogonalise":
        B, m, n = c["count"], min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
        # X X^T and its square are symmetric: half of each
        return {"bytes": B * m * n * (i + ELEM[c["out"]] * (1 + c["residual"]) + 8 * c["momentum"]),
                "flops": B * c["steps"] * (m * m * n + m * m * m + 2 * m * m * n)}
    if c["op"] == "rotary":
        tokens = c["batch"] * c["seq"]
        heads = tokens * (c["q_heads"] + c["k_heads"])
        return {"bytes": 2 * heads * c["head_dim"] * i + 4 * tokens, "flops": 3 * heads * c["rotary_dim"]}
    size, C = c["n"] * c["positions"] * c["channels"], c["channels"]
    if c["op"] == "group_norm":
        return {"bytes": 2 * size * i + 8 * C + 8 * c["n"] * c["groups"], "flops": 10 * size}
    return {"bytes": 3 * size * i + 16 * C + 8 * c["n"] * c["groups"], "flops": 20 * size}


def _exact_ortho(c, s):
    outs, moms = [], []
    for i in range(c["count"]):
        x = s["update"][i].double()
        if c["momentum"]:
            mom = MU * s["momentum"][i].double() + x
            moms.append(mom)
            x = x + MU * mom
        x = x / (torch.linalg.norm(x) + EPS_ORTHO)
        a, b, q = QUINTIC
        # whichever side is short: X p(X^T X) = p(X X^T) X, the polynomial by Horner's rule
        for _ in range(c["steps"]):
            if c["rows"] <= c["cols"]:
                h = x @ x.t()
                x = a * x + h @ (b * x + q * (h @ x))
            else:
                h = x.t() @ x
                x = a * x + (b * x + q * (x @ h)) @ h
        outs.append(DECAY * s["residual"][i].double() - LR * x if c["residual"] else LR * x)
    return {"out": torch.stack(outs), "momentum": torch.stack(moms) if c["momentum"] else None}


_FN = {"none": lambda z: z, "relu": torch.nn.functional.relu, "gelu": torch.nn.functional.gelu,
       "silu": torch.nn.functional.silu}


def _exact_norm(c, s):
    ys, means, rstds = [], [], []
    for i in range(c["n"]):
        x = s["x"][i].double().view(c["positions"], c["groups"], -1)
        var, mean = torch.var_mean(x, (0, 2), correction=0)
        rstd = torch.rsqrt(var + EPS_NORM)
        h = ((x - mean[None, :, None]) * rstd[None, :, None]).view(c["positions"], c["channels"])
        ys.append(_FN[c["act"]](h * s["gamma"].double() + s["beta"].double()))
        means.append(mean)
        rstds.append(rstd)
    return {"y": torch.stack(ys), "mean": torch.stack(means), "rstd": torch.stack(rstds)}


def _exact_norm_backward(c, s):
    """Gradients of the kept statistics' form, by the chain rule in its vector form: the part of
    the incoming gradient along the constant and along xhat is taken out."""
    P, G = c["positions"], c["groups"]
    dxs = []
    gamma, beta = s["gamma"].double(), s["beta"].double()
    d_gamma, d_beta = torch.zeros_like(gamma), torch.zeros_like(beta)
    for i in range(c["n"]):
        mean, rstd = s["mean"][i].double()[None, :, None], s["rstd"][i].double()[None, :, None]
        h = (s["x"][i].double().view(P, G, -1) - mean) * rstd
        z = (h.view(P, -1) * gamma + beta).requires_grad_()
        (dz,) = torch.autograd.grad(_FN[c["act"]](z), z, s["dout"][i].double())
        d_gamma += torch.einsum("pc,pc->c", dz, h.view(P, -1))
        d_beta += dz.sum(0)
        dh = (dz * gamma).view(P, G, -1)
        count = P * (c["channels"] // G)
        along = torch.einsum("pgc,pgc->g", dh, h) / count
        dxs.append((rstd * (dh - dh.sum((0, 2))[None, :, None] / count - h * along[None, :, None])).view(P, -1))
    return {"dx": torch.stack(dxs), "d_gamma": d_gamma, "d_beta": d_beta}


def _exact_rotary(c, s):
    """Each pair as a complex number, turned by a unit one."""
    r = c["rotary_dim"]
    angle = s["position"].double()[..., None, None] * _frequencies(c)
    turn = torch.polar(torch.ones_like(angle), -angle if c["inverse"] else angle)
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        if c["layout"] == "half":
            z = torch.complex(x[..., :r // 2], x[..., r // 2:r].contiguous()) * turn
            y = torch.cat((z.real, z.imag, x[..., r:]), -1)
        else:
            z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2)) * turn
            y = torch.cat((torch.view_as_real(z).flatten(-2), x[..., r:]), -1)
        out[name] = torch.where((s["position"] >= 0)[..., None, None], y, 0.0)
    return out


def exact(case, seed):
    if case["op"] == "orthogonalise" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "orthogonalise":
        return _exact_ortho(case, s)
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    return (_exact_norm if case["op"] == "group_norm" else _exact_norm_backward)(case, s)
