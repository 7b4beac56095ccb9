"""What the server-side training operators are measured on.

Two operators of the federated server, each in both directions:

  product   out = act(alpha * op(a) . op(b) + bias) + beta * residual and its gradients:
            the student's layers and head, the merge of an aggregated adapter into its
            frozen base, the weight step
  distill   the temperature-scaled divergence of a student's logits from the clients' top
            logits, weighted by the clients' sample counts, and its gradient

`listed` and `draw` give cases, `prepare` a case's inputs on the GPU, `run` one pass -- in
elementary fp32 torch operations, or with `own` through the package's calls -- `work` the
bytes and operations that a pass cannot do without, and `exact` its outputs in fp64.
"""
import math

import torch

own = False

ELEM = {"bf16": 2, "f32": 4}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}

_handle = None


def _work():
    """The library handle that a server process opens once and keeps."""
    global _handle
    if _handle is None:
        import server_side_fedavg_gb300 as fa
        _handle = fa.fa_work_open()
    return _handle


# ---------------------------------------------------------------- the cases
def _product(name, m, n, k, dtype, out, trans_a=False, trans_b=True, bias=False, act="none",
             residual=False, pre=False, alpha=1.0):
    return {"name": name, "op": "product", "m": m, "n": n, "k": k, "dtype": dtype, "out": out,
            "trans_a": trans_a, "trans_b": trans_b, "bias": bias, "act": act, "residual": residual,
            "pre": pre, "alpha": alpha}


def _backward(name, m, n, k, dtype, out, bias=False, act="none"):
    return {"name": name, "op": "product_backward", "m": m, "n": n, "k": k, "dtype": dtype,
            "out": out, "bias": bias, "act": act}


def _distill(name, op, rows, vocab, dtype, clients, topk, temperature=1.0, masked=False,
             absent=False, saved=False):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "dtype": dtype,
            "clients": clients, "topk": topk, "temperature": temperature, "masked": masked,
            "absent": absent, "saved": saved}


def listed():
    return [
        # the classifier of the small CNN (fc 10 x 256) on a batch of four: latency alone
        _product("fc_batch4", 4, 10, 256, "f32", "f32", bias=True),
        # the 7B decoder's head for one token: reads the whole 32000 x 4096 weight once
        _product("head_one_token", 1, 32000, 4096, "bf16", "bf16"),
        # the aggregated rank-16 adapter of one projection merged into its frozen base
        _product("merge_adapter", 4096, 4096, 16, "bf16", "bf16", trans_b=False, residual=True, alpha=2.0),
        # the vision tower's second layer over 8 images of 257 positions, with its residual
        _product("vit_fc2", 2056, 1024, 4096, "bf16", "bf16", bias=True, residual=True),
        # a decoder's gate projection over a training batch, pre-activation kept for backward
        _product("gate_train", 4096, 11008, 4096, "bf16", "bf16", act="silu", pre=True),
        # the projector in fp32 on an odd number of positions
        _product("projector_f32", 777, 4096, 1024, "f32", "f32", bias=True, act="gelu"),
        # gradients of the vision tower's first layer (activation, bias, both operands)
        _backward("vit_fc1_backward", 2056, 4096, 1024, "bf16", "bf16", bias=True, act="gelu"),
        # gradients of the 7B decoder's head, the weight's in fp32 for the server's master copy
        _backward("head_backward_f32", 1024, 32000, 4096, "bf16", "f32"),
        # one row's divergence from one client's list: latency alone
        _distill("loss_one_row", "distill_loss", 1, 32000, "bf16", 1, 32),
        # a public batch's loss on fp32 logits of an odd vocabulary, padded rows masked
        _distill("loss_f32_masked", "distill_loss", 1531, 32003, "f32", 5, 20, 2.0, masked=True, absent=True),
        # the training step: loss and gradient for eight clients' lists
        _distill("step_eight_clients", "distill_grad", 4096, 32000, "bf16", 8, 32, 2.0, masked=True, absent=True),
        # a vocabulary that no single SM's shared memory holds, gradient from a kept statistic
        _distill("grad_large_vocab", "distill_grad", 700, 131075, "bf16", 4, 64, 1.0, absent=True, saved=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case: sizes log-uniform over the listed range, odd ones as they fall."""
    dtype = rng.choice(("bf16", "bf16", "f32"))
    op = rng.choice(("product", "product_backward", "distill_loss", "distill_grad"))
    if op.startswith("product"):
        while True:
            m, n, k = _log(rng, 1, 8192), _log(rng, 8, 32000), _log(rng, 8, 11008)
            if rng.random() < 0.5:      # half of the cases on the usual multiples of eight
                n, k = (n + 7) // 8 * 8, (k + 7) // 8 * 8
            if m * n * k * (6 if dtype == "f32" else 1) * (2 if op != "product" else 1) <= 2 * 1024 * 32000 * 4096:
                break
        act = rng.choice(("none", "relu", "gelu", "silu"))
        out = "f32" if dtype == "f32" else rng.choice(("bf16", "bf16", "f32"))
        bias = rng.random() < 0.5
        if op == "product":
            c = _product("", m, n, k, dtype, out, rng.random() < 0.15, rng.random() < 0.75, bias, act,
                         rng.random() < 0.4, act != "none" and rng.random() < 0.5, rng.choice((1.0, 1.0, 0.5)))
        else:
            c = _backward("", m, n, k, dtype, out, bias, act)
    else:
        while True:
            rows, vocab = _log(rng, 1, 8192), _log(rng, 10, 200000)
            if rows * vocab * ELEM[dtype] <= 4096 * 32000 * 2:
                break
        topk = max(1, min(_log(rng, 1, 128), vocab // 2))
        c = _distill("", op, rows, vocab, dtype, rng.randint(1, 8), topk, rng.choice((1.0, 2.0, 4.0)),
                     rng.random() < 0.5, rng.random() < 0.5, op == "distill_grad" and rng.random() < 0.4)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _normal(g, shape, scale, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"].startswith("product"):
        m, n, k, t = c["m"], c["n"], c["k"], TORCH[c["dtype"]]
        trans_a, trans_b = c.get("trans_a", False), c.get("trans_b", True)
        # activations of unit scale, weights of the usual 1 / sqrt(fan in)
        s["a"] = _normal(g, (k, m) if trans_a else (m, k), 1.0, t)
        s["b"] = _normal(g, (n, k) if trans_b else (k, n), k ** -0.5, t)
        o = TORCH[c["out"]]
        if c["op"] == "product":
            s["bias"] = _normal(g, (n,), 0.5, t) if c["bias"] else None
            s["residual"] = _normal(g, (m, n), 1.0, o) if c["residual"] else None
            s["out"] = torch.empty((m, n), device="cuda", dtype=o)
            s["pre"] = torch.empty((m, n), device="cuda", dtype=o) if c["pre"] else None
        else:
            s["dout"] = _normal(g, (m, n), 1.0, t)
            s["pre"] = _normal(g, (m, n), 1.0, t) if c["act"] != "none" else None
            s["da"] = torch.empty((m, k), device="cuda", dtype=o)
            s["db"] = torch.empty((n, k), device="cuda", dtype=o)
            s["dbias"] = torch.empty((n,), device="cuda", dtype=o) if c["bias"] else None
        return s
    rows, vocab, J, topk = c["rows"], c["vocab"], c["clients"], c["topk"]
    s["logits"] = _normal(g, (rows, vocab), 2.5, TORCH[c["dtype"]])
    used = vocab
    if c["masked"] and vocab > 2 * topk + 8:      # a padded vocabulary: its last entries are closed
        used = vocab - 5
        s["logits"][:, used:] = float("-inf")
    # the clients' lists overlap: each takes topk of the 2 topk candidates of its row
    pool = min(2 * topk, used)
    step = next(p for p in (10007, 7919, 1009, 101, 7, 1) if math.gcd(p, used) == 1)
    first = torch.randint(0, used, (rows, 1), generator=g, device="cuda")
    cand = (first + step * torch.arange(pool, device="cuda")) % used
    s["index"], s["value"] = [], []
    for _ in range(J):
        at = torch.rand((rows, pool), generator=g, device="cuda").argsort(1)[:, :topk]
        idx = torch.gather(cand, 1, at).to(torch.int32)
        val = _normal(g, (rows, topk), 2.0, torch.float32).sort(1, descending=True).values
        if c["absent"]:                            # a client that has nothing for some rows
            gone = torch.rand((rows, 1), generator=g, device="cuda") < 0.2
            idx = torch.where(gone, torch.full_like(idx, -1), idx)
        s["index"].append(idx.contiguous())
        s["value"].append(val.contiguous())
    s["weight"] = [float(v) for v in torch.randint(100, 1001, (J,), generator=g, device="cuda").tolist()]
    w = torch.full((rows,), 1.0 / rows, device="cuda")
    if c["masked"]:
        w = torch.where(torch.rand((rows,), generator=g, device="cuda") < 0.1, torch.zeros_like(w), w)
    s["row_weight"] = w
    s["lse"] = torch.empty((rows,), device="cuda")
    s["loss"] = torch.empty((rows,), device="cuda")
    if c["op"] == "distill_grad":
        s["grad"] = torch.empty_like(s["logits"])
        if c["saved"]:                             # kept by the forward call
            s["lse"] = torch.logsumexp(s["logits"].double() / c["temperature"], 1).float()
    return s


# ---------------------------------------------------------------- the plain form
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
    sig = 1 / (1 + torch.exp(-z))
    return sig * (1 + z * (1 - sig))


def _plain_product(s):
    c = s["case"]
    a, b, o = s["a"].float(), s["b"].float(), TORCH[c["out"]]
    z = c["alpha"] * torch.matmul(a.t() if c["trans_a"] else a, b.t() if c["trans_b"] else b)
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(c["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"out": y.to(o), "pre": z.to(o) if c["pre"] else None}


def _plain_backward(s):
    c, o = s["case"], TORCH[s["case"]["out"]]
    a, b, dz = s["a"].float(), s["b"].float(), s["dout"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(c["act"], s["pre"].float())
    return {"da": torch.matmul(dz, b).to(o), "db": torch.matmul(dz.t(), a).to(o),
            "dbias": dz.sum(0).to(o) if c["bias"] else None}


def _plain_distill(s):
    c = s["case"]
    T, w, live = c["temperature"], s["row_weight"], s["row_weight"] > 0
    z = s["logits"].float() / T
    if c["saved"]:
        lse = s["lse"]
    else:
        top = z.amax(1)
        lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    zero = torch.zeros_like(w)
    total, loss, parts = zero, zero, []
    for idx, val, n in zip(s["index"], s["value"], s["weight"]):
        ok = idx >= 0
        u = torch.where(ok, val / T, -torch.inf)
        peak = u.amax(1, keepdim=True)
        present = peak > -torch.inf
        u = u - torch.where(present, peak, 0.0)
        e = torch.exp(u)
        sums = torch.where(present, e.sum(1, keepdim=True), 1.0)
        p = e / sums
        at = idx.clamp(min=0).long()
        kl = p * (u - torch.log(sums) - (torch.gather(z, 1, at) - lse[:, None]))
        total = total + n * present[:, 0]
        loss = loss + n * torch.where(p > 0, kl, 0.0).sum(1)
        parts.append((at, n * p))
    some = torch.where(total > 0, total, 1.0)
    loss = torch.where(live & (total > 0), w * T * T * loss / some, 0.0)
    if c["op"] == "distill_loss":
        return {"loss": loss, "lse": torch.where(live, lse, 0.0)}
    d = torch.exp(z - lse[:, None])
    for at, p in parts:
        d.scatter_add_(1, at, -p / some[:, None])
    d = torch.where((live & (total > 0))[:, None], (w * T)[:, None] * d, 0.0)
    return {"grad": d.to(s["logits"].dtype), "loss": loss}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import server_side_fedavg_gb300 as fa
    c = s["case"]
    work, stream = _work(), torch.cuda.current_stream()
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        fa.fa_product(work, m, n, k, s["a"], m if c["trans_a"] else k, s["b"], k if c["trans_b"] else n,
                      s["out"], n, c["dtype"], c["out"], c["trans_a"], c["trans_b"], c["alpha"], s["bias"],
                      c["act"], s["residual"], n, 1.0, s["pre"], stream)
        return {"out": s["out"], "pre": s["pre"]}
    if c["op"] == "product_backward":
        m, n, k = c["m"], c["n"], c["k"]
        fa.fa_product_backward(work, m, n, k, s["a"], k, s["b"], k, s["dout"], n, s["da"], k, s["db"], k,
                               c["dtype"], c["dtype"], c["out"], False, True, 1.0, c["act"], s["pre"], n,
                               s["dbias"], stream)
        return {"da": s["da"], "db": s["db"], "dbias": s["dbias"]}
    rows, vocab = c["rows"], c["vocab"]
    lists = fa.distill_lists(s["index"], s["value"], [c["topk"]] * c["clients"], s["weight"], "f32")
    if c["op"] == "distill_loss":
        fa.fa_distill_loss(work, rows, vocab, s["logits"], vocab, c["dtype"], lists, c["temperature"],
                           s["row_weight"], s["loss"], s["lse"], stream)
        return {"loss": s["loss"], "lse": s["lse"]}
    fa.fa_distill_grad(work, rows, vocab, s["logits"], vocab, c["dtype"], lists, c["temperature"],
                       s["row_weight"], s["lse"] if c["saved"] else None, s["loss"], s["grad"], vocab, stream)
    return {"grad": s["grad"], "loss": s["loss"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "product":
        return _plain_product(state)
    if op == "product_backward":
        return _plain_backward(state)
    return _plain_distill(state)


# ---------------------------------------------------------------- bytes, operations, fp64
def work(case):
    c = case
    i = ELEM[c["dtype"]]
    if c["op"].startswith("product"):
        m, n, k, o = c["m"], c["n"], c["k"], ELEM[c["out"]]
        if c["op"] == "product":
            return {"bytes": (m * k + n * k) * i + m * n * o * (1 + c["pre"] + c["residual"]) + n * i * c["bias"],
                    "flops": 2 * m * n * k}
        return {"bytes": (m * k + n * k + m * n * (1 + (c["act"] != "none"))) * i + (m * k + n * k + n * c["bias"]) * o,
                "flops": 4 * m * n * k}
    rows, vocab = c["rows"], c["vocab"]
    lists = rows * c["clients"] * c["topk"] * 8
    if c["op"] == "distill_loss":
        return {"bytes": rows * vocab * i + lists + 12 * rows, "flops": 4 * rows * vocab}
    return {"bytes": 2 * rows * vocab * i + lists + 12 * rows, "flops": 7 * rows * vocab}


_FN = {"none": lambda z: z, "relu": torch.nn.functional.relu, "gelu": torch.nn.functional.gelu,
       "silu": torch.nn.functional.silu}


def _chunks(n, size):
    return [(i, min(n, i + size)) for i in range(0, n, size)]


def exact(case, seed):
    if case["op"].startswith("product") and work(case)["flops"] > 6e12:
        return None
    c, s = case, prepare(case, seed)
    if c["op"] == "product":
        a = s["a"].double().t() if c["trans_a"] else s["a"].double()
        b = s["b"].double().t() if c["trans_b"] else s["b"].double()
        z = (a @ b).mul_(c["alpha"])
        if c["bias"]:
            z += s["bias"].double()
        y = _FN[c["act"]](z)
        if c["residual"]:
            y = y + s["residual"].double()
        return {"out": y, "pre": z if c["pre"] else None}
    if c["op"] == "product_backward":
        dz = s["dout"].double()
        if c["act"] != "none":
            z = s["pre"].double().requires_grad_()
            (dz,) = torch.autograd.grad(_FN[c["act"]](z), z, dz)
        return {"da": dz @ s["b"].double(), "db": dz.t() @ s["a"].double(),
                "dbias": dz.sum(0) if c["bias"] else None}
    # the divergence from its definition: a dense target of each row, a block of rows at a time
    T, rows, vocab = c["temperature"], c["rows"], c["vocab"]
    losses, lses, grads = [], [], []
    for r0, r1 in _chunks(rows, max(1, (1 << 28) // (8 * vocab))):
        z = s["logits"][r0:r1].double() / T
        lse = s["lse"][r0:r1].double() if c["saved"] else torch.logsumexp(z, 1)
        logq = z - lse[:, None]
        target = torch.zeros_like(z)
        entropy = torch.zeros_like(lse)
        total = torch.zeros_like(lse)
        for idx, val, n in zip(s["index"], s["value"], s["weight"]):
            here = idx[r0:r1, 0] >= 0
            p = torch.softmax(val[r0:r1].double() / T, 1) * (n * here)[:, None]
            target.scatter_add_(1, idx[r0:r1].clamp(min=0).long(), p)
            entropy += n * here * (torch.softmax(val[r0:r1].double() / T, 1)
                                   * torch.log_softmax(val[r0:r1].double() / T, 1)).sum(1)
            total += n * here
        w = s["row_weight"][r0:r1].double() * (total > 0)
        some = torch.where(total > 0, total, 1.0)
        cross = torch.where(target > 0, target * logq, 0.0).sum(1)
        losses.append(w * T * T * (entropy - cross) / some)
        lses.append(torch.where(s["row_weight"][r0:r1] > 0, lse, 0.0))
        if c["op"] == "distill_grad":
            grads.append((w * T)[:, None] * (torch.exp(logq) - target / some[:, None]))
    if c["op"] == "distill_loss":
        return {"loss": torch.cat(losses), "lse": torch.cat(lses)}
    return {"grad": torch.cat(grads), "loss": torch.cat(losses)}
