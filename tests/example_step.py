"""A server's training step of two students from the clients' top logits, run as written by the GPU
tests: a decoder layer with rotary positions, and an image student with group norm.  Each forward
call's gradient is the call beside it; the weight gradients, and a mean of the clients' deltas,
become orthogonalised weight steps."""
import torch
import server_side_fedavg_gb300 as fa

f32, bf16, dev = torch.float32, torch.bfloat16, "cuda"
gen = torch.Generator(device=dev).manual_seed(11)
rand = lambda *s, scale=1.0, dtype=f32: (torch.randn(s, generator=gen, device=dev) * scale).to(dtype)  # noqa: E731
new = lambda *s, dtype=f32: torch.empty(s, device=dev, dtype=dtype)  # noqa: E731
work = fa.fa_work_open()

# ---------------------------------------------------------------- a decoder layer, and its head
batch, seq, heads, dim, vocab, topk = 2, 64, 4, 32, 500, 8
hidden, tokens = heads * dim, batch * seq
x, w_qkv, head = rand(tokens, hidden), rand(3 * hidden, hidden, scale=hidden ** -0.5), rand(vocab, hidden, scale=hidden ** -0.5)
length = torch.tensor([seq, seq - 10], device=dev)               # the second row is padded
place = torch.arange(seq, device=dev, dtype=torch.int32).repeat(batch, 1)
live = place < length[:, None]
position = torch.where(live, place, -1).to(torch.int32)
index = [torch.rand((tokens, vocab), generator=gen, device=dev).topk(topk).indices.int() for _ in range(3)]
value = [rand(tokens, topk, scale=2.0) for _ in range(3)]
lists = fa.distill_lists(index, value, [topk] * 3, [100.0, 250.0, 400.0])
weight = live.flatten().float() / live.sum()
turns = fa.rotary_turns(dim, 10000.0, "banded", factor=4.0, context=32, low=1.0, high=4.0)      # once per model

qkv = new(tokens, 3 * hidden)
fa.fa_product(work, tokens, 3 * hidden, hidden, x, hidden, w_qkv, hidden, qkv, 3 * hidden, "f32", "f32", trans_b=True)
# q and k are turned where they lie in qkv
at = (seq * 3 * hidden, 3 * hidden, dim)
q, k, v = (qkv[:, i * hidden:] for i in range(3))
fa.fa_rotary(work, batch, seq, dim, turns, "f32", q, heads, q, k, heads, k, position=position, q_strides=at, k_strides=at)

# the attention between them is the student's own
leaf = qkv.clone().requires_grad_()
qs, ks, vs = leaf.view(batch, seq, 3, heads, dim).permute(2, 0, 3, 1, 4)
score = qs @ ks.transpose(-1, -2) * dim ** -0.5
score = score.masked_fill(~live[:, None, None, :], -torch.inf)
h_graph = (torch.softmax(score, -1) @ vs).transpose(1, 2).reshape(tokens, hidden)
h = h_graph.detach().contiguous()

logits, loss, d_h, d_head = new(tokens, vocab), new(tokens), new(tokens, hidden), new(vocab, hidden)
fa.fa_product(work, tokens, vocab, hidden, h, hidden, head, hidden, logits, vocab, "f32", "f32", trans_b=True)
fa.fa_distill_grad(work, tokens, vocab, logits, vocab, "f32", lists, 2.0, weight, None, loss, logits, vocab)
fa.fa_product_backward(work, tokens, vocab, hidden, h, hidden, head, hidden, logits, vocab, d_h, hidden, d_head, hidden, "f32", "f32",
                       "f32", trans_b=True)
(d_qkv,) = torch.autograd.grad(h_graph, leaf, d_h)
d_qkv = d_qkv.contiguous()
# the gradient of the turned q and k is turned back; v's stays
dq, dk = d_qkv, d_qkv[:, hidden:]
fa.fa_rotary(work, batch, seq, dim, turns, "f32", dq, heads, dq, dk, heads, dk, position=position, inverse=True, q_strides=at,
             k_strides=at)
d_w = new(3 * hidden, hidden)
fa.fa_product_backward(work, tokens, 3 * hidden, hidden, x, hidden, w_qkv, hidden, d_qkv, 3 * hidden, None, hidden, d_w, hidden, "f32",
                       "f32", "f32", trans_b=True)
# W_q, W_k and W_v as three matrices: W = 0.999 W - 0.02 orthogonalised(d_W), momentum from 0
momentum, w_next = new(3, hidden, hidden), new(3, hidden, hidden)
fa.fa_orthogonalise(work, 3, hidden, hidden, d_w, w_next, "f32", "f32", momentum_out=momentum, mu=0.95, nesterov=True, residual=w_qkv,
                    alpha=-0.02, beta=0.999)

# ---------------------------------------------------------------- an image student: 1 x 1 x 1 convolution, group norm
n, side, c_in, c_out, groups = 2, 12, 16, 32, 8
P = side ** 3
u, w_conv, gamma, beta = rand(n, P, c_in), rand(c_out, c_in, scale=0.25), 1 + rand(c_out, scale=0.1), rand(c_out, scale=0.1)
d_y = rand(n, P, c_out)                          # from the layers above
z, y, mean, rstd = new(n, P, c_out), new(n, P, c_out), new(n, groups), new(n, groups)
fa.fa_product(work, n * P, c_out, c_in, u, c_in, w_conv, c_in, z, c_out, "f32", "f32", trans_b=True)
fa.fa_group_norm(work, n, P, c_out, groups, z, y, "f32", gamma, beta, "f32", act="silu", mean=mean, rstd=rstd)
d_z, d_gamma, d_beta, d_conv, d_u = new(n, P, c_out), new(c_out), new(c_out), new(c_out, c_in), new(n, P, c_in)
fa.fa_group_norm_backward(work, n, P, c_out, groups, z, d_y, d_z, "f32", gamma, beta, "f32", mean, rstd, act="silu", d_gamma=d_gamma,
                          d_beta=d_beta)
fa.fa_product_backward(work, n * P, c_out, c_in, u, c_in, w_conv, c_in, d_z, c_out, d_u, c_in, d_conv, c_in, "f32", "f32", "f32",
                       trans_b=True)
conv_next = new(c_out, c_in)
fa.fa_orthogonalise(work, 1, c_out, c_in, d_conv, conv_next, "f32", "f32", residual=w_conv, alpha=-0.02)

# ---------------------------------------------------------------- the clients' mean as the update
# three clients' deltas of two keys, averaged; the mean of the first key steps the server's matrix
layout, deltas = [("w", c_out * c_in), ("b", c_out)], [rand(c_out * c_in + c_out, scale=1e-3) for _ in range(3)]
ctx = fa.fa_open(layout, "f32", "f32", 3)
outs = [new(numel) for _, numel in layout]
for j, delta in enumerate(deltas):
    fa.fa_accumulate(ctx, j, [100.0, 200.0, 300.0][j], fa.FA_KEY_FLAT, 0, delta, delta.numel(), torch.cuda.current_stream())
fa.fa_finalize(ctx, outs, torch.cuda.current_stream())
server_next = new(c_out, c_in)
fa.fa_orthogonalise(work, 1, c_out, c_in, outs[0], server_next, "f32", "f32", residual=w_conv, alpha=0.02)
fa.fa_sync(ctx)
fa.fa_close(ctx)
fa.fa_work_sync(work)
fa.fa_work_close(work)
print("loss", loss.sum().item())
