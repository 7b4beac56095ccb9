"""A server's distillation step, run as written by the GPU tests: an aggregated adapter is
merged into its frozen layer, the student's layer and head are applied to a public batch,
the clients' top logits give the loss and its gradient, and the head is updated."""
import torch
import server_side_fedavg_gb300 as fa

tokens, hidden, vocab, rank, topk, clients = 512, 1024, 32000, 16, 32, 8
bf16, dev = torch.bfloat16, "cuda"
g = torch.Generator(device=dev).manual_seed(7)
rand = lambda *s, scale=1.0: (torch.randn(s, generator=g, device=dev) * scale).to(bf16)  # noqa: E731

work = fa.fa_work_open()

# W += 2 B A: B [hidden, rank] and A [rank, hidden] as fa_reduce_subsets averaged them
layer, lora_b, lora_a = rand(hidden, hidden, scale=0.03), rand(hidden, rank, scale=0.1), rand(rank, hidden, scale=0.1)
fa.fa_product(work, hidden, hidden, rank, lora_b, rank, lora_a, hidden, layer, hidden, "bf16", "bf16",
              alpha=2.0, residual=layer, ldr=hidden)

# the student on the public batch: h = x + silu(x W^T), logits = h H^T
x, head = rand(tokens, hidden), rand(vocab, hidden, scale=0.03)
h, logits = torch.empty_like(x), torch.empty((tokens, vocab), device=dev, dtype=bf16)
fa.fa_product(work, tokens, hidden, hidden, x, hidden, layer, hidden, h, hidden, "bf16", "bf16", trans_b=True,
              act="silu", residual=x, ldr=hidden)
fa.fa_product(work, tokens, vocab, hidden, h, hidden, head, hidden, logits, vocab, "bf16", "bf16", trans_b=True)

# what the clients sent for it: their top logits, and their sample counts as weights
index = [torch.rand((tokens, vocab), generator=g, device=dev).topk(topk).indices.int() for _ in range(clients)]
value = [torch.randn((tokens, topk), generator=g, device=dev) * 2 for _ in range(clients)]
lists = fa.distill_lists(index, value, [topk] * clients, [100.0 + 50 * j for j in range(clients)])
weight = torch.full((tokens,), 1.0 / tokens, device=dev)      # 0 in padded rows

losses, lr = [], 0.05
loss, d_h = torch.empty(tokens, device=dev), torch.empty_like(h)
for _ in range(3):
    fa.fa_product(work, tokens, vocab, hidden, h, hidden, head, hidden, logits, vocab, "bf16", "bf16", trans_b=True)
    # the gradient takes the logits' place
    fa.fa_distill_grad(work, tokens, vocab, logits, vocab, "bf16", lists, 2.0, weight, None, loss, logits, vocab)
    # the gradient of h, for the layers below, and the head's step: H -= lr dlogits^T h
    fa.fa_product_backward(work, tokens, vocab, hidden, h, hidden, head, hidden, logits, vocab, d_h, hidden, None, hidden,
                           "bf16", "bf16", "bf16", trans_b=True)
    fa.fa_product(work, vocab, hidden, tokens, logits, vocab, h, hidden, head, hidden, "bf16", "bf16", trans_a=True,
                  alpha=-lr, residual=head, ldr=hidden)
    losses.append(loss.sum().item())
fa.fa_work_sync(work)
print("losses", losses)
fa.fa_work_close(work)
