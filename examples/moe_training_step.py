"""A mixture-of-experts layer trained on one GPU with the library's operators:

    python examples/moe_training_step.py [--steps 30]

The model maps each token to a vector, y = W2_e relu(W1_e E[token]), with e the
token's expert, and learns a table of random targets.  One step is

  sort_ids           the batch's positions by expert, and where each expert starts
  embedding_lookup   the tokens' rows of E, in that order
  expert_matmul      up and down projections; on the way back the input gradients
  expert_weight_grad into the flat gradient buffer of the owner step
  embedding_grad     into the flat gradient of the AdamW tail
  grad_clip          both buffers by their common norm, in place
  muon_owner_step_apply on the experts' matrices, adamw_tail_step on E

All buffers are made once, and a step neither allocates nor waits for the GPU.
(Squared error, relu and the router, which looks a token's expert up, are torch.)
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from matrix_optimizers_under_gb300 import binding as m  # noqa: E402


class MoeLayer:
    def __init__(self, vocab=2000, dim=256, hidden=512, experts=8, batch=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.dim, self.hidden, self.experts, self.batch = vocab, dim, hidden, experts, batch

        def new(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device="cuda")

        # the matrices of the owner step: E up projections, then E down projections, one flat buffer
        size = dim * hidden
        table = [(i, hidden, dim) for i in range(experts)] + [(experts + i, dim, hidden) for i in range(experts)]
        self.shards = [m.make_shard(i * size, rows, cols, i) for i, rows, cols in table]
        self.weights = torch.randn(2 * experts * size, generator=g, device="cuda") * dim ** -0.5
        self.weights_bf16 = self.weights.bfloat16()           # what the products read
        self.grads = torch.zeros_like(self.weights)
        self.momentum = torch.zeros_like(self.weights)

        def stacks(flat):
            return (flat[:experts * size].view(experts, hidden, dim), flat[experts * size:].view(experts, dim, hidden))

        self.w1, self.w2 = stacks(self.weights_bf16)
        self.dw1, self.dw2 = stacks(self.grads)
        # the AdamW tail: the embedding
        self.emb = torch.randn(vocab, dim, generator=g, device="cuda")
        self.demb, self.m1, self.m2 = (torch.zeros_like(self.emb) for _ in range(3))
        self.targets = torch.randn(vocab, dim, generator=g, device="cuda")
        self.expert_of = torch.randint(0, experts, (vocab,), generator=g, device="cuda")

        n = batch
        self.order, self.starts = new(n, dtype=torch.int32), new(experts + 1, dtype=torch.int32)
        self.x, self.dy, self.want = (new(n, dim, dtype=torch.bfloat16) for _ in range(3))
        self.z, self.a, self.dz = (new(n, hidden, dtype=torch.bfloat16) for _ in range(3))
        self.y, self.dx = new(n, dim), new(n, dim)
        self.norm = new(2)
        self.grad_set = m.grad_set([self.grads, self.demb.view(-1)])

        def scratch(size):
            return new(max(1, size), dtype=torch.uint8)

        self.sort_ws = scratch(m.sort_ids_workspace_bytes(n, experts))
        self.up_ws = scratch(m.expert_workspace_bytes(experts, hidden, dim, n))
        self.down_ws = scratch(m.expert_workspace_bytes(experts, dim, hidden, n))
        self.emb_ws = scratch(m.embedding_grad_workspace_bytes(n, vocab, dim))
        self.clip_ws = scratch(m.grad_clip_workspace_bytes(self.grad_set))
        self.muon_ws = scratch(m.muon_workspace_bytes(self.shards))
        self.steps = 0

    def gradients(self, ids):
        """Fills the gradient buffers for a batch of tokens; returns the loss (a device scalar)."""
        m.sort_ids(self.expert_of[ids], self.experts, self.order, self.starts, self.sort_ws)
        self.ids = ids[self.order]                            # tokens, expert by expert
        m.embedding_lookup(self.emb, self.ids, self.x)
        m.embedding_lookup(self.targets, self.ids, self.want)
        m.expert_matmul(self.x, self.w1, self.starts, self.z, self.up_ws)
        self.a.copy_(self.z).relu_()
        m.expert_matmul(self.a, self.w2, self.starts, self.y, self.down_ws)

        err = self.y - self.want
        self.dy.copy_(err * (2.0 / err.numel()))
        m.expert_weight_grad(self.dy, self.a, self.starts, self.dw2, self.down_ws)
        m.expert_matmul(self.dy, self.w2, self.starts, self.dz, self.down_ws, input_grad=True)
        self.dz.mul_(self.z > 0)
        m.expert_weight_grad(self.dz, self.x, self.starts, self.dw1, self.up_ws)
        m.expert_matmul(self.dz, self.w1, self.starts, self.dx, self.up_ws, input_grad=True)
        m.embedding_grad(self.dx, self.ids, self.demb, self.emb_ws)
        return err.square().mean()

    def step(self, ids, max_norm=1.0, lr=0.02, adam_lr=1e-2):
        loss = self.gradients(ids)
        m.grad_clip(self.grad_set, self.norm, self.clip_ws, max_norm=max_norm)
        self.steps += 1
        m.muon_owner_step_apply(self.shards, self.grads, self.momentum, None, self.weights, self.muon_ws, lr=lr)
        m.adamw_tail_step(self.emb.view(-1), self.demb.view(-1), self.m1.view(-1), self.m2.view(-1), lr=adam_lr,
                          beta1=0.9, beta2=0.95, eps=1e-8, wd=0.0, step=self.steps)
        self.weights_bf16.copy_(self.weights)
        return loss


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--batch", type=int, default=4096)
    args = ap.parse_args()
    layer = MoeLayer(batch=args.batch)
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, layer.vocab, (args.steps, args.batch), generator=g, device="cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    losses = [layer.step(ids[0])]
    start.record()
    for t in range(1, args.steps):
        losses.append(layer.step(ids[t]))
    end.record()
    end.synchronize()
    for ws in (layer.up_ws, layer.down_ws, layer.emb_ws):
        assert m.op_device_status(ws)[0] == 0
    for t, loss in enumerate(losses):
        if t % 5 == 0 or t == args.steps - 1:
            print(f"step {t:3d}  loss {float(loss):.4f}")
    print(f"gradient norm {float(layer.norm[0]):.4f}, clipped by {float(layer.norm[1]):.4f}; "
          f"{start.elapsed_time(end) / max(1, args.steps - 1):.3f} ms a step")


if __name__ == "__main__":
    main()
