"""Train a small next-token model whose unit keeps its activations in 8 bits.

    python examples/unit_saved8.py [--steps 100]

One flat parameter holds the embedding, a gated feed-forward layer and the output
layer.  Every step goes round as a rank's does: the optimizer's INT8 payload is
"gathered", the tokens' rows are read straight from it, the matrices are views of
the restored flat parameter; the feed-forward layer keeps 8-bit checkpoints of
its input, its gate and its other factor; the backward pass takes the gradients
from those and writes them, and the embedding's by sorted tokens, into the flat
gradient; the fused AdamW step updates the fp32 master and writes the next
payload.  The host waits for nothing inside a step.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fsdp_sharded_mixed_flatparameter_amd as zf  # noqa: E402

VOCAB, DIM, HIDDEN = 1000, 128, 320
SHAPES = [(VOCAB, DIM), (2 * HIDDEN, DIM), (DIM, HIDDEN), (VOCAB, DIM)]
HP = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, max_grad_norm=1.0)


class Unit:
    """The parameters, the unit's buffers for `tokens` tokens, and its passes."""

    def __init__(self, tokens, seed=0, loss_scale=2.0 ** 10):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.layout = zf.zero_flat_layout([math.prod(s) for s in SHAPES], 1, align=256)
        n = self.layout["shard"]
        master = torch.zeros(n, device="cuda")
        for w in zf.unflatten(master, SHAPES):
            w.copy_(torch.randn(w.shape, generator=gen, device="cuda") / math.sqrt(w.shape[1]))
        self.opt = zf.ShardOptimizer(master, HP, loss_scale=loss_scale, dynamic=True, quant_block=256)
        self.flat = master.to(torch.bfloat16)                 # the slot, then the gathered flat parameter
        self.codes = torch.empty(n, dtype=torch.int8, device="cuda")
        self.scales = torch.empty(-(-n // 256), device="cuda")
        zf.zero_quant_allgather_slot(self.flat, self.codes, self.scales)
        self.grad = torch.zeros(n, device="cuda")
        self.grads = zf.unflatten(self.grad, SHAPES)
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.x, self.dx = torch.empty(tokens, DIM, **bf16), torch.empty(tokens, DIM, **bf16)
        self.h = torch.empty(tokens, HIDDEN, **bf16)
        self.both = torch.empty(tokens, 2 * HIDDEN, **bf16)   # the gradients of gate and up, side by side
        self.saved = {k: zf.Saved8(tokens, c) for k, c in
                      (("x", DIM), ("gate", HIDDEN), ("up", HIDDEN), ("h", HIDDEN), ("y", DIM))}

    def gather(self):
        """The payload restored; the matrices are views of it, and the embedding is
        not needed: its rows are read from the payload."""
        n = self.layout["shard"]
        zf.zero_dequant_allgather(self.codes, self.scales, 1, n, self.flat)
        self.weights = zf.unflatten(self.flat, SHAPES)

    def forward(self, tokens):
        """The logits (fp32) of each token's successor."""
        s, (_, inner, outer, head) = self.saved, self.weights
        zf.zero_embed_lookup_int8(tokens, self.codes, self.scales, 1, self.layout["shard"], 0, VOCAB, self.x,
                                  scale=math.sqrt(DIM))
        zf.zero_act_save8(self.x, s["x"])
        packed = self.x @ inner.t()
        zf.zero_act_forward8(zf.ZERO_SILU, packed[:, :HIDDEN], self.h, s["gate"], up=packed[:, HIDDEN:],
                             saved_up=s["up"])
        y = self.x + self.h @ outer.t()
        zf.zero_act_save8(y, s["y"])
        return (y @ head.t()).float()

    def backward(self, tokens, dlogits):
        """The gradients of a forward pass into the flat gradient, from dlogits."""
        s, (_, inner, outer, head) = self.saved, self.weights
        d = dlogits.to(torch.bfloat16)
        zf.zero_weight_grad8(d, s["y"], self.grads[3])
        dy = d @ head
        dh = dy @ outer
        zf.zero_act_backward8(zf.ZERO_SILU, dh, s["gate"], self.both[:, :HIDDEN], saved_up=s["up"],
                              dup=self.both[:, HIDDEN:], again=s["h"])
        zf.zero_weight_grad8(dy, s["h"], self.grads[2])
        zf.zero_weight_grad8(self.both, s["x"], self.grads[1])
        torch.add(dy, self.both @ inner, out=self.dx)
        zf.zero_embed_grad(tokens, self.dx, self.grads[0], scale=math.sqrt(DIM))

    def step(self):
        self.opt.step_from_reduced(self.grad, self.flat, 0, q_buf=self.codes, q_scales=self.scales)


def loss_and_gradient(logits, targets, scale):
    """The mean cross-entropy and the gradient of scale times it."""
    lse = torch.logsumexp(logits, 1)
    loss = (lse - logits.gather(1, targets[:, None])[:, 0]).mean()
    p = torch.exp(logits - lse[:, None])
    p.scatter_add_(1, targets[:, None], torch.full_like(p[:, :1], -1.0))
    return loss, p * (scale / logits.shape[0])


def train(steps=100, batch=64, length=32, seed=0):
    """Returns the losses (a list of floats) and the unit."""
    unit = Unit(batch * length, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    losses = []
    for _ in range(steps):
        # every token has one successor; a sequence begins anywhere, frequent tokens first
        first = (torch.rand(batch, generator=gen, device="cuda") ** 3 * VOCAB).long()
        tokens = (first[:, None] + 7 * torch.arange(length + 1, device="cuda")) % VOCAB
        inputs, targets = tokens[:, :-1].reshape(-1), tokens[:, 1:].reshape(-1)
        unit.gather()
        loss, d = loss_and_gradient(unit.forward(inputs), targets, unit.opt.state.field("loss_scale"))
        unit.backward(inputs, d)
        unit.step()
        losses.append(loss)
    return [float(v) for v in losses], unit


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=100)
    args = ap.parse_args()
    losses, unit = train(args.steps)
    st = unit.opt.state.read()
    kept = sum(s.codes.numel() + s.exponents.numel() for s in unit.saved.values())
    print("loss %.4f -> %.4f in %d steps, %d applied, gradient norm %.3f, loss scale %g; %d bytes of activations kept"
          % (losses[0], losses[-1], len(losses), st.step, st.last_norm, st.loss_scale, kept))
