"""Train a small MLP with the optimizer over a list of tensors.

    python examples/list_adamw.py [--state-bits 8] [--steps 200]

The fp16 parameters and their gradients are views of two packed buffers, as a
rank holds them after a gather and before a scatter.  Each step scales the loss
by the device's loss scale, and TensorListOptimizer takes the statistics of
every gradient (norm, overflow), clips, updates the fp32 master weights with
32-bit or 8-bit AdamW states and writes the fp16 parameters back.  The host
never waits inside a step.  Biases take no weight decay, the output layer half
the learning rate.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fsdp_sharded_mixed_flatparameter_amd as zf  # noqa: E402

SHAPES = [(61, 256), (256,), (256, 256), (256,), (256, 3), (3,)]


def train(state_bits=8, steps=200, batch=512, seed=0):
    """Returns the losses (a list of floats) and the optimizer."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    numels = [math.prod(s) for s in SHAPES]
    params = torch.zeros(sum(numels), dtype=torch.float16, device="cuda")
    grads = torch.zeros_like(params)
    masters = [torch.randn(n, generator=gen, device="cuda") / math.sqrt(s[0]) if len(s) == 2
               else torch.zeros(n, device="cuda") for n, s in zip(numels, SHAPES)]
    hp = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.01, max_grad_norm=1.0)
    opt = zf.TensorListOptimizer(masters, hp, state_bits=state_bits, loss_scale=2.0 ** 12, dynamic=True,
                                 lr_mult=[1.0] * 4 + [0.5] * 2, decay_mult=[1.0, 0.0] * 3,
                                 grad_dtype=torch.float16, param_dtype=torch.float16)
    # the parameters: views of the packed buffer, each with its gradient's view
    weights = zf.unflatten(params, SHAPES)
    for w, m, g in zip(weights, masters, zf.unflatten(grads, SHAPES)):
        w.copy_(m.view(w.shape))
        w.requires_grad_()
        w.grad = g
    opt.bind([w.grad for w in weights], [w.detach() for w in weights])

    x = torch.randn(batch, SHAPES[0][0], generator=gen, device="cuda")
    y = torch.stack((x[:, 0] * x[:, 1], x[:, 2].abs(), x[:, 3:8].sum(1) / 2), 1)
    x, losses = x.half(), []
    for _ in range(steps):
        h = x
        for w, b in zip(weights[::2], weights[1::2]):
            h = h @ w + b
            if w is not weights[-2]:
                h = torch.nn.functional.gelu(h)
        loss = (h.float() - y).square().mean()
        (loss * opt.state.field("loss_scale")).backward()      # adds into w.grad in place
        opt.step()
        grads.zero_()
        losses.append(loss.detach())
    return [float(v) for v in losses], opt


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    ap.add_argument("--steps", type=int, default=200)
    args = ap.parse_args()
    losses, opt = train(args.state_bits, args.steps)
    st = opt.state.read()
    print("loss %.4f -> %.4f in %d steps, %d applied, gradient norm %.3f, loss scale %g"
          % (losses[0], losses[-1], len(losses), st.step, st.last_norm, st.loss_scale))
    print("norm of each tensor's gradient:",
          " ".join("%.3g" % v for v in opt.plan.tensor_sumsq.sqrt().tolist()))
