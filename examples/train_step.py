"""A small language model trained with the library alone: one residual layer
between a tied embedding and head, in FP32.

    x = E[ids]                          embedding
    a = layer_norm(x)                   layer_norm
    y = x + a W                         sgemm with beta = 1
    h = layer_norm(y)                   layer_norm
    loss = mean cross entropy of h E^T  linear_cross_entropy (no logits in memory)

and back: linear_cross_entropy_backward, layer_norm_backward and two transposed
sgemm calls; embedding_backward adds the lookup's gradient to the head's, which
share E; clip_grad_norm scales all gradients by their common norm.  torch holds
the memory and takes the plain gradient step.

The data: each token is followed by one fixed other token.

    python examples/train_step.py --steps 60
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))
import dense_fp32_gemm_07_gb300 as b2g  # noqa: E402

EPS = 1e-5


def parameters(vocab, width, seed=0, device="cuda"):
    """Embedding (and head), layer, and the two norms' weights and biases."""
    g = torch.Generator().manual_seed(seed)
    p = {"embed": torch.randn(vocab, width, generator=g) * width ** -0.5,
         "layer": torch.randn(width, width, generator=g) * width ** -0.5}
    for n in ("norm1", "norm2"):
        p[n + ".weight"], p[n + ".bias"] = torch.ones(width), torch.zeros(width)
    return {name: t.to(device) for name, t in p.items()}


def batch(vocab, tokens, seed, device="cuda"):
    """`tokens` ids and the ids that follow them."""
    follows = torch.randperm(vocab, generator=torch.Generator().manual_seed(1))
    ids = torch.randint(vocab, (tokens,), generator=torch.Generator().manual_seed(seed))
    return ids.to(device), follows[ids].to(device)


def step(p, ids, target, max_norm):
    """(mean loss, gradients by name, their norm before clipping) of one batch."""
    n = ids.numel()
    x = b2g.embedding(ids, p["embed"])
    a, mean1, rstd1 = b2g.layer_norm(x, p["norm1.weight"], p["norm1.bias"], EPS)
    y = b2g.sgemm(a, p["layer"], x.clone(), beta=1.0)
    h, mean2, rstd2 = b2g.layer_norm(y, p["norm2.weight"], p["norm2.bias"], EPS)
    loss, lse = b2g.linear_cross_entropy(h, p["embed"], target)

    each = torch.full((n,), 1.0 / n, device=ids.device)
    dh, dembed = b2g.linear_cross_entropy_backward(h, p["embed"], target, lse, each)
    dy, dw2, db2 = b2g.layer_norm_backward(dh, y, p["norm2.weight"], mean2, rstd2)
    dlayer = b2g.sgemm(a, dy, torch.empty_like(p["layer"]), transA=True)
    da = b2g.sgemm(dy, p["layer"], torch.empty_like(dy), transB=True)
    dx, dw1, db1 = b2g.layer_norm_backward(da, x, p["norm1.weight"], mean1, rstd1)
    for part in (dx, dy):  # through the layer, and past it
        b2g.embedding_backward(ids, part, p["embed"].shape[0], out=dembed, accumulate=True)

    grads = {"embed": dembed, "layer": dlayer, "norm1.weight": dw1, "norm1.bias": db1,
             "norm2.weight": dw2, "norm2.bias": db2}
    norm = b2g.clip_grad_norm(list(grads.values()), max_norm)
    return loss.mean(), grads, norm


def train(vocab=1000, width=256, tokens=2048, steps=60, rate=2.0, max_norm=1.0, report=None):
    """The mean loss of each step."""
    p = parameters(vocab, width)
    losses = []
    for i in range(steps):
        ids, target = batch(vocab, tokens, seed=2 + i)
        loss, grads, norm = step(p, ids, target, max_norm)
        for name, g in grads.items():
            p[name].sub_(g, alpha=rate)
        losses.append(loss)
        if report:
            report(i, float(loss), float(norm))
    rc, bits = b2g.b2g_status()
    if rc:
        raise b2g.B2GError(rc)
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("vocab", 1000), ("width", 256), ("tokens", 2048), ("steps", 60)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    train(a.vocab, a.width, a.tokens, a.steps,
          report=lambda i, loss, norm: print(f"step {i:4d}  loss {loss:.4f}  norm {norm:.4f}"))


if __name__ == "__main__":
    main()
