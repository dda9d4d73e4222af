"""A small language model whose training step keeps its activations in 8 bits: one
residual layer between a tied embedding and head, in FP32.

    x = E[ids]                              embedding
    y = rms_norm(x)                         rms_norm_8bit: y for the product, y and x kept
    z = y W^T                               sgemm
    t = x + z,  h = rms_norm(t)             rms_norm_8bit with the residual: t kept
    loss = mean cross entropy of h E^T      linear_cross_entropy (no logits in memory)

Between the two passes there are h (the loss reads it again), codes and scales of x, y and
t, and each row's 1 / rms; x, y and t themselves are gone.  The backward pass reads the
8-bit forms: rms_norm_backward the norms' inputs, with the gradient that goes past the
norm added on the way, and linear_weight_grad_8bit the layer's input.

The data: each token is followed by one fixed other token.

    python examples/kept_step.py --steps 60
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))
import dense_fp32_gemm_07_gb300 as b2g  # noqa: E402

EPS = 1e-5


def parameters(vocab, width, seed=0, device="cuda"):
    """Embedding (and head), layer, and the two norms' weights."""
    g = torch.Generator().manual_seed(seed)
    p = {"embed": torch.randn(vocab, width, generator=g) * width ** -0.5,
         "layer": torch.randn(width, width, generator=g) * width ** -0.5,
         "norm1": torch.ones(width), "norm2": torch.ones(width)}
    return {name: t.to(device) for name, t in p.items()}


def batch(vocab, tokens, seed, device="cuda"):
    """`tokens` ids and the ids that follow them."""
    follows = torch.randperm(vocab, generator=torch.Generator().manual_seed(1))
    ids = torch.randint(vocab, (tokens,), generator=torch.Generator().manual_seed(seed))
    return ids.to(device), follows[ids].to(device)


def forward(p, ids, target):
    """(loss of each token, what the backward pass reads)."""
    x = b2g.embedding(ids, p["embed"])
    y, _, rstd1, y8, x8 = b2g.rms_norm_8bit(x, p["norm1"], eps=EPS, with_y=True, keep_total=True)
    z = b2g.sgemm(y, p["layer"], torch.empty_like(x), transB=True)
    h, _, rstd2, _, t8 = b2g.rms_norm_8bit(z, p["norm2"], residual=x, eps=EPS, with_y=True,
                                           keep_total=True)
    loss, lse = b2g.linear_cross_entropy(h, p["embed"], target)
    return loss, dict(h=h, lse=lse, y8=y8, x8=x8, t8=t8, rstd1=rstd1, rstd2=rstd2)


def backward(p, ids, target, kept):
    """Gradients of the mean loss by name."""
    n = ids.numel()
    each = torch.full((n,), 1.0 / n, device=ids.device)
    dh, dembed = b2g.linear_cross_entropy_backward(kept["h"], p["embed"], target, kept["lse"], each)
    dt, dnorm2 = b2g.rms_norm_backward(dh, kept["t8"], p["norm2"], kept["rstd2"])
    dlayer = b2g.linear_weight_grad_8bit(dt, *kept["y8"])
    dy = b2g.sgemm(dt, p["layer"], torch.empty_like(dt))
    # past the layer, x is the residual: its gradient there is added to that through the norm
    dx, dnorm1 = b2g.rms_norm_backward(dy, kept["x8"], p["norm1"], kept["rstd1"], dtotal=dt)
    b2g.embedding_backward(ids, dx, p["embed"].shape[0], out=dembed, accumulate=True)
    return {"embed": dembed, "layer": dlayer, "norm1": dnorm1, "norm2": dnorm2}


def train(vocab=1000, width=256, tokens=2048, steps=60, rate=2.0, max_norm=1.0, report=None):
    """The mean loss of each step."""
    p = parameters(vocab, width)
    losses = []
    for i in range(steps):
        ids, target = batch(vocab, tokens, seed=2 + i)
        loss, kept = forward(p, ids, target)
        grads = backward(p, ids, target, kept)
        norm = b2g.clip_grad_norm(list(grads.values()), max_norm)
        for name, g in grads.items():
            p[name].sub_(g, alpha=rate)
        losses.append(loss.mean())
        if report:
            report(i, float(losses[-1]), float(norm))
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
