"""The training-step operators beside the SGEMM, as cases that can be timed and compared.

Layer norm, embedding lookup, softmax cross entropy of a linear layer and
gradient clipping are what a training or scoring step runs around its matrix
products.  Each case below is one pass through one of them as a program makes
it.  ``run`` computes it in a plain form (elementary torch operations, in 32
bits, rounded once at the end) or, where ``own`` is true, through the package's
entry points; ``exact`` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5         # layer norm
IGNORE = -100      # cross entropy: rows with this target carry no loss and no gradient
SKIP = 3072        # a drawn size never takes this value


def listed():
    return [
        # --- layer norm: y, mean and 1/std of each row; backward dx, dweight, dbias
        # one token of a decoding step: launch latency is all there is
        dict(name="norm 1 token", op="layer_norm", mode="forward", rows=1, cols=4096, dtype="bf16"),
        # one layer's norm in a training step, both directions
        dict(name="norm train 8192x4096", op="layer_norm", mode="train", rows=8192, cols=4096,
             dtype="bf16"),
        # odd width (rows at every alignment) in the SGEMM's own type
        dict(name="norm train ragged f32", op="layer_norm", mode="train", rows=1000, cols=1025,
             dtype="f32"),
        # --- embedding lookup, scaled; its gradient, one dense table
        # sixteen sequences, one new token each
        dict(name="embed 16 tokens", op="embedding", mode="forward", tokens=16, vocab=32768,
             width=4096, dtype="bf16"),
        # a small training batch on a mid-sized table with an odd number of rows
        dict(name="embed train f32", op="embedding", mode="train", tokens=4095, vocab=50001,
             width=512, dtype="f32"),
        # a large training batch; frequent tokens make segments of thousands of rows
        dict(name="embed train large", op="embedding", mode="train", tokens=32768, vocab=131072,
             width=4096, dtype="bf16"),
        # --- softmax cross entropy of h w^T: loss and log-sum-exp; backward dh, dw
        # scoring sixteen positions (one new token of sixteen sequences): reads the head once
        dict(name="xent score 16", op="linear_cross_entropy", mode="forward", tokens=16,
             vocab=32768, width=4096, dtype="bf16"),
        # small training batch, odd sizes everywhere, FP32
        dict(name="xent train ragged f32", op="linear_cross_entropy", mode="train", tokens=1000,
             vocab=11007, width=777, dtype="f32"),
        # an ordinary training batch
        dict(name="xent train 2048", op="linear_cross_entropy", mode="train", tokens=2048,
             vocab=32768, width=2048, dtype="bf16"),
        # a large training batch on a large vocabulary
        dict(name="xent train 8192", op="linear_cross_entropy", mode="train", tokens=8192,
             vocab=131072, width=4096, dtype="bf16"),
        # --- global gradient norm and clipping of a list of tensors
        # a small model's gradients as views of one flat buffer, odd sizes
        dict(name="clip small f32", op="clip_grad_norm", layers=4, width=129, vocab=1025, flat=True,
             dtype="f32"),
        # a mid-sized model's gradients, one tensor each
        dict(name="clip large bf16", op="clip_grad_norm", layers=12, width=2048, vocab=65536,
             flat=False, dtype="bf16"),
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number of [lo, hi], its logarithm uniform, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = max(lo, min(hi, max(step, v // step * step)))
    return v + step if v == SKIP else v


def draw(rng):
    op = rng.choice(["layer_norm", "embedding", "linear_cross_entropy", "clip_grad_norm"])
    dtype = rng.choice(["bf16", "f32"])
    step = rng.choice([1, 8, 8, 64])
    if op == "layer_norm":
        return dict(op=op, mode=rng.choice(["forward", "train"]), rows=_spread(rng, 1, 16384),
                    cols=_spread(rng, 64, 8192, step), dtype=dtype)
    if op == "embedding":
        return dict(op=op, mode=rng.choice(["forward", "train"]), tokens=_spread(rng, 1, 32768),
                    vocab=_spread(rng, 1024, 131072), width=_spread(rng, 64, 4096, step),
                    dtype=dtype)
    if op == "linear_cross_entropy":
        mode = rng.choice(["forward", "train"])
        most = 2 ** 42 if dtype == "bf16" else 2 ** 37
        while True:
            c = dict(op=op, mode=mode, tokens=_spread(rng, 1, 8192),
                     vocab=_spread(rng, 1024, 131072), width=_spread(rng, 128, 4096, step),
                     dtype=dtype)
            if c["tokens"] * c["vocab"] * c["width"] <= most:
                return c
    return dict(op=op, layers=rng.randint(1, 14), width=_spread(rng, 64, 2048, step),
                vocab=_spread(rng, 1024, 65536), flat=rng.random() < 0.5, dtype=dtype)


def _parameter_shapes(case):
    """The tensors of a small transformer's layers, ending with its embedding."""
    w = case["width"]
    per_layer = [(w,), (w,), (w, 4 * w), (4 * w, w)]
    return per_layer * case["layers"] + [(case["vocab"], w)]


def _token_ids(gen, tokens, vocab, dev):
    """Ids whose frequency falls like 1 / rank, as words' does."""
    u = torch.rand(tokens, generator=gen, device=dev, dtype=torch.float64)
    return (torch.exp(u * math.log(vocab)).long() - 1).clamp_(0, vocab - 1)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        x = torch.randn(*shape, generator=gen, device=dev)
        return x.mul_(std).add_(mean).to(dt)

    s = {"case": case}
    if case["op"] == "layer_norm":
        r, c = case["rows"], case["cols"]
        s["x"] = normal(r, c, std=1.5, mean=0.3)
        s["weight"], s["bias"] = normal(c, std=0.2, mean=1.0), normal(c, std=0.1)
        if case["mode"] == "train":
            s["dy"] = normal(r, c, std=0.01)
    elif case["op"] == "embedding":
        n, v, d = case["tokens"], case["vocab"], case["width"]
        s["ids"] = _token_ids(gen, n, v, dev)
        s["table"] = normal(v, d, std=0.02)
        s["scale"] = math.sqrt(d)
        if case["mode"] == "train":
            s["dout"] = normal(n, d, std=0.01)
    elif case["op"] == "linear_cross_entropy":
        n, v, d = case["tokens"], case["vocab"], case["width"]
        w = torch.randn(v, d, generator=gen, device=dev).mul_(0.02)
        target = _token_ids(gen, n, v, dev)
        # normalised hidden states; about half of the tokens are predicted well
        h = torch.randn(n, d, generator=gen, device=dev)
        known = (torch.rand(n, 1, generator=gen, device=dev) < 0.5).float()
        h += known * w[target] * (7.0 / (0.0004 * d))
        ignored = torch.rand(n, generator=gen, device=dev) < 0.05
        s["target"] = torch.where(ignored, torch.full_like(target, IGNORE), target)
        s["h"], s["w"] = h.to(dt), w.to(dt)
        if case["mode"] == "train":  # the mean over the rows that count
            valid = (s["target"] != IGNORE).sum().clamp(min=1).float()
            s["grad_loss"] = torch.ones(n, device=dev) / valid
    else:
        shapes = _parameter_shapes(case)
        if case["flat"]:
            flat = normal(sum(math.prod(x) for x in shapes), std=1e-3)
            s["grads"] = [x.view(y) for x, y in zip(flat.split([math.prod(y) for y in shapes]), shapes)]
        else:
            s["grads"] = [normal(*x, std=1e-3) for x in shapes]
        s["out"] = [torch.empty_like(x) for x in s["grads"]]
        s["max_norm"] = 1.0 if sum(x.numel() for x in s["grads"]) > 1e6 else 0.25
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import dense_fp32_gemm_07_gb300 as b2g

    case = s["case"]
    train = case.get("mode") == "train"
    if case["op"] == "layer_norm":
        y, mean, rstd = b2g.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
        out = {"y": y, "mean": mean, "rstd": rstd}
        if train:
            out["dx"], out["dweight"], out["dbias"] = b2g.layer_norm_backward(
                s["dy"], s["x"], s["weight"], mean, rstd)
        return out
    if case["op"] == "embedding":
        out = {"out": b2g.embedding(s["ids"], s["table"], scale=s["scale"])}
        if train:
            out["dtable"] = b2g.embedding_backward(s["ids"], s["dout"], case["vocab"],
                                                   scale=s["scale"])
        return out
    if case["op"] == "linear_cross_entropy":
        loss, lse = b2g.linear_cross_entropy(s["h"], s["w"], s["target"], ignore_index=IGNORE)
        out = {"loss": loss, "lse": lse}
        if train:
            out["dh"], out["dw"] = b2g.linear_cross_entropy_backward(
                s["h"], s["w"], s["target"], lse, s["grad_loss"], ignore_index=IGNORE)
        return out
    norm = b2g.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])
    return {"norm": norm, "grads": s["out"]}


def _run_plain(s):
    case = s["case"]
    train = case.get("mode") == "train"
    dt = DTYPES[case["dtype"]]
    if case["op"] == "layer_norm":
        x, w, b = s["x"].float(), s["weight"].float(), s["bias"].float()
        mean = x.mean(1)
        centred = x - mean[:, None]
        rstd = torch.rsqrt((centred * centred).mean(1) + EPS)
        xhat = centred * rstd[:, None]
        out = {"y": (xhat * w + b).to(dt), "mean": mean, "rstd": rstd}
        if train:
            dy = s["dy"].float()
            g = dy * w
            dx = (g - g.mean(1)[:, None] - xhat * (g * xhat).mean(1)[:, None]) * rstd[:, None]
            out["dx"] = dx.to(dt)
            out["dweight"], out["dbias"] = (dy * xhat).sum(0).to(dt), dy.sum(0).to(dt)
        return out
    if case["op"] == "embedding":
        out = {"out": (s["table"][s["ids"]].float() * s["scale"]).to(dt)}
        if train:
            d = torch.zeros(case["vocab"], case["width"], device=s["ids"].device)
            d.index_add_(0, s["ids"], s["dout"].float())
            out["dtable"] = (d * s["scale"]).to(dt)
        return out
    if case["op"] == "linear_cross_entropy":
        h, w, target = s["h"].float(), s["w"].float(), s["target"]
        valid = target != IGNORE
        at = torch.where(valid, target, torch.zeros_like(target))[:, None]
        z = h @ w.t()
        top = z.max(1, keepdim=True).values
        lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
        loss = torch.where(valid, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
        out = {"loss": loss, "lse": lse}
        if train:
            g = torch.where(valid, s["grad_loss"], torch.zeros_like(lse))[:, None]
            dz = torch.exp(z - lse[:, None]) * g
            dz.scatter_add_(1, at, -g)
            out["dh"], out["dw"] = (dz @ w).to(dt), (dz.t() @ h).to(dt)
        return out
    norm = torch.stack([(x.float() * x.float()).sum() for x in s["grads"]]).sum().sqrt()
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm, "grads": [(x.float() * coef).to(dt) for x in s["grads"]]}


# ------------------------------------------------------- the same in 64 bits

def exact(case, seed):
    if case["op"] == "linear_cross_entropy":
        passes = 3 if case["mode"] == "train" else 1
        if passes * 2 * case["tokens"] * case["vocab"] * case["width"] > 8e12:
            return None  # 64-bit products would take too long
    s = prepare(case, seed)
    train = case.get("mode") == "train"
    F = torch.nn.functional

    def leaf(x):
        return x.double().requires_grad_(train)

    if case["op"] == "layer_norm":
        x, w, b = leaf(s["x"]), leaf(s["weight"]), leaf(s["bias"])
        y = F.layer_norm(x, x.shape[1:], w, b, EPS)
        var, mean = torch.var_mean(x.detach(), 1, correction=0)
        out = {"y": y.detach(), "mean": mean, "rstd": 1 / torch.sqrt(var + EPS)}
        if train:
            y.backward(s["dy"].double())
            out.update(dx=x.grad, dweight=w.grad, dbias=b.grad)
        return out
    if case["op"] == "embedding":
        table = leaf(s["table"])
        y = F.embedding(s["ids"], table) * s["scale"]
        out = {"out": y.detach()}
        if train:
            y.backward(s["dout"].double())
            out["dtable"] = table.grad
        return out
    if case["op"] == "linear_cross_entropy":
        h, w = leaf(s["h"]), leaf(s["w"])
        z = F.linear(h, w)
        loss = F.cross_entropy(z, s["target"], ignore_index=IGNORE, reduction="none")
        out = {"loss": loss.detach(), "lse": torch.logsumexp(z.detach(), 1)}
        if train:
            loss.backward(s["grad_loss"].double())
            out.update(dh=h.grad, dw=w.grad)
        return out
    norm = torch.linalg.vector_norm(torch.cat([x.flatten().double() for x in s["grads"]]))
    coef = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    return {"norm": norm, "grads": [x.double() * coef for x in s["grads"]]}


# ------------------------------------- what a pass reads, writes and computes

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    train = case.get("mode") == "train"
    if case["op"] == "layer_norm":
        n, c = case["rows"] * case["cols"], case["cols"]
        b, f = 2 * n * es + 2 * c * es + 8 * case["rows"], 8 * n  # x; y, weight, bias, statistics
        if train:
            b, f = b + 2 * n * es + 2 * c * es, f + 14 * n        # dy; dx, dweight, dbias
        return {"bytes": b, "flops": f}
    if case["op"] == "embedding":
        n, v, d = case["tokens"], case["vocab"], case["width"]
        b, f = 8 * n + (min(n, v) + n) * d * es, n * d            # ids, rows; out
        if train:
            b, f = b + (n + v) * d * es, f + 2 * n * d            # dout; dtable
        return {"bytes": b, "flops": f}
    if case["op"] == "linear_cross_entropy":
        n, v, d = case["tokens"], case["vocab"], case["width"]
        b, f = (n + v) * d * es + 16 * n, 2 * n * v * d           # h, w, target; loss, lse
        if train:
            b, f = b + (n + v) * d * es + 4 * n, 3 * f            # grad_loss; dh, dw
        return {"bytes": b, "flops": f}
    n = sum(math.prod(x) for x in _parameter_shapes(case))
    return {"bytes": 2 * n * es + 4, "flops": 3 * n}
