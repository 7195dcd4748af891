"""Cases of the layers whose parameters the AdamW lane steps: the token
embedding, the LayerNorms and the output head with its loss, each with the
gradients that the lane reads.

Kinds of a case:

* lookup       out[t] = scale * table[token[t]]
* lookup_grad  dtable[v] = scale * sum of grad[t] over the tokens t that are v
* norm         y = (x - mean) / sqrt(var + eps) * weight + bias, with the
               statistics that a backward pass needs
* norm_grad    dx, dweight, dbias
* loss         softmax cross entropy of hidden . weight^T, per token
* loss_train   the loss and the gradients of hidden and weight

Sizes: GPT-2's embedding and head (vocabulary 50257, width 768), Llama-8B's
(128256, 4096), the MoE set's width (7168), and odd ones.
"""
import math

import torch

own = False

PAD = 0           # the padding token of the cases that have one
IGNORE = -100     # the target of a token that takes no part in the loss
EPS = 1e-5
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one decoding step of 16 sequences: fp32 master table, bf16 activations
        {"name": "lookup-16", "kind": "lookup", "tokens": 16, "vocab": 50257, "dim": 768, "table": "f32",
         "out": "bf16", "scale": 1.0},
        # a training batch of Llama-8B's embedding, scaled by sqrt(dim)
        {"name": "lookup-llama", "kind": "lookup", "tokens": 16384, "vocab": 128256, "dim": 4096, "table": "bf16",
         "out": "bf16", "scale": 64.0},
        # GPT-2's token embedding after one micro-batch of 8 x 1024 tokens
        {"name": "lookup-grad-gpt2", "kind": "lookup_grad", "tokens": 8192, "vocab": 50257, "dim": 768,
         "grad": "bf16", "out": "bf16", "scale": 1.0, "pad": False},
        # Llama-8B's, with padded sequences
        {"name": "lookup-grad-llama", "kind": "lookup_grad", "tokens": 16384, "vocab": 128256, "dim": 4096,
         "grad": "bf16", "out": "bf16", "scale": 64.0, "pad": True},
        # a small fp32 model with an odd width and vocabulary
        {"name": "lookup-grad-odd", "kind": "lookup_grad", "tokens": 1237, "vocab": 5003, "dim": 333,
         "grad": "f32", "out": "f32", "scale": 2.5, "pad": True},
        # a decoding step: few rows, latency counts
        {"name": "norm-16", "kind": "norm", "rows": 16, "dim": 4096, "x": "bf16", "weight": "bf16", "bias": True},
        # a training batch at Llama-8B's width
        {"name": "norm-16384", "kind": "norm", "rows": 16384, "dim": 4096, "x": "bf16", "weight": "f32",
         "bias": True},
        # GPT-2's LayerNorm backward, 16 x 1024 tokens, fp32 master parameters
        {"name": "norm-grad-gpt2", "kind": "norm_grad", "rows": 16384, "dim": 768, "x": "bf16", "weight": "f32",
         "bias": True},
        # fp32 activations, ragged rows and width, no bias
        {"name": "norm-grad-odd", "kind": "norm_grad", "rows": 4099, "dim": 1025, "x": "f32", "weight": "f32",
         "bias": False},
        # evaluation of a short prompt on a small vocabulary
        {"name": "loss-61", "kind": "loss", "tokens": 61, "vocab": 5003, "dim": 256, "masked": 0.0},
        # GPT-2's head on a micro-batch of 8 x 1024 tokens
        {"name": "loss-train-gpt2", "kind": "loss_train", "tokens": 8192, "vocab": 50257, "dim": 768, "masked": 0.0},
        # Llama-8B's head, an instruction-tuning batch: a quarter of the tokens are prompt
        {"name": "loss-train-llama", "kind": "loss_train", "tokens": 4096, "vocab": 128256, "dim": 4096,
         "masked": 0.25},
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    kind = rng.choice(["lookup", "lookup_grad", "norm", "norm_grad", "loss", "loss_train"])
    kinds = ["f32", "bf16"]
    if kind in ("lookup", "lookup_grad"):
        c = {"kind": kind, "tokens": _spread(rng, 16, 16384), "vocab": _spread(rng, 1000, 128256),
             "dim": _spread(rng, 333, 4096, rng.choice([1, 8, 64])), "out": rng.choice(kinds),
             "scale": rng.choice([1.0, 2.5, 64.0])}
        if kind == "lookup":
            return {**c, "table": rng.choice(kinds)}
        return {**c, "grad": rng.choice(kinds), "pad": rng.random() < 0.5}
    if kind in ("norm", "norm_grad"):
        dim = _spread(rng, 333, 7168, rng.choice([1, 8, 64]))
        return {"kind": kind, "rows": _spread(rng, 16, 16384), "dim": dim, "x": rng.choice(kinds),
                "weight": rng.choice(kinds), "bias": rng.random() < 0.7}
    # the head: any token count and vocabulary, a width in steps of 8 (16 bytes of bf16)
    return {"kind": kind, "tokens": _spread(rng, 61, 4096), "vocab": _spread(rng, 5003, 128256),
            "dim": _spread(rng, 256, 4096, 8), "masked": rng.choice([0.0, 0.0, 0.25, 0.6])}


def _tokens(case, g):
    """Token ids whose frequencies fall as a language's do (1 / rank), the
    ranks in a random order; with padding, about a tenth of the tokens."""
    n, v = case["tokens"], case["vocab"]
    # the quantile function of a density of 1 / (rank + 2.7)
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = (2.7 * ((v + 2.7) / 2.7) ** u - 2.7).long().clamp_(0, v - 1)
    ids = torch.randperm(v, generator=g, device="cuda")[rank]
    if case.get("pad"):
        ids[torch.rand(n, generator=g, device="cuda") < 0.1] = PAD
    return ids


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = case["kind"]

    def normal(*shape, to, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(to)

    if kind == "lookup":
        return {"case": case, "ids": _tokens(case, g),
                "table": normal(case["vocab"], case["dim"], to=_TYPES[case["table"]], scale=0.02)}
    if kind == "lookup_grad":
        return {"case": case, "ids": _tokens(case, g),
                "grad": normal(case["tokens"], case["dim"], to=_TYPES[case["grad"]], scale=1e-3)}
    if kind in ("norm", "norm_grad"):
        n, d = case["rows"], case["dim"]
        # activations with a mean of their own and some wide channels
        x = torch.randn((n, d), generator=g, device="cuda")
        x = x * (0.5 + torch.rand((1, d), generator=g, device="cuda") * 2) + 0.3
        wt = _TYPES[case["weight"]]
        s = {"case": case, "x": x.to(_TYPES[case["x"]]),
             "weight": (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(wt),
             "bias": normal(d, to=wt, scale=0.1) if case["bias"] else None}
        if kind == "norm_grad":
            # the forward pass has left its statistics
            x32 = s["x"].float()
            mean = x32.mean(1)
            s["mean"] = mean
            s["rstd"] = torch.rsqrt((x32 - mean[:, None]).square().mean(1) + EPS)
            s["grad"] = normal(n, d, to=s["x"].dtype, scale=1e-3)
        return s
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    weight = normal(v, d, to=torch.bfloat16, scale=0.02)
    targets = _tokens(case, g)
    # a trained model's hidden states lean towards their target's row
    h = torch.randn((n, d), generator=g, device="cuda")
    h += weight[targets].float() * (7.0 / (0.02 * 0.02 * d))
    if case["masked"]:
        # masked as prompts are: a run at the start of each stretch of 256 tokens
        at = torch.arange(n, device="cuda") % 256
        targets[at < int(256 * case["masked"])] = IGNORE
    count = (targets != IGNORE).sum().clamp(min=1)
    return {"case": case, "hidden": h.to(torch.bfloat16), "weight": weight, "targets": targets,
            "dloss": torch.ones(n, device="cuda") / count}


# ---- plain forms ---------------------------------------------------------------


def _plain_lookup(s):
    c = s["case"]
    return (s["table"][s["ids"]].float() * c["scale"]).to(_TYPES[c["out"]])


def _plain_lookup_grad(s):
    c = s["case"]
    g = s["grad"].float() * c["scale"]
    if c["pad"]:
        g = torch.where((s["ids"] == PAD)[:, None], torch.zeros_like(g), g)
    out = torch.zeros((c["vocab"], c["dim"]), device=g.device)
    return out.index_add_(0, s["ids"], g).to(_TYPES[c["out"]])


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = torch.rsqrt(xc.square().mean(1) + EPS)
    y = xc * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_grad(s):
    g, rstd = s["grad"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    q = g * s["weight"].float()
    dx = (q - q.mean(1, keepdim=True) - xh * (q * xh).mean(1, keepdim=True)) * rstd
    wt = s["weight"].dtype
    db = g.sum(0).to(wt) if s["bias"] is not None else None
    return [v for v in (dx.to(s["x"].dtype), (g * xh).sum(0).to(wt), db) if v is not None]


def _plain_logits(s):
    valid = s["targets"] != IGNORE
    logits = s["hidden"].float() @ s["weight"].float().T
    top = logits.max(1).values
    lse = top + (logits - top[:, None]).exp().sum(1).log()
    at = torch.where(valid, s["targets"], torch.zeros_like(s["targets"]))
    loss = lse - logits.gather(1, at[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return valid, at, logits, torch.where(valid, loss, zero), torch.where(valid, lse, zero)


def _plain_loss_train(s):
    valid, at, p, loss, lse = _plain_logits(s)
    p -= lse[:, None]
    p.exp_()
    p[torch.arange(p.shape[0], device=p.device), at] -= 1.0
    p *= torch.where(valid, s["dloss"], torch.zeros_like(lse))[:, None]
    dh = p @ s["weight"].float()
    dw = p.T @ s["hidden"].float()
    return loss, dh.to(s["hidden"].dtype), dw.to(s["weight"].dtype)


# ---- the framework's calls -------------------------------------------------------


def _own(s):
    import matrix_orthogonalizing_optimizer_step_b200 as mo
    c = s["case"]
    kind = c["kind"]
    if kind == "lookup":
        return mo.muon_embedding(s["ids"], s["table"], scale=c["scale"], out_dtype=_TYPES[c["out"]])
    if kind == "lookup_grad":
        return mo.muon_embedding_backward(s["ids"], s["grad"], c["vocab"], scale=c["scale"],
                                          padding_idx=PAD if c["pad"] else None, grad_dtype=_TYPES[c["out"]])
    if kind == "norm":
        return mo.muon_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
    if kind == "norm_grad":
        got = mo.muon_layer_norm_backward(s["grad"], s["x"], s["mean"], s["rstd"], s["weight"], bias=c["bias"])
        return [v for v in got if v is not None]
    loss, lse = mo.muon_head_loss(s["hidden"], s["weight"], s["targets"], ignore_index=IGNORE)
    if kind == "loss":
        return loss, lse
    dh, dw = mo.muon_head_loss_backward(s["hidden"], s["weight"], s["targets"], lse, s["dloss"],
                                        ignore_index=IGNORE)
    return loss, dh, dw


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "lookup":
        return _plain_lookup(state)
    if kind == "lookup_grad":
        return _plain_lookup_grad(state)
    if kind == "norm":
        return _plain_norm(state)
    if kind == "norm_grad":
        return _plain_norm_grad(state)
    if kind == "loss":
        return _plain_logits(state)[3:]
    return _plain_loss_train(state)


def work(case):
    kind, d = case["kind"], case["dim"]
    if kind in ("lookup", "lookup_grad"):
        n, v = case["tokens"], case["vocab"]
        # the tokens; then rows read once (at most the table's) and all rows written
        if kind == "lookup":
            return {"bytes": n * 8 + min(n, v) * d * _BYTES[case["table"]] + n * d * _BYTES[case["out"]],
                    "flops": n * d}
        return {"bytes": n * 8 + n * d * _BYTES[case["grad"]] + v * d * _BYTES[case["out"]], "flops": n * d}
    if kind in ("norm", "norm_grad"):
        n, e, w = case["rows"], _BYTES[case["x"]], _BYTES[case["weight"]]
        both = 2 if case["bias"] else 1
        if kind == "norm":
            return {"bytes": 2 * n * d * e + both * d * w + 8 * n, "flops": 8 * n * d}
        return {"bytes": 3 * n * d * e + (1 + both) * d * w + 8 * n, "flops": 14 * n * d}
    n, v = case["tokens"], case["vocab"]
    counted = n
    if case["masked"]:
        run_of = int(256 * case["masked"])
        counted = n - (n // 256) * run_of - min(n % 256, run_of)
    moved = n * d * 2 + v * d * 2 + n * 8
    if kind == "loss":
        return {"bytes": moved + 8 * n, "flops": 2 * counted * v * d}
    # logits, and the products that give the two gradients
    return {"bytes": 2 * moved + 4 * n, "flops": 6 * counted * v * d}


# ---- the definitions in 64 bits ----------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    kind = case["kind"]
    if kind == "lookup":
        return torch.index_select(s["table"].to(f64), 0, s["ids"]) * case["scale"]
    if kind == "lookup_grad":
        keep = s["ids"] != PAD if case["pad"] else torch.ones_like(s["ids"], dtype=torch.bool)
        total = torch.zeros((case["vocab"], case["dim"]), dtype=f64, device="cuda")
        total.index_add_(0, s["ids"][keep], s["grad"][keep].to(f64))
        return total * case["scale"]
    if kind in ("norm", "norm_grad"):
        x, w = s["x"].to(f64), s["weight"].to(f64)
        var, mean = torch.var_mean(x, dim=1, correction=0)
        sd = torch.sqrt(var + EPS)
        xh = (x - mean.unsqueeze(1)) / sd.unsqueeze(1)
        if kind == "norm":
            y = xh * w if s["bias"] is None else torch.addcmul(s["bias"].to(f64), xh, w)
            return y, mean, 1.0 / sd
        g = s["grad"].to(f64)
        d = x.shape[1]
        gw = g * w
        # the gradient through x, through the mean and through the variance
        dvar = (gw * (x - mean.unsqueeze(1))).sum(1) * -0.5 / sd ** 3
        dmean = -(gw.sum(1) / sd)
        dx = gw / sd.unsqueeze(1) + (dmean / d).unsqueeze(1) + dvar.unsqueeze(1) * 2 * (x - mean.unsqueeze(1)) / d
        out = [dx, torch.einsum("nd,nd->d", g, xh)]
        return out + [torch.einsum("nd->d", g)] if case["bias"] else out
    n = case["tokens"]
    w = s["weight"].to(f64)
    loss = torch.zeros(n, dtype=f64, device="cuda")
    lse = torch.zeros(n, dtype=f64, device="cuda")
    dh = torch.zeros((n, case["dim"]), dtype=f64, device="cuda")
    dw = torch.zeros_like(w) if kind == "loss_train" else None
    rows = torch.nonzero(s["targets"] != IGNORE)[:, 0]
    for part in torch.split(rows, 1024):
        h, y = s["hidden"][part].to(f64), s["targets"][part]
        z = h @ w.T
        norm = torch.logsumexp(z, 1)
        lse[part] = norm
        loss[part] = norm - z[torch.arange(len(part), device="cuda"), y]
        if dw is not None:
            q = torch.softmax(z, 1)
            q[torch.arange(len(part), device="cuda"), y] -= 1
            q *= s["dloss"][part].to(f64)[:, None]
            dh[part] = q @ w
            dw += q.T @ h
    return (loss, lse) if kind == "loss" else (loss, dh, dw)
