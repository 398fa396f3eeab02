"""Operators on the tied int8 embedding / LM-head matrix, measured: many-token int8 linear, embedding
lookup and its gradient, and the cross entropy over the vocabulary with its gradient.

The matrix is int8 codes W [V][d] with one fp32 scale per row.  `run` computes each operator either in plain
torch operations (own false) or through the framework's entry points (own true), on the same inputs.
Default sizes are those of the framework's 1.3B-shaped configuration (V = 50288, d = 2048, in_proj with 8512
rows); the others are generic.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decoded token's logits: 103 MB of codes read once, the latency of a serving step
        {"name": "linear-1-f32", "op": "linear", "m": 1, "v": 50288, "d": 2048, "type": "f32", "out": "f32", "norm": True},
        # a batch of 16 sequences decoded together, bf16 activations
        {"name": "linear-16-bf16", "op": "linear", "m": 16, "v": 50288, "d": 2048, "type": "bf16", "out": "f32", "norm": True},
        # an odd batch through a projection-sized matrix, rows and width that fill no tile
        {"name": "linear-333-odd", "op": "linear", "m": 333, "v": 8511, "d": 2032, "type": "f32", "out": "f32", "norm": False},
        # every logit of a 2048-token prompt, stored in bf16
        {"name": "linear-2048-bf16", "op": "linear", "m": 2048, "v": 50288, "d": 2048, "type": "bf16", "out": "bf16", "norm": True},
        # the embedding of a few sequences' next tokens
        {"name": "embed-16-f32", "op": "embed", "m": 16, "v": 50288, "d": 2048, "type": "f32"},
        # the embedding of a training batch
        {"name": "embed-16384-bf16", "op": "embed", "m": 16384, "v": 50288, "d": 2048, "type": "bf16"},
        # its gradient for a short batch over a small vocabulary (repeated tokens)
        {"name": "embed-grad-500-f32", "op": "embed_grad", "m": 500, "v": 8191, "d": 1040, "type": "f32"},
        # its gradient for a training batch: the dense [V][d] gradient is written once
        {"name": "embed-grad-16384-bf16", "op": "embed_grad", "m": 16384, "v": 50288, "d": 2048, "type": "bf16"},
        # scoring a handful of tokens (the answer of a multiple-choice question)
        {"name": "score-7-f32", "op": "score", "m": 7, "v": 50288, "d": 2048, "type": "f32", "norm": True},
        # scoring a 2048-token passage: perplexity, no gradient
        {"name": "score-2048-bf16", "op": "score", "m": 2048, "v": 50288, "d": 2048, "type": "bf16", "norm": True},
        # loss and gradients of a short, odd batch with ignored labels, fp32 activations
        {"name": "train-333-f32", "op": "train", "m": 333, "v": 20011, "d": 1040, "type": "f32", "norm": True},
        # loss and gradients of a 2048-token training batch
        {"name": "train-2048-bf16", "op": "train", "m": 2048, "v": 50288, "d": 2048, "type": "bf16", "norm": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "embed", "embed_grad", "score", "train"])
    c = {"op": op, "type": rng.choice(["f32", "bf16"]),
         "v": min(50288, _log(rng, 1000, 60000)), "d": 16 * _log(rng, 16, 128)}
    if op in ("embed", "embed_grad"):
        c["m"] = _log(rng, 1, 16384)
    else:
        c["m"] = _log(rng, 1, 2048)
        c["norm"] = rng.random() < 0.5
        if op == "linear":
            c["out"] = rng.choice(["f32", "bf16"])
    return c


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dev = "cuda"
    m, v, d = case["m"], case["v"], case["d"]
    t = TYPES[case["type"]]
    st = dict(case)
    st["W"] = torch.randint(-127, 128, (v, d), generator=g, device=dev, dtype=torch.int8)
    st["s_row"] = torch.rand(v, generator=g, device=dev) * 9e-4 + 1e-4
    if case["op"] in ("embed", "embed_grad"):
        # token frequencies fall off as in text: a few tokens make up much of a batch
        u = torch.rand(m, generator=g, device=dev, dtype=torch.float64)
        st["tokens"] = (torch.exp(u * math.log(v + 1.0)) - 1.0).long().clamp_(0, v - 1).int()
        if case["op"] == "embed_grad":
            st["dh"] = torch.randn(m, d, generator=g, device=dev).to(t)
    else:
        st["norm_w"] = torch.rand(d, generator=g, device=dev) + 0.5 if case["norm"] else None
        x = torch.randn(m, d, generator=g, device=dev)
        if case["op"] in ("score", "train"):
            # a trained model's tokens: the hidden state leans towards its label's row, by a varying amount
            y = torch.randint(0, v, (m,), generator=g, device=dev)
            lean = torch.rand(m, 1, generator=g, device=dev) * 0.35
            x = x + lean * st["W"][y].float() / 73.0
            y[torch.rand(m, generator=g, device=dev) < 0.08] = -1  # padding and prompt tokens: ignored
            st["labels"] = y.int()
            st["dloss"] = torch.full((m,), 1.0 / m, device=dev)
        st["x"] = x.to(t)
    if own:
        from bit_quantized_mamba_b200 import dfssm as D
        ops = {"linear": (D.OP_LINEAR_INT8,), "embed": (D.OP_EMBED_TOKENS,), "embed_grad": (D.OP_EMBED_BACKWARD,),
               "score": (D.OP_HEAD_LOSS,), "train": (D.OP_HEAD_LOSS, D.OP_HEAD_LOSS_BACKWARD)}[case["op"]]
        st["ws"] = [D.workspace(D.workspace_size(op, m, d, v)) for op in ops]
    return st


# ------------------------------------------------------------------------------------ plain forms


def _normed(x, norm_w):
    """fp32 rows, normalised when there is a weight: u = fl(fl(x r) w), r = fl(1 / sqrt(mean x^2 + eps))."""
    x = x.float()
    if norm_w is None:
        return x, None
    r = (1.0 / torch.sqrt(x.double().square().mean(1, keepdim=True) + EPS)).float()
    return x * r * norm_w, r


def _quantized(u):
    """int8 codes (as fp32) and scale of every row: s = fl(absmax / 127), q = rint(fl(u / s)) within +-127."""
    s = (u.abs().amax(1, keepdim=True).double() / 127.0).float()
    q = torch.where(s > 0, torch.round(u / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(u))
    return q.clamp(-127, 127), s


def _plain_linear(st):
    u, _ = _normed(st["x"], st["norm_w"])
    q, s = _quantized(u)
    return (q @ st["W"].float().t() * s * st["s_row"]).to(TYPES[st["out"]])


def _plain_embed(st):
    i = st["tokens"].long()
    return (st["W"][i].float() * st["s_row"][i, None]).to(TYPES[st["type"]])


def _plain_embed_grad(st):
    i, dh, W = st["tokens"].long(), st["dh"].float(), st["W"]
    dE = torch.zeros(W.shape, device=dh.device).index_add_(0, i, dh)
    ds = torch.zeros(W.shape[0], device=dh.device).index_add_(0, i, (dh * W[i].float()).sum(1))
    return {"dE": dE, "ds_row": ds}


def _plain_head(st, grad):
    W, s_row, y = st["W"].float(), st["s_row"], st["labels"].long()
    u, r = _normed(st["x"], st["norm_w"])
    q, s = _quantized(u)
    logits = q @ W.t() * s * s_row
    kept = y >= 0
    at = y.clamp(min=0)[:, None]
    ly = logits.gather(1, at)
    logits = logits.scatter(1, at, float("-inf"))           # the other rows of the vocabulary
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    others = top + torch.log(e.sum(1, keepdim=True))
    z = others - ly                                          # loss = log(1 + exp(z))
    loss = torch.where(kept, torch.nn.functional.softplus(z[:, 0], threshold=80.0), torch.zeros_like(s[:, 0]))
    if not grad:
        return {"loss": loss}
    g = torch.where(kept, st["dloss"], torch.zeros_like(loss))[:, None]
    lse = torch.logaddexp(others, ly)
    p = torch.exp(logits - lse)                              # zero at the label
    dl = (p.scatter(1, at, -torch.sigmoid(z))) * g           # p - 1 at the label, without cancellation
    out = {"loss": loss}
    acc_s = q @ W.t() * s
    out["ds_row"] = (dl * acc_s).sum(0)
    du = _long_product(dl * s_row, W)
    return out | _plain_norm_grad(st, u, r, du)


def _long_product(a, b):
    """a @ b over a long inner axis: products of pieces of 2048, then their sum (fp32 over the whole axis at
    once is about 1e-5 off)."""
    n = -(-a.shape[1] // 2048) * 2048
    a = torch.nn.functional.pad(a, (0, n - a.shape[1])).reshape(a.shape[0], -1, 2048).transpose(0, 1)
    b = torch.nn.functional.pad(b, (0, 0, 0, n - b.shape[0])).reshape(-1, 2048, b.shape[1])
    return torch.bmm(a, b).sum(0)


def _plain_norm_grad(st, u, r, du):
    t = TYPES[st["type"]]
    if r is None:
        return {"dx": du.to(t)}
    x, w = st["x"].float(), st["norm_w"]
    dot = (du * w * x).sum(1, keepdim=True)
    dx = r * (du * w) - x * (r * r * r) * (dot / x.shape[1])
    return {"dx": dx.to(t), "dnorm_w": (du * x * r).sum(0)}


def run(st):
    op = st["op"]
    if own:
        from bit_quantized_mamba_b200 import dfssm as D
        ws = st["ws"]
        if op == "linear":
            return D.linear_int8(st["W"], st["s_row"], st["x"], norm_w=st["norm_w"], out_dtype=TYPES[st["out"]], ws=ws[0])
        if op == "embed":
            return D.embed_tokens(st["W"], st["s_row"], st["tokens"], dtype=TYPES[st["type"]], ws=ws[0])
        if op == "embed_grad":
            dE, ds = D.embed_tokens_backward(st["W"], st["tokens"], st["dh"], ws=ws[0])
            return {"dE": dE, "ds_row": ds}
        loss, stats = D.head_loss(st["W"], st["s_row"], st["x"], st["labels"], norm_w=st["norm_w"], ws=ws[0])
        if op == "score":
            return {"loss": loss}
        dx, ds, dn = D.head_loss_backward(st["W"], st["s_row"], st["x"], st["labels"], stats, st["dloss"],
                                          norm_w=st["norm_w"], ws=ws[1])
        out = {"loss": loss, "ds_row": ds, "dx": dx}
        return out if dn is None else out | {"dnorm_w": dn}
    if op == "linear":
        return _plain_linear(st)
    if op == "embed":
        return _plain_embed(st)
    if op == "embed_grad":
        return _plain_embed_grad(st)
    return _plain_head(st, op == "train")


def work(case):
    """Each input read once, each output written once; multiply-adds count as two operations."""
    m, v, d = case["m"], case["v"], case["d"]
    size = 4 if case["type"] == "f32" else 2
    table = v * d + 4 * v
    op = case["op"]
    if op == "linear":
        return {"bytes": table + m * d * size + m * v * (4 if case["out"] == "f32" else 2), "flops": 2 * m * v * d}
    # distinct tokens to expect of m draws from prepare()'s distribution: each table row is read once
    n = math.log(v + 1.0)
    rows = sum(1.0 - (1.0 - math.log1p(1.0 / (k + 1.0)) / n) ** m for k in range(v))
    if op == "embed":
        return {"bytes": rows * (d + 4) + 4 * m + m * d * size, "flops": m * d}
    if op == "embed_grad":
        return {"bytes": 4 * m + m * d * size + rows * d + 4 * v * d + 4 * v, "flops": 3 * m * d}
    if op == "score":
        return {"bytes": table + m * d * size + 8 * m, "flops": 2 * m * v * d}
    # the logits once more and the product with the table for dx
    return {"bytes": 2 * table + 2 * m * d * size + 16 * m + 4 * v, "flops": 6 * m * v * d}


# ------------------------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    st = prepare(dict(case), seed)
    op, W = case["op"], st["W"]
    f8 = torch.float64
    if op == "embed":
        i = st["tokens"].long()
        return W.index_select(0, i).to(f8).mul(st["s_row"].index_select(0, i).to(f8).unsqueeze(1))
    if op == "embed_grad":
        i = st["tokens"].long()
        dE = torch.zeros(W.shape, dtype=f8, device=W.device)
        order = torch.argsort(i, stable=True)
        dE.index_put_((i[order],), st["dh"][order].to(f8), accumulate=True)
        ds = torch.zeros(W.shape[0], dtype=f8, device=W.device)
        for a in range(0, W.shape[0], 8192):
            ds[a:a + 8192] = (dE[a:a + 8192] * W[a:a + 8192]).sum(1)
        return {"dE": dE, "ds_row": ds}
    # the codes are whole numbers that the definition fixes through single fp32 operations
    h = st["x"].to(f8)
    if st["norm_w"] is not None:
        inv = (h.pow(2).sum(1) / h.shape[1] + EPS).rsqrt()
        u = torch.mul(torch.mul(st["x"].float(), inv.float().unsqueeze(1)), st["norm_w"])
    else:
        inv, u = None, st["x"].float()
    top = u.abs().max(1).values
    s = top.to(f8).div(127).float()
    q = torch.div(u, s.unsqueeze(1)).nan_to_num(0.0, 0.0, 0.0).round().clamp(-127, 127).to(f8)
    zq = q * s.to(f8).unsqueeze(1)
    if op == "linear":
        return torch.cat([zq @ W[a:a + 8192].to(f8).t() * st["s_row"][a:a + 8192].to(f8) for a in range(0, W.shape[0], 8192)], 1)
    T = W.to(f8) * st["s_row"].to(f8).unsqueeze(1)
    y = st["labels"].long()
    L = zq @ T.t()
    rows = torch.arange(len(y), device=y.device)
    yc = torch.where(y < 0, 0, y)
    ly = L[rows, yc].clone()
    L[rows, yc] = -math.inf
    rest = torch.logsumexp(L, 1)
    keep = (y >= 0).to(f8)
    loss = torch.logaddexp(torch.zeros_like(ly), rest - ly) * keep
    if op == "score":
        return {"loss": loss}
    G = L.sub_(torch.logaddexp(rest, ly).unsqueeze(1)).exp_()
    G[rows, yc] = -1.0 / (1.0 + torch.exp(ly - rest))
    G *= (st["dloss"].to(f8) * keep).unsqueeze(1)
    ds = torch.cat([(G[:, a:a + 4096] * (zq @ W[a:a + 4096].to(f8).t())).sum(0) for a in range(0, W.shape[0], 4096)])
    du = G @ T
    res = {"loss": loss, "ds_row": ds}
    if inv is None:
        return res | {"dx": du}
    w = st["norm_w"].to(f8)
    n = h * inv.unsqueeze(1)
    v = du * w
    res["dx"] = inv.unsqueeze(1) * (v - n * (v * n).mean(1, keepdim=True))
    res["dnorm_w"] = (du * n).sum(0)
    return res
