"""Cases, plain forms and exact values of the operators around the layers: token
ids to rows and their gradient, products with 4-bit weights, tokens from logits.

  embed   txl_embed_forward: out[t] = scale * table[token[t]], zeros for a token
          outside 0 .. V-1 (padding); what a segment's first layer reads
  grad    txl_embed_backward: dtable[v] (+)= scale * sum of dout[t] over the t
          with token[t] == v, the table overwritten or added to
  dense4  txl_dense_w4: y = x W (+ bias) (ReLU) for a few tokens, W in 4 bits:
          W[j, i] = scales[j / group, i] * (code - 8), codes [n, k/2], the low
          four bits of a byte for the even j
  sample  txl_sample: a token per row of logits, by temperature, top-k, top-p
          and min-p, from a given uniform number

Where `own` is false, run() computes them with elementary torch operations.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # The token of each of 64 decoding streams: latency.
        dict(name="embed tokens", op="embed", T=64, V=32768, d=1024, table="bf16", out="bf16", pad=0.0),
        # The base evaluation's segments (22 of 512 tokens), rows of a master copy in fp32 rounded for the first layer.
        dict(name="embed segments", op="embed", T=11264, V=32768, d=512, table="f32", out="bf16", pad=0.0),
        # The gradient of the base evaluation's segments, the table's gradient written whole.
        dict(name="grad segments", op="grad", T=11264, V=32768, d=512, out="bf16", pad=0.0, accumulate=False),
        # The wide evaluation's segments (8 of 768 tokens), added to the gradient that a tied output product has left in a larger table.
        dict(name="grad tied", op="grad", T=6144, V=131072, d=1024, out="f32", pad=0.0, accumulate=True),
        # A ragged batch with padding, a width off every vector size.
        dict(name="grad ragged", op="grad", T=4999, V=10007, d=333, out="f32", pad=0.1, accumulate=False),
        # A single stream's token through a projection of the base layer: latency.
        dict(name="product token", op="dense4", m=1, k=512, n=512, group=32, out="bf16", bias=False, relu=False),
        # A few streams through the first product of a feed-forward part.
        dict(name="product layer", op="dense4", m=4, k=1024, n=4096, group=64, out="bf16", bias=True, relu=True),
        # A serving batch through the second.
        dict(name="product batch", op="dense4", m=32, k=4096, n=1024, group=128, out="bf16", bias=True, relu=False),
        # The logits of a few streams over a large vocabulary: bound by reading the weights.
        dict(name="product vocabulary", op="dense4", m=8, k=1024, n=131072, group=128, out="f32", bias=False, relu=False),
        # A single stream's next token: latency.
        dict(name="sample one", op="sample", B=1, V=32768, logits="bf16", k=50, p=0.9, minp=0.0, greedy=0.0),
        # A serving batch, every row with settings of its own, some greedy, a large vocabulary.
        dict(name="sample batch", op="sample", B=64, V=131072, logits="bf16", k=200, p=0.95, minp=0.02, greedy=0.1),
        # Rows with top-p alone, over all of an odd vocabulary, logits in fp32.
        dict(name="sample nucleus", op="sample", B=128, V=50021, logits="f32", k=0, p=0.97, minp=0.0, greedy=0.0),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["embed", "grad", "grad", "dense4", "dense4", "dense4", "sample", "sample", "sample"])
    case = dict(op=op)
    kind = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    if op in ("embed", "grad"):
        d = _log(rng, 1, 2048)
        if rng.random() < 0.6:
            d = max(8, d // 8 * 8)
        V = _log(rng, 2, min(200000, 60_000_000 // d))
        case.update(T=_log(rng, 1, 16384), V=V, d=d, out=kind(), pad=rng.choice([0.0, 0.0, 0.05, 0.5]))
        case.update(dict(table=kind()) if op == "embed" else dict(accumulate=rng.random() < 0.5))
    elif op == "dense4":
        group = rng.choice([32, 64, 128])
        k = group * _log(rng, 1, 4096 // group)
        case.update(m=_log(rng, 1, 32), k=k, n=8 * _log(rng, 1, min(16384, 16_000_000 // k)), group=group, out=kind(), bias=rng.random() < 0.5, relu=rng.random() < 0.3)
    else:
        V = _log(rng, 2, 131072)
        case.update(B=_log(rng, 1, min(256, 8_000_000 // V)), V=V, logits=kind(), k=rng.choice([0, 0, 1, _log(rng, 1, 1000)]), p=rng.choice([1.0, round(rng.uniform(0.05, 0.999), 3)]),
                    minp=rng.choice([0.0, 0.0, round(rng.uniform(0.001, 0.3), 4)]), greedy=rng.choice([0.0, 0.0, 0.2]))
    return case


def _touched(case):
    """About how many rows of the table the tokens name (they are spread over the logarithm of the row)."""
    T, V = case["T"] * (1 - case["pad"]), case["V"]
    total, lo = 0.0, 1
    while lo <= V:
        hi = min(V, lo * 2 - 1)
        p = math.log((hi + 1) / lo) / math.log(V + 1) / (hi - lo + 1)
        total += (hi - lo + 1) * (1 - (1 - p) ** T)
        lo = hi + 1
    return total


def work(case):
    size = lambda x: 4 if case[x] == "f32" else 2  # noqa: E731
    if case["op"] == "embed":
        T, d = case["T"], case["d"]
        return {"bytes": 4 * T + _touched(case) * d * size("table") + T * d * size("out"), "flops": T * d}
    if case["op"] == "grad":
        T, d = case["T"], case["d"]
        rows = 2 * _touched(case) if case["accumulate"] else case["V"]
        return {"bytes": 4 * T + T * (1 - case["pad"]) * d * size("out") + rows * d * 4, "flops": T * d}
    if case["op"] == "dense4":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": n * k / 2 + 2 * n * (k // case["group"]) + 2 * m * k + m * n * size("out") + 4 * n * case["bias"], "flops": 2 * m * k * n}
    return {"bytes": case["B"] * (case["V"] * size("logits") + 24), "flops": 4 * case["B"] * case["V"]}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    normal = lambda *shape: torch.empty(shape, device="cuda").normal_(generator=g)  # noqa: E731
    rand = lambda *shape: torch.rand(shape, device="cuda", generator=g)  # noqa: E731
    s = dict(case)
    if case["op"] in ("embed", "grad"):
        T, V, d = case["T"], case["V"], case["d"]
        # ids by frequency, as vocabularies are numbered: the common ones come again and again
        ids = ((V + 1.0) ** rand(T).double()).floor().long().clamp(1, V) - 1
        s["tokens"] = torch.where(rand(T) < case["pad"], -1, ids).int()
        s["scale"] = d ** 0.5
        if case["op"] == "embed":
            s["table"] = (normal(V, d) * d ** -0.5).to(TYPES[case["table"]])
            s["o"] = torch.empty(T, d, device="cuda", dtype=TYPES[case["out"]])
        else:
            s["dout"] = (0.01 * normal(T, d)).to(TYPES[case["out"]])
            s["dtable"] = 0.01 * normal(V, d)
    elif case["op"] == "dense4":
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = normal(m, k).to(torch.bfloat16)
        s["codes"] = torch.randint(0, 256, (n, k // 2), device="cuda", generator=g, dtype=torch.uint8)
        s["scales"] = ((0.5 + rand(k // case["group"], n)) * (0.2 * k ** -0.5)).to(torch.bfloat16)
        s["b"] = 0.1 * normal(n) if case["bias"] else None
        s["y"] = torch.empty(m, n, device="cuda", dtype=TYPES[case["out"]])
    else:
        B, V = case["B"], case["V"]
        # a few likely tokens over a broad rest
        z = 2.0 * normal(B, V)
        z += 8.0 * (rand(B, V) < 20.0 / V)
        s["z"] = z.to(TYPES[case["logits"]])
        s["u"] = rand(B)
        s["temperature"] = torch.where(rand(B) < case["greedy"], 0.0, 0.6 + 0.8 * rand(B))
        s["top_k"] = (case["k"] * (0.5 + rand(B))).ceil().int() if case["k"] else None
        s["top_p"] = case["p"] * (1 - 0.1 * rand(B)) if case["p"] < 1 else None
        s["min_p"] = case["minp"] * (0.5 + rand(B)) if case["minp"] else None
        s["tokens"] = torch.empty(B, device="cuda", dtype=torch.int32)
        s["prob"] = torch.empty(B, device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _embed(s):
    t = s["tokens"].long()
    inside = (t >= 0) & (t < s["V"])
    rows = s["table"][t.clamp(0, s["V"] - 1)].float() * s["scale"]
    s["o"].copy_(torch.where(inside[:, None], rows, 0.0))
    return s["o"]


def _embed_grad(s):
    t = s["tokens"].long()
    inside = (t >= 0) & (t < s["V"])
    if not s["accumulate"]:
        s["dtable"].zero_()
    rows = s["dout"].float() * torch.where(inside, s["scale"], 0.0)[:, None]
    return s["dtable"].index_add_(0, t.clamp(0, s["V"] - 1), rows)


def _dense4(s):
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], 2).flatten(1).float() - 8.0  # [n, k]
    w = codes.unflatten(1, (-1, s["group"])) * s["scales"].float().t()[:, :, None]
    y = s["x"].float() @ w.flatten(1).t()
    if s["bias"]:
        y += s["b"]
    if s["relu"]:
        y = y.clamp(min=0.0)
    s["y"].copy_(y)
    return s["y"]


def _sample(s):
    z = s["z"].double()  # in 64 bits: a number next to a border decides a token
    z = torch.where(z.isnan(), -torch.inf, z).clamp(max=torch.finfo(torch.float32).max)
    B, V = z.shape
    z, order = torch.sort(z, dim=1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    w = torch.where(z > -torch.inf, ((z - z[:, :1]) / torch.where(t > 0, t, 1.0)).exp(), 0.0)
    rank = torch.arange(V, device="cuda")
    keep = (t > 0) | (rank == 0)
    if s["top_k"] is not None:
        keep = keep & (rank < torch.where(s["top_k"] > 0, s["top_k"], V)[:, None])
    w = w * keep
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        w = w * ((w.cumsum(1) - w < torch.where(p < 1, p, torch.inf) * w.sum(1, keepdim=True)) | (rank == 0))
    if s["min_p"] is not None:
        w = w * (w >= s["min_p"].double()[:, None])
    w = torch.zeros_like(w).scatter_(1, order, w)  # by token again
    upto = w.cumsum(1)
    token = (upto > s["u"].double()[:, None] * upto[:, -1:]).int().argmax(1)
    s["tokens"].copy_(token)
    s["prob"].copy_(w.gather(1, token[:, None])[:, 0] / upto[:, -1])
    return dict(tokens=s["tokens"], prob=s["prob"])


def _library(s):
    import transformer_xl_relative_txl_gb300 as txl

    if s["op"] == "embed":
        return txl.txl_embed_forward(s["tokens"], s["table"], s["o"], scale=s["scale"])
    if s["op"] == "grad":
        return txl.txl_embed_backward(s["tokens"], s["dout"], s["dtable"], scale=s["scale"], accumulate=s["accumulate"])
    if s["op"] == "dense4":
        return txl.txl_dense_w4(s["x"], s["codes"], s["scales"], s["y"], bias=s["b"], relu=s["relu"])
    txl.txl_sample(s["z"], s["u"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], prob=s["prob"])
    return dict(tokens=s["tokens"], prob=s["prob"])


def run(s):
    if own:
        return _library(s)
    return dict(embed=_embed, grad=_embed_grad, dense4=_dense4, sample=_sample)[s["op"]](s)


# ---------------------------------------------------------------------------
# exact values
# ---------------------------------------------------------------------------
def exact(case, seed):
    """Each operator by its definition in 64 bits: rows by a product with the tokens' indicator (in blocks) or row by
    row, weights from their digits in base 16, a row's tokens one filter after the other on the sorted list."""
    s = prepare(case, seed)
    if case["op"] == "embed":
        out = torch.zeros(case["T"], case["d"], dtype=torch.float64, device="cuda")
        real = (s["tokens"] >= 0).nonzero()[:, 0]
        out[real] = s["table"].double().index_select(0, s["tokens"][real]) * math.sqrt(case["d"])
        return out
    if case["op"] == "grad":
        out = s["dtable"].double() if case["accumulate"] else torch.zeros(case["V"], case["d"], dtype=torch.float64, device="cuda")
        seen, at = s["tokens"].unique(return_inverse=True)
        rows = torch.zeros(len(seen), case["d"], dtype=torch.float64, device="cuda")
        for a in range(0, case["T"], 1024):
            named = (at[a:a + 1024][None] == torch.arange(len(seen), device="cuda")[:, None]).double()
            rows += named @ s["dout"][a:a + 1024].double()
        out[seen[seen >= 0].long()] += rows[seen >= 0] * math.sqrt(case["d"])
        return out
    if case["op"] == "dense4":
        y = torch.zeros(case["m"], case["n"], dtype=torch.float64, device="cuda")
        x, group = s["x"].double(), case["group"]
        for j in range(0, case["k"], group):
            byte = s["codes"][:, j // 2:(j + group) // 2].long()
            part = x[:, j:j + group:2] @ (byte % 16 - 8).double().t() + x[:, j + 1:j + group:2] @ (byte // 16 - 8).double().t()
            y += part * s["scales"][j // group].double()
        if case["bias"]:
            y += s["b"].double()
        return torch.relu(y) if case["relu"] else y
    tokens, prob = [], []
    setting = lambda name, b: None if s[name] is None else s[name][b].item()  # noqa: E731
    for b in range(case["B"]):
        z = s["z"][b].double()
        t, k, p, least = (setting(x, b) for x in ("temperature", "top_k", "top_p", "min_p"))
        order = torch.argsort(-z, stable=True)
        if t == 0:
            order = order[:1]
        if k:
            order = order[:k]
        w = torch.exp(z[order] / (t or 1.0) - z[order[0]] / (t or 1.0))
        if p is not None and p < 1:
            order = order[:int((w.cumsum(0) < p * w.sum()).sum()) + 1]
            w = w[:len(order)]
        if least:
            order, w = order[w >= least], w[w >= least]
        order, by = order.sort()
        upto = w[by].cumsum(0)
        at = min(int(torch.searchsorted(upto, s["u"][b].double() * upto[-1], right=True)), len(order) - 1)
        tokens.append(int(order[at]))
        prob.append(float(w[by][at] / upto[-1]))
    return dict(tokens=torch.tensor(tokens, dtype=torch.int32), prob=torch.tensor(prob, dtype=torch.float64))
