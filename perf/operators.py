"""Workloads of the token-path operators: embedding lookup and its gradient,
tokens sorted by expert and back (with the gradients of both ways), and
sampling of the next token. Each case is one call of an operator as a program
that trains or serves a language model makes it; `run` has the plain form in
elementary torch operations beside the library's calls."""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
DEV = "cuda"


def listed():
    return [
        # one decoding step of a small batch: latency of a lookup
        {"name": "embed_decode", "op": "embed", "n": 32, "vocab": 32000, "width": 4096, "dtype": "bf16", "pad": 0.0},
        # the lookup of a training batch, with padding ids
        {"name": "embed_train", "op": "embed", "n": 32768, "vocab": 131072, "width": 4096, "dtype": "bf16", "pad": 0.05},
        # gradient of a small model's table in fp32, odd sizes everywhere
        {"name": "embed_grad_ragged", "op": "embed_grad", "n": 4999, "vocab": 10007, "width": 257, "dtype": "fp32", "pad": 0.1},
        # gradient of a training batch over a large vocabulary
        {"name": "embed_grad_train", "op": "embed_grad", "n": 65536, "vocab": 131072, "width": 2048, "dtype": "bf16", "pad": 0.02},
        # decoding step: 16 tokens to 8 of 128 experts
        {"name": "to_experts_decode", "op": "dispatch", "n": 16, "per": 8, "experts": 128, "width": 4096, "dtype": "bf16", "drop": 0.0},
        # training or prompt batch to 8 of 64 experts, a few assignments dropped by capacity
        {"name": "to_experts_train", "op": "dispatch", "n": 16384, "per": 8, "experts": 64, "width": 2048, "dtype": "bf16", "drop": 0.03},
        # decoding step: the experts' rows weighted and summed back
        {"name": "back_decode", "op": "combine", "n": 16, "per": 8, "experts": 128, "width": 4096, "dtype": "bf16", "drop": 0.0},
        # prompt batch back, odd width
        {"name": "back_ragged", "op": "combine", "n": 9973, "per": 6, "experts": 160, "width": 1451, "dtype": "fp16", "drop": 0.05},
        # gradients of a small fp32 model: both ways
        {"name": "experts_grad_ragged", "op": "routed_grad", "n": 1021, "per": 2, "experts": 8, "width": 769, "dtype": "fp32", "drop": 0.1},
        # gradients of a training batch: both ways
        {"name": "experts_grad_train", "op": "routed_grad", "n": 8192, "per": 8, "experts": 128, "width": 4096, "dtype": "bf16", "drop": 0.0},
        # one sequence being decoded, fp32 logits of a large vocabulary
        {"name": "sample_one", "op": "sample", "n": 1, "vocab": 131072, "dtype": "fp32", "spread": 2.5, "plain_rows": 0.0},
        # a serving batch, each row with settings of its own
        {"name": "sample_batch", "op": "sample", "n": 256, "vocab": 131072, "dtype": "bf16", "spread": 2.5, "plain_rows": 0.25},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "dispatch", "combine", "routed_grad", "sample"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    es = BYTES[dtype]
    if op == "sample":
        rows = _log(rng, 1, 256)
        return {"op": op, "n": rows, "vocab": _log(rng, 1000, 131072 * 2 // es), "dtype": dtype,
                "spread": rng.uniform(0.5, 5.0), "plain_rows": rng.choice([0.0, 0.25, 1.0])}
    width = _log(rng, 64, 4096)
    if rng.random() < 0.5:
        width = (width + 63) // 64 * 64
    if op in ("embed", "embed_grad"):
        vocab = _log(rng, 1000, 131072)
        vocab = min(vocab, 131072 * 2048 * 2 // (width * es))
        n = min(_log(rng, 1, 65536), 65536 * 2048 * 2 // (width * es))
        return {"op": op, "n": n, "vocab": vocab, "width": width, "dtype": dtype, "pad": rng.choice([0.0, 0.1, 0.5])}
    experts = _log(rng, 4, 256)
    per = rng.randint(1, min(8, experts))
    n = min(_log(rng, 1, 32768), 8192 * 8 * 4096 * 2 // (per * width * es))
    return {"op": op, "n": n, "per": per, "experts": experts, "width": width, "dtype": dtype, "drop": rng.choice([0.0, 0.05, 0.3])}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n, op = case["n"], case["op"]
    dt = DTYPES[case["dtype"]]

    def rand(*shape):
        return torch.rand(*shape, device=DEV, generator=g)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, device=DEV, generator=g) * scale).to(dt)

    s = {"op": op}
    if op in ("embed", "embed_grad"):
        vocab, width = case["vocab"], case["width"]
        # token frequencies fall with the rank, as in text; padding is -1
        ids = torch.exp(rand(n).double() * math.log(vocab + 1)).sub_(1).floor_().long().clamp_(0, vocab - 1)
        ids[rand(n) < case["pad"]] = -1
        s.update(ids=ids, vocab=vocab, scale=math.sqrt(width) if op == "embed" else 1.0 / 8)
        if op == "embed":
            s["table"] = randn(vocab, width, scale=0.02)
        else:
            s["dout"] = randn(n, width)
        return s
    if op == "sample":
        vocab = case["vocab"]
        s["logits"] = randn(n, vocab, scale=case["spread"])
        if n > 3:
            s["logits"][2, rand(vocab) < 0.7] = float("-inf")  # a grammar's mask
        s["u"] = rand(n)
        plain = rand(n) < case["plain_rows"]
        s["temperature"] = torch.where(rand(n) < 0.05, torch.zeros_like(s["u"]), 0.4 + rand(n))
        s["top_k"] = torch.where(plain | (rand(n) < 0.4), torch.zeros_like(s["u"]), 1 + 200 * rand(n)).int()
        s["top_p"] = torch.where(plain, torch.ones_like(s["u"]), 0.5 + 0.49 * rand(n))
        s["min_p"] = torch.where(plain | (rand(n) < 0.6), torch.zeros_like(s["u"]), 0.1 * rand(n))
        return s
    per, experts, width = case["per"], case["experts"], case["width"]
    score = torch.randn(n, experts, device=DEV, generator=g) + torch.randn(experts, device=DEV, generator=g)
    top, ids = torch.topk(score, per, dim=1)
    ids[rand(n, per) < case["drop"]] = -1
    s.update(ids=ids, experts=experts)
    if op == "dispatch":
        s["x"] = randn(n, width)
        s["rows"] = torch.zeros(n * per, width, dtype=dt, device=DEV)
        return s
    s["ranks"] = _group_plain(ids, experts)[0]
    s["weights"] = torch.softmax(top, dim=1).contiguous()
    s["y"] = randn(n * per, width)
    if op == "routed_grad":
        s["dout"] = randn(n, width)
        s["drows"] = randn(n * per, width)
        s["dy"] = torch.zeros(n * per, width, dtype=dt, device=DEV)
    return s


def _group_plain(ids, groups):
    """(ranks, offsets) of the stable grouping of ids, -1 for ids outside."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < groups), flat, groups)
    _, order = torch.sort(key, stable=True)
    ranks = torch.empty_like(order)
    ranks[order] = torch.arange(order.numel(), device=order.device)
    ranks = torch.where(key < groups, ranks, -1).int().reshape(ids.shape)
    count = torch.bincount(key, minlength=groups + 1)[:groups]
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)]).int()
    return ranks, offsets


def _sample_plain(s):
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    top, vocab = x[:, :1], x.shape[1]
    place = torch.arange(vocab, device=x.device)
    t = s["temperature"].double()[:, None]
    w = torch.exp((x.double() - top.double()) / torch.where(t > 0, t, 1.0))
    w = torch.where(x == -math.inf, 0.0, w)
    k = torch.where(t[:, 0] > 0, s["top_k"], 1)[:, None]
    keep = (x > -math.inf) & ((k <= 0) | (place < k))
    w = torch.where(keep, w, 0.0)
    run = w.cumsum(1)
    p = s["top_p"].double()[:, None]
    keep &= (p >= 1) | (run - w < p * run[:, -1:]) | (place == 0)
    keep &= (w >= s["min_p"].double()[:, None]) | (place == 0)
    w = torch.where(keep, w, 0.0)
    by_index = torch.zeros_like(w).scatter_(1, order, w)
    run = by_index.cumsum(1)
    total = run[:, -1:]
    token = (run <= s["u"].double()[:, None] * total).sum(1, keepdim=True).clamp_(max=vocab - 1)
    kept = keep.sum(1)
    logprob = torch.log(by_index.gather(1, token) / total)[:, 0]
    none = kept == 0
    return (torch.where(none, -1, token[:, 0]).int(), kept.int(), torch.where(none, -math.inf, logprob).float())


def run(s):
    op = s["op"]
    if own:
        import scan_stream_compaction_amd as ssc
        if op == "embed":
            return ssc.embed_rows(s["table"], s["ids"], s["scale"])
        if op == "embed_grad":
            order, _, offsets = ssc.group_by_key(s["ids"], s["vocab"], ranks=False)
            return ssc.embed_rows_grad(s["dout"], s["ids"], order, offsets, s["scale"])
        if op == "dispatch":
            _, ranks, offsets = ssc.group_by_key(s["ids"], s["experts"], order=False)
            return ranks, offsets, ssc.dispatch_rows(s["x"], ranks, out=s["rows"])
        if op == "combine":
            return ssc.combine_rows(s["y"], s["ranks"], s["weights"])
        if op == "routed_grad":
            dy, dweights = ssc.combine_rows_grad(s["dout"], s["y"], s["ranks"], s["weights"], dy=s["dy"])
            return dy, dweights, ssc.dispatch_rows_grad(s["drows"], s["ranks"])
        return ssc.sample_rows(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    if op == "embed":
        ids, table = s["ids"], s["table"]
        inside = (ids >= 0) & (ids < s["vocab"])
        return (table[torch.where(inside, ids, 0)].float() * (inside * s["scale"])[:, None]).to(table.dtype)
    if op == "embed_grad":
        ids, dout = s["ids"], s["dout"]
        inside = (ids >= 0) & (ids < s["vocab"])
        grad = torch.zeros(s["vocab"] + 1, dout.shape[1], dtype=torch.float32, device=dout.device)
        grad.index_add_(0, torch.where(inside, ids, s["vocab"]), dout.float())
        return (grad[:-1] * s["scale"]).to(dout.dtype)
    if op == "dispatch":
        ranks, offsets = _group_plain(s["ids"], s["experts"])
        t, k = torch.nonzero(ranks >= 0, as_tuple=True)
        s["rows"][ranks[t, k].long()] = s["x"][t]
        return ranks, offsets, s["rows"]
    if op == "sample":
        return _sample_plain(s)
    ranks = s["ranks"].long()
    inside = ranks >= 0
    at = ranks.clamp(min=0)
    if op == "combine":
        return (s["y"][at].float() * (s["weights"] * inside)[:, :, None]).sum(1).to(s["y"].dtype)
    dout = s["dout"].float()[:, None]
    dweights = torch.where(inside, (dout * s["y"][at].float()).sum(2), 0.0)
    s["dy"][ranks[inside]] = (dout * s["weights"][:, :, None]).to(s["dy"].dtype)[inside]
    dx = (s["drows"][at].float() * inside[:, :, None]).sum(1).to(s["drows"].dtype)
    return s["dy"], dweights, dx


def work(case):
    n, es = case["n"], BYTES[case["dtype"]]
    if case["op"] == "sample":
        return {"bytes": n * case["vocab"] * es + 32 * n, "flops": 4 * n * case["vocab"]}
    row = case["width"] * es
    if case["op"] in ("embed", "embed_grad"):
        inside = n * (1 - case["pad"])
        if case["op"] == "embed":
            v = np.arange(1, case["vocab"] + 1)
            p = np.log1p(1 / v) / math.log(case["vocab"] + 1)
            distinct = float((1 - (1 - p) ** inside).sum())
            return {"bytes": 8 * n + (distinct + n) * row, "flops": n * case["width"]}
        return {"bytes": 8 * n + (inside + case["vocab"]) * row, "flops": inside * case["width"]}
    slots = n * case["per"]
    kept = slots * (1 - case["drop"])
    if case["op"] == "dispatch":
        return {"bytes": 8 * slots + 4 * slots + 4 * (case["experts"] + 1) + (n + kept) * row, "flops": slots}
    if case["op"] == "combine":
        return {"bytes": 8 * slots + (n + kept) * row, "flops": 2 * kept * case["width"]}
    return {"bytes": 12 * slots + (2 * n + 3 * kept) * row, "flops": 4 * kept * case["width"]}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "embed":
        t = torch.cat([s["table"], torch.zeros_like(s["table"][:1])])
        return t[s["ids"]].double() * s["scale"]  # -1 is the last row, of zeros
    if op == "embed_grad":
        kept = s["ids"] >= 0
        ids = s["ids"][kept]
        out = torch.zeros(s["vocab"], s["dout"].shape[1], dtype=torch.float64, device=DEV)
        return out.index_put_((ids,), s["dout"][kept].double() * s["scale"], accumulate=True)
    if op == "dispatch":
        return None  # whole numbers, and rows moved as they are
    if op == "sample":
        return None, None, torch.from_numpy(_sample_exact(s))
    n, per = s["ranks"].shape
    zero = torch.zeros_like(s["y"][:1])
    ranks = s["ranks"].long()
    y = torch.cat([s["y"], zero])
    w = s["weights"].double()
    if op == "combine":
        out = torch.zeros(n, y.shape[1], dtype=torch.float64, device=DEV)
        for k in range(per):
            out += w[:, k, None] * y[ranks[:, k]].double()
        return out
    dout = s["dout"].double()
    dy = torch.zeros(y.shape, dtype=torch.float64, device=DEV)
    dx = torch.zeros_like(dout)
    dw = torch.zeros_like(w)
    drows = torch.cat([s["drows"], zero])
    for k in range(per):
        dy[ranks[:, k]] = w[:, k, None] * dout
        dw[:, k] = (dout * y[ranks[:, k]].double()).sum(1)
        dx += drows[ranks[:, k]].double()
    return dy[:-1], dw, dx


def _sample_exact(s):
    """The log-probabilities row by row, with numpy's sort and sums in 64 bits."""
    logits = s["logits"].double().cpu().numpy()
    u, t, k, p, m = (s[name].double().cpu().numpy() for name in ("u", "temperature", "top_k", "top_p", "min_p"))
    out = np.empty(len(logits), np.float64)
    for r, row in enumerate(logits):
        order = np.argsort(-row, kind="stable")
        order = order[: int(k[r]) if k[r] > 0 and t[r] > 0 else len(row) if t[r] > 0 else 1]
        order = order[row[order] > -np.inf]
        w = np.exp((row[order] - row[order[0]]) / (t[r] if t[r] > 0 else 1.0))
        if p[r] < 1:
            before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
            nucleus = max(1, int((before < p[r] * w.sum()).sum()))
            order, w = order[:nucleus], w[:nucleus]
        large = w >= min(m[r], 1.0)
        order, w = order[large], w[large]
        by = np.argsort(order)
        cum = np.cumsum(w[by])
        at = min(int(np.searchsorted(cum, u[r] * cum[-1], side="right")), len(cum) - 1)
        out[r] = np.log(w[by][at] / cum[-1])
    return out
