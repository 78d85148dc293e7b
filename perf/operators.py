"""Operators around a vocabulary row, with their plain forms and the cases they are measured on.

Three operators of the library, the last with its gradient:

* sample   one token per row from given uniform numbers: temperature, then top-k, top-p and min-p in
           the library's total order (logit descending, token id ascending), then the first token whose
           inclusive share of the support's mass exceeds the row's number;
* topk     a teacher's top k: ids in the same order and their log-probabilities over the whole row;
* distill  Kullback-Leibler loss against a teacher's top log-probabilities, and its gradient with
           respect to the student's logits.

`run` takes the plain forms below, or the library's calls where `own` is true.
"""

import torch

own = False

VOCAB = 151_936  # the vocabulary of the repository's benchmark


def listed():
    return [
        # one sequence being decoded: latency
        {"name": "sample_one_row", "op": "sample", "rows": 1, "vocab": VOCAB, "dtype": "bf16", "filter": "topk", "masked": False},
        # a serving batch of the benchmark's shape, nucleus only: the support holds thousands of tokens
        {"name": "sample_batch_topp", "op": "sample", "rows": 128, "vocab": VOCAB, "dtype": "bf16", "filter": "topp", "masked": False},
        # fp32 logits, constrained decoding (most tokens masked), every request with its own settings, odd sizes
        {"name": "sample_ragged_f32", "op": "sample", "rows": 37, "vocab": 50_021, "dtype": "f32", "filter": "mixed", "masked": True},
        # a rollout batch in fp32 without any filter: the support is the vocabulary
        {"name": "sample_full_f32", "op": "sample", "rows": 64, "vocab": VOCAB, "dtype": "f32", "filter": "none", "masked": False},
        # a large rollout batch, every request with its own settings
        {"name": "sample_rollout", "op": "sample", "rows": 512, "vocab": VOCAB, "dtype": "bf16", "filter": "mixed", "masked": False},
        # the smallest teacher call (the tiny workload's shape)
        {"name": "topk_tiny", "op": "topk", "rows": 8, "vocab": 1024, "dtype": "f32", "k": 20},
        # wide lists over an odd vocabulary
        {"name": "topk_ragged_f32", "op": "topk", "rows": 61, "vocab": 50_021, "dtype": "f32", "k": 257},
        # a teacher's logits for a training batch
        {"name": "topk_teacher", "op": "topk", "rows": 2048, "vocab": VOCAB, "dtype": "bf16", "k": 64},
        # the smallest loss call, forward alone (an evaluation)
        {"name": "distill_tiny_fwd", "op": "distill", "rows": 8, "vocab": 1024, "dtype": "f32", "k": 20, "tail": False, "step": "fwd"},
        # lists of uneven length, some empty, an odd vocabulary: forward, then backward
        {"name": "distill_ragged_f32", "op": "distill", "rows": 133, "vocab": 50_021, "dtype": "f32", "k": 257, "tail": False, "step": "two"},
        # a training step whose loss weights are known beforehand: loss and gradient in one call
        {"name": "distill_fused", "op": "distill", "rows": 2048, "vocab": VOCAB, "dtype": "bf16", "k": 64, "tail": True, "step": "fused"},
        # a training step through automatic differentiation: forward, then backward
        {"name": "distill_train", "op": "distill", "rows": 4096, "vocab": VOCAB, "dtype": "bf16", "k": 64, "tail": True, "step": "two"},
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, int(lo * (hi / lo) ** rng.random() + rng.random()))


def draw(rng):
    op = rng.choice(["sample", "sample", "topk", "distill"])
    dtype = rng.choice(["bf16", "f32"])
    vocab = _spread(rng, 1000, VOCAB)
    if op == "sample":
        return {"op": op, "rows": _spread(rng, 1, 512), "vocab": vocab, "dtype": dtype,
                "filter": rng.choice(["topk", "topp", "minp", "mixed", "none"]), "masked": rng.random() < 0.25}
    if op == "topk":
        return {"op": op, "rows": _spread(rng, 1, 1024), "vocab": vocab, "dtype": dtype, "k": _spread(rng, 1, 1000)}
    return {"op": op, "rows": _spread(rng, 1, 1500), "vocab": vocab, "dtype": dtype, "k": _spread(rng, 1, 512),
            "tail": rng.random() < 0.5, "step": rng.choice(["fwd", "two", "fused"])}


def work(case):
    rows, vocab, size = case["rows"], case["vocab"], 2 if case["dtype"] == "bf16" else 4
    row = float(rows) * vocab
    if case["op"] == "sample":  # logits, the row's number and settings in; token, log-probability and size out
        return {"bytes": row * size + 32.0 * rows, "flops": 4.0 * row}
    if case["op"] == "topk":
        return {"bytes": row * size + rows * (4.0 + 8.0 * case["k"]), "flops": 4.0 * row}
    lists = rows * (8.0 * case["k"] + 12.0)
    if case["step"] == "fwd":
        return {"bytes": row * size + lists, "flops": 4.0 * row}
    reads = 2 if case["step"] == "two" else 1  # two calls read the logits twice, the gradient is written once
    return {"bytes": row * size * (reads + 1) + lists * reads, "flops": 8.0 * row}


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _logits(case, gen, sigma=3.0):
    """Rows of N(0, sigma) with 8 raised tokens each, rows padded to 16 bytes as the library wants them."""
    rows, vocab = case["rows"], case["vocab"]
    ld = (vocab + 7) // 8 * 8
    x = torch.randn((rows, ld), device="cuda", generator=gen).mul_(sigma)
    at = torch.randint(0, vocab, (rows, 8), device="cuda", generator=gen)
    x.scatter_(1, at, torch.gather(x, 1, at) + 8.0)
    return x.to(_dtype(case))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rows, vocab = case["rows"], case["vocab"]

    def uniform(*shape):
        return torch.rand(shape, device="cuda", generator=gen)

    if case["op"] == "topk":
        return {"case": case, "logits": _logits(case, gen), "temperature": 0.8 + 0.4 * uniform(rows)}
    if case["op"] == "sample":
        x = _logits(case, gen)
        if case["masked"]:  # a grammar allows about one token in sixteen, and always token 1
            banned = uniform(rows, x.shape[1]) > 1 / 16
            banned[:, 1] = False
            x.masked_fill_(banned, float("-inf"))
        t = 0.6 + 0.6 * uniform(rows)
        k = torch.zeros(rows, dtype=torch.int32, device="cuda")
        p, m = torch.ones(rows, device="cuda"), torch.zeros(rows, device="cuda")
        kind = case["filter"]
        if kind == "topk":
            k.fill_(50)
            p.fill_(0.95)
        elif kind == "topp":
            p.fill_(0.95)
        elif kind == "minp":
            m.fill_(0.05)
        elif kind == "mixed":  # a tenth greedy; each filter on for half of the rows
            t = torch.where(uniform(rows) < 0.1, torch.zeros_like(t), t)
            k = torch.where(uniform(rows) < 0.5, (uniform(rows) * 200 + 1).to(torch.int32), k)
            p = torch.where(uniform(rows) < 0.5, 0.5 + 0.49 * uniform(rows), p)
            m = torch.where(uniform(rows) < 0.5, 0.001 + 0.1 * uniform(rows), m)
        return {"case": case, "logits": x, "temperature": t, "top_k": k, "top_p": p, "min_p": m, "uniform": uniform(rows)}
    student = _logits(case, gen)
    k = min(case["k"], vocab)
    ids = torch.empty((rows, k), dtype=torch.int32, device="cuda")
    lp = torch.empty((rows, k), device="cuda")
    for lo in range(0, rows, 512):  # the teacher: the student's logits and noise, 512 rows at a time
        x = student[lo:lo + 512, :vocab].float()
        x = x + torch.randn(x.shape, device="cuda", generator=gen).mul_(0.7)
        v, i = torch.topk(x, k, dim=1)
        lp[lo:lo + 512] = v - torch.logsumexp(x, 1, keepdim=True)
        ids[lo:lo + 512] = i.to(torch.int32)
    width = torch.where(uniform(rows) < 0.75, torch.full((rows,), k, device="cuda"), (uniform(rows) * (k + 1)).long())
    ids.masked_fill_(torch.arange(k, device="cuda")[None] >= width[:, None], -1)  # a quarter of the lists is shorter
    weight = uniform(rows)
    return {"case": case, "logits": student, "ids": ids, "logprob": lp, "temperature": 0.9 + 0.2 * uniform(rows),
            "g_loss": weight / weight.sum()}


# ---------------------------------------------------------------------------------------------
# plain forms


def _plain_sample(s):
    """In 64 bits: the decisions are cuts of a cumulative sum, next to which 32 bits would choose."""
    x = s["logits"][:, :s["case"]["vocab"]].double()
    vocab = x.shape[1]
    v, order = x.sort(dim=1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    greedy = t == 0
    w = torch.exp((v - v[:, :1]) / torch.where(greedy, torch.ones_like(t), t))
    k = s["top_k"].long()[:, None]
    nk = torch.where((k <= 0) | (k > vocab), torch.full_like(k, vocab), k)
    nk = torch.minimum(nk, (v > float("-inf")).sum(1, keepdim=True))
    place = torch.arange(vocab, device=x.device)[None]
    w = torch.where(place < nk, w, torch.zeros_like(w))
    c = torch.cumsum(w, 1)
    p = s["top_p"].double()[:, None]
    n = torch.minimum(nk, torch.where(p < 1, (c < p * c[:, -1:]).sum(1, keepdim=True) + 1, nk))
    n = torch.minimum(n, torch.where(s["min_p"][:, None] > 0, (w >= s["min_p"].double()[:, None]).sum(1, keepdim=True), nk))
    n = torch.where(greedy, torch.ones_like(n), n)
    z = torch.gather(c, 1, n - 1)
    at = torch.minimum((c <= s["uniform"].double()[:, None] * z).sum(1, keepdim=True), n - 1)
    logprob = torch.log(torch.gather(w, 1, at) / z)
    return {"token": torch.gather(order, 1, at)[:, 0].to(torch.int32), "logprob": logprob[:, 0].float(),
            "support_size": n[:, 0].to(torch.int32)}


def _plain_topk(s):
    x = s["logits"][:, :s["case"]["vocab"]].float()
    k = min(s["case"]["k"], x.shape[1])
    v, order = x.sort(dim=1, descending=True, stable=True)
    z = v / s["temperature"][:, None]
    z = z - z[:, :1]
    logprob = z[:, :k] - torch.log(torch.exp(z).sum(1, keepdim=True))
    return {"ids": order[:, :k].to(torch.int32), "logprob": logprob}


def _plain_distill(s):
    case = s["case"]
    x, ids = s["logits"][:, :case["vocab"]].float(), s["ids"]
    t = s["temperature"][:, None]
    kept = ids >= 0
    at = ids.clamp(min=0).long()
    here = kept.any(1, keepdim=True)
    z = x / t
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    zk = torch.gather(z, 1, at).double() - top.double()
    # the teacher's masses, in 64 bits: what its list leaves is a difference next to 1
    lp = torch.where(kept, s["logprob"].double(), torch.full_like(zk, float("-inf")))
    if case["tail"]:
        rest = (1.0 - torch.exp(lp).sum(1, keepdim=True)).clamp(min=0.0)
    else:
        lp = torch.where(here, lp - torch.logsumexp(lp, 1, keepdim=True), lp)
        rest = torch.zeros_like(top).double()
    a = torch.exp(lp)
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    others = torch.scatter_reduce(e, 1, at, torch.where(kept, torch.zeros_like(a), torch.full_like(a, float("inf"))).float(), "amin")
    others_total = others.sum(1, keepdim=True, dtype=torch.float64)  # summed apart: a difference would lose a small rest
    logq = zk - torch.log(total)
    loss = torch.where(kept & (a > 0), a * (lp - logq), torch.zeros_like(a)).sum(1, keepdim=True)
    has = (rest > 0) & (others_total > 0) & here
    one = torch.ones_like(rest)
    loss = loss + torch.where(has, rest * (torch.log(torch.where(has, rest, one)) - torch.log(torch.where(has, others_total / total, one))), torch.zeros_like(rest))
    out = {"loss": loss[:, 0].float(), "valid": here[:, 0].to(torch.uint8)}
    if case["step"] == "fwd":
        return out
    g = torch.where(here, s["g_loss"][:, None] / t, torch.zeros_like(t))
    if case["tail"]:
        share = torch.where(others_total > 0, 1.0 / total - rest / torch.where(others_total > 0, others_total, one), torch.zeros_like(total))
        grad = others * (g * share).float()
    else:
        grad = e * (g / total).float()
    listed_grad = ((torch.exp(logq) - a) * g).float()
    rows, slots = kept.nonzero(as_tuple=True)
    grad[rows, at[rows, slots]] = listed_grad[rows, slots]
    out["grad"] = grad.to(s["logits"].dtype)
    return out


def _own(s):
    import sampling_support_b200 as vs

    case = s["case"]
    vocab = case["vocab"]
    if case["op"] == "sample":
        out = vs.sample(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                        min_p=s["min_p"], vocab=vocab)
        return {n: out[n] for n in ("token", "logprob", "support_size")}
    if case["op"] == "topk":
        out = vs.topk_logprob(s["logits"], min(case["k"], vocab), temperature=s["temperature"], vocab=vocab)
        return {n: out[n] for n in ("ids", "logprob")}
    kw = {"temperature": s["temperature"], "tail": case["tail"], "vocab": vocab}
    if case["step"] == "fused":
        out = vs.distill_fwd(s["logits"], s["ids"], s["logprob"], g_loss=s["g_loss"], grad_dtype=s["logits"].dtype, **kw)
        return {"loss": out["loss"], "valid": out["valid"], "grad": out["grad"][:, :vocab]}
    out = vs.distill_fwd(s["logits"], s["ids"], s["logprob"], want_grad=case["step"] == "two", **kw)
    got = {"loss": out["loss"], "valid": out["valid"]}
    if case["step"] == "two":
        got["grad"] = vs.distill_bwd(s["logits"], s["ids"], s["logprob"], out["ctx"], s["g_loss"],
                                     grad_dtype=s["logits"].dtype, **kw)[:, :vocab]
    return got


def run(state):
    if own:
        return _own(state)
    return {"sample": _plain_sample, "topk": _plain_topk, "distill": _plain_distill}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, row by row


def _exact_sample_row(x, t, k, p, m, u):
    ids = torch.nonzero(x > float("-inf"))[:, 0]
    x = x[ids]
    by = torch.argsort(-x, stable=True)
    if t == 0:
        return int(ids[by[0]]), 0.0, 1
    logw = (x[by] - x[by[0]]) / t
    if 0 < k < len(by):
        logw = logw[:k]
    share = torch.softmax(logw, 0)
    n = len(share)
    if p < 1:
        before = torch.cumsum(share, 0) - share
        n = min(n, int((before < p).sum()))
    if m > 0:
        n = min(n, int((torch.exp(logw) >= m).sum()))
    share = torch.softmax(logw[:n], 0)
    upto = torch.cumsum(share, 0)
    at = min(int(torch.searchsorted(upto, torch.tensor([u], dtype=upto.dtype, device=upto.device), right=True)), n - 1)
    return int(ids[by[at]]), float(logw[at] - torch.logsumexp(logw[:n], 0)), n


def _exact_distill_row(x, t, ids, lp, tail, g):
    keep = ids >= 0
    ids, lp = ids[keep].long(), lp[keep].double()
    if len(ids) == 0:
        return torch.zeros((), dtype=torch.float64, device=x.device), 0, torch.zeros_like(x)
    logq = torch.log_softmax(x / t, 0)
    if not tail:
        a = torch.softmax(lp, 0)
        loss = (torch.special.xlogy(a, a) - a * logq[ids]).sum()
        grad = torch.exp(logq)
        grad[ids] -= a
        return loss, 1, grad * (g / t)
    a = torch.exp(lp)
    out = torch.ones(len(x), dtype=torch.bool, device=x.device)
    out[ids] = False
    rest = max(0.0, 1.0 - float(a.sum()))
    loss = (torch.special.xlogy(a, a) - a * logq[ids]).sum()
    grad = torch.exp(logq)
    if bool(out.any()):
        log_out = torch.logsumexp(logq[out], 0)
        if rest > 0:
            loss = loss + rest * (torch.log(torch.tensor(rest, dtype=x.dtype, device=x.device)) - log_out)
        grad = torch.where(out, torch.exp(logq - log_out) * (torch.exp(log_out) - rest), grad)
    grad[ids] -= a
    return loss, 1, grad * (g / t)


def exact(case, seed):
    s = prepare(case, seed)
    x = s["logits"][:, :case["vocab"]]
    rows = range(case["rows"])
    if case["op"] == "sample":
        t, k, p, m, u = (s[n].double().tolist() for n in ("temperature", "top_k", "top_p", "min_p", "uniform"))
        got = [_exact_sample_row(x[r].double(), t[r], int(k[r]), p[r], m[r], u[r]) for r in rows]
        return {"token": torch.tensor([g[0] for g in got], dtype=torch.int32),
                "logprob": torch.tensor([g[1] for g in got], dtype=torch.float64),
                "support_size": torch.tensor([g[2] for g in got], dtype=torch.int32)}
    if case["op"] == "topk":
        k = min(case["k"], case["vocab"])
        t = s["temperature"].double().tolist()
        ids = torch.empty((len(x), k), dtype=torch.int32, device=x.device)
        lp = torch.empty((len(x), k), dtype=torch.float64, device=x.device)
        for r in rows:
            y = x[r].double()
            ids[r] = torch.argsort(-y, stable=True)[:k].to(torch.int32)
            lp[r] = torch.log_softmax(y / t[r], 0)[ids[r].long()]
        return {"ids": ids, "logprob": lp}
    t, g = s["temperature"].double().tolist(), s["g_loss"].double().tolist()
    loss = torch.empty(len(x), dtype=torch.float64, device=x.device)
    valid = torch.empty(len(x), dtype=torch.uint8, device=x.device)
    grad = torch.empty(x.shape, dtype=torch.float64, device=x.device) if case["step"] != "fwd" else None
    for r in rows:
        loss[r], valid[r], d = _exact_distill_row(x[r].double(), t[r], s["ids"][r], s["logprob"][r], case["tail"], g[r])
        if grad is not None:
            grad[r] = d
    out = {"loss": loss, "valid": valid}
    if grad is not None:
        out["grad"] = grad
    return out
