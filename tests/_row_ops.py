"""Plain 64-bit forms of the row operators (numpy), written from their
formulas, one row at a time: sampling from a given uniform number, top-k
log-probabilities, and distillation from a teacher's list with its gradient."""

from __future__ import annotations

import numpy as np
import torch

MASKED = -np.inf


def widen(t: torch.Tensor) -> np.ndarray:
    return t.double().cpu().numpy()


def order_of(x: np.ndarray) -> np.ndarray:
    """Unmasked token ids in the total order: value descending, id ascending."""
    ids = np.flatnonzero(x > MASKED)
    return ids[np.argsort(-x[ids], kind="stable")]


def sample_row(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, logprob, support size) of one row in fp64."""
    by = order_of(x)
    if len(by) == 0 or np.isnan(x).any() or np.isposinf(x).any():
        return -1, np.nan, 0
    if t == 0:
        return int(by[0]), 0.0, 1
    z = (x[by] - x[by[0]]) / t
    if 0 < k < len(z):
        z = z[:k]
    w = np.exp(z)
    c = np.cumsum(w)
    n = len(w)
    if p < 1:
        n = min(n, int(np.count_nonzero(c < p * c[-1])) + 1)
    if m > 0:
        n = min(n, int(np.count_nonzero(w >= m)))
    at = min(int(np.count_nonzero(c[:n] <= u * c[n - 1])), n - 1)
    return int(by[at]), float(z[at] - np.log(c[n - 1])), n


def topk_row(x, k, t=1.0):
    """(ids, logprobs) of one row, padded with -1 and -inf."""
    ids, lp = np.full(k, -1, np.int64), np.full(k, -np.inf)
    by = order_of(x)
    z = (x[by] - x[by[0]]) / t
    n = min(k, len(by))
    ids[:n] = by[:n]
    lp[:n] = z[:n] - np.log(np.exp(z).sum())
    return ids, lp


def distill_row(x, ids, lp, t=1.0, tail=False):
    """(loss, valid, gradient, q, a over the vocabulary) of one row."""
    vocab = len(x)
    seen, keep = set(), []
    for s, i in enumerate(ids):
        if 0 <= i < vocab and i not in seen:
            seen.add(i)
            keep.append(s)
    ids, lp = ids[keep], lp[keep].astype(np.float64)
    zero = np.zeros(vocab)
    z = x / t
    e = np.exp(z - z.max())
    q = e / e.sum()
    with np.errstate(divide="ignore"):
        logq = z - z.max() - np.log(e.sum())
    if len(ids) == 0 or (not tail and not (lp > -np.inf).any()):
        return 0.0, 0, zero, q, zero
    if tail:
        la = lp
    else:
        top = lp.max()
        la = lp - top - np.log(np.exp(lp - top).sum())
    a = np.exp(la)
    has = a > 0
    loss = float((a[has] * (la[has] - logq[ids[has]])).sum())
    full = zero.copy()
    full[ids] = a
    grad = q - full
    if tail:
        out = np.ones(vocab, bool)
        out[ids] = False
        rest, qt = max(0.0, 1.0 - a.sum()), q[out].sum()
        if out.any() and e[out].sum() > 0:
            log_qt = np.log(e[out].sum()) - np.log(e.sum())
            if rest > 0:
                loss += rest * (np.log(rest) - log_qt)
            grad[out] = e[out] / e[out].sum() * (qt - rest)
    return loss, 1, grad / t, q, full


def logits_on(device, rows, vocab, dtype, seed, sigma=3.0, spikes=4, ld=None, pad=float("nan")):
    """[rows, ld] logits of N(0, sigma) with raised tokens; the pad columns hold `pad`."""
    per = 8 if dtype == torch.bfloat16 else 4
    ld = (vocab + per - 1) // per * per if ld is None else ld
    g = torch.Generator().manual_seed(seed)
    x = torch.full((rows, ld), pad)
    x[:, :vocab] = torch.randn((rows, vocab), generator=g) * sigma
    at = torch.randint(0, vocab, (rows, spikes), generator=g)
    x.scatter_add_(1, at, torch.full(at.shape, 6.0))
    return x.to(dtype).to(device)
