"""vs_distill_fwd / vs_distill_bwd over the whole range of their inputs: masks
by a finite value, logits with a common offset, small and large temperatures,
teacher values of any size, almost all of the teacher's mass on the list, a
loss near zero.

The bounds.  The factor log2(e) / T is rounded to fp32 (a relative d of at most
2^-23); logits are subtracted before they are multiplied, or the product's
rounding is put back, so

* loss: d moves log q_k by d |z_k - E z|; the a-weighted sum of those distances
  is at most the loss, plus the entropies (log 1,024, log of the vocabulary:
  below 30 together).  The normaliser's fp32 exponentials are worth at most
  1.5e-5 (2^-22 each, 2^-23 of an argument of at most 60, 2^-24 for each of at
  most 96 additions), the tail's the same.  With the rounding of the result,
  |error| <= 4e-5 + 2^-22 |loss|.
* gradient of element j, over g / T: q_j and a_j relative to themselves by the
  normaliser's 1e-5 and by d |z_j - z_max| <= 2^-23 * 87 = 1e-5 (beyond 87 nats
  q_j is below 2^-125): 2e-5 in all; outside the list the same of the product
  r_j (q_t - a_t); the stored value by half a step of its type."""

import numpy as np
import pytest
import torch

import sampling_support_b200 as vsb
from _row_ops import logits_on, widen

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def two_calls(x, ids, lp, t, tail, vocab, grad_dtype, g):
    """(loss, valid, status, gradient) of a forward and a backward call."""
    kw = dict(temperature=t, tail=tail, vocab=vocab)
    out = vsb.distill_fwd(x, ids, lp, want_grad=True, **kw)
    grad = vsb.distill_bwd(x, ids, lp, out["ctx"], g, grad_dtype=grad_dtype, **kw)
    return out["loss"], out["valid"], out["status"], grad[:, :vocab]


def log_sum(z):
    top = z.max()
    return top + np.log(np.exp(z - top).sum())


def plain_row(x, ids, lp, t, tail):
    """(loss, valid, gradient, q, a over the vocabulary) of a row without masked tokens whose list has different
    ids in the vocabulary; a share far below fp64's range keeps its logarithm."""
    with np.errstate(over="ignore"):
        z = x / t
    z = z - z.max()
    logq = z - log_sum(z)
    lp = lp.astype(np.float64)
    la = lp if tail else lp - lp.max() - log_sum(lp - lp.max())
    a = np.exp(la)
    loss = float((a * (la - logq[ids])).sum())
    full = np.zeros(len(x))
    full[ids] = a
    q = np.exp(logq)
    grad = q - full
    off = np.ones(len(x), bool)
    off[ids] = False
    if tail and off.any():
        rest, log_qt = max(0.0, 1.0 - a.sum()), log_sum(logq[off])
        if rest > 0:
            loss += rest * (np.log(rest) - log_qt)
        r = np.exp(z[off] - z[off].max())
        grad[off] = r / r.sum() * (np.exp(log_qt) - rest)
    return loss, 1, grad / t, q, full


def one_call(x, ids, lp, t, tail, vocab, grad_dtype, g):
    out = vsb.distill_fwd(x, ids, lp, temperature=t, tail=tail, vocab=vocab, g_loss=g, grad_dtype=grad_dtype)
    return out["loss"], out["valid"], out["status"], out["grad"][:, :vocab]


WAYS = [two_calls, one_call]


def check(x, ids, lp, t, tail, vocab, grad_dtype=F32, g=1.0):
    xs, li, ll = widen(x[:, :vocab]), ids.cpu().numpy(), lp.cpu().numpy()
    gs = torch.full((len(x),), g, device="cuda")
    ways = [f(x, ids, lp, t, tail, vocab, grad_dtype, gs) for f in WAYS]
    torch.cuda.synchronize()
    tr, gr = float(np.float32(t)), float(np.float32(g))
    half = torch.finfo(grad_dtype).eps / 2
    for r in range(len(xs)):
        want, ok, d, q, a = plain_row(xs[r], li[r], ll[r], tr, tail)
        d = d * gr
        tol = 2e-5 * gr / tr * (q + a) + 2e-5 * np.abs(d) + half * np.abs(d) * (1 + 1e-4) + 1e-37
        for way, (loss, valid, status, grad) in zip([f.__name__ for f in WAYS], ways):
            assert int(valid[r]) == ok and int(status[r]) == 0, (way, r)
            got = float(loss[r])
            assert abs(got - want) <= 4e-5 + 2.0 ** -22 * abs(want), (way, r, got, want)
            off = np.abs(widen(grad[r]) - d) - tol
            worst = int(np.argmax(np.where(np.isnan(off), np.inf, off)))
            assert off[worst] <= 0, (way, r, worst, float(grad[r, worst]), d[worst])


def listed(rows, vocab, k, seed):
    """k different ids per row and log-probabilities that leave about a fifth of the mass."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(rows)]).to(torch.int32)
    lp = torch.log(0.8 * torch.softmax(torch.randn((rows, k), generator=g), 1))
    return ids, lp


MASKS = [-1e4, -1e6, -1e7, -1e9, -1e10, -1e14, -1e30]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("vocab", [1003, 20_011])
def test_finite_masks(dtype, tail, mask, vocab):
    """Constrained decoding with a finite mask: every token off the list masked,
    most of them, the whole row, and listed tokens too."""
    rows, k = 4, 20
    x = logits_on("cpu", rows, vocab, F32, seed=vocab, ld=vocab + (-vocab) % 8)
    ids, lp = listed(rows, vocab, k, seed=31)
    on = torch.zeros((rows, x.shape[1]), dtype=torch.bool).scatter_(1, ids.long(), True)
    some = torch.rand((rows, x.shape[1]), generator=torch.Generator().manual_seed(32)) < 0.9
    x[0] = torch.where(on[0], x[0], torch.tensor(mask))
    x[1] = torch.where(~on[1] & some[1], torch.tensor(mask), x[1])
    x[2] = mask
    x[3] = torch.where(some[3], torch.tensor(mask), x[3])
    check(x.to(dtype).cuda(), ids.cuda(), lp.cuda(), 1.0, tail, vocab, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_finite_masks_of_the_largest_vocabularies(dtype):
    rows, vocab, k = 2, 1 << 20, 20
    x = logits_on("cpu", rows, vocab, F32, seed=3)
    ids, lp = listed(rows, vocab, k, seed=33)
    on = torch.zeros((rows, vocab), dtype=torch.bool).scatter_(1, ids.long(), True)
    x[0] = torch.where(on[0], x[0], torch.tensor(-1e9))
    x[1, ::2] = -1e9
    check(x.to(dtype).cuda(), ids.cuda(), lp.cuda(), 1.0, True, vocab, dtype)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("offset", [1e3, -1e4, 1e6, -1e6, 1e7])
@pytest.mark.parametrize("vocab", [1003, 20_011])
def test_common_offsets(tail, offset, vocab):
    x = logits_on("cuda", 3, vocab, F32, seed=7) + offset
    ids, lp = listed(3, vocab, 30, seed=34)
    check(x, ids.cuda(), lp.cuda(), 1.0, tail, vocab)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("t", [1e-2, 1e-3, 1e-5, 1e-6, 1e-9, 1e-12])
@pytest.mark.parametrize("vocab", [1003, 20_011])
def test_small_temperatures(dtype, tail, t, vocab):
    """The row's largest token on the list, off it, and shared by both."""
    x = logits_on("cuda", 3, vocab, dtype, seed=8, spikes=0)
    ids, lp = listed(3, vocab, 30, seed=35)
    x[0, int(ids[0, 3])] = 14.0
    out = next(j for j in range(500, vocab) if j not in ids[1].tolist())
    x[1, out] = 14.0
    x[2, int(ids[2, 0])] = x[2, next(j for j in range(700, vocab) if j not in ids[2].tolist())] = 14.0
    check(x, ids.cuda(), lp.cuda(), t, tail, vocab)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("vocab", [1003, 20_011, 1 << 20])
def test_differences_beyond_fp32(dtype, tail, vocab):
    """Logits at both ends of the type: their difference overflows fp32, their
    difference over T does not."""
    g = torch.Generator().manual_seed(9)
    x = ((torch.rand((3, vocab + (-vocab) % 8), generator=g) * 2 - 1) * 3.0e38).to(dtype).cuda()
    x[1, :vocab] = -3.0e38
    x[1, 5] = 3.0e38
    x[2, :vocab:2] = 3.0e38
    ids, lp = listed(3, vocab, 30, seed=36)
    check(x, ids.cuda(), lp.cuda(), 1e38, tail, vocab, g=1e30)


@pytest.mark.parametrize("offset", [30.0, -1e3, 1e4, 1e6, -1e9, 1e30])
@pytest.mark.parametrize("vocab", [1003, 1 << 20])
def test_teacher_logits_of_any_size(offset, vocab):
    """List mode takes any logits: a common offset (and what it rounds away
    from the values, which the plain form sees too) changes nothing."""
    x = logits_on("cuda", 3, vocab, F32, seed=10)
    ids, lp = listed(3, vocab, 30, seed=37)
    check(x, ids.cuda(), (lp + offset).cuda(), 1.0, False, vocab)


@pytest.mark.parametrize("vocab", [1003, 20_011])
def test_a_list_with_almost_all_of_the_mass(vocab):
    """The list leaves 1e-6, the student almost nothing: outside the list the
    gradient is -a_t r_j, so a_t = 1 - sum a has to hold to 2e-5 of itself,
    2e-11 of the sum.  The shares lie half way between powers of two, where a
    polynomial in the exponent's fraction is at its worst."""
    share = [2.0 ** -0.5, 2.0 ** -2.5, 2.0 ** -3.5]
    share.append(1 - 1e-6 - sum(share))
    lp = torch.log(torch.tensor([share, share[::-1]], dtype=torch.float64)).float()
    ids = torch.tensor([[3, 501, 77, 1002], [7, 9, 1000, 6]], dtype=torch.int32)
    x = logits_on("cpu", 2, vocab, F32, seed=11, sigma=1.0, spikes=0)
    x.scatter_(1, ids.long(), lp + 30.0)
    check(x.cuda(), ids.cuda(), lp.cuda(), 1.0, True, vocab)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [1003, 20_011, 151_936])
def test_a_loss_near_zero(dtype, vocab):
    """A teacher close to its student.  The loss is a difference of logarithms
    of about its square in size, so it is taken in fp64, and the fp32 parts
    enter by derivatives that vanish with it: the share outside the list (off by
    e <= 5e-6: 2^-22 for the exponential, 2^-24 of an argument of at most 60,
    2^-24 for each of at most 24 additions, 2^-22 and 2^-23 * 30 for a thread's
    reference) by (q_t - a_t) e, the factor 1 / T (2^-23) by the difference of
    the means of z under q and under a.  The result is rounded once; 1e-11 for
    the squares and for fp64."""
    rows, k = 6, 64
    x = logits_on("cuda", rows, vocab, dtype, seed=12)
    g = torch.Generator().manual_seed(38)
    xs = x[:, :vocab].double().cpu()
    y = xs + 0.03 * torch.randn(xs.shape, generator=g, dtype=torch.float64)
    v, ids = torch.topk(y, k, dim=1)
    lp = (v - torch.logsumexp(y, 1, keepdim=True)).float()
    out = vsb.distill_fwd(x, ids.to(torch.int32).cuda(), lp.cuda(), tail=True, vocab=vocab)
    for r in range(rows):
        li, ll = ids[r].numpy(), lp[r].numpy()
        z = xs[r].numpy()
        want, _, _, q, a = plain_row(z, li, ll, 1.0, True)
        off = np.ones(vocab, bool)
        off[li] = False
        qt, at = q[off].sum(), 1 - a.sum()
        mean = ((q[li] - a[li]) * z[li]).sum() + (qt - at) * (q[off] * z[off]).sum() / qt
        tol = 5e-6 * abs(qt - at) + 2.0 ** -23 * abs(mean) + 2.0 ** -24 * want + 1e-11
        assert want < 2e-3 and tol < 2e-7
        assert abs(float(out["loss"][r]) - want) <= tol, (r, float(out["loss"][r]), want, tol)


def test_one_row_of_lists_of_different_widths():
    x = logits_on("cuda", 1, 1003, F32, seed=13)
    ids, lp = listed(2, 1003, 30, seed=39)
    wide = torch.zeros((2, 50))
    wide[:, :30] = lp
    check(x, ids.cuda()[1:], wide.cuda()[1:, :30], 1.0, True, 1003)
