"""vs_topk_logprob over the whole range of its logits and temperatures: masks by
a finite value, common offsets, small temperatures.

Ids are equal.  The row's sum is off by at most 1.5e-5 (2^-22 for each fp32
exponential, 2^-23 of an argument of at most 60, 2^-24 for each of at most 96
additions); the difference, the quotient and the result are rounded once each,
and the factor log2(e) / T (2^-23) moves log Z by at most 2^-23 of a mean distance
below 60 nats: 2^-22 of the value and 2.5e-5 in all."""

import numpy as np
import pytest
import torch

import sampling_support_b200 as vsb
from _row_ops import logits_on, topk_row, widen

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def check(x, k, vocab, t):
    out = vsb.topk_logprob(x, k, temperature=t, vocab=vocab)
    torch.cuda.synchronize()
    xs = widen(x[:, :vocab])
    for r in range(len(xs)):
        ids, lp = topk_row(xs[r], k, float(np.float32(t)))
        assert int(out["status"][r]) == 0 and out["ids"][r].tolist() == ids.tolist()
        got = out["logprob"][r].double().cpu().numpy()
        off = np.abs(got - lp) - (2.5e-5 + 2.0 ** -22 * np.abs(lp))
        assert (off <= 0).all(), (r, got[off > 0], lp[off > 0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [1003, 20_011, 1 << 20])
@pytest.mark.parametrize("mask", [-1e4, -1e6, -1e9, -1e10, -1e30])
def test_finite_masks(dtype, vocab, mask):
    x = logits_on("cuda", 3, vocab, F32, seed=vocab, ld=vocab + (-vocab) % 8)
    x[0, 30:] = mask
    x[1, torch.rand(x.shape[1], generator=torch.Generator().manual_seed(1)).cuda() < 0.9] = mask
    x[2] = mask
    check(x.to(dtype), 60, vocab, 1.0)


@pytest.mark.parametrize("vocab", [1003, 20_011])
@pytest.mark.parametrize("offset", [1e3, -1e4, 1e6, 1e7])
def test_common_offsets(vocab, offset):
    check(logits_on("cuda", 3, vocab, F32, seed=5) + offset, 60, vocab, 1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [1003, 20_011])
@pytest.mark.parametrize("t", [1e-2, 1e-3, 1e-6, 1e-9, 1e-12])
def test_small_temperatures(dtype, vocab, t):
    check(logits_on("cuda", 3, vocab, dtype, seed=6), 60, vocab, t)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [1003, 20_011, 1 << 20])
def test_differences_beyond_fp32(dtype, vocab):
    """Logits at both ends of the type: their difference overflows fp32, their
    difference over T does not."""
    g = torch.Generator().manual_seed(9)
    x = ((torch.rand((3, vocab + (-vocab) % 8), generator=g) * 2 - 1) * 3.0e38).to(dtype).cuda()
    x[1, :vocab] = -3.0e38
    x[1, 5] = 3.0e38
    check(x, 60, vocab, 1e38)
