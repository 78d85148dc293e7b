"""vs_topk_logprob against the 64-bit plain form.

Ids are equal.  A log-probability is (l - max) / T - log Z with Z summed in
fp32: each of its terms is off by 2^-22 (exponential) and by 2^-22 |argument|
(its rounded factor and product), whose mean over the terms is at most
log2(vocab) <= 18, and a thread adds at most 160 of them one after another
(2^-24 each) before a tree of at most 20: below 1.6e-5 of Z in all; the
rounded difference, quotient and result add 2^-22 of the value."""

import numpy as np
import pytest
import torch

import sampling_support_b200 as vsb
from _row_ops import logits_on, topk_row, widen

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def check(x, k, vocab=None, temperature=1.0, **kw):
    vocab = x.shape[1] if vocab is None else vocab
    out = vsb.topk_logprob(x, k, temperature=temperature, vocab=vocab, **kw)
    torch.cuda.synchronize()
    xs = widen(x[:, :vocab])
    for r in range(len(xs)):
        t = float(temperature[r]) if isinstance(temperature, torch.Tensor) else float(np.float32(temperature))
        ids, lp = topk_row(xs[r], k, t)
        assert out["ids"][r].tolist() == ids.tolist()
        got = out["logprob"][r].double().cpu().numpy()
        fin = np.isfinite(lp)
        assert np.array_equal(got[~fin], lp[~fin])
        assert (np.abs(got[fin] - lp[fin]) <= 2e-5 + 2.0 ** -22 * np.abs(lp[fin])).all()
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab,k", [(1, 1), (7, 7), (33, 8), (1000, 1), (1000, 1000), (4097, 64), (20_011, 1024),
                                     (20_011, 257), (151_936, 64), (151_936, 1000)])
@pytest.mark.parametrize("rows", [3, 80])
def test_sizes(dtype, vocab, k, rows):
    x = logits_on("cuda", rows, vocab, dtype, seed=vocab + k)
    check(x, k, vocab, temperature=0.9)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab,k,rows", [(2876, 727, 58), (2785, 161, 300), (4096, 192, 200), (4099, 193, 40),
                                          (4096, 768, 30), (4096, 769, 30), (8001, 1024, 20), (1100, 1024, 9)])
def test_wide_lists_of_small_vocabularies(dtype, vocab, k, rows):
    x = logits_on("cuda", rows, vocab, dtype, seed=vocab + k)
    x[0, : vocab // 2] = float("-inf")
    x[1, k // 2 : vocab] = float("-inf")  # fewer than k tokens
    x[2, : vocab - 5] = torch.randint(0, 3, (vocab - 5,), generator=torch.Generator().manual_seed(k)).to(dtype).cuda()
    check(x, k, vocab, temperature=1.1)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [1, 20, 700])
def test_ties_and_crowds(dtype, k):
    """Equal values beyond any list's room, sorted rows, few distinct values,
    values near the type's ends."""
    rows, vocab = 7, 50_000
    g = torch.Generator().manual_seed(k)
    x = torch.randn((rows, vocab), generator=g)
    x[0] = 0.0
    x[1] = torch.arange(vocab, 0, -1) / vocab
    x[2] = torch.arange(vocab) / vocab
    x[3] = torch.randint(0, 2, (vocab,), generator=g).float()
    x[4, :300] = 9.0
    x[5] = x[5].sign() * 3.0e38
    x[6, 1000:] = 2.0
    check(x.to(dtype).cuda(), k)
    check(x.to(dtype).cuda(), k, temperature=50.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [1, 256, 1024])
def test_largest_vocabulary(dtype, k):
    """Rows that no cluster's shared memory holds, and one in between, one of
    them a crowd."""
    for vocab in (1 << 20, 300_001):
        x = logits_on("cuda", 3, vocab, dtype, seed=k)
        x[1, :vocab] = 1.0
        x[1, 1000:vocab:1000] = 2.0
        check(x, k, vocab)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_and_bad_rows(dtype):
    rows, vocab, k = 8, 5003, 40
    x = logits_on("cuda", rows, vocab, dtype, seed=2)
    x[0, 10:] = float("-inf")  # ten tokens
    x[1] = float("-inf")
    x[1, 77] = 1.0
    good = x.clone()
    good[2:] = logits_on("cuda", rows - 2, vocab, dtype, seed=3)
    check(good, k, vocab)
    x[2] = float("-inf")
    x[3, 5002] = float("nan")
    x[4, 0] = float("inf")
    t = torch.ones(rows, device="cuda")
    t[5], t[6] = 0.0, float("nan")
    out = vsb.topk_logprob(x, k, temperature=t, vocab=vocab)
    assert out["status"].tolist() == [0, 0, vsb.ROW_EMPTY_SUPPORT, vsb.ROW_NONFINITE_INPUT, vsb.ROW_NONFINITE_INPUT,
                                      vsb.ROW_BAD_PARAM, vsb.ROW_BAD_PARAM, 0]
    assert (out["ids"][2:7] == -1).all()
    assert (out["logprob"][2] == float("-inf")).all() and torch.isnan(out["logprob"][3:7]).all()


def test_views_temperatures_stream_and_capture():
    big = logits_on("cuda", 20, 4096, BF, seed=5)
    view = big[1:20:3, 8:8 + 3001]
    t = torch.rand(view.shape[0], generator=torch.Generator().manual_seed(1)).cuda() + 0.3
    check(view, 33, temperature=t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check(view, 33, temperature=t, stream=side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = vsb.topk_logprob(view, 33, temperature=t)
    big.copy_(logits_on("cuda", 20, 4096, BF, seed=6))
    g.replay()
    torch.cuda.synchronize()
    again = check(view, 33, temperature=t)
    assert torch.equal(out["ids"], again["ids"]) and torch.equal(out["logprob"], again["logprob"])


def test_agrees_with_the_fused_head():
    """The list from logits in memory and the one from hidden states name the
    same tokens where the fp32 products decide alike."""
    g = torch.Generator().manual_seed(3)
    h = torch.randn((32, 128), generator=g).to(BF).cuda()
    w = (torch.randn((2048, 128), generator=g) * 0.2).to(BF).cuda()
    y = torch.zeros(32, dtype=torch.int32, device="cuda")
    head = vsb.fused_lmhead_score(h, w, y, 0.8, 16, 1.0, 0.0)
    logits = h.float() @ w.float().t()
    out = vsb.topk_logprob(logits.contiguous(), 16, temperature=0.8)
    same = out["ids"] == head["topk_ids"]
    assert same.float().mean() > 0.95  # neighbours within fp32 rounding may trade places
    assert (out["logprob"] - head["topk_logprob"])[same].abs().max() < 1e-4
