"""vs_sample against the 64-bit plain form: tokens and support sizes equal,
log-probabilities within their rounding.

The kernel's masses are fp64 exponentials in fixed point, vocab * 2^fx <= 2^62:
each is off by at most 2^-(fx+1) of the largest (1), so a support's mass, at
least 1, is off by at most vocab * 2^-(fx+1) <= 2^21 * 2^-42 relative, below
2^-21 for the largest vocabulary and below 2^-28 for the ones here; the result
is rounded once to fp32 (2^-24 relative)."""

import numpy as np
import pytest
import torch

import sampling_support_b200 as vsb
from _row_ops import logits_on, sample_row, widen
from sampling_support_b200 import _binding as B

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def close_logprob(got, want):
    got = got.double().cpu().numpy()
    both = np.isnan(got) & np.isnan(want)
    bad = ~both & ~(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -28)
    assert not bad.any(), (got[bad], want[bad])


def per_row(v, r):
    return float(v[r]) if isinstance(v, torch.Tensor) else v


def check(x, u, vocab=None, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
    vocab = x.shape[1] if vocab is None else vocab
    out = vsb.sample(x, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, vocab=vocab,
                     stream=stream)
    torch.cuda.synchronize()
    compare(out, x, u, vocab, temperature, top_k, top_p, min_p)
    return out


def compare(out, x, u, vocab, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    xs = widen(x[:, :vocab])
    f32 = lambda v, r: per_row(v, r) if isinstance(v, torch.Tensor) else float(np.float32(v))
    want = [sample_row(xs[r], per_row(u, r), f32(temperature, r), int(per_row(top_k, r)), f32(top_p, r),
                       f32(min_p, r)) for r in range(len(xs))]
    assert out["support_size"].tolist() == [w[2] for w in want]
    assert out["token"].tolist() == [w[0] for w in want]
    close_logprob(out["logprob"], np.array([w[1] for w in want]))


def numbers(rows, seed):
    return torch.rand(rows, generator=torch.Generator().manual_seed(seed)).cuda()


FILTERS = {
    "none": {}, "k1": dict(top_k=1), "k50": dict(top_k=50, top_p=0.95), "p": dict(top_p=0.9),
    "p_small": dict(top_p=1e-6), "m": dict(min_p=0.05), "all": dict(top_k=40, top_p=0.8, min_p=0.02),
    "pm": dict(top_p=0.97, min_p=0.01), "big_k": dict(top_k=700, top_p=0.99), "huge_k": dict(top_k=5000, min_p=1e-5),
}


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [1, 7, 8, 33, 1000, 4097, 20_011])
@pytest.mark.parametrize("name", sorted(FILTERS))
def test_sizes_and_filters(dtype, vocab, name):
    rows = 9
    x = logits_on("cuda", rows, vocab, dtype, seed=vocab)
    check(x, numbers(rows, 1), vocab, temperature=0.85, **FILTERS[name])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 40, 149])
def test_benchmark_vocabulary(dtype, rows):
    """One row on a whole cluster, a few CTAs per row, one CTA per row."""
    vocab = 151_936
    x = logits_on("cuda", rows, vocab, dtype, seed=rows)
    g = torch.Generator().manual_seed(rows)
    pick = lambda a, b: torch.where(torch.rand(rows, generator=g) < 0.5, a, b).cuda()
    one = torch.ones(rows)
    check(x, numbers(rows, 2), vocab, temperature=pick(0.7 * one, 1.1 * one),
          top_k=pick(0 * one, 60 * one).to(torch.int32), top_p=pick(one, 0.95 * one), min_p=pick(0 * one, 0.02 * one))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_ends_of_the_uniform_number(dtype):
    x = logits_on("cuda", 6, 5000, dtype, seed=3)
    u = torch.tensor([0.0, 1.0, 1 - 2.0 ** -24, 2.0 ** -24, 0.5, 2.0 ** -126]).cuda()
    for kw in (dict(), dict(top_k=30), dict(top_p=0.9), dict(min_p=0.1)):
        check(x, u, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [4, 4096, 20_000, 131_072])
def test_equal_logits_cut_exactly(dtype, vocab):
    """Every token the same: shares are exact, so are the cuts, and one value
    is shared by more tokens than any list holds."""
    x = torch.zeros((5, max(vocab, 8)), dtype=dtype, device="cuda")
    x[4] = -torch.finfo(dtype).max  # all at the type's lowest value: a uniform row too
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0]).cuda()
    for kw in (dict(), dict(top_p=0.5), dict(top_k=vocab // 2), dict(min_p=0.5)):
        check(x, u, vocab, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("temperature", [1e-40, 1e-30, 1e-3, 0.05, 30.0, 1e6])
def test_temperatures(dtype, temperature):
    x = logits_on("cuda", 8, 12_000, dtype, seed=4)
    for kw in (dict(), dict(top_p=0.7), dict(top_k=20), dict(top_k=3000), dict(min_p=0.3)):
        check(x, numbers(8, 5), temperature=temperature, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_values_far_apart_and_crowded(dtype):
    """An outlier far above a crowd of nearby values (the crowd falls into few
    bins), values near the type's ends, tiny values of both signs, and few
    distinct values."""
    rows, vocab = 6, 30_000
    g = torch.Generator().manual_seed(8)
    x = torch.randn((rows, vocab), generator=g)
    x[0] = x[0] * 1e-3
    x[0, 7] = 900.0
    x[1] = x[1].sign() * 3.0e38
    x[2] = x[2] * 1e-30
    x[3] = torch.randint(0, 3, (vocab,), generator=g).float()
    x[4] = 300.0 + x[4] * 0.01
    x[5, :] = -3.0e38
    x[5, 100:110] = 3.0e38
    x = x.to(dtype).cuda()
    for t in (0.5, 1.0, 400.0):
        for kw in (dict(), dict(top_p=0.6), dict(top_k=9), dict(top_k=10_001), dict(min_p=0.9), dict(top_p=0.9999)):
            check(x, numbers(rows, 9), temperature=t, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_tokens(dtype):
    """-inf is in no set: a few tokens left, one, none; the type's lowest value
    is an ordinary logit."""
    rows, vocab = 7, 9001
    x = logits_on("cuda", rows, vocab, dtype, seed=6)
    keep = torch.rand((rows, x.shape[1]), generator=torch.Generator().manual_seed(7)).cuda() < 0.01
    x = torch.where(keep, x, torch.full_like(x, float("-inf")))
    x[1] = float("-inf")
    x[1, 8999] = -5.0
    x[2] = float("-inf")
    x[3] = torch.where(keep[3], x[3], torch.full_like(x[3], -torch.finfo(dtype).max))
    for kw in (dict(), dict(top_k=200), dict(top_k=2000), dict(top_p=0.9), dict(min_p=0.001)):
        out = check(x, numbers(rows, 3), vocab, **kw)
        assert out["status"].tolist() == [0, 0, vsb.ROW_EMPTY_SUPPORT, 0, 0, 0, 0]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("top_k", [0, 5])
def test_rows_without_a_token(dtype, top_k):
    x = logits_on("cuda", 12, 3001, dtype, seed=1)
    x[0, 3000] = float("nan")
    x[1, 17] = float("inf")
    x[2, :3001] = float("nan")
    x[11, 5] = -float("nan")
    u = numbers(12, 1)
    t = torch.full((12,), 0.9, device="cuda")
    p, m = torch.ones(12, device="cuda"), torch.zeros(12, device="cuda")
    u[3], u[4], u[5] = -0.1, 1.5, float("nan")
    t[6], t[7] = -1.0, float("nan")
    p[8], m[9] = 0.0, 1.5
    t[10] = float("inf")
    out = vsb.sample(x, u, temperature=t, top_p=p, min_p=m, top_k=top_k, vocab=3001)
    torch.cuda.synchronize()
    assert out["token"].tolist() == [-1] * 12
    assert out["support_size"].tolist() == [0] * 12
    assert torch.isnan(out["logprob"]).all()
    assert out["status"].tolist() == [vsb.ROW_NONFINITE_INPUT] * 3 + [vsb.ROW_BAD_PARAM] * 8 + [vsb.ROW_NONFINITE_INPUT]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_greedy_and_per_row_settings(dtype):
    rows, vocab = 16, 6007
    x = logits_on("cuda", rows, vocab, dtype, seed=11)
    x[0, :vocab] = 1.5  # ties: the lowest id
    g = torch.Generator().manual_seed(2)
    t = torch.rand(rows, generator=g).cuda() + 0.2
    t[::4] = 0.0
    k = torch.randint(-1, 900, (rows,), generator=g).to(torch.int32).cuda()
    p = (torch.rand(rows, generator=g) + 0.3).cuda()  # some above 1: disabled
    m = (torch.rand(rows, generator=g) * 0.2 - 0.1).cuda()  # some below 0: disabled
    m[5], t[5] = 1.0, 1.0  # only the largest
    out = check(x, numbers(rows, 4), vocab, t, k, p, m)
    assert out["token"][0] == 0 and out["logprob"][0] == 0 and (out["support_size"][::4] == 1).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_views_and_batch_independence(dtype):
    big = logits_on("cuda", 24, 2048, dtype, seed=12)
    view = big[3:21:2, 64:64 + 1777]  # every other row, an offset of whole vectors, an odd width
    u = numbers(9, 6)
    a = check(view, u, top_p=0.9)
    one = vsb.sample(view[4:5], u[4:5], top_p=0.9)
    assert one["token"].item() == a["token"][4].item() and one["logprob"].item() == a["logprob"][4].item()


def test_another_stream_and_a_captured_call():
    x = logits_on("cuda", 5, 30_000, BF, seed=13)
    u = numbers(5, 7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check(x, u, top_p=0.95, stream=side)
    vsb.sample(x, u, top_k=40)
    graphs = []
    for kw in (dict(top_p=0.9), dict(top_k=40)):  # two graphs of the same inputs, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = vsb.sample(x, u, **kw)
        graphs.append((g, out, kw))
    for turn in range(3):
        x.copy_(logits_on("cuda", 5, 30_000, BF, seed=20 + turn))
        u.copy_(numbers(5, 30 + turn))
        for g, out, kw in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, out, kw in graphs:
            compare(out, x, u, 30_000, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [515, 40_000])
def test_zeros_of_either_sign_are_equal(dtype, vocab):
    x = logits_on("cuda", 6, vocab, dtype, seed=15)
    x[x.abs() < 0.7] = 0.0
    x[:, ::3] *= -1.0  # zeros of both signs, in no order
    x[2:] = x[2:].clamp(max=0.0)  # and as the largest values
    x[4:, 5::7] = 2.0 ** -40  # next to values near them
    u = numbers(6, 9)
    for kw in (dict(top_k=3), dict(top_k=vocab // 5), dict(top_p=0.3), dict(min_p=0.9), dict(temperature=0.0), {}):
        check(x, u, vocab, **kw)


def test_calls_at_once_from_two_threads():
    import threading

    x = [logits_on("cuda", rows, 60_000, dtype, seed=16) for rows, dtype in ((3, BF), (20, F32))]
    y = [t.to(BF) for t in x]
    u = [numbers(3, 10), numbers(20, 11)]
    kw = [dict(top_p=0.9), dict(top_k=30)]
    torch.cuda.synchronize()
    outs = [[], []]

    def work(i):
        stream = torch.cuda.Stream()
        for _ in range(40):
            outs[i].append(vsb.sample(x[i], u[i], stream=stream, **kw[i]))
            outs[i].append(vsb.topk_logprob(y[i], (50, 900)[i], stream=stream))  # of different shared memory
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        compare(outs[i][0], x[i], u[i], 60_000, **kw[i])
        for j, out in enumerate(outs[i]):
            for name, t in out.items():
                assert torch.equal(t, outs[i][j % 2][name]), (i, j, name)


def test_a_top_k_beyond_32_bits_keeps_every_token():
    x, u = logits_on("cuda", 2, 1000, F32, seed=17), numbers(2, 12)
    out = vsb.sample(x, u, top_k=(1 << 32) + 1, vocab=1000)
    assert out["support_size"].tolist() == [1000, 1000]
    with pytest.raises(vsb.VsError):
        vsb.topk_logprob(x, (1 << 32) + 1)


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows read their own logits."""
    vocab = 151_936
    rows = 2 ** 31 // vocab + 8
    x = torch.zeros((rows, vocab), dtype=BF, device="cuda")
    tail = logits_on("cuda", 4, vocab, BF, seed=14)
    x[-4:] = tail
    u = numbers(rows, 8)
    out = vsb.sample(x, u, top_k=40)
    out2 = vsb.sample(x, u, top_p=0.9)
    top = vsb.topk_logprob(x, 8)
    torch.cuda.synchronize()
    compare({n: v[-4:] for n, v in out.items()}, tail, u[-4:], vocab, top_k=40)
    compare({n: v[-4:] for n, v in out2.items()}, tail, u[-4:], vocab, top_p=0.9)
    assert top["ids"][:-4].eq(torch.arange(8, device="cuda", dtype=torch.int32)).all()
    assert torch.equal(top["ids"][-4:], vsb.topk_logprob(tail, 8)["ids"])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_largest_vocabulary(dtype):
    """Rows that no cluster's shared memory holds, and one in between."""
    for vocab in (1 << 20, 300_001):
        x = logits_on("cuda", 2, vocab, dtype, seed=16)
        for kw in (dict(top_k=100, top_p=0.9), dict(top_p=0.9), dict(), dict(min_p=0.1), dict(top_k=2000)):
            check(x, numbers(2, 9), vocab, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("top_k", [3, 256, 300, 512])
def test_lists_of_crowded_rows(dtype, top_k):
    """More equal or nearly equal tokens than a list holds, cut by top-k: a
    crowd at the top, one that the k-th token falls into, one in a single slice."""
    rows, vocab = 4, 40_000
    g = torch.Generator().manual_seed(top_k)
    x = torch.randn((rows, vocab), generator=g)
    x[0] = 2.0
    x[0, ::7] = 2.0 - 1e-3
    x[1, 5000:9000] = 6.0
    x[1, 100:100 + top_k // 2] = 7.0
    x[2] = torch.arange(vocab) % 3
    x[3, :1500] = 9.0 + torch.arange(1500) % 5
    check(x.to(dtype).cuda(), numbers(rows, 10), top_k=top_k, temperature=0.8)


def test_no_rows():
    out = vsb.sample(torch.empty((0, 64), device="cuda"), torch.empty(0, device="cuda"))
    assert out["token"].numel() == 0
    with pytest.raises(vsb.VsError) as e:
        vsb.sample(torch.zeros((2, 64), device="cuda"), torch.zeros(2, device="cuda"), top_p=0.0)
    assert e.value.code == B.VS_ERR_INVALID_ARG


def test_frequencies_follow_the_support():
    """Stratified numbers draw each token in proportion to its share: with
    u = (i + 1/2) / N a token of share s is drawn s N times, within one."""
    n, vocab = 4096, 64
    x = logits_on("cuda", 1, vocab, F32, seed=15, spikes=2).expand(n, vocab).contiguous()
    u = ((torch.arange(n, dtype=torch.float32) + 0.5) / n).cuda()
    out = vsb.sample(x, u, temperature=1.3, top_p=0.98)
    counts = torch.bincount(out["token"], minlength=vocab).double().cpu().numpy()
    z = widen(x[0]) / float(np.float32(1.3))
    w = np.exp(z - z.max())
    by = np.argsort(-w, kind="stable")
    size = out["support_size"][0].item()
    share = np.zeros(vocab)
    share[by[:size]] = w[by[:size]] / w[by[:size]].sum()
    assert (np.abs(counts - share * n) <= 1.0).all()
