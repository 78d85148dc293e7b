"""vs_sample over the whole range of its settings: min-p of any size,
the uniform number 1, and one answer for a row whatever the batch around it."""

import pytest
import torch

import sampling_support_b200 as vsb
from _row_ops import logits_on
from test_gpu_row_sample import compare

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def tensors(rows, t, k, p, m):
    """Settings as per-row tensors: the kernel is chosen by the number of rows."""
    return dict(temperature=torch.full((rows,), t, device="cuda"),
                top_k=torch.full((rows,), k, dtype=torch.int32, device="cuda"),
                top_p=torch.full((rows,), p, device="cuda"), min_p=torch.full((rows,), m, device="cuda"))


def check_both(x, u, vocab, t=1.0, k=0, p=1.0, m=0.0):
    """Against the plain form as scalars and as per-row settings, in a call of
    their own and among more rows (the rows again, in another order)."""
    rows = len(x)
    compare(vsb.sample(x, u, temperature=t, top_k=k, top_p=p, min_p=m, vocab=vocab), x, u, vocab, t, k, p, m)
    kw = tensors(rows, t, k, p, m)
    few = vsb.sample(x, u, vocab=vocab, **kw)
    compare(few, x, u, vocab, *kw.values())
    times = 40 // rows
    many = vsb.sample(x.repeat(times, 1), u.repeat(times), vocab=vocab, **tensors(rows * times, t, k, p, m))
    for name, v in few.items():
        assert torch.equal(many[name].view(times, rows).view(torch.int32),
                           v.view(torch.int32)[None].expand(times, rows)), name


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("min_p", [1e-19, 1e-21, 1e-25, 1e-30, 1e-38, 1e-44])
@pytest.mark.parametrize("top_k", [0, 400, 3000])
def test_smallest_min_p(dtype, min_p, top_k):
    """Tokens down to 100 nats below the maximum: those with w >= min_p stay,
    also where their mass rounds to nothing."""
    vocab = 5003
    x = logits_on("cuda", 8, vocab, dtype, seed=21, sigma=5.0)
    x[1, :vocab] = torch.linspace(20.0, -25.0, vocab).to(dtype).cuda()
    u = torch.linspace(0.03, 0.97, 8).cuda()
    check_both(x, u, vocab, t=0.3, k=top_k, m=min_p)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("min_p", [0.0, 1e-22, 1e-30, 1e-40])
def test_far_negative_logits(dtype, min_p):
    """Values below -2^17 that min-p tells apart, and the last of them drawn."""
    vocab = 3001
    x = torch.full((4, 3008), float("nan"), device="cuda")
    x[:, :vocab] = torch.linspace(0.0, -3.0e5, vocab).cuda()
    x[1, :vocab] = x[1, :vocab].flip(0)
    x[2, 100:vocab] = -1.5e5
    x[3, 200:vocab] = float("-inf")
    u = torch.tensor([0.3, 1.0, 1.0, 1.0]).cuda()
    for t in (2500.0, 1.0, 1e5):
        check_both(x.to(dtype), u, vocab, t=t, m=min_p)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [1003, 5003, 50_021])
@pytest.mark.parametrize("kw", [{}, dict(k=300), dict(k=900), dict(p=0.9), dict(k=500, p=0.9999), dict(m=1e-9),
                                dict(m=1e-30), dict(k=900, m=1e-30)], ids=str)
def test_the_number_one_takes_the_last_token(dtype, vocab, kw):
    """u = 1 is the support's last token also where the masses at its end round
    to nothing: values spread over 300 nats, a crowd of equal values at the
    end, masked tokens behind, zeros and values next to them."""
    x = logits_on("cuda", 5, vocab, dtype, seed=22)
    x[1, vocab // 2:vocab] = -60.0
    x[2, 64:vocab] = float("-inf")
    x[3, :vocab:3] = 0.0
    x[3, 1:vocab:3] = 2.0 ** -40
    x[4, :vocab] = x[4, :vocab] * 20
    u = torch.tensor([1.0, 1.0, 1.0, 1.0, 1.0]).cuda()
    check_both(x, u, vocab, t=0.25, **kw)


# Rows of two tokens, 0 and v, whose first token's share 1 / (1 + exp(v / t)) lies within 6e-15 of the number u, with
# v / t half way between two 64ths of an octave, where a mass by table and polynomial is off by up to 4e-14: (v, t, u).
CLOSE = [(-0.3547404408454895, 1.981567144393921, 0.5446358919143677),
         (-1.068514347076416, 0.744685173034668, 0.807656466960907),
         (-1.775558352470398, 0.996565043926239, 0.8559039831161499),
         (-2.5069146156311035, 0.8252211809158325, 0.9542559385299683),
         (-0.4350297451019287, 1.3174697160720825, 0.5818082690238953),
         (-0.7860302925109863, 0.5241159200668335, 0.8175336122512817),
         (-0.22042067348957062, 0.6893056631088257, 0.5792686939239502),
         (-0.17568178474903107, 0.5495159029960632, 0.5792518258094788),
         (-0.2530349791049957, 0.5500776171684265, 0.6130138635635376)]


@pytest.mark.parametrize("crowd", [False, True])
@pytest.mark.parametrize("settings", [dict(k=2), dict(k=0), dict(k=2, p=1.0 - 2.0 ** -24), dict(k=2, m=1e-3)], ids=str)
def test_one_answer_whatever_the_batch(settings, crowd):
    """A row with a small top-k is listed in a small batch and goes another way
    in a large one: the same masses, so the same token also where their last
    units decide."""
    n, vocab = len(CLOSE), 6000
    v, t, u = (torch.tensor(a).cuda() for a in zip(*CLOSE))
    x = torch.full((n, vocab), float("-inf"), device="cuda")
    x[:, 17] = 0.0
    x[:, 900] = v
    kw = dict(k=0, p=1.0, m=0.0)
    kw.update(settings)
    if crowd:  # below the two tokens, out of the support
        kw["m"] = max(kw["m"], 1e-3)
        x[:, 1000:] = -50.0
    few = vsb.sample(x, u, **{**tensors(n, 1.0, **kw), "temperature": t})
    many = vsb.sample(x.repeat(4, 1), u.repeat(4), **{**tensors(4 * n, 1.0, **kw), "temperature": t.repeat(4)})
    listed = vsb.sample(x.repeat(4, 1), u.repeat(4), temperature=t.repeat(4), top_k=kw["k"], top_p=kw["p"],
                        min_p=kw["m"])
    assert few["support_size"].eq(2).all()
    for name in ("token", "support_size", "logprob"):
        for other in (many, listed):
            assert torch.equal(other[name].view(4, n).view(torch.int32),
                               few[name].view(torch.int32)[None].expand(4, n)), name


@pytest.mark.parametrize("top_k", [350, 512])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_answer_for_crowded_rows(top_k, dtype):
    """The cut falls among more equal tokens than a list holds, below values
    that share the zeros' bin: taken by digits of the key in a small batch, from
    the values' counts in a large one."""
    vocab, n = 30_000, 32
    g = torch.Generator().manual_seed(42)
    x = torch.full((n, vocab), -1.0)
    x[:, 100:400] = (torch.rand((n, 300), generator=g) * 2 - 1) * 2.0 ** -24
    x[:, 150:200] = 0.0
    x[:, 5] = 12.0
    x[::2, 5] = 1e-3
    x = x.to(dtype).cuda()
    u = torch.rand(n, generator=g).cuda()
    u[::4] = 1.0
    for t in (1.0, 0.5):
        many = vsb.sample(x, u, **tensors(n, t, top_k, 1.0, 0.0))
        for r in range(0, n, 16):
            few = vsb.sample(x[r:r + 16], u[r:r + 16], **tensors(16, t, top_k, 1.0, 0.0))
            for name, w in few.items():
                assert torch.equal(w.view(torch.int32), many[name][r:r + 16].view(torch.int32)), name
        compare(many, x, u, vocab, *tensors(n, t, top_k, 1.0, 0.0).values())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_captured_call_whose_rows_change_kernels(dtype):
    """Up to 16 rows with per-row settings take two kernels in one call, each
    its share of the rows by their top-k: replayed after the settings change,
    rows go from one to the other, and become greedy or refused."""
    rows, vocab = 16, 20_011
    x = logits_on("cuda", rows, vocab, dtype, seed=51)
    u, kw = torch.full((rows,), 0.4, device="cuda"), tensors(rows, 0.8, 20, 0.9, 0.0)
    vsb.sample(x, u, vocab=vocab, **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = vsb.sample(x, u, vocab=vocab, **kw)
    gen = torch.Generator().manual_seed(52)
    for turn in range(4):
        x.copy_(logits_on("cuda", rows, vocab, dtype, seed=60 + turn))
        u.copy_(torch.rand(rows, generator=gen))
        kw["top_k"].copy_(torch.randint(-1, 3, (rows,), generator=gen) * 300)  # off, 300 (listed), 600 (not)
        kw["temperature"].copy_(torch.randint(0, 3, (rows,), generator=gen) * 0.5)
        kw["min_p"].copy_(torch.randint(0, 2, (rows,), generator=gen) * 1e-3)
        if turn == 3:
            u[5] = 2.0
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        if turn == 3:
            assert int(out["token"][5]) == -1 and int(out["status"][5]) == vsb.ROW_BAD_PARAM
            keep = [r for r in range(rows) if r != 5]
            compare({n: v[keep] for n, v in out.items()}, x[keep], u[keep], vocab, *(v[keep] for v in kw.values()))
        else:
            compare(out, x, u, vocab, *kw.values())
