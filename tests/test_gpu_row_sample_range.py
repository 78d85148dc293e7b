"""vs_sample over the whole range of its settings: min-p of any size,
and the uniform number 1."""

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
