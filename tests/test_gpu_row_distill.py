"""vs_distill_fwd / vs_distill_bwd against the 64-bit plain form.

The loss: teacher masses and the listed student terms are fp64; the row's
normaliser sums fp32 exponentials (each off by 2^-22, and by 2^-24 of an
argument of at most 60 in log2 units; at most 64 partial sums of a thread, 2^-24
each): below 8e-6; the factor log2(e) / T is rounded twice, which moves log q_k
by at most 2^-23 |z_k - E z| <= 1e-5 for values within 80 of the mean; the
loss is rounded once (2^-24).  A tail's share has such a normaliser of its own,
weighted by at most one.  So |error| <= 3e-5 + 2^-23 |loss|.

The gradient of element j, over g / T: q_j and the listed a_j are each off by
at most 2e-5 relative (the normaliser's 8e-6, its rounded logarithm 2^-24 * 60,
the exponential 2^-22, the factor above); the stored value is rounded by half a
step of its type."""

import numpy as np
import pytest
import torch

import sampling_support_b200 as vsb
from _row_ops import distill_row, logits_on, sample_row, topk_row, widen

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def lists(rows, vocab, k, seed, x=None, noise=0.7):
    """A teacher's list per row (its own top k of noisy student logits), uneven
    widths, pads in the middle, an empty row."""
    g = torch.Generator().manual_seed(seed)
    y = (torch.randn((rows, vocab), generator=g) * 3.0) if x is None else \
        x.float().cpu() + noise * torch.randn((rows, vocab), generator=g)
    v, i = torch.topk(y, k, dim=1)
    lp = (v - torch.logsumexp(y, 1, keepdim=True)).float()
    ids = i.to(torch.int32)
    drop = torch.rand((rows, k), generator=g) < torch.rand((rows, 1), generator=g) * 0.5
    ids[drop] = -1
    if rows > 2:
        ids[2] = -1
    return ids.cuda(), lp.cuda()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def compare(x, ids, lp, t, tail, g, vocab, loss, valid, grad, before=None):
    xs, li, ll = widen(x[:, :vocab]), ids.cpu().numpy(), lp.cpu().numpy()
    for r in range(len(xs)):
        tr = float(t[r]) if isinstance(t, torch.Tensor) else float(np.float32(t))
        want, ok, d, q, a = distill_row(xs[r], li[r], ll[r], tr, tail)
        assert int(valid[r]) == ok
        assert abs(float(loss[r]) - want) <= 3e-5 + 2.0 ** -23 * abs(want), (r, float(loss[r]), want)
        if grad is None:
            continue
        gr = 1.0 if g is None else float(g[r])
        d = d * gr
        old = 0.0 if before is None else widen(before[r, :vocab])
        full = old + d
        tol = 2e-5 * abs(gr) / tr * (q + a) + 2e-5 * np.abs(d) + half_step(grad.dtype) * np.abs(full) * (1 + 1e-4) + 1e-37
        if before is not None:
            tol = tol + 2.0 ** -23 * np.abs(old)  # the fp32 addition
        got = widen(grad[r, :vocab])
        worst = np.abs(got - full) - tol
        assert worst.max() <= 0, (r, int(worst.argmax()), got[worst.argmax()], full[worst.argmax()])


def check(x, ids, lp, t=1.0, tail=False, g=None, vocab=None, grad_dtype=None, stream=None):
    """Forward, backward and the call that does both."""
    vocab = x.shape[1] if vocab is None else vocab
    grad_dtype = x.dtype if grad_dtype is None else grad_dtype
    kw = dict(temperature=t, tail=tail, vocab=vocab, stream=stream)
    out = vsb.distill_fwd(x, ids, lp, want_grad=True, **kw)
    grad = vsb.distill_bwd(x, ids, lp, out["ctx"], g, grad_dtype=grad_dtype, **kw)
    both = vsb.distill_fwd(x, ids, lp, g_loss=g, grad_dtype=grad_dtype, **kw)
    torch.cuda.synchronize()
    compare(x, ids, lp, t, tail, g, vocab, out["loss"], out["valid"], grad)
    compare(x, ids, lp, t, tail, g, vocab, both["loss"], both["valid"], both["grad"])
    assert torch.equal(out["loss"], both["loss"]) and torch.equal(out["status"], both["status"])
    return out, grad


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("vocab,k", [(1, 1), (7, 3), (33, 33), (1000, 20), (4097, 64), (20_011, 1024), (20_011, 257)])
def test_sizes(dtype, tail, vocab, k):
    rows = 6
    x = logits_on("cuda", rows, vocab, dtype, seed=vocab)
    ids, lp = lists(rows, vocab, k, seed=k, x=x[:, :vocab])
    g = torch.rand(rows, generator=torch.Generator().manual_seed(1)).cuda() - 0.3
    t = torch.rand(rows, generator=torch.Generator().manual_seed(2)).cuda() + 0.5
    check(x, ids, lp, t, tail, g, vocab)


@pytest.mark.parametrize("dtype,grad_dtype", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("tail", [False, True])
def test_gradient_types(dtype, grad_dtype, tail):
    x = logits_on("cuda", 5, 3001, dtype, seed=4)
    ids, lp = lists(5, 3001, 30, seed=5, x=x[:, :3001])
    check(x, ids, lp, 0.9, tail, None, 3001, grad_dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 20, 160])
def test_benchmark_vocabulary(dtype, rows):
    vocab = 151_936
    x = logits_on("cuda", rows, vocab, dtype, seed=rows)
    ids, lp = lists(rows, vocab, 64, seed=3, x=x)
    check(x, ids, lp, 1.0, True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_vocabularies_beyond_shared_memory(dtype):
    """The largest vocabulary, whose row no cluster's shared memory holds, and
    one in between with an odd end."""
    for vocab in (1 << 20, 640_003):
        x = logits_on("cuda", 3, vocab, dtype, seed=5)
        ids, lp = lists(3, vocab, 300, seed=6, x=x[:, :vocab])
        check(x, ids, lp, 0.9, True, None, vocab)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("grad_dtype", [BF, F32])
def test_accumulates(tail, grad_dtype):
    rows, vocab = 5, 2003
    x = logits_on("cuda", rows, vocab, BF, seed=6)
    ids, lp = lists(rows, vocab, 40, seed=7, x=x[:, :vocab])
    ids[0, 5] = ids[0, 4].clamp(min=0)  # a repeat
    g = torch.rand(rows, generator=torch.Generator().manual_seed(3)).cuda()
    out = vsb.distill_fwd(x, ids, lp, tail=tail, want_grad=True, vocab=vocab)
    acc = torch.randn((rows, 2008), generator=torch.Generator().manual_seed(4)).to(grad_dtype).cuda() * 0.01
    before = acc.clone()
    got = vsb.distill_bwd(x, ids, lp, out["ctx"], g, tail=tail, mode=vsb.VS_GRAD_ACCUMULATE, out=acc, vocab=vocab)
    torch.cuda.synchronize()
    assert got is acc and torch.equal(acc[:, vocab:], before[:, vocab:])
    compare(x, ids, lp, 1.0, tail, g, vocab, out["loss"], out["valid"], acc, before)
    with pytest.raises(ValueError):
        vsb.distill_bwd(x, ids, lp, out["ctx"], g, tail=tail, mode=vsb.VS_GRAD_ACCUMULATE, vocab=vocab)


@pytest.mark.parametrize("tail", [False, True])
def test_repeats_bad_ids_and_pads(tail):
    vocab = 1000
    x = logits_on("cuda", 4, vocab, F32, seed=8)
    ids = torch.tensor([[5, 5, 7, -1, 999, 5], [1000, -2, 3, 2 ** 31 - 1, 4, -2 ** 31], [-1] * 6, [0, 1, 2, 3, 4, 4]],
                       dtype=torch.int32).cuda()
    lp = torch.log(torch.tensor([[.1, .9, .2, .3, .05, .4]] * 4)).cuda()
    out, _ = check(x, ids, lp, 0.7, tail)
    dup, bad, empty = vsb.ROW_DUP_SUPPORT_ID, vsb.ROW_BAD_SUPPORT_ID, vsb.ROW_EMPTY_SUPPORT
    assert out["status"].tolist() == [dup, bad, empty, dup]
    assert out["loss"][2] == 0 and out["valid"].tolist() == [1, 1, 0, 1]


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_list(tail, dtype):
    x = logits_on("cuda", 3, 500, dtype, seed=9)
    ids, lp = torch.empty((3, 0), dtype=torch.int32, device="cuda"), torch.empty((3, 0), device="cuda")
    out, grad = check(x, ids, lp, 1.0, tail, vocab=500)
    assert out["valid"].tolist() == [0, 0, 0] and (grad[:, :500] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_small_shares_outside_the_list(dtype):
    """A confident student: the mass outside the list is far below fp32's step
    at 1, and its logarithm and the gradient there still hold."""
    vocab = 4000
    x = logits_on("cuda", 3, vocab, dtype, seed=10, sigma=1.0, spikes=0)
    x[:, 11] = 40.0
    x[1, 11] = 70.0
    x[2, 12] = 39.5
    ids = torch.tensor([[11, 12, 13]] * 3, dtype=torch.int32).cuda()
    lp = torch.log(torch.tensor([[.7, .1, .05], [.999, 1e-4, 1e-4], [.5, .4, .1]])).cuda()
    check(x, ids, lp, 1.0, True)
    check(x, ids, lp, 1.0, False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
def test_values_at_the_ends_of_the_type(dtype, tail):
    """Rows whose logits times log2(e) / T overflow fp32: all at the lowest
    value (uniform), tokens masked by it, and both ends in one row."""
    vocab, low = 1003, -torch.finfo(dtype).max
    x = logits_on("cuda", 4, vocab, dtype, seed=23, spikes=0)
    x[0, :vocab] = low
    x[1, 20:vocab] = low
    x[2, :vocab] = -low
    x[3, 7:vocab:3] = low
    x[3, 0:vocab:2] = -low
    ids = torch.tensor([[0, 5, 900], [3, 19, 18], [1, 2, 1002], [0, 2, 4]], dtype=torch.int32).cuda()
    lp = torch.log(torch.tensor([[.5, .2, .1]] * 4)).cuda()
    for t in (0.5, 1.0):
        check(x, ids, lp, t, tail, None, vocab)


def test_identical_teacher_and_student():
    """The loss is zero to rounding and so is the gradient, when the list is
    the vocabulary and when it is the top of it."""
    vocab = 600
    x = logits_on("cuda", 4, vocab, F32, seed=11)
    top = vsb.topk_logprob(x, vocab)
    for tail in (False, True):
        out, grad = check(x, top["ids"], top["logprob"], 1.0, tail)
        assert out["loss"].abs().max() < 3e-5
    few = vsb.topk_logprob(x, 50)
    out, grad = check(x, few["ids"], few["logprob"], 1.0, True)
    assert out["loss"].abs().max() < 3e-5


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_student_tokens(dtype):
    """-inf has no share: outside the list nothing changes, on the list without
    teacher mass neither, and with it the loss is infinite."""
    vocab = 2001
    x = logits_on("cuda", 4, vocab, dtype, seed=12)
    x[:, 1500:vocab] = float("-inf")
    x[1, 3] = float("-inf")
    x[2, 4] = float("-inf")
    x[3, :vocab] = float("-inf")
    x[3, 1], x[3, 2] = 1.0, 0.5  # only listed tokens are left: no tail
    ids = torch.tensor([[1, 2, 1700], [1, 2, 3], [1, 4, 3], [1, 2, 3]], dtype=torch.int32).cuda()
    lp = torch.log(torch.tensor([[.5, .2, 0], [.5, .2, 0], [.5, .2, .1], [.5, .2, 0]])).cuda()
    for tail in (False, True):
        kw = dict(tail=tail, vocab=vocab)
        out = vsb.distill_fwd(x, ids, lp, want_grad=True, **kw)
        grad = vsb.distill_bwd(x, ids, lp, out["ctx"], grad_dtype=F32, **kw)
        assert out["loss"][2] == float("inf") and out["valid"].tolist() == [1, 1, 1, 1]
        assert torch.isfinite(grad[:, :vocab]).all() and (grad[0, 1500:vocab] == 0).all()
        rows = [0, 1, 3]
        compare(x[rows], ids[rows], lp[rows], 1.0, tail, None, vocab, out["loss"][rows], out["valid"][rows], grad[rows])


@pytest.mark.parametrize("tail", [False, True])
def test_rows_without_a_loss(tail):
    vocab = 901
    x = logits_on("cuda", 8, vocab, F32, seed=13)
    x[0, 900] = float("nan")
    x[1, 5] = float("inf")
    x[2, :vocab] = float("-inf")
    x[3, 7] = float("nan")  # on the list
    ids = torch.full((8, 2), 7, dtype=torch.int32).cuda()
    ids[:, 1] = 8
    lp = torch.full((8, 2), -1.0).cuda()
    lp[4, 1], lp[5, 0] = float("nan"), float("inf")
    t = torch.ones(8).cuda()
    t[6], t[7] = 0.0, float("nan")
    kw = dict(temperature=t, tail=tail, vocab=vocab)
    out = vsb.distill_fwd(x, ids, lp, want_grad=True, grad_dtype=F32, **kw)
    grad = vsb.distill_bwd(x, ids, lp, out["ctx"], **kw)
    torch.cuda.synchronize()
    assert torch.isnan(out["loss"]).all() and out["valid"].sum() == 0
    assert out["status"].tolist() == [vsb.ROW_NONFINITE_INPUT] * 6 + [vsb.ROW_BAD_PARAM] * 2
    assert (grad[:, :vocab] == 0).all() and (out["grad"][:, :vocab] == 0).all()


def test_smallest_temperatures():
    vocab = 901
    x = logits_on("cuda", 2, vocab, F32, seed=13)
    x[1, :vocab] = 3.0  # every difference is zero, whatever T
    ids, lp = torch.full((2, 1), 7, dtype=torch.int32).cuda(), torch.full((2, 1), -1.0).cuda()
    kw = dict(temperature=torch.tensor([2.0 ** -127, 2.0 ** -126]).cuda(), tail=True, vocab=vocab)
    out = vsb.distill_fwd(x, ids, lp, want_grad=True, grad_dtype=F32, **kw)
    grad = vsb.distill_bwd(x, ids, lp, out["ctx"], **kw)
    torch.cuda.synchronize()
    assert out["status"].tolist() == [vsb.ROW_BAD_PARAM, 0] and (grad[0, :vocab] == 0).all()
    assert torch.isnan(out["loss"][0]) and torch.isfinite(out["loss"][1])
    assert torch.isfinite(grad[:, :vocab]).all() and torch.isfinite(out["grad"][:, :vocab]).all()


def test_gradient_by_differences():
    """The gradient predicts how the kernel's own loss moves: along a direction
    d of unit steps of 2^-6, the central difference of the fp32 losses is off by
    two roundings of the loss (3e-5 each side, correlated far below that) over
    the step, and by the third derivative's h^2 / 6."""
    vocab, h = 300, 2.0 ** -6
    g = torch.Generator().manual_seed(14)
    x = (torch.randn((1, vocab), generator=g) * 2).cuda()
    ids, lp = lists(1, vocab, 12, seed=15, x=x)
    for tail in (False, True):
        out = vsb.distill_fwd(x, ids, lp, tail=tail, grad_dtype=F32)
        grad = out["grad"][0, :vocab].double().cpu()
        for s in range(4):
            d = torch.randn(vocab, generator=g).sign()
            up = vsb.distill_fwd(x + h * d.cuda(), ids, lp, tail=tail)["loss"].double()
            dn = vsb.distill_fwd(x - h * d.cuda(), ids, lp, tail=tail)["loss"].double()
            diff = ((up - dn) / (2 * h)).item()
            want = float((grad * d.double()).sum())
            assert abs(diff - want) <= 6e-5 / (2 * h) + h * h


def test_views_stream_and_capture():
    big = logits_on("cuda", 12, 4096, BF, seed=16)
    view = big[1:12:2, 16:16 + 2005]
    wide_i, wide_l = lists(6, 2005, 50, seed=17, x=view)
    ids, lp = wide_i[:, 10:40], wide_l[:, 10:40]  # a window of wider lists
    check(view, ids, lp, 1.0, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check(view, ids, lp, 1.0, True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    gl = torch.ones(6, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = vsb.distill_fwd(view, ids, lp, tail=True, want_grad=True)
        grad = vsb.distill_bwd(view, ids, lp, out["ctx"], gl, tail=True, grad_dtype=F32)
    big.copy_(logits_on("cuda", 12, 4096, BF, seed=18))
    gl.copy_(torch.rand(6))
    g.replay()
    torch.cuda.synchronize()
    compare(view, ids, lp, 1.0, True, gl, 2005, out["loss"], out["valid"], grad)


def test_offsets_beyond_32_bits():
    vocab = 151_936
    rows = 2 ** 31 // vocab + 4
    x = torch.zeros((rows, vocab), dtype=BF, device="cuda")
    last = logits_on("cuda", 2, vocab, BF, seed=19)
    x[-2:] = last
    ids, lp = lists(2, vocab, 16, seed=20, x=last)
    ids, lp = ids.repeat(rows // 2 + 1, 1)[-rows:].contiguous(), lp.repeat(rows // 2 + 1, 1)[-rows:].contiguous()
    out = vsb.distill_fwd(x, ids, lp, tail=True, want_grad=True, grad_dtype=BF)
    compare(last, ids[-2:], lp[-2:], 1.0, True, None, vocab, out["loss"][-2:], out["valid"][-2:], out["grad"][-2:])
    ctx = out["ctx"]
    del out
    grad = vsb.distill_bwd(x, ids, lp, ctx, tail=True, grad_dtype=BF)
    loss = vsb.distill_fwd(last, ids[-2:], lp[-2:], tail=True)
    compare(last, ids[-2:], lp[-2:], 1.0, True, None, vocab, loss["loss"], loss["valid"], grad[-2:])


def test_a_distillation_step():
    """As used together: sample a rollout's tokens from the student, list the
    teacher's top tokens, take the loss beside the sampled tokens' score, and
    accumulate both gradients into one buffer; one captured step gives the same
    bits as an eager one."""
    rows, vocab, k = 12, 8003, 32
    student = logits_on("cuda", rows, vocab, BF, seed=21)
    teacher = logits_on("cuda", rows, vocab, BF, seed=22)
    u = torch.rand(rows, generator=torch.Generator().manual_seed(5)).cuda()
    gl = torch.full((rows,), 1.0 / rows, device="cuda")
    neg = torch.full((rows,), -0.1 / rows, device="cuda")

    def step():
        s = vsb.sample(student, u, temperature=0.9, top_p=0.95, vocab=vocab)
        top = vsb.topk_logprob(teacher, k, vocab=vocab)
        f = vsb.distill_fwd(student, top["ids"], top["logprob"], tail=True, want_grad=True, vocab=vocab)
        sc = vsb.score_fwd(student, s["token"], want_grad=True, vocab=vocab)
        d = vsb.score_bwd(student, s["token"], sc["ctx"], g_lp_full=neg, vocab=vocab)
        d = vsb.distill_bwd(student, top["ids"], top["logprob"], f["ctx"], gl, tail=True, out=d,
                            mode=vsb.VS_GRAD_ACCUMULATE, vocab=vocab)
        return s, top, f, sc, d

    s, top, f, sc, d = step()
    torch.cuda.synchronize()
    xs, ys = widen(student[:, :vocab]), widen(teacher[:, :vocab])
    for r in range(rows):
        tok, lp, size = sample_row(xs[r], float(u[r]), float(np.float32(0.9)), p=float(np.float32(0.95)))
        assert s["token"][r] == tok and s["support_size"][r] == size
        ids, _ = topk_row(ys[r], k)
        assert top["ids"][r].tolist() == ids.tolist()
        li, ll = top["ids"][r].cpu().numpy(), top["logprob"][r].cpu().numpy()
        want, _, grad, q, a = distill_row(xs[r], li, ll, 1.0, True)
        assert abs(float(f["loss"][r]) - want) <= 3e-5 + 2.0 ** -23 * want
        logq = xs[r] - xs[r].max() - np.log(np.exp(xs[r] - xs[r].max()).sum())
        assert abs(float(sc["lp_full"][r]) - logq[tok]) < 1e-4
        hit = np.zeros(vocab)
        hit[tok] = 1.0
        full = grad / rows - 0.1 / rows * (hit - q)
        # score_bwd's element is within 2e-3 of its row's largest, here at most 0.1 / rows
        assert np.abs(widen(d[r, :vocab]) - full).max() <= 2e-3 * 0.1 / rows + 3e-5 / rows
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = step()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again[0]["token"], s["token"]) and torch.equal(again[2]["loss"], f["loss"])
    assert torch.equal(again[4][:, :vocab], d[:, :vocab])
