"""Row operators without a GPU: what the entry points refuse, and the plain
64-bit forms that the GPU tests compare with."""

import ctypes

import numpy as np
import pytest
import torch

import sampling_support_b200 as vsb
from _row_ops import distill_row, sample_row, topk_row
from sampling_support_b200 import _binding as B

FAKE = 0x10000  # 16-byte aligned, never dereferenced by a rejected call
INV, UNS = B.VS_ERR_INVALID_ARG, B.VS_ERR_UNSUPPORTED


def _sample(token=FAKE, **kw):
    a = B.SampleArgs(rows=4, vocab=1000, ld=1000, dtype=B.VS_BF16, logits=FAKE, temperature_scalar=1.0,
                     top_p_scalar=1.0, uniform=FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return vsb.load().vs_sample(ctypes.byref(a), token, None, None, None, None)


@pytest.mark.parametrize("field,value,code", [
    ("rows", -1, INV), ("vocab", 0, INV), ("ld", 999, INV), ("ld", 1001, INV), ("dtype", 2, INV),
    ("logits", 0, INV), ("logits", FAKE + 2, INV), ("uniform", 0, INV), ("token", 0, INV),
    ("temperature_scalar", -1.0, INV), ("temperature_scalar", float("nan"), INV),
    ("temperature_scalar", float("inf"), INV), ("top_p_scalar", 0.0, INV), ("top_p_scalar", 1.01, INV),
    ("top_p_scalar", float("nan"), INV), ("min_p_scalar", 1.0, INV), ("min_p_scalar", -0.1, INV),
])
def test_sample_refuses(field, value, code):
    assert _sample(**{field: value}) == code
    assert vsb.load().vs_last_error().decode() != ""


def test_sample_refuses_a_large_vocabulary_and_takes_no_rows():
    big = B.VS_MAX_ROW_VOCAB + 8
    assert _sample(vocab=big, ld=big) == UNS
    assert _sample(rows=0, logits=0, uniform=0, token=0) == B.VS_OK
    assert vsb.load().vs_sample(None, FAKE, None, None, None, None) == INV


def _topk(rows=4, vocab=1000, ld=1000, dtype=B.VS_F32, logits=FAKE, temp=1.0, k=8, ids=FAKE, out_ld=8):
    return vsb.load().vs_topk_logprob(rows, vocab, ld, dtype, logits, None, temp, k, ids, None, out_ld,
                                      None, None)


def test_topk_refuses():
    for kw in (dict(rows=-1), dict(vocab=0), dict(ld=998), dict(ld=1002), dict(dtype=9), dict(logits=0),
               dict(logits=FAKE + 4), dict(temp=0.0), dict(temp=float("nan")), dict(k=0), dict(k=1001, out_ld=1001),
               dict(out_ld=7), dict(ids=0)):
        assert _topk(**kw) == INV, kw
    assert _topk(temp=2.0 ** -127) == INV  # 1 / T is not finite in fp32
    assert _topk(rows=(1 << 24) + 1) == UNS
    assert _topk(vocab=4000, ld=4000, k=1025, out_ld=1025) == UNS
    assert _topk(vocab=B.VS_MAX_ROW_VOCAB + 4, ld=B.VS_MAX_ROW_VOCAB + 4) == UNS
    assert _topk(rows=0, logits=0, ids=0) == B.VS_OK


def _distill_args(**kw):
    a = B.DistillArgs(rows=4, vocab=1000, ld=1000, dtype=B.VS_BF16, logits=FAKE, temperature_scalar=1.0,
                      teacher_ids=FAKE, teacher_logprob=FAKE, teacher_width=8, teacher_ld=8, tail=0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_DISTILL = [
    (dict(rows=-1), INV), (dict(vocab=0), INV), (dict(ld=999), INV), (dict(ld=1004), INV), (dict(dtype=5), INV),
    (dict(logits=0), INV), (dict(logits=FAKE + 8), INV), (dict(temperature_scalar=0.0), INV),
    (dict(temperature_scalar=float("inf")), INV), (dict(temperature_scalar=2.0 ** -127), INV),
    (dict(rows=(1 << 24) + 1), UNS), (dict(teacher_ids=0), INV), (dict(teacher_logprob=0), INV),
    (dict(teacher_ld=7), INV), (dict(tail=2), INV), (dict(teacher_width=-1), UNS),
    (dict(teacher_width=1025, teacher_ld=1025), UNS),
    (dict(vocab=B.VS_MAX_ROW_VOCAB + 8, ld=B.VS_MAX_ROW_VOCAB + 8), UNS),
]


@pytest.mark.parametrize("kw,code", BAD_DISTILL)
def test_distill_refuses_bad_arguments(kw, code):
    lib = vsb.load()
    a, o = _distill_args(**kw), B.DistillOut()
    assert lib.vs_distill_fwd(ctypes.byref(a), ctypes.byref(o), None) == code
    assert lib.vs_distill_bwd(ctypes.byref(a), FAKE, None, FAKE << 8, B.VS_F32, 1000, B.VS_GRAD_DENSE, None) == code


def test_distill_refuses_bad_outputs():
    lib = vsb.load()
    a = _distill_args()
    far = FAKE << 8
    fwd = lambda **kw: lib.vs_distill_fwd(ctypes.byref(a), ctypes.byref(B.DistillOut(**kw)), None)
    assert lib.vs_distill_fwd(ctypes.byref(a), None, None) == INV
    assert fwd(ctx=FAKE + 8) == INV
    assert fwd(g_loss=FAKE) == INV  # an upstream gradient without a gradient to write
    assert fwd(dlogits=far, dl_dtype=7, grad_ld=1000) == INV
    assert fwd(dlogits=far, dl_dtype=B.VS_F32, grad_ld=999) == INV
    assert fwd(dlogits=far, dl_dtype=B.VS_F32, grad_ld=1001) == INV
    assert fwd(dlogits=far + 4, dl_dtype=B.VS_F32, grad_ld=1000) == INV
    for at in (FAKE, FAKE + 2 * 1000 * 3, FAKE - 2 * 1000 * 2):  # in place, or over some of the rows
        assert fwd(dlogits=at, dl_dtype=B.VS_BF16, grad_ld=1000) == INV
        assert "overlap" in lib.vs_last_error().decode()
    bwd = lambda ctx=FAKE, dl=far, dt=B.VS_F32, ld=1000, mode=B.VS_GRAD_DENSE: lib.vs_distill_bwd(
        ctypes.byref(a), ctx, None, dl, dt, ld, mode, None)
    for kw in (dict(ctx=0), dict(ctx=FAKE + 4), dict(dl=0), dict(dl=FAKE), dict(dt=3), dict(ld=996),
               dict(ld=1001), dict(mode=B.VS_GRAD_SPARSE), dict(mode=9)):
        assert bwd(**kw) == INV, kw


def test_distill_zero_rows_is_a_no_op():
    lib = vsb.load()
    a, o = _distill_args(rows=0, logits=0, teacher_ids=0, teacher_logprob=0), B.DistillOut()
    assert lib.vs_distill_fwd(ctypes.byref(a), ctypes.byref(o), None) == B.VS_OK
    assert lib.vs_distill_bwd(ctypes.byref(a), 0, None, 0, B.VS_F32, 1000, B.VS_GRAD_DENSE, None) == B.VS_OK


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(2, 16)
    with pytest.raises(ValueError):
        vsb.sample(x, torch.zeros(2))  # host memory
    with pytest.raises(ValueError):
        vsb.sample(x, torch.zeros(3))
    with pytest.raises(ValueError):
        vsb.sample(x, torch.zeros(2, dtype=torch.float64))
    with pytest.raises(ValueError):
        vsb.sample(x, torch.zeros(2), top_k=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        vsb.sample(x, torch.zeros(2), vocab=17)
    with pytest.raises(ValueError):
        vsb.sample(x.t(), torch.zeros(16))
    with pytest.raises(ValueError):
        vsb.sample(x, torch.zeros(2), vocab=-(1 << 32) + 16)
    with pytest.raises(ValueError):
        vsb.sample(torch.zeros(1, 8).expand((1 << 24) + 1, 8), torch.zeros(1).expand((1 << 24) + 1))
    assert [B._int32(v) for v in (7, (1 << 32) + 1, -(1 << 40))] == [7, (1 << 31) - 1, -(1 << 31)]
    with pytest.raises(ValueError):
        vsb.topk_logprob(x, 4)
    with pytest.raises(TypeError):
        vsb.topk_logprob(torch.zeros(2, 16, dtype=torch.float16), 4) if torch.cuda.is_available() else \
            B._dtype_code(torch.zeros(2, 16, dtype=torch.float16))
    ids, lp = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4)
    with pytest.raises(ValueError):
        vsb.distill_fwd(x, ids, lp)
    with pytest.raises(ValueError):
        vsb.distill_fwd(x, ids.long(), lp)
    with pytest.raises(ValueError):
        vsb.distill_fwd(x, ids, lp[:, :3])
    with pytest.raises(ValueError):
        vsb.distill_fwd(x, ids, lp, g_loss=torch.zeros(2))


# --- the plain forms --------------------------------------------------------


def test_plain_sample_on_hand_made_rows():
    x = np.zeros(4)  # four equal tokens: cuts fall exactly on the shares
    assert [sample_row(x, u)[0] for u in (0.0, 0.2499, 0.25, 0.5, 0.75, 1.0)] == [0, 0, 1, 2, 3, 3]
    assert sample_row(x, 0.9, p=0.5)[::2] == (1, 2)  # inclusive: two tokens hold exactly one half
    assert sample_row(x, 0.9, k=3)[::2] == (2, 3)
    y = np.array([0.0, np.log(0.25), np.log(0.25), -np.inf])
    assert sample_row(y, 0.99, m=0.25)[::2] == (2, 3)
    assert sample_row(y, 0.7, t=0)[0] == 0
    assert sample_row(np.full(3, -np.inf), 0.5)[0] == -1


def test_plain_topk_pads_past_the_unmasked_tokens():
    ids, lp = topk_row(np.array([-np.inf, 1.0, 1.0, -np.inf]), 3)
    assert ids.tolist() == [1, 2, -1] and np.allclose(lp[:2], -np.log(2)) and lp[2] == -np.inf


@pytest.mark.parametrize("tail", [False, True])
def test_plain_distill_gradient_by_differences(tail):
    rng = np.random.default_rng(4)
    x = rng.normal(0, 2, 40)
    ids = np.array([3, 17, -1, 5, 17, 39], np.int32)
    lp = np.log(np.array([0.3, 0.2, 0.9, 0.25, 0.7, 0.1])).astype(np.float32)
    t = 0.8
    _, valid, grad, _, _ = distill_row(x, ids, lp, t, tail)
    assert valid == 1
    h = 1e-6
    for j in range(40):
        d = np.zeros(40)
        d[j] = h
        diff = (distill_row(x + d, ids, lp, t, tail)[0] - distill_row(x - d, ids, lp, t, tail)[0]) / (2 * h)
        assert abs(diff - grad[j]) < 1e-8
    assert abs(grad.sum()) < 1e-12  # a softmax's gradient has no common part


def test_plain_distill_equals_full_kl_when_the_list_is_the_vocabulary():
    rng = np.random.default_rng(5)
    x, y = rng.normal(0, 2, 30), rng.normal(0, 2, 30)
    ly = y - np.log(np.exp(y).sum())
    lx = x - np.log(np.exp(x).sum())
    want = (np.exp(ly) * (ly - lx)).sum()
    ids = np.arange(30)
    assert abs(distill_row(x, ids, ly, 1.0, False)[0] - want) < 1e-12
    assert abs(distill_row(x, ids, ly, 1.0, True)[0] - want) < 1e-12
    assert abs(distill_row(y, ids, ly, 1.0, False)[0]) < 1e-12
