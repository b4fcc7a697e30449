"""Routing to experts without a GPU: every refusal of qmm_moe_topk and of the
Python call, before any HIP call."""
import pytest

torch = pytest.importorskip("torch")

import quantized_matmul_qgemv_amd as qmm  # noqa: E402
from quantized_matmul_qgemv_amd import _lib  # noqa: E402

INV, UNS = _lib.QMM_ERR_INVALID_ARG, _lib.QMM_ERR_UNSUPPORTED
A = 0x10000  # a fake, aligned, never dereferenced device address
NAN, INF = float("nan"), float("inf")


def call(logits=A, bias=None, ids=A, weights=A, t=4, e=128, top_k=8, score=0, groups=1, keep=1, top=1,
         renorm=1, scale=1.0):
    return _lib.lib().qmm_moe_topk(logits, bias, ids, weights, t, e, top_k, score, groups, keep, top, renorm,
                                   scale, None)


@pytest.mark.parametrize("kw, status, text", [
    (dict(t=-1), INV, "t=-1"),
    (dict(t=1 << 26), INV, "t=67108864"),
    (dict(e=0), INV, "e=0"),
    (dict(e=1025), INV, "e=1025"),
    (dict(score=2), UNS, "score=2"),
    (dict(groups=0), INV, "groups=0"),
    (dict(groups=3), INV, "divide e=128"),
    (dict(groups=128), INV, "groups=128"),
    (dict(groups=8, keep=0), INV, "group_keep=0"),
    (dict(groups=8, keep=9), INV, "group_keep=9"),
    (dict(keep=2), INV, "group_keep=2"),
    (dict(groups=8, keep=4, top=0), INV, "group_top=0"),
    (dict(groups=8, keep=4, top=3), INV, "group_top=3"),
    (dict(e=8, groups=8, keep=8, top=2), INV, "group_top=2"),
    (dict(top_k=0), INV, "top_k=0"),
    (dict(top_k=65), INV, "top_k=65"),
    (dict(e=4, top_k=5), INV, "top_k=5"),
    (dict(e=32, groups=8, keep=1, top_k=5), INV, "top_k=5 must be in [1, 4]"),
    (dict(renorm=2), INV, "renormalize"),
    (dict(scale=NAN), INV, "scale must be finite"),
    (dict(scale=INF), INV, "scale must be finite"),
    (dict(logits=None), INV, "null pointer logits"),
    (dict(logits=A + 2), INV, "logits is not 4-byte aligned"),
    (dict(bias=A + 1), INV, "bias is not 4-byte aligned"),
    (dict(ids=None), INV, "null pointer expert_ids"),
    (dict(weights=A + 2), INV, "weights is not 4-byte aligned"),
])
def test_refusals(kw, status, text):
    assert call(**kw) == status, _lib.last_error()
    assert text in _lib.last_error()


def test_no_tokens_is_no_work():
    assert call(t=0, logits=None, ids=None, weights=None) == 0
    assert _lib.last_error() == ""


def test_python_refusals():
    l = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="device tensor"):
        qmm.moe_topk(l, 2)
    with pytest.raises(ValueError, match=r"\[T, E\]"):
        qmm.moe_topk(l[0], 2)
    with pytest.raises(ValueError, match="score must be"):
        qmm.moe_topk(l, 2, score="tanh")
    with pytest.raises(ValueError, match=r"bias must be \[16\]"):
        qmm.moe_topk(l, 2, bias=torch.zeros(15))
    with pytest.raises(ValueError, match="expert_ids must be"):
        qmm.moe_topk(l, 2, expert_ids=torch.zeros(4, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="weights must be"):
        qmm.moe_topk(l, 2, weights=torch.zeros(5, 2))
