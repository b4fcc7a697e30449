"""Routing to experts: calls that stand at the edge of what the header promises."""
import numpy as np
import pytest

from qmm_testlib import dev, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import quantized_matmul_qgemv_amd as qmm  # noqa: E402
from test_gpu_moe_topk import INF, compare  # noqa: E402


@pytest.mark.parametrize("e", [48, 64, 112, 256])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [1, 2, 4, 8])
def test_masks_infinities_and_nan(e, score, biased, groups):
    """Numbers of experts whose groups are whole lanes of sixteen."""
    say("moe_topk masks", e, score, biased, groups)
    r = np.random.default_rng([78, e])
    size = e // groups
    l = (r.standard_normal((30, e)) * 2).astype(np.float32)
    l[0] = -INF                       # every expert switched off
    l[1, 3:] = -INF                   # fewer left than are chosen
    l[2, :e - 3] = -INF
    l[3, ::2] = -INF
    l[4] = np.finfo(np.float32).min   # a mask of the lowest value, everywhere
    l[5, 1:] = np.finfo(np.float32).min
    l[6, 7] = np.nan
    l[7] = np.nan
    l[8, 5] = INF
    l[9, [5, 30]] = INF
    l[10] = 1e4 * r.standard_normal(e)
    l[11] = 3e38
    l[12] = -3e38
    l[13] = 0
    l[14] = np.float32(1e-45) * r.integers(0, 5, e)  # smallest subnormals, apart
    l[15, 9] = -np.float32(0)
    l[16] = -200 - np.arange(e)       # scores below the smallest fp32
    l[17] = 100 + np.arange(e)
    l[18, :size] = -INF               # the first group switched off, the last, all but one
    l[19, e - size:] = -INF
    l[20, size:] = -INF
    l[21, size - 1:] = -INF           # and but for one expert
    l[22] = -INF
    l[22, e - 1] = -3
    l[23, e - 1] = np.nan
    l[24, 0] = np.nan
    l[24, e - 1] = INF
    bias = (r.standard_normal(e) * 0.1).astype(np.float32) if biased else None
    for renorm in (True, False):
        for top in ((1,) if groups == 1 else (1, 2)):
            compare(l, 6, bias, score=score, groups=groups, group_keep=max(1, groups - 1), group_top=top, renormalize=renorm)


@pytest.mark.parametrize("e", [64, 128, 256, 512])
@pytest.mark.parametrize("kw", [dict(), dict(score="sigmoid", groups=8, group_keep=4, group_top=2),
                                dict(renormalize=False)], ids=str)
def test_rows_that_start_off_sixteen_bytes(e, kw):
    """Logits, and a bias, one float into a buffer: the same as aligned ones."""
    say("moe_topk unaligned", e, kw)
    r = np.random.default_rng([80, e])
    t = 37
    l = (r.standard_normal((t, e)) * 2).astype(np.float32)
    b = (r.standard_normal(e) * 0.1).astype(np.float32)

    def shifted(a):
        buf = torch.empty(a.size + 1, device="cuda")
        v = buf[1:].view(a.shape)
        v.copy_(dev(a))
        assert v.data_ptr() % 16 == 4
        return v

    for bias in (None, b):
        compare(l, 8, bias, **kw)
        want = qmm.moe_topk(dev(l), 8, bias=None if bias is None else dev(bias), **kw)
        for L in (dev(l), shifted(l)):
            for B in ((None,) if bias is None else (dev(bias), shifted(bias))):
                got = qmm.moe_topk(L, 8, bias=B, **kw)
                torch.cuda.synchronize()
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("e, top_k, kw", [(6, 2, dict(groups=3, group_keep=2)),      # a wave a token
                                          (4, 1, dict(score="sigmoid"))])            # sixteen lanes a token
def test_the_most_tokens_a_call_takes(e, top_k, kw):
    """2^26 - 1 tokens, whose last workgroup is not full: rows of 1021 kinds, each
    token has what its kind has in a call of its own."""
    say("moe_topk most tokens", e, top_k, kw)
    t, kinds = 2 ** 26 - 1, 1021
    r = np.random.default_rng([94, e])
    rows = (r.standard_normal((kinds, e)) * 2).astype(np.float32)
    compare(rows, top_k, **kw)
    ids, weights = qmm.moe_topk(dev(rows), top_k, **kw)
    kind = torch.arange(t, device="cuda") % kinds
    logits = dev(rows)[kind]
    got_ids, got_weights = qmm.moe_topk(logits, top_k, **kw)
    torch.cuda.synchronize()
    assert torch.equal(got_ids, ids[kind])
    assert torch.equal(got_weights, weights[kind])
    del logits, got_ids, got_weights, kind
    torch.cuda.empty_cache()
