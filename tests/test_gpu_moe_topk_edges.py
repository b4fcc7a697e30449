"""Routing to experts: calls that stand at the edge of what the header promises."""
import numpy as np
import pytest

from qmm_testlib import dev, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import quantized_matmul_qgemv_amd as qmm  # noqa: E402
from test_gpu_moe_topk import compare  # noqa: E402


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
