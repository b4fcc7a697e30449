"""Low-rank adapters: calls that stand at the edge of what the header promises."""
import numpy as np
import pytest

from qmm_testlib import dev, host, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import quantized_matmul_qgemv_amd as qmm  # noqa: E402


def weights(r, slots, rank, k, n):
    a = (r.standard_normal((slots, rank, k)) / np.sqrt(k)).astype(np.float16)
    b = (r.standard_normal((slots, n, rank)) * 0.1).astype(np.float16)
    return a, b


@pytest.mark.parametrize("t", [2, 40, 300, 700])
@pytest.mark.parametrize("rank", [8, 16, 24, 40, 64])
@pytest.mark.parametrize("k", [64, 1024, 2112])
def test_an_infinite_weight_gives_the_same_alone_and_among_others(t, rank, k):
    """One infinity among the first weights of a row of A: A x has it times a
    finite x there, B A x likewise, whatever rows stand beside and however many."""
    say("lora infinite weight", t, rank, k)
    r = np.random.default_rng([93, t, rank, k])
    n = 70
    a, b = weights(r, 2, rank, k, n)
    a[0, rank // 2, 3] = np.inf
    x = r.standard_normal((t, k)).astype(np.float16)
    x[:, 3] = np.where(np.abs(x[:, 3]) < 0.1, np.float16(1), x[:, 3])
    b[0, :, rank // 2] = np.where(np.abs(b[0, :, rank // 2]) < 0.01, np.float16(0.5), b[0, :, rank // 2])
    ids = r.integers(0, 2, t).astype(np.int32)
    ids[:2] = 0
    got = host(qmm.lora(dev(x), dev(a), dev(b), dev(ids)))
    torch.cuda.synchronize()
    sign = np.sign(x[:, 3].astype(np.float32))[:, None] * np.sign(b[0, :, rank // 2].astype(np.float32))[None, :]
    at = ids == 0
    assert np.array_equal(got[at], np.float32(np.inf) * sign[at])
    assert np.isfinite(got[~at]).all()
    alone = host(qmm.lora(dev(x[:1]), dev(a), dev(b), dev(ids[:1])))
    assert np.array_equal(alone[0], got[0])
