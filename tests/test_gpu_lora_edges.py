"""Low-rank adapters: calls that stand at the edge of what the header promises."""
import numpy as np
import pytest

from qmm_testlib import Guarded, dev, host, say

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


# rows, slots, (k, n, rank) of each problem: every way a call can take
WAYS = [
    (1, 8, [(1024, 2048, 16)]),                          # dot products
    (64, 9, [(320, 100, 16), (320, 33, 64), (64, 1, 8)]),
    (512, 3, [(192, 130, 16)]),
    (200, 2, [(10240, 40, 40)]),                         # two products, tiles by ballots
    (256, 300, [(64, 64, 128), (704, 20, 256)]),
    (600, 500, [(256, 140, 24)]),                        # sorted, dot products
    (600, 500, [(256, 140, 24), (512, 9, 8)]),
    (700, 60, [(192, 65, 64)]),                          # sorted, both products in one launch
    (4096, 400, [(64, 20, 16)]),
    (4097, 400, [(64, 20, 16)]),                         # and in chunks
    (700, 3, [(1088, 65, 64), (64, 7, 8)]),              # sorted, tiles of 16, two products
    (513, 2, [(128, 64, 256)]),
    (9000, 4096, [(128, 24, 72)]),
    (1500, 3, [(704, 600, 64), (704, 10, 24)]),          # tiles of 64
    (40000, 5, [(2112, 36, 128)]),
]


@pytest.mark.parametrize("t, adapters, shapes", WAYS, ids=lambda v: str(v).replace(" ", ""))
@pytest.mark.parametrize("kind", ["apart", "same", "none and bad"])
def test_nothing_is_written_past_the_workspace(t, adapters, shapes, kind):
    """A workspace of just the size that is asked for, between guard bands, and
    the result of a larger one."""
    say("lora workspace", t, adapters, shapes, kind)
    r = np.random.default_rng([95, t, adapters])
    ids = {"apart": np.arange(t) % adapters, "same": np.full(t, adapters - 1),
           "none and bad": r.choice([-1, adapters, 0], t)}[kind].astype(np.int32)
    problems, I = [], dev(r.permutation(ids))
    for k, n, rank in shapes:
        a, b = weights(r, adapters, rank, k, n)
        problems.append((dev(r.standard_normal((t, k)).astype(np.float16)), dev(a), dev(b), None, None))
    need = qmm.lora_workspace(problems, I).numel()
    ws = Guarded((need,), torch.uint8)
    got = qmm.lora_batched(problems, I, workspace=ws.t)
    torch.cuda.synchronize()
    ws.check("workspace")
    for g, w in zip(got, qmm.lora_batched(problems, I, workspace=torch.empty(2 * need + 4096, dtype=torch.uint8, device="cuda"))):
        assert torch.equal(g.view(torch.int32), w.view(torch.int32))  # bit by bit, NaN among them


def test_two_calls_at_once_with_workspaces_of_their_own():
    """Workspaces and results that the program keeps, one of each for a stream."""
    say("lora two streams, given workspaces")
    r = np.random.default_rng(96)
    parts = []
    for t, k, n, rank in ((3000, 512, 640, 32), (5000, 768, 512, 16)):
        a, b = weights(r, 4, rank, k, n)
        ids = r.integers(-1, 4, t).astype(np.int32)
        parts.append((dev(r.standard_normal((t, k)).astype(np.float16)), dev(a), dev(b), dev(ids)))
    alone = [qmm.lora(*p) for p in parts]
    ws = [qmm.lora_workspace([p[:3] + (None, None)], p[3]) for p in parts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in parts]
    for _ in range(5):
        ys = [torch.zeros_like(a) for a in alone]
        torch.cuda.synchronize()
        for _ in range(3):
            for p, st, w, y in zip(parts, streams, ws, ys):
                qmm.lora(*p, y=y, workspace=w, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(y, a) for y, a in zip(ys, alone))


def test_flattened_weights_are_those_by_adapter_and_expert():
    say("lora flattened experts")
    r = np.random.default_rng(97)
    t, top_k, adapters, experts, k, n, rank = 60, 3, 3, 8, 128, 36, 16
    a, b = weights(r, adapters * experts, rank, k, n)
    a, b = dev(a), dev(b)
    a4, b4 = a.view(adapters, experts, rank, k), b.view(adapters, experts, n, rank)
    x = dev(r.standard_normal((t, k)).astype(np.float16))
    ids, expert_ids = dev(r.integers(-1, adapters, t).astype(np.int32)), dev(r.integers(0, experts, (t, top_k)).astype(np.int32))
    scales = dev((r.random(adapters) + 0.5).astype(np.float32))
    for s in (None, scales):
        want = qmm.lora(x, a4, b4, ids, scales=s, expert_ids=expert_ids)
        for A, B, kw in ((a, b, dict(experts=experts)), (a, b4, {}), (a4, b, {}), (a4, b4, dict(experts=experts))):
            assert torch.equal(qmm.lora(x, A, B, ids, scales=s, expert_ids=expert_ids, **kw), want)
    assert torch.equal(qmm.lora(x, a, b, ids, scales=scales, expert_ids=expert_ids), want)
