"""Low-rank adapters without a GPU: calls that cannot be meant are refused, with
what is meant beside them taken, before any HIP call."""
import pytest

torch = pytest.importorskip("torch")

import quantized_matmul_qgemv_amd as qmm  # noqa: E402
from quantized_matmul_qgemv_amd import _lib  # noqa: E402
from quantized_matmul_qgemv_amd._lib import LoraProblem  # noqa: E402
from test_lora_cpu import A, INV, Y, call, problem  # noqa: E402

X = 0x80000000  # more fake addresses
T, N = 4, 64
ROWS = T * N * 4  # bytes of a y or base


# ------------------------------------------------ problems of one call that overlap

@pytest.mark.parametrize("problems, text", [
    ([problem(), problem()], "problem 1: y overlaps the y of problem 0"),
    ([problem(), problem(y=Y + ROWS - 4)], "problem 1: y overlaps the y of problem 0"),
    ([problem(y=Y + ROWS - 4), problem()], "problem 1: y overlaps the y of problem 0"),
    ([problem(), problem(y=Y + ROWS), problem(y=Y + 2 * ROWS - 4)], "problem 2: y overlaps the y of problem 1"),
    # two adapters stacked in one call: the second would read what the first has, or has not yet, written
    ([problem(), problem(base=Y, y=Y + ROWS)], "problem 0: y overlaps the base of problem 1"),
    ([problem(base=Y + ROWS), problem(y=Y + ROWS)], "problem 1: y overlaps the base of problem 0"),
    ([problem(), problem(base=Y + ROWS - 4, y=Y + 2 * ROWS)], "problem 0: y overlaps the base of problem 1"),
    ([problem(x=Y)], "problem 0: y overlaps the x of problem 0"),
    ([problem(), problem(x=Y + ROWS - 16, y=Y + ROWS)], "problem 0: y overlaps the x of problem 1"),
    ([problem(x=X), problem(x=X - ROWS + 16, y=X - ROWS + 16)], "problem 1: y overlaps the x of problem 0"),
])
def test_problems_that_overlap(problems, text):
    assert call(problems=problems) == INV, _lib.last_error()
    assert text in _lib.last_error(), _lib.last_error()


@pytest.mark.parametrize("problems", [
    [problem(), problem(y=Y + ROWS)],
    [problem(base=Y), problem(base=Y + ROWS, y=Y + ROWS)],             # each in place
    [problem(base=X), problem(base=X, y=Y + ROWS)],                    # one base of both
    [problem(x=X), problem(x=X, y=X + T * 64 * 2)],                    # y right behind x
    [problem(x=X), problem(x=X, y=X - ROWS)],                          # and right before
    [problem(x=X, x_row_per_pair=0), problem(x=X, y=X + 64 * 64 * 2)],
])
def test_problems_side_by_side(problems):
    """Taken as far as the last check before the launch, the workspace's alignment."""
    assert call(problems=problems, ws=A + 8) == INV
    assert "workspace is not 16-byte aligned" in _lib.last_error(), _lib.last_error()


def test_the_rows_of_pairs_count():
    ps = [problem(x=X, x_row_per_pair=1, y=X + T * 64 * 2)]  # x has a row for every pair: twice as many
    kw = dict(top_k=2, experts=4, experts_ids=A, ws=A + 8)
    assert call(problems=ps, **kw) == INV
    assert "problem 0: y overlaps the x of problem 0" in _lib.last_error()
    assert call(problems=[problem(x=X, x_row_per_pair=0, y=X + T * 64 * 2)], **kw) == INV
    assert "workspace is not 16-byte aligned" in _lib.last_error()


# ------------------------------------------------ what the workspace's size depends on

def size(rows, slots, *ps):
    arr = (LoraProblem * len(ps))(*ps)
    return _lib.lib().qmm_lora_workspace_size(arr, len(ps), rows, slots)


@pytest.mark.parametrize("rows", [4, 300, 5000])
def test_the_workspace_depends_on_k_and_rank_alone(rows):
    assert call(t=0) == 0
    need = size(rows, 8, problem(k=4096, rank=16), problem(k=64, rank=128))
    assert need > 0
    bare = [LoraProblem(None, None, None, None, None, 0, 4096, 16, 0), LoraProblem(None, None, None, None, None, -1, 64, 128, 7)]
    assert size(rows, 8, *bare) == need
    for bad in (dict(k=0), dict(k=65), dict(rank=0), dict(rank=12), dict(rank=264)):
        assert size(rows, 8, problem(**bad)) == 0
        assert _lib.last_error() == ""  # asking for a size is no failed call
    # the call itself looks at everything
    assert call(problems=[problem(n=0)]) == INV and "n=0" in _lib.last_error()
    assert call(problems=[problem(x_row_per_pair=7)]) == INV and "x_row_per_pair" in _lib.last_error()


# ------------------------------------------------ experts that are named in part

def test_expert_ids_without_a_number_of_experts():
    assert call(experts=0, experts_ids=A, ws=A + 8) == INV
    assert "expert_ids without experts" in _lib.last_error(), _lib.last_error()
    assert call(experts=4, experts_ids=A, ws=A + 8) == INV
    assert "workspace is not 16-byte aligned" in _lib.last_error()


# ------------------------------------------------ the Python call's shapes

def h(*shape):
    return torch.zeros(*shape, dtype=torch.float16)


IDS, EXPERT_IDS = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32)


def test_weights_for_experts_without_expert_ids():
    """[adapters, experts, ...] weights in a call without expert_ids: not adapters x experts of them."""
    a, b = h(2, 3, 8, 64), h(2, 3, 10, 8)
    with pytest.raises(ValueError, match=r"problem 0: a must be \[adapters, rank, k\] without expert_ids"):
        qmm.lora(h(4, 64), a, b, IDS)
    with pytest.raises(ValueError, match="without expert_ids"):
        qmm.lora_workspace([(h(4, 64), a, b, None, None)], IDS)
    with pytest.raises(ValueError, match="device tensor"):
        qmm.lora(h(4, 64), a, b, IDS, expert_ids=EXPERT_IDS)
    with pytest.raises(ValueError, match="device tensor"):
        qmm.lora(h(4, 64), a[:, 0], b[:, 0], IDS)


def test_weights_laid_out_otherwise():
    """Every a and b holds its weights by adapter and expert as the call has them;
    an equal number of values is not enough."""
    x, a, b = h(4, 64), h(2, 3, 8, 64), h(2, 3, 10, 8)
    kw = dict(expert_ids=EXPERT_IDS)
    flat_a, flat_b, scales = h(6, 8, 64), h(6, 10, 8), torch.ones(2)
    for args, other in [
        ((x, a, h(3, 2, 10, 8), IDS), kw),              # b by expert and adapter
        ((x, a, h(6, 1, 10, 8), IDS), kw),
        ((x, a, h(2, 3, 1, 10, 8), IDS), kw),
        ((x, h(2, 8, 64), h(2, 1, 10, 8), IDS), {}),
        ((x, h(2, 8, 64), h(2, 0, 10, 8), IDS), {}),
        ((x, flat_a, h(3, 2, 10, 8), IDS), dict(kw, scales=scales, experts=3)),
    ]:
        with pytest.raises(ValueError, match="problem 0: a .* and b .* must be"):
            qmm.lora(*args, **other)
    for second in [(x, h(3, 2, 8, 64), b, None, None), (x, h(3, 2, 8, 64), h(3, 2, 10, 8), None, None),
                   (x, h(2, 8, 64), h(2, 10, 8), None, None)]:
        with pytest.raises(ValueError, match="problem 1: a .* and b .* must be"):
            qmm.lora_batched([(x, a, b, None, None), second], IDS, **kw)
    # each way of holding the same weights, and both in one call
    for args, other in [((x, a, b, IDS), kw), ((x, a, flat_b, IDS), kw), ((x, flat_a, flat_b, IDS), dict(kw, scales=scales)),
                        ((x, flat_a, b, IDS), dict(kw, scales=scales))]:
        with pytest.raises(ValueError, match="device tensor"):
            qmm.lora(*args, **other)


def test_the_number_of_experts_of_flattened_weights():
    """Flattened weights do not say how many experts they are of: the call can,
    and scales of another length are then refused; so do weights of another
    problem that are not flattened.  Otherwise scales [adapters] say it."""
    x, a, b = h(4, 64), h(12, 8, 64), h(12, 10, 8)
    kw = dict(expert_ids=EXPERT_IDS)
    for scales in (torch.ones(6), torch.ones(2), torch.ones(12), torch.ones(5)):
        with pytest.raises(ValueError, match=r"scales must be \[4\]"):
            qmm.lora(x, a, b, IDS, scales=scales, experts=3, **kw)
        with pytest.raises(ValueError, match=r"scales must be \[4\]"):
            qmm.lora(x, a, b.view(4, 3, 10, 8), IDS, scales=scales, **kw)
        with pytest.raises(ValueError, match=r"scales must be \[4\]"):
            qmm.lora_batched([(x, a, b, None, None), (x, a.view(4, 3, 8, 64), b, None, None)], IDS, scales, EXPERT_IDS)
    for scales in (None, torch.ones(4)):
        with pytest.raises(ValueError, match="device tensor"):
            qmm.lora(x, a, b, IDS, scales=scales, experts=3, **kw)
    with pytest.raises(ValueError, match="device tensor"):
        qmm.lora(x, a, b, IDS, scales=torch.ones(6), **kw)
    with pytest.raises(ValueError, match="12 sets of weights are not a multiple of 5 experts"):
        qmm.lora(x, a, b, IDS, experts=5, **kw)
    with pytest.raises(ValueError, match="problem 0: a .* and b .* must be"):
        qmm.lora(x, a.view(4, 3, 8, 64), b, IDS, experts=4, **kw)
    with pytest.raises(ValueError, match="experts=3 without expert_ids"):
        qmm.lora(x, a, b, IDS, experts=3)
    for wrong in (0, -3):
        with pytest.raises(ValueError, match="experts="):
            qmm.lora(x, a, b, IDS, experts=wrong, **kw)
