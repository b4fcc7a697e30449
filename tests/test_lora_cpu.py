"""Low-rank adapters without a GPU: every refusal of qmm_lora and of the Python
calls, before any HIP call, and the workspace's size."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

import quantized_matmul_qgemv_amd as qmm  # noqa: E402
from quantized_matmul_qgemv_amd import _lib  # noqa: E402
from quantized_matmul_qgemv_amd._lib import LoraProblem  # noqa: E402

INV, WSP = _lib.QMM_ERR_INVALID_ARG, _lib.QMM_ERR_WORKSPACE
A = 0x100000  # a fake, aligned, never dereferenced device address
Y = 0x40000000


def problem(**kw):
    f = dict(x=A, a=A, b=A, base=None, y=Y, n=64, k=64, rank=8, x_row_per_pair=0)
    f.update(kw)
    return LoraProblem(*[f[k] for k, _ in LoraProblem._fields_])


def call(problems=None, count=None, ids=A, experts_ids=None, scales=None, t=4, top_k=1, adapters=3, experts=0,
         ws=A, ws_bytes=1 << 40, **kw):
    ps = problems if problems is not None else [problem(**kw)]
    arr = (LoraProblem * max(1, len(ps)))(*ps)
    return _lib.lib().qmm_lora(arr, len(ps) if count is None else count, ids, experts_ids, scales, t, top_k,
                               adapters, experts, ws, ws_bytes, None)


@pytest.mark.parametrize("kw, status, text", [
    (dict(count=0), INV, "count=0"),
    (dict(problems=[problem()] * 9), INV, "count=9"),
    (dict(t=-1), INV, "t=-1"),
    (dict(top_k=0), INV, "top_k=0"),
    (dict(top_k=2), INV, "without experts"),
    (dict(adapters=0), INV, "adapters=0"),
    (dict(adapters=4097), INV, "4097 sets"),
    (dict(experts=-1), INV, "experts=-1"),
    (dict(adapters=64, experts=128, experts_ids=A), INV, "8192 sets"),
    (dict(t=0x7FFFFFFF), INV, "too many rows"),
    (dict(n=0), INV, "n=0"),
    (dict(n=(1 << 21) + 1), INV, "n=2097153"),
    (dict(k=0), INV, "k=0"),
    (dict(k=96), INV, "k=96"),
    (dict(k=(1 << 24) + 64), INV, "k=16777280"),
    (dict(rank=0), INV, "rank=0"),
    (dict(rank=12), INV, "rank=12"),
    (dict(rank=264), INV, "rank=264"),
    (dict(x_row_per_pair=2), INV, "x_row_per_pair"),
    (dict(ids=None), INV, "null pointer adapter_ids"),
    (dict(ids=A + 2), INV, "adapter_ids is not 4-byte aligned"),
    (dict(experts=8), INV, "null pointer expert_ids"),
    (dict(scales=A + 1), INV, "scales is not 4-byte aligned"),
    (dict(x=None), INV, "problem 0 has a null pointer"),
    (dict(y=None), INV, "problem 0 has a null pointer"),
    (dict(a=A + 8), INV, "not 16-byte aligned"),
    (dict(base=A + 2), INV, "base or y is not 4-byte aligned"),
    (dict(base=Y + 64), INV, "y overlaps base"),
    (dict(problems=[problem(), problem(rank=9)]), INV, "problem 1: rank=9"),
    (dict(ws=None), WSP, "workspace of 0 bytes"),
    (dict(ws_bytes=64), WSP, "workspace of 64 bytes"),
    (dict(ws=A + 8), INV, "workspace is not 16-byte aligned"),
])
def test_refusals(kw, status, text):
    assert call(**kw) == status, _lib.last_error()
    assert text in _lib.last_error(), _lib.last_error()


def test_null_problems_and_no_tokens():
    assert _lib.lib().qmm_lora(None, 1, A, None, None, 4, 1, 3, 0, A, 1 << 40, None) == INV
    assert call(t=0, ids=None, ws=None) == 0
    assert _lib.last_error() == ""


def size(rows, slots, *ps):
    arr = (LoraProblem * len(ps))(*ps)
    return _lib.lib().qmm_lora_workspace_size(arr, len(ps), rows, slots)


def test_workspace_size():
    one = size(64, 8, problem(k=4096, rank=16))
    assert one >= 64 * 16 * 4
    assert size(64, 8, problem(k=4096, rank=16), problem(k=4096, rank=16)) > one
    # sorted rows, their tiles and the partial products
    assert size(100000, 64, problem(k=4096, rank=16)) >= 100000 * (4 + 16 * 4)
    assert size(100000, 64, problem(k=4096, rank=16)) >= size(4096, 64, problem(k=4096, rank=16))
    for bad in (size(0, 8, problem()), size(4, 0, problem()), size(4, 4097, problem()), size(4, 4, problem(k=65)),
                size(1 << 30, 4, problem()), _lib.lib().qmm_lora_workspace_size(None, 1, 4, 4)):
        assert bad == 0


@pytest.mark.parametrize("rows", [1, 256, 257, 4096, 4097, 65536, 1 << 20])
@pytest.mark.parametrize("slots", [1, 64, 4096])
def test_workspace_holds_what_the_call_asks_for(rows, slots):
    ps = [problem(k=2560, rank=24), problem(k=64, rank=256, n=7)]
    need = size(rows, slots, *ps)
    assert need > 0
    assert call(problems=ps, t=rows, adapters=slots, ws_bytes=need - 1) == WSP
    assert f"{need} needed" in _lib.last_error()


def test_python_refusals():
    h = torch.float16
    x, a, b = torch.zeros(4, 64, dtype=h), torch.zeros(3, 8, 64, dtype=h), torch.zeros(3, 10, 8, dtype=h)
    ids = torch.zeros(4, dtype=torch.int32)
    for args, kw, text in [
        ((x, a, b, ids.view(2, 2)), {}, r"adapter_ids must be \[T\]"),
        ((x[:3], a, b, ids), {}, r"x must be \[4, 64\]"),
        ((x, a, b[:2], ids), {}, "must be"),
        ((x, a, torch.zeros(3, 10, 16, dtype=h), ids), {}, "must be"),
        ((x, a, b, ids), dict(base=torch.zeros(4, 11)), "base must be"),
        ((x, a, b, ids), dict(y=torch.zeros(5, 10)), "y must be"),
        ((x, a, b, ids), dict(scales=torch.ones(2)), r"scales must be \[3\]"),
        ((x, a, b, ids), dict(expert_ids=torch.zeros(4, 2, dtype=torch.int32)), "experts, rank, k"),
        ((x, a, b, ids), dict(expert_ids=torch.zeros(3, 2, dtype=torch.int32)), "expert_ids must be"),
        ((x, a, b, ids), {}, "device tensor"),
    ]:
        with pytest.raises(ValueError, match=text):
            qmm.lora(*args, **kw)
    with pytest.raises(ValueError, match="no problems"):
        qmm.lora_batched([], ids)
    assert C.sizeof(LoraProblem) == 56
