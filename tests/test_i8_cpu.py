"""Products in 8-bit integers without a GPU: every refusal of the C entry points
and of the Python calls, before any HIP call, and the workspaces' sizes."""
import pytest

torch = pytest.importorskip("torch")

import quantized_matmul_qgemv_amd as qmm  # noqa: E402
from quantized_matmul_qgemv_amd import _lib  # noqa: E402
from quantized_matmul_qgemv_amd._lib import I8Problem  # noqa: E402

INV, UNS, WSP = _lib.QMM_ERR_INVALID_ARG, _lib.QMM_ERR_UNSUPPORTED, _lib.QMM_ERR_WORKSPACE
F32, F16, BF16, I8 = _lib.QMM_F32, _lib.QMM_F16, _lib.QMM_BF16, _lib.QMM_I8
A, X, Y = 0x100000, 0x80000000, 0x40000000  # fake, aligned, never dereferenced device addresses
M, N, K = 20, 64, 64  # more rows than the product rounds itself


def problem(**kw):
    f = dict(w=A, w_scales=A, x=X, x_scales=None, bias=None, y=Y, m=M, n=N, k=K, x_type=F16, y_type=F32)
    f.update(kw)
    return I8Problem(*[f[k] for k, _ in I8Problem._fields_])


def call(problems=None, count=None, ws=A, ws_bytes=1 << 40, **kw):
    ps = problems if problems is not None else [problem(**kw)]
    arr = (I8Problem * max(1, len(ps)))(*ps)
    return _lib.lib().qmm_i8_gemm(arr, len(ps) if count is None else count, ws, ws_bytes, None)


@pytest.mark.parametrize("kw, status, text", [
    (dict(count=0), INV, "count=0"),
    (dict(problems=[problem()] * 9), INV, "count=9"),
    (dict(m=-1), INV, "m=-1"),
    (dict(m=1 << 24), INV, "m=16777216"),
    (dict(n=0), INV, "n=0"),
    (dict(n=(1 << 21) + 1), INV, "n=2097153"),
    (dict(k=0), INV, "k=0"),
    (dict(k=24), INV, "k=24"),
    (dict(k=131024), INV, "k=131024"),
    (dict(x_type=4), UNS, "type 4 of x"),
    (dict(x_type=-1), UNS, "type -1 of x"),
    (dict(y_type=I8), UNS, "type 3 of the output"),
    (dict(m=1 << 23, n=4097), INV, "too many outputs"),
    (dict(problems=[problem(m=1 << 23, n=1), problem(m=1 << 23, n=1, y=Y + (1 << 30))]), INV, "too many rows"),
    (dict(w=None), INV, "null pointer"),
    (dict(w_scales=None), INV, "null pointer"),
    (dict(x=None), INV, "null pointer"),
    (dict(y=None), INV, "null pointer"),
    (dict(x_type=I8), INV, "x_scales belong"),
    (dict(x_scales=A), INV, "x_scales belong"),
    (dict(w=A + 8), INV, "w or x is not 16-byte aligned"),
    (dict(x=X + 2), INV, "w or x is not 16-byte aligned"),
    (dict(w_scales=A + 2), INV, "not 4-byte aligned"),
    (dict(bias=A + 1), INV, "not 4-byte aligned"),
    (dict(x_type=I8, x_scales=A + 2), INV, "not 4-byte aligned"),
    (dict(y=Y + 2), INV, "y is not 4-byte aligned"),
    (dict(y=Y + 1, y_type=F16), INV, "y is not 2-byte aligned"),
    (dict(ws=None), WSP, "workspace of 0 bytes"),
    (dict(ws_bytes=1535), WSP, "workspace of 1535 bytes, 1536 needed"),
    (dict(ws=A + 8), INV, "workspace is not 16-byte aligned"),
])
def test_refusals(kw, status, text):
    assert call(**kw) == status, _lib.last_error()
    assert text in _lib.last_error(), _lib.last_error()


ROWS = M * N * 4  # bytes of a y


@pytest.mark.parametrize("problems, text", [
    ([problem(), problem()], "problem 1: y overlaps the y of problem 0"),
    ([problem(), problem(y=Y + ROWS - 4)], "problem 1: y overlaps the y of problem 0"),
    ([problem(x=Y)], "problem 0: y overlaps the x of problem 0"),
    ([problem(), problem(x=Y + ROWS - 16, y=Y + ROWS * 2)], "problem 0: y overlaps the x of problem 1"),
    ([problem(w=Y + ROWS - 16)], "problem 0: y overlaps the w of problem 0"),
    ([problem(w_scales=Y + 4)], "problem 0: y overlaps the scales of problem 0"),
    ([problem(x_type=I8, x_scales=Y + ROWS - 4)], "problem 0: y overlaps the scales of problem 0"),
    ([problem(bias=Y)], "problem 0: y overlaps the bias of problem 0"),
])
def test_outputs_on_operands(problems, text):
    assert call(problems=problems) == INV, _lib.last_error()
    assert text in _lib.last_error(), _lib.last_error()


@pytest.mark.parametrize("problems", [
    [problem(), problem(y=Y + ROWS)],
    [problem(x=Y + ROWS)],
    [problem(w=Y - N * K)],
    [problem(), problem(m=0, x=None, y=None, w=None)],  # nothing to do beside something
])
def test_side_by_side(problems):
    """Taken as far as the last check before the launch, the workspace's alignment."""
    assert call(problems=problems, ws=A + 8) == INV
    assert "workspace is not 16-byte aligned" in _lib.last_error(), _lib.last_error()


def size(*ps):
    return _lib.lib().qmm_i8_gemm_workspace_size((I8Problem * len(ps))(*ps), len(ps))


def test_workspace_sizes():
    assert call(m=0) == 0  # clears the message
    one = size(problem())
    assert one == 1536  # 20 x 64 codes, 20 scales, each on 256
    assert size(problem(), problem(n=9, w=None, y=None)) == one  # one x, rounded once
    assert size(problem(), problem(x=X + 4096)) == 2 * one
    assert size(problem(), problem(m=M - 1)) > one
    assert size(problem(), problem(m=0)) == one
    assert size(problem(x_type=I8)) == 0
    assert size(problem(m=2)) == 0  # rounded by the product
    assert size(problem(m=2), problem(m=2, x_type=BF16)) == 4 * 256  # of two types: before it
    # k in parts: int32 sums of each part
    parts = size(problem(x_type=I8, n=1024, k=8192))
    assert parts >= 2 * M * 1024 * 4 and parts % (M * 1024 * 4) == 0
    for bad in (dict(k=0), dict(k=17), dict(n=0), dict(m=-1), dict(x_type=7)):
        assert size(problem(**bad)) == 0
        assert _lib.last_error() == ""
    assert _lib.lib().qmm_i8_gemm_workspace_size(None, 1) == 0
    grouped = _lib.lib().qmm_i8_grouped_workspace_size
    assert grouped(4, 64, F16) == 512 and grouped(4, 64, I8) == 0 and grouped(-1, 64, F16) == 0 and grouped(4, 8, F16) == 0


def test_nothing_to_do():
    assert call(m=0, x=None, y=None) == 0
    assert _lib.lib().qmm_i8_quantize(None, F16, None, None, 0, 64, None) == 0


def quantize(x=X, x_type=F16, codes=A, scales=Y, m=M, k=K):
    return _lib.lib().qmm_i8_quantize(x, x_type, codes, scales, m, k, None)


@pytest.mark.parametrize("kw, status, text", [
    (dict(x_type=I8), UNS, "type 3 of x"),
    (dict(x_type=9), UNS, "type 9 of x"),
    (dict(m=-1), INV, "m=-1"),
    (dict(m=1 << 24), INV, "m=16777216"),
    (dict(k=8), INV, "k=8"),
    (dict(k=131024), INV, "k=131024"),
    (dict(x=None), INV, "null pointer x"),
    (dict(x=X + 8), INV, "x is not 16-byte aligned"),
    (dict(codes=None), INV, "null pointer codes"),
    (dict(codes=A + 4), INV, "codes is not 16-byte aligned"),
    (dict(scales=None), INV, "null pointer scales"),
    (dict(scales=Y + 2), INV, "scales is not 4-byte aligned"),
    (dict(codes=X), INV, "overlap"),
    (dict(scales=X + M * K * 2 - 4), INV, "overlap"),
    (dict(scales=A + 16), INV, "overlap"),
])
def test_rounding_refusals(kw, status, text):
    assert quantize(**kw) == status, _lib.last_error()
    assert text in _lib.last_error(), _lib.last_error()


def routed(gated, **kw):
    f = dict(w=A, ws=A, w2=A, ws2=A, a=X, sa=None, a_type=F16, per_pair=0, plan=A, plan_bytes=1 << 30, y=Y, y_type=F32,
             t=M, top_k=2, e=4, n=N, k=K, wsp=A, wsp_bytes=1 << 40)
    f.update(kw)
    tail = (f["plan"], f["plan_bytes"], f["y"], f["y_type"], f["t"], f["top_k"], f["e"], f["n"], f["k"], f["wsp"],
            f["wsp_bytes"], None)
    if gated:
        return _lib.lib().qmm_i8_moe_gate_up_swiglu(f["w"], f["ws"], f["w2"], f["ws2"], f["a"], f["sa"], f["a_type"], *tail)
    return _lib.lib().qmm_i8_gemm_grouped(f["w"], f["ws"], f["a"], f["sa"], f["a_type"], f["per_pair"], *tail)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kw, status, text", [
    (dict(t=-1), INV, "t=-1"),
    (dict(top_k=0), INV, "top_k=0"),
    (dict(e=0), INV, "e=0"),
    (dict(e=1025), INV, "e=1025"),
    (dict(n=0), INV, "n=0"),
    (dict(k=40), INV, "k=40"),
    (dict(k=131024), INV, "k=131024"),
    (dict(a_type=5), UNS, "type 5 of x"),
    (dict(y_type=I8), UNS, "type 3 of the output"),
    (dict(t=1 << 23), INV, "too many pairs"),
    (dict(t=1 << 22, k=1024), INV, "rows * k must be below 2^32"),
    (dict(t=1 << 22, n=1 << 13, k=16), INV, "too many outputs"),
    (dict(w=None), INV, "null pointer w"),
    (dict(w=A + 8), INV, "w is not 16-byte aligned"),
    (dict(ws=None), INV, "null pointer w_scales"),
    (dict(a=None), INV, "null pointer x"),
    (dict(a=X + 4), INV, "x is not 16-byte aligned"),
    (dict(a_type=I8), INV, "null pointer x_scales"),
    (dict(sa=A), INV, "scales belong to rows of type QMM_I8"),
    (dict(plan=None), INV, "null pointer plan"),
    (dict(plan=A + 4), INV, "plan is not 16-byte aligned"),
    (dict(y=None), INV, "null pointer y"),
    (dict(y=Y + 2), INV, "y is not 4-byte aligned"),
    (dict(plan_bytes=64), WSP, "plan of 64 bytes"),
    (dict(wsp=None), WSP, "workspace of 0 bytes"),
    (dict(wsp_bytes=8), WSP, "workspace of 8 bytes"),
    (dict(wsp=A + 4), INV, "workspace is not 16-byte aligned"),
    (dict(y=X), INV, "the output overlaps its rows"),
])
def test_routed_refusals(gated, kw, status, text):
    assert routed(gated, **kw) == status, _lib.last_error()
    assert text in _lib.last_error(), _lib.last_error()


@pytest.mark.parametrize("gated", [False, True])
def test_refusal_of_a_grid_past_32_bits(gated):
    """1024 experts by 2^21 columns: at least 2048 row tiles by 8192 column tiles."""
    assert routed(gated, t=8192, top_k=2, e=1024, n=1 << 21, k=16, y=1 << 45, plan_bytes=1 << 30) == INV
    assert "too many tiles" in _lib.last_error(), _lib.last_error()


def test_refusals_of_one_routed_call_only():
    assert routed(False, per_pair=2) == INV and "a_row_per_pair" in _lib.last_error()
    # with a row for each pair there are twice as many
    assert routed(False, per_pair=1, t=1 << 21, k=1024) == INV and "rows * k" in _lib.last_error()
    assert routed(True, w2=None) == INV and "null pointer w2" in _lib.last_error()
    assert routed(True, ws2=A + 1) == INV and "w2_scales is not 4-byte aligned" in _lib.last_error()
    assert routed(False, t=0, a=None) == 0 and routed(True, t=0, a=None) == 0


# ------------------------------------------------------------------ from Python

def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


W, WS, XF = z(8, 64, dtype=torch.int8), z(8), z(3, 64, dtype=torch.float16)


@pytest.mark.parametrize("error, text, f", [
    (ValueError, "no problems", lambda: qmm.i8_gemm_batched([])),
    (ValueError, "must be \\[n, k\\]", lambda: qmm.i8_gemm(W, WS, z(3, 32, dtype=torch.float16))),
    (ValueError, "x must be \\[m, k\\]", lambda: qmm.i8_gemm(W, WS, z(64, dtype=torch.float16))),
    (ValueError, "w_scales must be \\[8\\]", lambda: qmm.i8_gemm(W, z(7), XF)),
    (ValueError, "x_scales must be \\[3\\]", lambda: qmm.i8_gemm(W, WS, XF, z(4))),
    (ValueError, "bias must be \\[8\\]", lambda: qmm.i8_gemm(W, WS, XF, bias=z(1))),
    (ValueError, "y must be \\[3, 8\\]", lambda: qmm.i8_gemm(W, WS, XF, y=z(8, 3))),
    (ValueError, "x must be a device tensor", lambda: qmm.i8_gemm(W, WS, XF, y=z(3, 8))),
    (TypeError, "x has dtype torch.float64", lambda: qmm.i8_gemm_workspace([(W, WS, z(3, 64, dtype=torch.float64), None, None, None)])),
    (TypeError, "x has dtype torch.int32", lambda: qmm.i8_grouped_workspace(z(3, 64, dtype=torch.int32))),
    (ValueError, "x must be \\[m, k\\]", lambda: qmm.i8_quantize(z(64))),
    (ValueError, "codes must be", lambda: qmm.i8_quantize(XF, codes=z(3, 32, dtype=torch.int8))),
    (ValueError, "scales must be", lambda: qmm.i8_quantize(XF, scales=z(4))),
    (ValueError, "x must be a device tensor", lambda: qmm.i8_quantize(XF)),
])
def test_python_refusals(error, text, f):
    with pytest.raises(error, match=text):
        f()


@pytest.mark.parametrize("error, text, kw", [
    (ValueError, "expert_ids must be", dict(expert_ids=z(6, dtype=torch.int32))),
    (ValueError, "must be \\[E, n, k\\]", dict(w=W)),
    (ValueError, "must be \\[E, n, k\\]", dict(a=z(3, 32, dtype=torch.float16))),
    (ValueError, "and their scales", dict(ws=z(2, 7))),
    (ValueError, "there must be 3 rows", dict(a=z(6, 64, dtype=torch.float16))),
    (ValueError, "rows' scales must be \\[3\\]", dict(sa=z(6))),
    (ValueError, "the output must be \\[6, 8\\]", dict(y=z(3, 8))),
    (ValueError, "x must be a device tensor", dict()),
])
def test_python_routed_refusals(error, text, kw):
    f = dict(w=z(2, 8, 64, dtype=torch.int8), ws=z(2, 8), a=XF, expert_ids=z(3, 2, dtype=torch.int32), sa=None, y=None)
    f.update(kw)
    plan = z(256, dtype=torch.uint8)
    with pytest.raises(error, match=text):
        qmm.i8_gemm_grouped(f["w"], f["ws"], f["a"], f["expert_ids"], plan, False, a_scales=f["sa"], y=f["y"])
    with pytest.raises(error, match=text):
        qmm.i8_moe_gate_up_swiglu((f["w"], f["ws"]), (f["w"], f["ws"]), f["a"], f["expert_ids"], plan, x_scales=f["sa"],
                                  h=f["y"])


# ------------------------------------------- outputs and workspaces on what a call reads

OUT = M * 2 * N * 4  # bytes of a routed call's output
W_BYTES = 4 * N * K


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kw, text", [
    (dict(w=Y), "the weights"),
    (dict(w=Y - W_BYTES + 16), "the weights"),
    (dict(ws=Y + OUT - 4), "the weights' scales"),
    (dict(ws=Y - 4 * N * 4 + 4), "the weights' scales"),
    (dict(a_type=I8, sa=Y + 4), "its rows' scales"),
    (dict(plan=Y), "the plan"),
    (dict(plan=Y + OUT - 16), "the plan"),
])
def test_routed_outputs_on_operands(gated, kw, text):
    assert routed(gated, **kw) == INV, _lib.last_error()
    assert _lib.last_error().endswith("the output overlaps " + text), _lib.last_error()


@pytest.mark.parametrize("kw, text", [(dict(w2=Y + OUT - 16), "the weights"), (dict(ws2=Y), "the weights' scales")])
def test_routed_outputs_on_the_second_weights(kw, text):
    assert routed(True, **kw) == INV, _lib.last_error()
    assert _lib.last_error().endswith("the output overlaps " + text), _lib.last_error()


BIG, BIG_OUT, BIG_W, BIG_S = 1 << 45, 16384 * (1 << 21) * 4, 1024 * (1 << 21) * 16, 1024 * (1 << 21) * 4


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kw", [dict(w=BIG - BIG_W), dict(w=BIG + BIG_OUT), dict(ws=BIG + BIG_OUT), dict(ws=BIG - BIG_S),
                                dict(plan=BIG + BIG_OUT), dict(w2=BIG + BIG_OUT, ws2=BIG - BIG_S),
                                dict(a_type=I8, sa=BIG + BIG_OUT), dict(a_type=I8, sa=BIG - 8192 * 4)])
def test_routed_outputs_beside_operands(gated, kw):
    """Taken as far as the number of tiles, which is refused behind every overlap of the output."""
    assert routed(gated, t=8192, top_k=2, e=1024, n=1 << 21, k=16, y=BIG, plan_bytes=1 << 30, **kw) == INV
    assert "too many tiles" in _lib.last_error(), _lib.last_error()


NEED = 1536  # bytes of the workspace of 20 x 64 rows: codes and scales
SPACE = 0x60000000


@pytest.mark.parametrize("kw, text", [
    (dict(x=SPACE), "x"),
    (dict(x=SPACE + NEED - 16), "x"),
    (dict(w=SPACE - N * K + 16), "w"),
    (dict(w_scales=SPACE + NEED - 4), "scales"),
    (dict(bias=SPACE), "bias"),
    (dict(y=SPACE + NEED - 4), "y"),
    (dict(y=SPACE - ROWS + 4), "y"),
])
def test_workspaces_on_operands(kw, text):
    assert call(ws=SPACE, **kw) == INV, _lib.last_error()
    assert _lib.last_error().endswith(f"the workspace overlaps the {text} of problem 0"), _lib.last_error()


def test_workspaces_on_the_operands_of_other_problems():
    """A workspace that the sums of parts of k need, on the scales of given codes."""
    ps = [problem(x_type=I8, x_scales=A, n=1024, k=8192), problem(x_type=I8, x_scales=SPACE + 64, n=1024, k=8192, y=Y + (1 << 24))]
    assert call(problems=ps, ws=SPACE) == INV, _lib.last_error()
    assert _lib.last_error().endswith("the workspace overlaps the scales of problem 1"), _lib.last_error()
    # no rows, nothing read: what such a problem names does not matter
    ps = [problem(), problem(m=0, x=SPACE, w=SPACE), problem(y=SPACE, m=M)]
    assert call(problems=ps, ws=SPACE) == INV, _lib.last_error()
    assert _lib.last_error().endswith("the workspace overlaps the y of problem 2"), _lib.last_error()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kw, text", [
    (dict(a=SPACE), "its rows"),
    (dict(w=SPACE), "the weights"),
    (dict(ws=SPACE + NEED - 4), "the weights' scales"),
    (dict(plan=SPACE + NEED - 16), "the plan"),
    (dict(y=SPACE + NEED - 4), "the output"),
    (dict(y=SPACE - OUT + 4), "the output"),
])
def test_routed_workspaces_on_operands(gated, kw, text):
    assert routed(gated, wsp=SPACE, **kw) == INV, _lib.last_error()
    assert _lib.last_error().endswith("the workspace overlaps " + text), _lib.last_error()


def test_routed_workspaces_on_the_second_weights():
    for kw, text in ((dict(w2=SPACE), "the weights"), (dict(ws2=SPACE), "the weights' scales")):
        assert routed(True, wsp=SPACE, **kw) == INV, _lib.last_error()
        assert _lib.last_error().endswith("the workspace overlaps " + text), _lib.last_error()


@pytest.mark.parametrize("kw", [dict(x=SPACE + NEED), dict(x=SPACE - M * K * 2), dict(w=SPACE - N * K), dict(w_scales=SPACE + NEED), dict(bias=SPACE - N * 4)])
def test_workspaces_beside_operands(kw):
    """Only the y of the second problem, the last that is looked at, is on the workspace."""
    ps = [problem(**kw), problem(n=1, x=kw.get("x", X), y=SPACE + 256)]
    assert call(problems=ps, ws=SPACE) == INV
    assert _lib.last_error().endswith("the workspace overlaps the y of problem 1"), _lib.last_error()


# --------------------------------------------------- sizes that 32 bits do not hold

def far(*shape, dtype=torch.int8):
    """A tensor without memory: only its sizes are looked at."""
    return torch.empty(shape, dtype=dtype, device="meta")


LONG = (1 << 32) + 16  # 16 in 32 bits


@pytest.mark.parametrize("text, f", [
    ("m=4294967312", lambda: qmm.i8_quantize(far(LONG, 16, dtype=torch.float16))),
    ("m=4294967312", lambda: qmm.i8_quantize(far((1 << 28) + 1, 16, 16, dtype=torch.float16))),
    ("k=4294967312", lambda: qmm.i8_quantize(far(1, LONG, dtype=torch.float16))),
    ("m=4294967312", lambda: qmm.i8_gemm(far(8, 16), far(8, dtype=torch.float32), far(LONG, 16), far(LONG, dtype=torch.float32))),
    ("n=4294967312", lambda: qmm.i8_gemm(far(LONG, 16), far(LONG, dtype=torch.float32), far(3, 16, dtype=torch.float16))),
    ("k=4294967312", lambda: qmm.i8_gemm(far(8, LONG), far(8, dtype=torch.float32), far(3, LONG, dtype=torch.float16))),
    ("m=4294967312", lambda: qmm.i8_gemm_workspace([(far(8, 16), None, far(LONG, 16), None, None, None)])),
    ("n=4294967312", lambda: qmm.i8_gemm_workspace([(far(LONG, 16), None, far(3, 16), None, None, None)])),
    ("rows=4294967312", lambda: qmm.i8_grouped_workspace(far(LONG, 16, dtype=torch.float16))),
    ("k=4294967312", lambda: qmm.i8_grouped_workspace(far(3, LONG, dtype=torch.float16))),
])
def test_sizes_past_32_bits(text, f):
    with pytest.raises(ValueError, match=text + " must be below 2"):
        f()


@pytest.mark.parametrize("text, t, top_k, e, n, k", [
    ("t=4294967312", LONG, 1, 2, 8, 16), ("top_k=4294967312", 1, LONG, 2, 8, 16), ("pairs=4294967312", LONG // 16, 16, 2, 8, 16),
    ("e=4294967312", 3, 2, LONG, 8, 16), ("n=4294967312", 3, 2, 2, LONG, 16), ("k=4294967312", 3, 2, 2, 8, LONG)])
def test_routed_sizes_past_32_bits(text, t, top_k, e, n, k):
    w, ws = far(e, n, k), far(e, n, dtype=torch.float32)
    x, ids, plan = far(t, k, dtype=torch.float16), far(t, top_k, dtype=torch.int32), far(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match=text + " must be below 2"):
        qmm.i8_gemm_grouped(w, ws, x, ids, plan, False)
    with pytest.raises(ValueError, match=text + " must be below 2"):
        qmm.i8_moe_gate_up_swiglu((w, ws), (w, ws), x, ids, plan)


@pytest.mark.parametrize("text, f", [
    ("no problems", lambda: qmm.i8_gemm_workspace([])),
    ("problem 0: x must be \\[m, k\\]", lambda: qmm.i8_gemm_workspace([(W, WS, z(64, dtype=torch.float16), None, None, None)])),
    ("problem 1: w .* and x .* must be", lambda: qmm.i8_gemm_workspace([(W, WS, XF, None, None, None),
                                                                     (z(8, 32, dtype=torch.int8), WS, XF, None, None, None)])),
    ("problem 0: w .* and x .* must be", lambda: qmm.i8_gemm_workspace([(z(8, dtype=torch.int8), WS, XF, None, None, None)])),
    ("x must be \\[rows, k\\]", lambda: qmm.i8_grouped_workspace(z(64, dtype=torch.float16))),
    ("x must be \\[rows, k\\]", lambda: qmm.i8_grouped_workspace(z(3, 2, 64, dtype=torch.float16))),
])
def test_workspaces_for_operands_of_the_wrong_shape(text, f):
    """Refused as by the calls that they are for."""
    with pytest.raises(ValueError, match=text):
        f()
