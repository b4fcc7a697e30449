"""The experts' products in 8-bit integers against their formulas in 64 bits."""
import numpy as np
import pytest

import i8_testlib as ref
from qmm_testlib import Guarded, dev, say
from test_gpu_i8_gemm import BF16, F16, F32, activations, f64, ids

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import quantized_matmul_qgemv_amd as qmm  # noqa: E402


def experts(r, e, n, k):
    return r.integers(-128, 128, (e, n, k)).astype(np.int8), (r.random((e, n)) * 2e-4 + 1e-6).astype(np.float32)


def some_ids(r, t, top_k, e, kind):
    if kind == "one":  # all pairs on one expert
        return np.full((t, top_k), e - 1, np.int32)
    ids = r.integers(0, e, (t, top_k)).astype(np.int32)
    if kind == "few":
        ids %= max(1, e // 3)
    if kind == "bad":
        ids[r.random((t, top_k)) < 0.2] = -1
        ids[r.random((t, top_k)) < 0.2] = e
        ids[r.random((t, top_k)) < 0.05] = -2 ** 31
    return ids


def want(weights, x, ids_, per_pair):
    """(y, off) of one product, or of gate and up, pair by pair's expert; NaN rows
    for ids outside."""
    q, s = x
    e, n = weights[0][0].shape[:2]
    flat = ids_.reshape(-1)
    rows = np.arange(flat.size) if per_pair else np.arange(flat.size) // ids_.shape[1]
    y, off = np.full((flat.size, n), np.nan), np.zeros((flat.size, n))
    for i in np.unique(flat[(flat >= 0) & (flat < e)]):
        at = np.flatnonzero(flat == i)
        v = [ref.product_f64(q[rows[at]], s[rows[at]], w[i], ws[i]) for w, ws in weights]
        y[at], off[at] = v[0] if len(v) == 1 else ref.swiglu_f64(*v)
    return y, off


# t, top_k, experts, n, k, ids
SIZES = [(1, 1, 1, 1, 16, "any"), (1, 8, 128, 768, 256, "any"), (3, 2, 5, 33, 48, "any"), (7, 4, 9, 130, 144, "bad"),
         (17, 8, 8, 65, 1040, "any"), (40, 3, 60, 100, 272, "few"), (33, 2, 4, 257, 208, "one"),
         (64, 8, 16, 128, 384, "bad"), (100, 8, 10, 515, 80, "any"), (160, 8, 8, 64, 640, "any"),
         (300, 4, 6, 96, 1296, "any"), (333, 4, 60, 517, 112, "few"), (512, 8, 9, 31, 128, "bad"), (2, 8, 4, 40, 64, "any"),
         (1000, 1, 3, 129, 96, "any"), (2000, 2, 7, 200, 144, "any"), (3000, 1, 5, 97, 48, "bad")]


@pytest.mark.parametrize("t,top_k,e,n,k,kind", SIZES)
@pytest.mark.parametrize("per_pair", [False, True])
def test_grouped_products(t, top_k, e, n, k, kind, per_pair):
    say("i8 grouped", t, top_k, e, n, k, kind, per_pair)
    r = np.random.default_rng([11, t, top_k, e, n, k])
    w, ws = experts(r, e, n, k)
    I = some_ids(r, t, top_k, e, kind)
    rows = t * top_k if per_pair else t
    q = r.integers(-128, 128, (rows, k)).astype(np.int8)
    s = (r.random(rows) * 0.1).astype(np.float32)
    D = dev(I)
    plan = qmm.moe_route(D, e)
    y = Guarded((t * top_k, n), F32)
    qmm.i8_gemm_grouped(dev(w), dev(ws), dev(q), D, plan, per_pair, a_scales=dev(s), y=y.t)
    torch.cuda.synchronize()
    y.check("y")
    ref.check(f64(y.t), want([(w, ws)], (q, s), I, per_pair), F32, (t, top_k, e, n, k))


@pytest.mark.parametrize("t,top_k,e,n,k,kind", SIZES)
@pytest.mark.parametrize("xt,ht", [(F16, F16), (BF16, BF16), (F32, F32)], ids=ids)
def test_gate_and_up(t, top_k, e, n, k, kind, xt, ht):
    say("i8 swiglu", t, top_k, e, n, k, kind, xt, ht)
    r = np.random.default_rng([12, t, top_k, e, n, k])
    gate, up = experts(r, e, n, k), experts(r, e, n, k)
    I = some_ids(r, t, top_k, e, kind)
    x = activations(r, t, k, xt)
    D = dev(I)
    plan = qmm.moe_route(D, e)
    h = Guarded((t * top_k, n), ht)
    ws = qmm.i8_grouped_workspace(x)
    ws.fill_(0xFF)
    qmm.i8_moe_gate_up_swiglu(tuple(map(dev, gate)), tuple(map(dev, up)), x, D, plan, h=h.t, workspace=ws)
    torch.cuda.synchronize()
    h.check("h")
    ref.check(f64(h.t), want([gate, up], ref.rows_f64(f64(x)), I, False), ht, (t, top_k, e, n, k))


@pytest.mark.parametrize("t,top_k,e,n,k,kind", [
    (1, 1, 3, 20, 16, "any"), (1, 8, 128, 200, 2048, "any"), (1, 8, 9, 65, 2064, "any"), (2, 4, 5, 33, 1040, "bad"),
    (4, 2, 2, 100, 272, "one"), (2, 8, 30, 48, 528, "any"), (4, 4, 6, 17, 4112, "few"), (16, 1, 3, 70, 96, "one"),
    (1, 16, 2, 2100, 64, "few"), (1, 2, 4, 16500, 48, "any")])
@pytest.mark.parametrize("xt", [F16, BF16, F32], ids=ids)
def test_few_pairs(t, top_k, e, n, k, kind, xt):
    """Every row of x in every type, rounded in the product and before it."""
    test_gate_and_up(t, top_k, e, n, k, kind, xt, F32)
    say("i8 grouped few", t, top_k, e, n, k, kind, xt)
    r = np.random.default_rng([23, t, top_k, e, n, k])
    w, ws = experts(r, e, n, k)
    I = some_ids(r, t, top_k, e, kind)
    a = activations(r, t * top_k, k, xt)
    D = dev(I)
    y = Guarded((t * top_k, n), F32)
    qmm.i8_gemm_grouped(dev(w), dev(ws), a, D, qmm.moe_route(D, e), True, y=y.t)
    torch.cuda.synchronize()
    y.check("y")
    ref.check(f64(y.t), want([(w, ws)], ref.rows_f64(f64(a)), I, True), F32, (t, top_k, e, n, k))


@pytest.mark.parametrize("shape", [0, 1])
@pytest.mark.parametrize("t,top_k,e,n,k,kind", SIZES)
def test_both_tile_shapes(t, top_k, e, n, k, kind, shape, monkeypatch):
    """A tile may take part of a row tile of the plan, one, or several."""
    monkeypatch.setenv("QMM_I8_MOE_FORCE", str(shape))
    test_grouped_products(t, top_k, e, n, k, kind, True)
    test_gate_and_up(t, top_k, e, n, k, kind, F16, BF16)


@pytest.mark.parametrize("rows", [32, 64, 128, 160])
@pytest.mark.parametrize("shape", [0, 1])
def test_plans_of_every_row_tile(rows, shape, monkeypatch):
    monkeypatch.setenv("QMM_MOE_FORCE", f"{rows},1")
    monkeypatch.setenv("QMM_I8_MOE_FORCE", str(shape))
    for size in [(100, 8, 10, 70, 80, "few"), (900, 2, 6, 30, 48, "bad"), (2, 2, 3, 20, 64, "any")]:
        test_grouped_products(*size, False)


@pytest.mark.parametrize("yt", [F32, F16, BF16], ids=ids)
def test_rows_rounded_in_the_call(yt):
    say("i8 grouped activations", yt)
    r = np.random.default_rng(13)
    for t in (1, 20, 300):
        e, n, k = 6, 100, 1040
        w, ws = experts(r, e, n, k)
        I = some_ids(r, t, 2, e, "any")
        a = activations(r, 2 * t, k, F16)
        D = dev(I)
        plan = qmm.moe_route(D, e)
        y = qmm.i8_gemm_grouped(dev(w), dev(ws), a, D, plan, True, dtype=yt)
        ref.check(f64(y), want([(w, ws)], ref.rows_f64(f64(a)), I, True), yt, t)
        q, s = qmm.i8_quantize(a)
        assert torch.equal(y, qmm.i8_gemm_grouped(dev(w), dev(ws), q, D, plan, True, a_scales=s, dtype=yt))


def test_a_plan_built_for_other_counts_gives_nan():
    say("i8 grouped foreign plan")
    r = np.random.default_rng(14)
    w, ws = experts(r, 4, 70, 64)
    a = activations(r, 30, 64, F16)
    I, J = dev(some_ids(r, 30, 2, 4, "any")), dev(some_ids(r, 31, 2, 4, "any"))
    other = qmm.moe_route(J, 4)
    y = qmm.i8_gemm_grouped(dev(w), dev(ws), a, I, other, False)
    h = qmm.i8_moe_gate_up_swiglu((dev(w), dev(ws)), (dev(w), dev(ws)), a, I, other)
    assert y.isnan().all() and h.isnan().all()


def test_no_tokens():
    w = torch.zeros(4, 8, 64, dtype=torch.int8, device="cuda")
    ws = torch.ones(4, 8, device="cuda")
    I = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    plan = torch.empty(256, dtype=torch.uint8, device="cuda")
    a = torch.zeros(0, 64, dtype=torch.float16, device="cuda")
    assert qmm.i8_gemm_grouped(w, ws, a, I, plan, False).shape == (0, 8)
    assert qmm.i8_moe_gate_up_swiglu((w, ws), (w, ws), a, I, plan).shape == (0, 8)


def test_a_routed_layer_end_to_end():
    """Router logits -> experts -> plan -> gate and up -> down -> weighted sum."""
    say("i8 routed layer")
    r = np.random.default_rng(15)
    for t in (1, 37, 400):
        e, top_k, hidden, inner = 12, 4, 272, 144
        gate, up, down = experts(r, e, inner, hidden), experts(r, e, inner, hidden), experts(r, e, hidden, inner)
        x = activations(r, t, hidden, F16)
        logits = torch.from_numpy(r.standard_normal((t, e)).astype(np.float32)).cuda()
        I, weights = qmm.moe_topk(logits, top_k)
        plan = qmm.moe_route(I, e)
        h = qmm.i8_moe_gate_up_swiglu(tuple(map(dev, gate)), tuple(map(dev, up)), x, I, plan)
        y = qmm.moe_combine(qmm.i8_gemm_grouped(dev(down[0]), dev(down[1]), h, I, plan, True), weights)
        # h is compared above; what follows is compared from the h that was computed
        pairs = want([down], ref.rows_f64(f64(h)), I.cpu().numpy(), True)[0].reshape(t, top_k, hidden)
        ww = f64(weights)[:, :, None]
        bound = (5 + top_k) * 1.1 * ref.HALF * (ww * np.abs(pairs)).sum(axis=1)
        assert np.all(np.abs(f64(y) - (ww * pairs).sum(axis=1)) <= bound + 1e-37)


@pytest.mark.parametrize("t,top_k,e,n,k,kind", SIZES + [(1, 8, 9, 65, 2064, "any"), (2, 8, 30, 48, 528, "bad"), (16, 1, 3, 70, 96, "one")])
def test_gate_and_up_of_given_codes(t, top_k, e, n, k, kind):
    """By the formulas, with codes down to -128, and the bits of the call that rounds x itself."""
    say("i8 swiglu codes", t, top_k, e, n, k, kind)
    r = np.random.default_rng([26, t, top_k, e, n, k])
    gate, up = experts(r, e, n, k), experts(r, e, n, k)
    G, U = tuple(map(dev, gate)), tuple(map(dev, up))
    I = some_ids(r, t, top_k, e, kind)
    D = dev(I)
    plan = qmm.moe_route(D, e)
    q, s = r.integers(-128, 128, (t, k)).astype(np.int8), (r.random(t) * 0.02).astype(np.float32)
    for ht in (F32, F16):
        h = Guarded((t * top_k, n), ht)
        qmm.i8_moe_gate_up_swiglu(G, U, dev(q), D, plan, x_scales=dev(s), h=h.t)
        torch.cuda.synchronize()
        h.check("h")
        ref.check(f64(h.t), want([gate, up], (q, s), I, False), ht, (t, top_k, e, n, k))
    x = activations(r, t, k, BF16)
    codes, scales = qmm.i8_quantize(x)
    a = qmm.i8_moe_gate_up_swiglu(G, U, x, D, plan, dtype=BF16)
    b = qmm.i8_moe_gate_up_swiglu(G, U, codes, D, plan, x_scales=scales, dtype=BF16)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("yt", [F32, F16, BF16], ids=ids)
@pytest.mark.parametrize("t,top_k", [(1, 8), (8, 2), (30, 2), (300, 4)])
def test_a_plan_built_for_other_counts_leaves_nothing_of_the_output(t, top_k, yt):
    """In few rows and in tiles, of one token more, of other pairs a token and of other
    experts: every value becomes NaN, and nothing beside the output changes."""
    say("i8 grouped foreign plans", t, top_k, yt)
    r = np.random.default_rng([27, t, top_k])
    e, n, k = 4, 70, 64
    w, ws = map(dev, experts(r, e, n, k))
    a = activations(r, t, k, F16)
    I = dev(some_ids(r, t, top_k, e, "any"))
    for J, other in ((some_ids(r, t + 1, top_k, e, "any"), e), (some_ids(r, t, top_k + 1, e, "any"), e), (some_ids(r, t, top_k, e, "any"), e + 5)):
        plan = qmm.moe_route(dev(J), other)
        for x, xs in ((a, None), qmm.i8_quantize(a)):
            for per_pair in (False, True):
                rows, scales = x, xs
                if per_pair:
                    rows = x.repeat_interleave(top_k, 0)
                    scales = None if xs is None else xs.repeat_interleave(top_k)
                y = Guarded((t * top_k, n), yt)
                y.t.fill_(1)
                qmm.i8_gemm_grouped(w, ws, rows, I, plan, per_pair, a_scales=scales, y=y.t)
                torch.cuda.synchronize()
                y.check("y")
                assert y.t.isnan().all()
            h = Guarded((t * top_k, n), yt)
            h.t.fill_(1)
            qmm.i8_moe_gate_up_swiglu((w, ws), (w, ws), x, I, plan, x_scales=xs, h=h.t)
            torch.cuda.synchronize()
            h.check("h")
            assert h.t.isnan().all()
