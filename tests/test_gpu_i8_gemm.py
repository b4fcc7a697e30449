"""Products in 8-bit integers against their formulas in 64 bits: every type, at
sizes with ragged edges, rows of zeros, infinities and NaN."""
import numpy as np
import pytest

import i8_testlib as ref
from qmm_testlib import Guarded, dev, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import quantized_matmul_qgemv_amd as qmm  # noqa: E402

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
FLOATS = [F32, F16, BF16]
ids = lambda v: str(v).split(".")[-1] if isinstance(v, torch.dtype) else None  # noqa: E731


def f64(t):
    return t.detach().double().cpu().numpy()


def activations(r, m, k, dtype):
    """Rows of very different size, as a device tensor of the type."""
    x = r.standard_normal((m, k)) * np.exp(r.standard_normal((m, 1)))
    return torch.from_numpy(x).to(dtype).cuda()


def weights(r, n, k):
    """Codes over the whole range, -128 among them, and scales."""
    return r.integers(-128, 128, (n, k)).astype(np.int8), (r.random(n) * 1e-3 + 1e-5).astype(np.float32)


# ------------------------------------------------------------------ rounding

@pytest.mark.parametrize("dtype", FLOATS, ids=ids)
@pytest.mark.parametrize("m,k", [(1, 16), (3, 48), (5, 1008), (4, 1024), (7, 1040), (2, 4096), (3, 4112),
                                 (2, 16384), (2, 16400), (1, 131008), (1000, 768), (257, 2560)])
def test_codes_are_those_of_the_exact_quotient(dtype, m, k):
    say("i8 quantize", dtype, m, k)
    r = np.random.default_rng([1, m, k])
    x = activations(r, m, k, dtype)
    codes, scales = Guarded((m, k), torch.int8), Guarded((m,), F32)
    qmm.i8_quantize(x, codes.t, scales.t)
    torch.cuda.synchronize()
    codes.check("codes")
    scales.check("scales")
    q, s = ref.rows_f64(f64(x))
    assert np.array_equal(scales.t.cpu().numpy(), s)
    assert np.array_equal(codes.t.cpu().numpy(), q)


@pytest.mark.parametrize("dtype", FLOATS, ids=ids)
def test_codes_at_and_beside_every_half(dtype):
    """Rows whose scale makes many quotients exact halves, and their neighbours in
    the type: 127 a, (n + 1/2) a and one step to each side."""
    r = np.random.default_rng(2)
    rows = []
    for e in range(-8, 9):
        for a in (1.0, 1.25, 1.0 + 2.0 ** -7, 1.5 - 2.0 ** -6):
            x = torch.tensor([(n + 0.5) * a * 2.0 ** e for n in range(-127, 127)] + [127.0 * a * 2.0 ** e] * 2,
                             dtype=torch.float64).to(dtype)
            bits = torch.int32 if dtype == F32 else torch.int16
            near = torch.cat([(x.view(bits) + d).view(dtype) for d in (-1, 0, 1)])
            near = torch.where(near.abs() > x[-1].abs(), x[-1], near)
            rows.append(torch.cat([near, x[-1:].repeat(768 - near.numel() % 768)])[:768])
    x = torch.stack(rows)[torch.from_numpy(r.permutation(len(rows)))].cuda()
    say("i8 quantize halves", dtype, tuple(x.shape))
    codes, scales = qmm.i8_quantize(x)
    q, s = ref.rows_f64(f64(x))
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), q)


@pytest.mark.parametrize("dtype", FLOATS, ids=ids)
@pytest.mark.parametrize("k", [16, 1040, 4112])
def test_rows_of_zeros_tiny_huge_and_not_finite(dtype, k):
    say("i8 quantize edges", dtype, k)
    big = float(torch.finfo(dtype).max)
    rows = [np.zeros(k)] + [np.full(k, v) for v in (big, -big, 1e-5, 2.0 ** -24)]
    if dtype != F16:
        rows += [np.full(k, v) for v in (2.0 ** -119, 2.0 ** -119 * (1 - 2.0 ** -8), 1e-38, 1e-40)]
    for bad in (np.nan, np.inf, -np.inf):
        for at in (0, k // 2, k - 1):
            x = np.linspace(-1, 1, k)
            x[at] = bad
            rows.append(x)
    x = torch.from_numpy(np.stack(rows)).to(dtype).cuda()
    codes, scales = qmm.i8_quantize(x)
    q, s = ref.rows_f64(f64(x))
    assert np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), q)


@pytest.mark.parametrize("k", [16, 2560])
def test_codes_beside_halves_of_the_smallest_scales(k):
    """Scales in [2^-126, 2^-125) that are an odd multiple of the smallest number, whose
    half is not a number of fp32: the numbers to both sides of 1/2 and 3/2 of it."""
    r = np.random.default_rng(3)
    unit = 2.0 ** -149
    top = np.float32(127.0 * unit * r.integers(8460000, 11100000, 512))
    s = np.float32(top / np.float32(127)).astype(np.float64) / unit
    j = np.floor(s / 2)
    near = [sign * (i * s + a) * unit for i in (0, 1) for a in (j, j + 1) for sign in (1, -1)]
    rows = np.stack(near + [top.astype(np.float64)] * (k - len(near)), axis=1)
    x = torch.from_numpy(rows.astype(np.float32))
    assert np.array_equal(f64(x), rows)
    say("i8 quantize smallest scales", k)
    codes, scales = qmm.i8_quantize(x.cuda())
    q, want = ref.rows_f64(rows)
    assert np.array_equal(scales.cpu().numpy(), want)
    assert np.array_equal(codes.cpu().numpy(), q)


def test_stacked_rows_and_no_rows():
    r = np.random.default_rng(4)
    x = torch.from_numpy(r.standard_normal((3, 5, 64)).astype(np.float32)).cuda()
    codes, scales = qmm.i8_quantize(x)
    q, s = ref.rows_f64(f64(x))
    assert np.array_equal(codes.cpu().numpy(), q) and np.array_equal(scales.cpu().numpy(), s)
    codes, scales = qmm.i8_quantize(x[:0])
    assert codes.shape == (0, 5, 64) and scales.shape == (0, 5)


# ------------------------------------------------------------------ products

SIZES = [(1, 1, 16), (1, 7, 48), (1, 1000, 2560), (2, 33, 64), (3, 64, 112), (4, 129, 128), (5, 31, 144),
         (8, 100, 4112), (15, 65, 240), (16, 256, 1088), (17, 257, 1040), (31, 2, 656), (33, 96, 384),
         (48, 515, 272), (64, 64, 2576), (65, 130, 400), (100, 1001, 208), (128, 128, 1024), (129, 387, 528),
         (200, 1, 4096), (255, 255, 80), (256, 512, 640), (257, 260, 1296), (300, 2049, 96), (513, 770, 352),
         (1030, 129, 176), (1, 40, 131008), (70, 4, 32)]


SHAPES = 7  # tile shapes a product can take


@pytest.mark.parametrize("m,n,k", SIZES)
def test_products_of_codes(m, n, k):
    codes_case(m, n, k)


@pytest.mark.parametrize("shape", range(SHAPES))
@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (65, 330, 112), (129, 387, 528), (257, 260, 1296), (513, 770, 352),
                                   (700, 1300, 272), (300, 2049, 128)])
def test_products_by_every_tile_shape(m, n, k, shape, monkeypatch):
    monkeypatch.setenv("QMM_I8_FORCE", str(shape))
    codes_case(m, n, k)


@pytest.mark.parametrize("splits", [2, 3, 8])
@pytest.mark.parametrize("shape", range(SHAPES))
def test_k_in_parts_gives_the_same_bits(shape, splits, monkeypatch):
    """Several products of a call, of odd and even widths, each k in parts."""
    say("i8 gemm parts", shape, splits)
    r = np.random.default_rng([24, shape, splits])
    for ns in ((100, 36, 260), (33, 130)):
        for yt in FLOATS:
            x = activations(r, 70, 1296, F16)
            monkeypatch.setenv("QMM_I8_FORCE", str(shape))
            monkeypatch.setenv("QMM_I8_SPLITS", str(splits))
            problems, wants = [], []
            for i, n in enumerate(ns):
                w, ws = weights(r, n, 1296)
                b = r.standard_normal(n).astype(np.float32) if i != 1 else None
                problems.append((dev(w), dev(ws), x, None, None if b is None else dev(b), Guarded((70, n), yt)))
                wants.append(ref.product_f64(*ref.rows_f64(f64(x)), w, ws, b))
            given = [p[:5] + (p[5].t,) for p in problems]
            wsp = qmm.i8_gemm_workspace(given)
            assert wsp.numel() >= splits * 70 * sum(ns) * 4
            guarded = Guarded((wsp.numel(),), torch.uint8)
            qmm.i8_gemm_batched(given, workspace=guarded.t)
            torch.cuda.synchronize()
            guarded.check("workspace")
            for p, want in zip(problems, wants):
                p[5].check("y")
                ref.check(f64(p[5].t), want, yt, (shape, splits))
            monkeypatch.setenv("QMM_I8_SPLITS", "1")
            for p, y in zip(problems, qmm.i8_gemm_batched([p[:5] + (None,) for p in problems], dtype=yt)):
                assert torch.equal(y, p[5].t)


@pytest.mark.parametrize("shape", range(SHAPES))
@pytest.mark.parametrize("yt", FLOATS, ids=ids)
def test_outputs_of_every_type_by_every_tile_shape(yt, shape, monkeypatch):
    """Widths that take whole pieces in every type, in some and in none, and a y
    off 16 bytes."""
    monkeypatch.setenv("QMM_I8_FORCE", str(shape))
    say("i8 gemm outputs", yt, shape)
    r = np.random.default_rng([21, shape])
    for n in (328, 332, 333):
        w, ws = weights(r, n, 80)
        b = r.standard_normal(n).astype(np.float32)
        x = activations(r, 270, 80, BF16)
        want = ref.product_f64(*ref.rows_f64(f64(x)), w, ws, b)
        y = Guarded((270, n), yt)
        qmm.i8_gemm(dev(w), dev(ws), x, bias=dev(b), y=y.t)
        off = torch.zeros(270 * n + 1, dtype=yt, device="cuda")
        qmm.i8_gemm(dev(w), dev(ws), x, bias=dev(b), y=off[1:].view(270, n))
        torch.cuda.synchronize()
        y.check(n)
        ref.check(f64(y.t), want, yt, n)
        assert torch.equal(off[1:].view(270, n), y.t) and off[0] == 0


def codes_case(m, n, k):
    say("i8 gemm codes", m, n, k)
    r = np.random.default_rng([5, m, n, k])
    w, ws = weights(r, n, k)
    q = r.integers(-128, 128, (m, k)).astype(np.int8)
    s = (r.random(m) * 0.1).astype(np.float32)
    y = Guarded((m, n), F32)
    qmm.i8_gemm(dev(w), dev(ws), dev(q), dev(s), y=y.t)
    torch.cuda.synchronize()
    y.check("y")
    ref.check(f64(y.t), ref.product_f64(q, s, w, ws), F32, (m, n, k))


@pytest.mark.parametrize("xt,yt", [(F32, F32), (F16, F32), (BF16, BF16), (F16, F16), (F32, BF16), (BF16, F16)], ids=ids)
@pytest.mark.parametrize("m,n,k,bias", [(1, 515, 2560, True), (3, 64, 1040, False), (16, 130, 4112, True),
                                        (40, 1000, 256, True), (130, 257, 1088, False), (300, 384, 768, True)])
def test_products_of_activations(xt, yt, m, n, k, bias):
    say("i8 gemm", xt, yt, m, n, k)
    r = np.random.default_rng([6, m, n, k])
    w, ws = weights(r, n, k)
    b = r.standard_normal(n).astype(np.float32) if bias else None
    x = activations(r, m, k, xt)
    y = Guarded((m, n), yt)
    qmm.i8_gemm(dev(w), dev(ws), x, bias=None if b is None else dev(b), y=y.t)
    torch.cuda.synchronize()
    y.check("y")
    ref.check(f64(y.t), ref.product_f64(*ref.rows_f64(f64(x)), w, ws, b), yt, (m, n, k))


@pytest.mark.parametrize("m", [1, 5, 16, 60, 300])
def test_given_codes_and_codes_formed_in_the_call_agree_bit_by_bit(m):
    say("i8 gemm both ways", m)
    r = np.random.default_rng([7, m])
    w, ws = weights(r, 333, 1040)
    x = activations(r, m, 1040, F16)
    q, s = qmm.i8_quantize(x)
    a = qmm.i8_gemm(dev(w), dev(ws), x)
    b = qmm.i8_gemm(dev(w), dev(ws), q, s)
    assert torch.equal(a, b)
    # and a row alone is the row among others
    assert torch.equal(qmm.i8_gemm(dev(w), dev(ws), x[:1].contiguous()), a[:1])


# (m, n, k): rounded by the product with 8, 4, 2 and 1 waves a row, one batch of k and
# several, k at the limit of what a workgroup rounds and past it; 8, 4 and 2 waves a
# column block; codes in few rows
FEW = [(1, 5, 16), (1, 33, 64), (1, 100, 2576), (1, 40, 16384), (1, 40, 16400), (2, 31, 8192), (2, 31, 8208), (3, 17, 4096),
       (4, 70, 1040), (4, 70, 4112), (5, 16, 2048), (7, 15, 2064), (8, 257, 528), (8, 64, 2048), (9, 65, 512), (12, 100, 336),
       (16, 48, 1296), (1, 16400, 144), (3, 20001, 80), (2, 33001, 272), (16, 16384, 48), (16, 16400, 48), (13, 30, 9728)]


@pytest.mark.parametrize("xt", FLOATS + [torch.int8], ids=ids)
@pytest.mark.parametrize("m,n,k", FEW)
def test_few_rows(m, n, k, xt):
    say("i8 gemm few rows", m, n, k, xt)
    r = np.random.default_rng([22, m, n, k])
    w, ws = weights(r, n, k)
    b = r.standard_normal(n).astype(np.float32)
    y = Guarded((m, n), F32)
    if xt == torch.int8:
        q, s = r.integers(-128, 128, (m, k)).astype(np.int8), (r.random(m) * 0.1).astype(np.float32)
        x, xs = dev(q), dev(s)
    else:
        x, xs = activations(r, m, k, xt), None
        q, s = ref.rows_f64(f64(x))
    qmm.i8_gemm(dev(w), dev(ws), x, xs, bias=dev(b), y=y.t)
    torch.cuda.synchronize()
    y.check("y")
    ref.check(f64(y.t), ref.product_f64(q, s, w, ws, b), F32, (m, n, k))


@pytest.mark.parametrize("m", [1, 7, 33, 300])
def test_largest_sums_are_exact(m):
    """All codes at -128 over the longest k: 128 * 128 * 131008 is below 2^31."""
    say("i8 gemm largest sums", m)
    k, n = 131008, 5
    w = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    x = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    x[:, 1::2] = 127
    x[0] = -128
    one = torch.ones(max(m, n), device="cuda")
    y = qmm.i8_gemm(w, one[:n].contiguous(), x, one[:m].contiguous())
    want = np.full((m, n), -128.0 * (127 - 128) * k / 2)
    want[0] = 128.0 * 128 * k
    assert np.array_equal(f64(y), np.float32(want).astype(np.float64))


def test_rows_that_are_not_finite_stay_their_own():
    say("i8 gemm not finite")
    r = np.random.default_rng(8)
    for m in (3, 40, 300):
        w, ws = weights(r, 70, 208)
        x = activations(r, m, 208, F16)
        clean = qmm.i8_gemm(dev(w), dev(ws), x)
        x[1, 5], x[m - 1, 207] = float("inf"), float("nan")
        y = qmm.i8_gemm(dev(w), dev(ws), x)
        assert y[1].isnan().all() and y[m - 1].isnan().all()
        keep = [i for i in range(m) if i not in (1, m - 1)]
        assert torch.equal(y[keep], clean[keep])


def test_several_products_of_one_call():
    say("i8 gemm batched")
    r = np.random.default_rng(9)
    for m in (1, 20, 200):
        x, x2 = activations(r, m, 1088, BF16), activations(r, m + 3, 96, F32)
        q, s = qmm.i8_quantize(x)
        problems, wants = [], []
        for i, (n, xi, si, yt) in enumerate([(300, x, None, F32), (65, x, None, F16), (1, q, s, BF16), (129, x2, None, F32)]):
            w, ws = weights(r, n, xi.shape[1])
            b = r.standard_normal(n).astype(np.float32) if i % 2 else None
            y = Guarded((xi.shape[0], n), yt)
            problems.append((dev(w), dev(ws), xi, si, None if b is None else dev(b), y))
            wants.append((ref.product_f64(*(ref.rows_f64(f64(xi)) if si is None else (f64(q), f64(s))), w, ws, b), yt))
        given = [p[:5] + (p[5].t,) for p in problems]
        ws_ = qmm.i8_gemm_workspace(given)
        ws_.fill_(0xFF)
        out = qmm.i8_gemm_batched(given, workspace=ws_)
        torch.cuda.synchronize()
        for i, (p, y, (want, yt)) in enumerate(zip(problems, out, wants)):
            p[5].check(i)
            ref.check(f64(y), want, yt, (m, i))


def test_no_rows_and_empty_problems_beside_others():
    r = np.random.default_rng(10)
    w, ws = weights(r, 9, 64)
    x = activations(r, 4, 64, F16)
    assert qmm.i8_gemm(dev(w), dev(ws), x[:0]).shape == (0, 9)
    a, b = qmm.i8_gemm_batched([(dev(w), dev(ws), x[:0], None, None, None), (dev(w), dev(ws), x, None, None, None)])
    assert a.shape == (0, 9) and torch.equal(b, qmm.i8_gemm(dev(w), dev(ws), x))


# (m, n, k), QMM_I8_FORCE, QMM_I8_SPLITS: few rows rounded in the product and before it, as codes,
# tiles with k whole and in parts (widths of 4 and odd ones)
STEPS = [((1, 1001, 2560), None, None), ((8, 260, 1040), None, None), ((12, 300, 528), None, None),
         ((64, 332, 1296), "0", "1"), ((64, 333, 1296), "0", "3"), ((64, 332, 1296), "2", "4"), ((300, 517, 400), "5", "1"),
         ((5, 333, 1296), "1", "1"), ((5, 333, 1296), "1", "2")]


@pytest.mark.parametrize("xt", [F16, torch.int8], ids=ids)
@pytest.mark.parametrize("size,force,splits", STEPS)
def test_every_way_rounds_after_each_scale_and_after_the_bias(size, force, splits, xt, monkeypatch):
    """Bit by bit what fp32 arithmetic gives step by step: the bias is about as large as
    the product, so that a product which is not rounded before the sum shows."""
    say("i8 gemm steps", size, force, splits, xt)
    if force is not None:
        monkeypatch.setenv("QMM_I8_FORCE", force)
        monkeypatch.setenv("QMM_I8_SPLITS", splits)
    m, n, k = size
    r = np.random.default_rng([25, m, n, k])
    w, ws = weights(r, n, k)
    if xt == torch.int8:
        q, s = r.integers(-128, 128, (m, k)).astype(np.int8), (r.random(m) * 0.1).astype(np.float32)
        x, xs = dev(q), dev(s)
    else:
        x, xs = activations(r, m, k, xt), None
        q, s = ref.rows_f64(f64(x))
    sums = q.astype(np.float64) @ w.astype(np.float64).T  # whole numbers
    product = sums.astype(np.float32) * s[:, None] * ws[None, :]
    b = (product[0] * (r.random(n) - 1.5)).astype(np.float32)
    want = product + b[None, :]
    apart = sums.astype(np.float32).astype(np.float64) * s[:, None]
    fused = (apart.astype(np.float32).astype(np.float64) * ws[None, :] + b[None, :]).astype(np.float32)
    assert want.dtype == np.float32 and (fused != want).sum() > want.size / 20  # the inputs tell one from the other
    y = qmm.i8_gemm(dev(w), dev(ws), x, xs, bias=dev(b))
    assert np.array_equal(y.cpu().numpy(), want)
