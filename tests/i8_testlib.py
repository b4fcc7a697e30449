"""The products in 8-bit integers by their formulas in 64 bits, and how far a
result may be off.

A sum of codes is exact.  It is rounded to fp32 and multiplied by two scales,
rounded each time: three half steps of 2^-24 (3.01 with their products); a bias
adds one of the sum's, a 16-bit type half a step of its own (torch.finfo(t).eps / 2,
or, where it is subnormal, half its smallest number; bf16's are fp32's)."""
import numpy as np

HALF = 2.0 ** -24


def rows_f64(x):
    """(codes, scales) of rows x, whose values are exact in float64."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(axis=-1)
    ok = np.isfinite(top)
    s = np.float32(np.where(ok, top, 0) / 127.0)
    s = np.where(np.where(ok, top, 0) < 2.0 ** -119, np.float32(0), s)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.rint(np.where(np.isfinite(x), x, 0) / np.where(s > 0, s, 1).astype(np.float64)[..., None])
    q = np.where((ok & (s > 0))[..., None], q, 0).astype(np.int8)
    return q, np.where(ok, s, np.float32(np.nan)).astype(np.float32)


def half_step(dtype):
    """(relative, absolute) error of the last rounding to a type named by torch."""
    name = str(dtype).split(".")[-1]
    return {"float32": (0.0, 0.0), "float16": (2.0 ** -11, 2.0 ** -25), "bfloat16": (2.0 ** -8, 2.0 ** -134)}[name]


def product_f64(q, s, w, ws, bias=None):
    """(y, the most its fp32 form may be off)."""
    y = (q.astype(np.float64) @ w.astype(np.float64).T) * s.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]
    off = 3.01 * HALF * np.abs(y)
    if bias is not None:
        y = y + bias.astype(np.float64)[None, :]
        off = off + 1.01 * HALF * np.abs(y)
    return y, off


def swiglu_f64(g, u):
    """silu(g) u of two products with what each may be off.  silu(g) = g / (1 + e),
    e = exp(-g): g's own error moves it by up to (1 + |g|) of it relatively, exp in
    fp32 by 2 |g| + 4 half steps, the sum, quotient and product by one each."""
    (g, dg), (u, du) = g, u
    with np.errstate(over="ignore"):
        y = g / (1.0 + np.exp(-g)) * u
    rel = 3.01 * HALF * (1 + np.abs(g)) + HALF * (2 * np.abs(g) + 4 + 3) + 3.01 * HALF
    # below -87 exp(-g) leaves fp32: silu is 0 there, off by less than 2^-118 |u|
    return y, 1.01 * rel * np.abs(y) + np.where(g < -86, 2.0 ** -118 * np.abs(u), 0)


def check(got, want, dtype, what=""):
    """got of `dtype` (as float64) against (y, off)."""
    y, off = want
    rel, least = half_step(dtype)
    got = np.asarray(got, np.float64)
    assert got.shape == y.shape, (what, got.shape, y.shape)
    assert np.array_equal(np.isnan(got), np.isnan(y)), what
    m = ~np.isnan(y)
    # fp16 holds what is below 65520 after fp32's rounding
    if str(dtype).endswith("float16") and not str(dtype).endswith("bfloat16"):
        big = np.abs(y) >= 65519.9
        assert np.all(np.isinf(got[m & big]) | (np.abs(got[m & big]) >= 65504)), what
        m &= ~big
    bound = off + rel * (np.abs(y) + off) + least + 2.0 ** -149
    bad = np.abs(got - y)[m] > bound[m]
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(got - y)[m] / bound[m]).max()))
