"""Low-rank adapters against the plain formula in 64 bits, row by row.

Tolerance.  Both products are sums of exact fp16 products in fp32.  A sum of
k terms is off by k half steps at worst, and the half steps of a sum of
random signs add up like a random walk: sqrt(k) of them, each of a partial sum
that stays within 3 of the final sums' rms.  The split of A x into two fp16
is off by 2^-23 of the row's largest value (at most 4 of its rms here).  So
the relative L2 error of the adapters' part is at most
    3 * 2^-24 * (sqrt(k) + sqrt(2 * rank)) + 4 * 2^-23
and what is added to the base is rounded once more (2^-24 of the sum).
No single element may be off by more than the worst case of the same sums."""
import numpy as np
import pytest

from qmm_testlib import Guarded, dev, host, rel_l2, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import quantized_matmul_qgemv_amd as qmm  # noqa: E402

HALF = 2.0 ** -24


def weights(r, slots, rank, k, n):
    a = (r.standard_normal((slots, rank, k)) / np.sqrt(k)).astype(np.float16)
    b = (r.standard_normal((slots, n, rank)) * 0.1).astype(np.float16)
    return a, b


def want(x, a, b, ids, scales=None, base=None, expert_ids=None, x_row_per_pair=False):
    """(y, the worst case of its error) in float64; rows of bad ids are NaN."""
    top_k = 1 if expert_ids is None else expert_ids.shape[1]
    rows, n = len(ids) * top_k, b.shape[-2]
    k, rank = a.shape[-1], a.shape[-2]
    adapters = a.shape[0]
    y = np.zeros((rows, n)) if base is None else base.astype(np.float64)
    y = y.copy()
    worst = HALF * np.abs(y)
    adapter = np.repeat(np.asarray(ids, np.int64), top_k)
    expert = np.zeros(rows, np.int64) if expert_ids is None else expert_ids.reshape(-1).astype(np.int64)
    experts = 1 if expert_ids is None else a.shape[1]
    bad = (adapter < -1) | (adapter >= adapters) | ((adapter >= 0) & ((expert < 0) | (expert >= experts)))
    y[bad] = np.nan
    slot = np.where(bad | (adapter < 0), -1, adapter * experts + expert)
    A_, B_ = a.reshape(-1, rank, k), b.reshape(-1, n, rank)
    for t in np.unique(slot[slot >= 0]):
        at = np.flatnonzero(slot == t)
        A, B = A_[t].astype(np.float64), B_[t].astype(np.float64)
        xr = x[at if x_row_per_pair else at // top_k].astype(np.float64)
        s = 1.0 if scales is None else float(scales[t // experts])
        v = xr @ A.T
        ev = 2 * HALF * k * (np.abs(xr) @ np.abs(A).T) + 2 * HALF * np.abs(v).max(axis=1, keepdims=True)
        y[at] += s * (v @ B.T)
        worst[at] += abs(s) * ((ev + 2 * HALF * (2 * rank + 2) * np.abs(v)) @ np.abs(B).T) + 2 * HALF * np.abs(y[at])
    return y, worst + 1e-37


def check(got, x, a, b, ids, what="", **kw):
    k, rank = a.shape[-1], a.shape[-2]
    y, worst = want(x, a, b, ids, **kw)
    got = host(got).astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(y)), what
    m = ~np.isnan(y)
    assert np.all(np.abs(got - y)[m] <= worst[m]), (what, float((np.abs(got - y)[m] - worst[m]).max()))
    base = kw.get("base")
    d, g = (y, got) if base is None else (y - base, got - base)
    if np.any(d[m]):
        tol = 3 * HALF * (np.sqrt(k) + np.sqrt(2 * rank)) + 8 * HALF
        if base is not None:  # the sum's own rounding, seen against the adapters' part
            tol += HALF * np.linalg.norm(y[m]) / np.linalg.norm(d[m])
        assert rel_l2(g[m], d[m]) <= tol, (what, rel_l2(g[m], d[m]), tol)


def run(x, a, b, ids, base=None, in_place=False, **kw):
    """One call into a guarded y, with a workspace full of NaN."""
    top_k = 1 if kw.get("expert_ids") is None else kw["expert_ids"].shape[1]
    y = Guarded((len(ids) * top_k, b.shape[-2]), torch.float32)
    B = None if base is None else dev(base)
    if in_place:
        y.t.copy_(B)
        B = y.t
    kw = {k: dev(v) if isinstance(v, np.ndarray) else v for k, v in kw.items()}
    X, A, Bw, I = dev(x), dev(a), dev(b), dev(ids)
    ws = qmm.lora_workspace([(X, A, Bw, B, y.t)], I, kw.get("expert_ids"))
    ws.fill_(0xFF)
    qmm.lora(X, A, Bw, I, base=B, y=y.t, workspace=ws, **kw)
    torch.cuda.synchronize()
    y.check("lora y")
    return y.t


def some_ids(r, t, adapters, kind):
    if kind == "same":
        return np.full(t, adapters - 1, np.int32)
    if kind == "none":
        return np.full(t, -1, np.int32)
    ids = r.integers(0, adapters, t).astype(np.int32)
    if kind == "runs":
        ids.sort()
    if kind == "holes":
        ids[r.random(t) < 0.4] = -1
    if kind == "bad":
        ids[r.random(t) < 0.2] = adapters
        ids[r.random(t) < 0.2] = -2
        ids[r.random(t) < 0.1] = -2 ** 31
        ids[r.random(t) < 0.1] = 2 ** 31 - 1
    return ids


# rows, k, n, rank, adapters, ids
SIZES = [
    (1, 64, 1, 8, 1, "same"),
    (1, 1024, 2048, 16, 8, "mixed"),
    (2, 128, 3, 16, 2, "mixed"),
    (16, 320, 15, 8, 1, "same"),
    (17, 320, 17, 24, 1, "same"),
    (33, 1088, 65, 32, 33, "mixed"),
    (64, 2560, 130, 16, 64, "holes"),
    (65, 192, 68, 40, 5, "bad"),
    (255, 576, 100, 64, 3, "mixed"),
    (256, 64, 64, 128, 300, "mixed"),
    (256, 512, 257, 16, 4, "same"),
    (100, 256, 31, 256, 7, "holes"),
    (50, 128, 48, 16, 4, "none"),
    (257, 64, 1, 8, 1, "same"),
    (257, 128, 5, 8, 300, "mixed"),
    (300, 2048, 260, 16, 5, "runs"),
    (333, 1088, 1001, 24, 7, "holes"),
    (500, 640, 97, 136, 4, "bad"),
    (700, 320, 128, 64, 3, "runs"),
    (513, 128, 64, 256, 2, "mixed"),
    (640, 4160, 64, 32, 2, "same"),
    (4096, 64, 20, 16, 40, "mixed"),
    (4097, 64, 20, 16, 40, "holes"),
    (9000, 128, 24, 8, 4096, "mixed"),
    (6000, 64, 12, 16, 9, "none"),
    # one launch: ranks that are no power of two, two and three rows a tile, its largest numbers of rows
    (7, 320, 100, 40, 4, "mixed"),
    (11, 576, 33, 48, 5, "mixed"),
    (30, 64, 700, 56, 12, "holes"),
    (128, 1600, 1025, 64, 60, "mixed"),
    (512, 192, 130, 16, 9, "bad"),
    (511, 128, 4100, 8, 3, "runs"),
    # A too large for one launch
    (5, 9728, 80, 64, 3, "mixed"),
    (200, 10240, 40, 40, 2, "holes"),
    # sorted, tiles of 2 and of 16
    (1030, 128, 200, 32, 900, "mixed"),
    (700, 192, 65, 64, 700, "holes"),
    (600, 256, 140, 24, 500, "bad"),
    (520, 64, 40, 64, 1000, "mixed"),
    # sorted, tiles of 64: every rank's kernel, k split and not, several turns of columns
    (1100, 1088, 301, 128, 2, "holes"),
    (1500, 704, 600, 64, 3, "runs"),
    (2100, 2048, 1030, 24, 5, "mixed"),
    (1024, 64, 256, 32, 1, "same"),
    (1300, 192, 36, 96, 4, "bad"),
    (17000, 64, 8200, 8, 3, "runs"),
]


@pytest.mark.parametrize("t, k, n, rank, adapters, kind", SIZES)
def test_parity(t, k, n, rank, adapters, kind):
    say("lora", t, k, n, rank, adapters, kind)
    r = np.random.default_rng([81, t, k, n, rank])
    a, b = weights(r, adapters, rank, k, n)
    x = r.standard_normal((t, k)).astype(np.float16)
    ids = some_ids(r, t, adapters, kind)
    base = r.standard_normal((t, n)).astype(np.float32)
    scales = (r.random(adapters) * 3 - 1).astype(np.float32)
    check(run(x, a, b, ids, base=base, scales=scales), x, a, b, ids, "base", base=base, scales=scales)
    check(run(x, a, b, ids, base=base, scales=scales, in_place=True), x, a, b, ids, "in place", base=base, scales=scales)
    check(run(x, a, b, ids), x, a, b, ids, "alone")


@pytest.mark.parametrize("t, top_k, experts, adapters, per_pair", [
    (1, 8, 16, 2, False), (5, 3, 8, 3, True), (32, 8, 128, 2, True), (40, 8, 16, 1, False), (200, 4, 32, 3, True),
    (700, 8, 64, 2, False)])
def test_experts(t, top_k, experts, adapters, per_pair):
    say("lora experts", t, top_k, experts, adapters, per_pair)
    r = np.random.default_rng([82, t, top_k])
    k, n, rank = 128, 52, 16
    a, b = weights(r, adapters * experts, rank, k, n)
    a, b = a.reshape(adapters, experts, rank, k), b.reshape(adapters, experts, n, rank)
    x = r.standard_normal((t * top_k if per_pair else t, k)).astype(np.float16)
    ids = some_ids(r, t, adapters, "holes")
    ex = np.argsort(r.random((t, experts)), axis=1)[:, :top_k].astype(np.int32)
    ex[r.random((t, top_k)) < 0.05] = -1
    ex[r.random((t, top_k)) < 0.05] = experts
    base = r.standard_normal((t * top_k, n)).astype(np.float32)
    scales = (r.random(adapters) + 0.5).astype(np.float32)
    kw = dict(expert_ids=ex, x_row_per_pair=per_pair, scales=scales, base=base)
    check(run(x, a, b, ids, **kw), x, a, b, ids, "experts", **kw)
    flat = run(x, a.reshape(-1, rank, k), b.reshape(-1, n, rank), ids, **kw)
    check(flat, x, a, b, ids, "flattened", **kw)


@pytest.mark.parametrize("t, adapters, last", [
    (40, 6, 128), (600, 6, 128), (1600, 6, 128),  # two products a call: tiles by ballots, sorted tiles of 16 and of 64
    (40, 6, 24), (100, 90, 24), (600, 900, 24), (600, 6, 24),  # one launch: dot products, the same over sorted rows, tiles of 16
])
def test_batched_projections(t, adapters, last):
    """Problems of one call: other inputs, widths and ranks; each as if alone."""
    say("lora batched", t, adapters, last)
    r = np.random.default_rng([83, t, adapters, last])
    ids = some_ids(r, t, adapters, "holes")
    parts = []
    for k, n, rank, with_base in [(320, 200, 16, True), (320, 33, 64, False), (128, 1, 8, True), (704, 64, last, True),
                                  (64, 2100, 8, False)]:
        a, b = weights(r, adapters, rank, k, n)
        x = r.standard_normal((t, k)).astype(np.float16)
        parts.append((x, a, b, r.standard_normal((t, n)).astype(np.float32) if with_base else None))
    I = dev(ids)
    ys = [Guarded((t, p[2].shape[1]), torch.float32) for p in parts]
    qmm.lora_batched([tuple(None if v is None else dev(v) for v in p) + (y.t,) for p, y in zip(parts, ys)], I)
    torch.cuda.synchronize()
    for i, ((x, a, b, base), y) in enumerate(zip(parts, ys)):
        y.check(f"problem {i}")
        check(y.t, x, a, b, ids, f"problem {i}", base=base)


@pytest.mark.parametrize("t", [20, 300])
def test_magnitudes(t):
    """A x from subnormal to 1e13: the split keeps its precision through the
    power of two that each row is scaled by."""
    say("lora magnitudes", t)
    r = np.random.default_rng([84, t])
    k, n, rank = 192, 40, 24
    a, b = weights(r, 3, rank, k, n)
    a = (np.sign(a.astype(np.float32)) * 6e4).astype(np.float16)
    x = r.standard_normal((t, k)).astype(np.float32)
    x = (x * 10.0 ** r.integers(-4, 5, (t, 1))).clip(-65504, 65504).astype(np.float16)
    ids = some_ids(r, t, 3, "mixed")
    for f in (1, 1e-7):
        af = (a.astype(np.float32) * f).astype(np.float16)
        got = host(run(x, af, b, ids)).astype(np.float64)
        y, worst = want(x, af, b, ids)
        assert np.all(np.abs(got - y) <= worst)
        tol = 3 * HALF * (np.sqrt(k) + np.sqrt(2 * rank)) + 8 * HALF
        for p in range(t):
            if np.linalg.norm(y[p]) > 1e-30:
                assert rel_l2(got[p], y[p]) <= 4 * tol, (f, p)  # a single row: 4 times its share


@pytest.mark.parametrize("t", [30, 400])
def test_what_is_not_finite_stays_in_its_row(t):
    say("lora not finite", t)
    r = np.random.default_rng([85, t])
    k, n, rank = 128, 30, 16
    a, b = weights(r, 4, rank, k, n)
    x = r.standard_normal((t, k)).astype(np.float16)
    ids = some_ids(r, t, 3, "mixed")  # slot 3 is not used
    ids[3] = 0
    ids[9] = -1
    a[3], b[3] = np.nan, np.inf
    clean = host(run(x, a, b, ids)).copy()
    x[3, 5], x[9, 7] = np.inf, np.nan
    got = host(run(x, a, b, ids))
    assert not np.isfinite(got[3]).any() and np.array_equal(got[9], np.zeros(n))
    rest = [i for i in range(t) if i != 3]
    assert np.array_equal(got[rest], clean[rest])
    x[3, 5] = np.nan
    assert np.isnan(host(run(x, a, b, ids))[3]).all()


def test_magnitudes_of_single_rows():
    """The same in tiles of one to three rows, subnormal x and A among them."""
    say("lora magnitudes, few rows")
    r = np.random.default_rng(91)
    k, n, rank, t = 576, 50, 16, 6
    a, b = weights(r, 3, rank, k, n)
    for xs, as_ in ((1e-6, 1.0), (1.0, 1e-5), (6e4, 6e4), (1e-7, 6e4)):
        af = np.clip(a.astype(np.float32) * 20 * as_, -65504, 65504).astype(np.float16)
        x = np.clip(r.standard_normal((t, k)) * xs, -65504, 65504).astype(np.float16)
        ids = np.array([0, 1, 1, 2, 2, 2], np.int32)
        check(run(x, af, b, ids), x, af, b, ids, (xs, as_))


def test_a_row_does_not_depend_on_the_others():
    say("lora rows alone")
    r = np.random.default_rng(86)
    k, n, rank = 1088, 70, 16
    a, b = weights(r, 5, rank, k, n)
    x = r.standard_normal((200, k)).astype(np.float16)
    ids = some_ids(r, 200, 5, "holes")
    ids[:6] = [3, 3, 3, 3, 3, 2]
    whole = host(run(x, a, b, ids))
    for p in (0, 1, 99, 199):
        assert np.array_equal(host(run(x[p:p + 1], a, b, ids[p:p + 1]))[0], whole[p])
    back = host(run(x[::-1].copy(), a, b, ids[::-1].copy()))[::-1]
    assert np.array_equal(back, whole)


def test_unaligned_columns():
    """A y and base that start one float into a buffer: the scalar epilogue."""
    say("lora unaligned")
    r = np.random.default_rng(87)
    for t in (30, 300):
        k, n, rank = 128, 64, 16
        a, b = weights(r, 3, rank, k, n)
        x = r.standard_normal((t, k)).astype(np.float16)
        ids = some_ids(r, t, 3, "mixed")
        base = r.standard_normal((t, n)).astype(np.float32)
        buf, bb = torch.empty(t * n + 1, device="cuda"), torch.empty(t * n + 1, device="cuda")
        y, B = buf[1:].view(t, n), bb[1:].view(t, n)
        B.copy_(dev(base))
        qmm.lora(dev(x), dev(a), dev(b), dev(ids), base=B, y=y)
        torch.cuda.synchronize()
        check(y, x, a, b, ids, base=base)


@pytest.mark.parametrize("t", [50, 5000])
def test_streams_graphs_and_repeats(t):
    say("lora graph", t)
    r = np.random.default_rng([88, t])
    k, n, rank = 192, 60, 16
    a, b = weights(r, 7, rank, k, n)
    X, A, B = dev(r.standard_normal((t, k)).astype(np.float16)), dev(a), dev(b)
    I = dev(some_ids(r, t, 7, "holes"))
    first = qmm.lora(X, A, B, I)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    ws = qmm.lora_workspace([(X, A, B, None, None)], I)
    other = torch.empty_like(first)
    st.wait_stream(torch.cuda.current_stream())
    qmm.lora(X, A, B, I, y=other, workspace=ws, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(first, other)
    y = torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.lora(X, A, B, I, y=y, workspace=ws)
    for i in range(3):
        X.copy_(torch.randn_like(X, dtype=torch.float32).half())
        I.copy_(dev(some_ids(r, t, 7, "mixed" if i else "none")))
        eager = qmm.lora(X, A, B, I)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own (given, or made by
    the call), over and over: every result is the one of a call alone."""
    say("lora two streams")
    r = np.random.default_rng(92)
    parts = []
    for t, k, n, rank in ((3000, 512, 640, 32), (2500, 768, 512, 16)):
        a, b = weights(r, 4, rank, k, n)
        parts.append((dev(r.standard_normal((t, k)).astype(np.float16)), dev(a), dev(b), dev(some_ids(r, t, 4, "holes"))))
    alone = [qmm.lora(*p) for p in parts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in parts]
    outs = [[], []]
    for _ in range(5):
        for i, (p, st) in enumerate(zip(parts, streams)):
            outs[i].append(qmm.lora(*p, stream=st))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(o, alone[i]) for o in outs[i])


def test_offsets_past_32_bits():
    """More than 2^31 values of y, and of the adapters' weights."""
    say("lora large offsets")
    t, n, k, rank = 70000, 32768, 64, 8
    gen = torch.Generator(device="cuda")
    gen.manual_seed(89)
    x = torch.randn(t, k, generator=gen, device="cuda").half()
    a = (torch.randn(3, rank, k, generator=gen, device="cuda") / 8).half()
    b = (torch.randn(3, n, rank, generator=gen, device="cuda") * 0.1).half()
    ids = (torch.arange(t, device="cuda") % 4 - 1).to(torch.int32)
    y = torch.ones(t, n, device="cuda")
    qmm.lora(x, a, b, ids, base=y, y=y)
    torch.cuda.synchronize()
    for p in (0, 1, 2, 3, 65535, 65537, 69997, 69998, 69999):
        i = int(ids[p])
        want_ = torch.ones(n, dtype=torch.float64, device="cuda")
        if i >= 0:
            want_ += b[i].double() @ (a[i].double() @ x[p].double())
        assert float((y[p].double() - want_).norm() / want_.norm()) < 1e-6, p
    del y, b
    slots, rank, k, n = 1100, 256, 8192, 64
    a = torch.zeros(slots, rank, k, dtype=torch.float16, device="cuda")
    b = (torch.randn(slots, n, rank, generator=gen, device="cuda") * 0.1).half()
    a[1099] = (torch.randn(rank, k, generator=gen, device="cuda") / 90).half()
    a[3] = (torch.randn(rank, k, generator=gen, device="cuda") / 90).half()
    x = torch.randn(300, k, generator=gen, device="cuda").half()
    for t in (9, 300):
        ids = torch.tensor([1099, 3, 500] * 100, dtype=torch.int32, device="cuda")[:t].contiguous()
        y = qmm.lora(x[:t].contiguous(), a, b, ids)
        torch.cuda.synchronize()
        want_ = torch.stack([b[i].double() @ (a[i].double() @ x[p].double()) for p, i in enumerate(ids.tolist())])
        assert float((y.double() - want_).norm() / want_.norm()) < 3 * HALF * (np.sqrt(k) + np.sqrt(2 * rank)) + 8 * HALF


def test_no_rows():
    z = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    assert qmm.lora(z(0, 64), z(2, 3, 8, 64), z(2, 3, 5, 8), torch.zeros(0, dtype=torch.int32, device="cuda"),
                    expert_ids=torch.zeros(0, 2, dtype=torch.int32, device="cuda")).shape == (0, 5)
    y = qmm.lora(z(0, 64), z(2, 8, 64), z(2, 5, 8), torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert y.shape == (0, 5)


def test_refusals_on_the_device():
    z = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(qmm.QmmError, match="rank=12"):
        qmm.lora(z(4, 64), z(2, 12, 64), z(2, 5, 12), ids)
    with pytest.raises(qmm.QmmError, match="k=96"):
        qmm.lora(z(4, 96), z(2, 8, 96), z(2, 5, 8), ids)
    with pytest.raises(ValueError, match="contiguous"):
        qmm.lora(z(64, 4).t(), z(2, 8, 64), z(2, 5, 8), ids)
    with pytest.raises(TypeError, match="dtype"):
        qmm.lora(z(4, 64).bfloat16(), z(2, 8, 64), z(2, 5, 8), ids)
    with pytest.raises(TypeError, match="dtype"):
        qmm.lora(z(4, 64), z(2, 8, 64), z(2, 5, 8), ids.long())
    with pytest.raises(qmm.QmmError, match="workspace of 16 bytes"):
        qmm.lora(z(4, 64), z(2, 8, 64), z(2, 5, 8), ids, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    big = torch.zeros(4 * 5 + 5, device="cuda")
    with pytest.raises(qmm.QmmError, match="overlaps base"):
        qmm.lora(z(4, 64), z(2, 8, 64), z(2, 5, 8), ids, base=big[5:].view(4, 5), y=big[:20].view(4, 5))


@pytest.mark.parametrize("t", [12, 90])
def test_adapted_routed_layer(t):
    """The parts as they are used: the router's product, the choice of experts,
    the experts' quantized down projection, each request's adapter on it, the
    weighted sum; and a quantized dense projection with adapters in place."""
    say("lora chain", t)
    import oracle
    import synth
    from qmm_testlib import assert_close, quantized
    e, top_k, n, k, bits, adapters, rank = 16, 4, 96, 128, 4, 3, 16
    r = np.random.default_rng([90, t])
    x = synth.draw_act((90, 0), t, k)
    h = synth.draw_act((90, 3), t * top_k, k)
    router = synth.draw_weight((90, 1), e, k).astype(np.float16)
    qs = [quantized((90, 2, i), n, k, bits) for i in range(e)]
    words, s, b = (np.stack([q[j] for q in qs]) for j in (2, 3, 4))
    la, lb = weights(r, adapters * e, rank, k, n)
    la, lb = la.reshape(adapters, e, rank, k), lb.reshape(adapters, e, n, rank)
    ids = some_ids(r, t, adapters, "holes")
    X, H, I = dev(x), dev(h), dev(ids)
    chosen, w = qmm.moe_topk(qmm.qgemm(dev(router.view(np.int32)), None, None, X, 16), top_k)
    plan = qmm.moe_route(chosen, e)
    pairs = qmm.qgemm_grouped(dev(words), dev(s), dev(b), H, chosen, bits, True, plan=plan)
    qmm.lora(H, dev(la), dev(lb), I, base=pairs, y=pairs, expert_ids=chosen, x_row_per_pair=True)
    out = qmm.moe_combine(pairs, w)
    torch.cuda.synchronize()
    ce = host(chosen)
    shared = oracle.grouped_f64(words, s, b, h, ce, bits, True)
    full, _ = want(h, la, lb, ids, base=shared, expert_ids=ce, x_row_per_pair=True)
    assert_close(host(out), oracle.moe_combine_f64(full, host(w).astype(np.float64)), "routed layer with adapters")

    dw = quantized((90, 9), n, k, bits)
    y = qmm.qgemm(dev(dw[2]), dev(dw[3]), dev(dw[4]), X, bits)
    qmm.lora(X, dev(la[:, 0]), dev(lb[:, 0]), I, base=y, y=y)
    torch.cuda.synchronize()
    full, _ = want(x, la[:, 0], lb[:, 0], ids, base=oracle.qmatmul_f64(dw[2], dw[3], dw[4], x, bits))
    assert_close(host(y), full, "dense projection with adapters")
