"""Products in 8-bit integers: calls that stand at the edge of what the header
promises.  Results do not depend on how a call runs, so most compare bit by bit."""
import numpy as np
import pytest

import i8_testlib as ref
from qmm_testlib import Guarded, dev, say
from test_gpu_i8_gemm import BF16, F16, F32, activations, f64, ids, weights
from test_gpu_i8_moe import experts, some_ids

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import quantized_matmul_qgemv_amd as qmm  # noqa: E402


# rows, columns, k of a call's problems: every way it can take
WAYS = [(1, [100, 33], 2560), (8, [64], 1024), (12, [300], 512), (64, [512], 8192), (70, [130, 1], 272), (300, [700], 400),
        (1000, [2560], 384)]


def calls(r, m, ns, k, xt=F16):
    x = activations(r, m, k, xt)
    problems = []
    for n in ns:
        w, ws = weights(r, n, k)
        problems.append((dev(w), dev(ws), x, None, None, torch.zeros(m, n, device="cuda")))
    return x, problems


@pytest.mark.parametrize("m,ns,k", WAYS)
def test_captured_and_replayed_with_new_inputs(m, ns, k):
    """Every replay takes the x that is there then; eager calls and
    synchronizations stand between."""
    say("i8 graph", m, ns, k)
    r = np.random.default_rng([30, m])
    x, problems = calls(r, m, ns, k)
    ws = qmm.i8_gemm_workspace(problems)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qmm.i8_gemm_batched(problems, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.i8_gemm_batched(problems, workspace=ws)
    for i in range(4):
        x.copy_(activations(r, m, k, F16))
        for p in problems:
            p[5].fill_(-1)
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        got = [p[5].clone() for p in problems]
        eager = qmm.i8_gemm_batched([p[:5] + (None,) for p in problems])
        for a, b in zip(got, eager):
            assert torch.equal(a, b), (m, i)


@pytest.mark.parametrize("t", [1, 2, 40, 600])
def test_routed_calls_captured_and_replayed(t):
    say("i8 routed graph", t)
    r = np.random.default_rng([31, t])
    e, n, k = 9, 72, 336
    gate, up, down = experts(r, e, n, k), experts(r, e, n, k), experts(r, e, k, n)
    gate, up, down = (tuple(map(dev, p)) for p in (gate, up, down))
    down = (down[0][:, :, :64].contiguous(), down[1])
    x, I = activations(r, t, k, BF16), dev(some_ids(r, t, 4, e, "any"))
    plan = torch.empty(qmm.moe_route_size(t, 4, e), dtype=torch.uint8, device="cuda")
    h = torch.empty(4 * t, n, dtype=F16, device="cuda")
    a = torch.empty(4 * t, 64, dtype=F16, device="cuda")
    y = torch.empty(4 * t, k, device="cuda")
    w1, w2 = qmm.i8_grouped_workspace(x), qmm.i8_grouped_workspace(a)

    def layer():
        qmm.moe_route(I, e, plan=plan)
        qmm.i8_moe_gate_up_swiglu(gate, up, x, I, plan, h=h, workspace=w1)
        a.copy_(h[:, :64])
        qmm.i8_gemm_grouped(*down, a, I, plan, True, y=y, workspace=w2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for _ in range(3):
        x.copy_(activations(r, t, k, BF16))
        I.copy_(dev(some_ids(r, t, 4, e, "any")))
        g.replay()
        torch.cuda.synchronize()
        got = h.clone(), y.clone()
        layer()
        torch.cuda.synchronize()
        assert torch.equal(got[0], h) and torch.equal(got[1], y)


@pytest.mark.parametrize("m,ns,k", WAYS)
def test_two_calls_at_once_on_two_streams(m, ns, k):
    say("i8 two streams", m, ns, k)
    r = np.random.default_rng([32, m])
    sets = [calls(r, m, ns, k)[1] for _ in range(2)]
    want = [qmm.i8_gemm_batched([p[:5] + (None,) for p in ps]) for ps in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [qmm.i8_gemm_workspace(ps) for ps in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for ps, st, ws in zip(sets, streams, spaces):
            qmm.i8_gemm_batched(ps, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for ps, ys in zip(sets, want):
        for p, y in zip(ps, ys):
            assert torch.equal(p[5], y)


def test_what_a_call_allocates_is_its_streams_own():
    say("i8 own memory")
    r = np.random.default_rng(33)
    x, problems = calls(r, 200, [300], 1040)
    want = qmm.i8_gemm(*problems[0][:3])
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs.append(qmm.i8_gemm(*problems[0][:3], stream=st))  # y and workspace of the side stream
        torch.full((1 << 16,), 7, dtype=torch.int32, device="cuda")  # the current stream's allocations beside it
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in outs)


def test_operands_that_are_not_contiguous_or_elsewhere_are_refused():
    r = np.random.default_rng(34)
    w, ws = weights(r, 64, 64)
    W, WS, x = dev(w), dev(ws), activations(r, 64, 64, F16)
    with pytest.raises(ValueError, match="w must be contiguous"):
        qmm.i8_gemm(W.t(), WS, x)
    with pytest.raises(ValueError, match="x must be contiguous"):
        qmm.i8_gemm(W, WS, x.t())
    with pytest.raises(TypeError, match="w has dtype"):
        qmm.i8_gemm(W.float(), WS, x)
    with pytest.raises(TypeError, match="y has dtype"):
        qmm.i8_gemm(W, WS, x, y=torch.empty(64, 64, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError, match="w_scales must be a device tensor"):
        qmm.i8_gemm(W, WS.cpu(), x)
    with pytest.raises(qmm.QmmError, match="x_scales belong"):
        qmm.i8_gemm(W, WS, x, WS)
    with pytest.raises(qmm.QmmError, match="k=24"):
        qmm.i8_gemm(W[:, :24].contiguous(), WS, x[:, :24].contiguous())
    with pytest.raises(qmm.QmmError, match="not 16-byte aligned"):
        qmm.i8_gemm(torch.zeros(64 * 64 + 8, dtype=torch.int8, device="cuda")[8:].view(64, 64), WS, x)
    with pytest.raises(qmm.QmmError, match="y overlaps the x"):
        y = torch.zeros(64, 64, device="cuda")
        qmm.i8_gemm(W, WS, y, y=y)
    with pytest.raises(qmm.QmmError, match="count=9"):
        qmm.i8_gemm_batched([(W, WS, x, None, None, None)] * 9)


def test_a_small_workspace_is_refused():
    r = np.random.default_rng(35)
    x, problems = calls(r, 64, [512], 8192)
    ws = qmm.i8_gemm_workspace(problems)
    with pytest.raises(qmm.QmmError, match="needed"):
        qmm.i8_gemm_batched(problems, workspace=ws[:-256])


@pytest.mark.parametrize("m,n,k", [(5, 40, 64), (40, 40, 64), (300, 520, 272)])
def test_rows_behind_the_last_and_columns_beside_stay(m, n, k):
    """Outputs in the middle of larger buffers, of every type, with sums of odd
    widths: nothing around them changes."""
    say("i8 guard", m, n, k)
    r = np.random.default_rng([36, m])
    for d in (0, 1, 3):
        w, ws = weights(r, n + d, k)
        x = activations(r, m, k, F16)
        for yt in (F32, F16, BF16):
            y = Guarded((m, n + d), yt)
            qmm.i8_gemm(dev(w), dev(ws), x, y=y.t)
            torch.cuda.synchronize()
            y.check((m, n + d, yt))


@pytest.mark.parametrize("m", [3, 300])
def test_a_scale_that_is_not_finite_is_its_columns_own(m):
    r = np.random.default_rng([37, m])
    w, ws = weights(r, 90, 128)
    x = activations(r, m, 128, F16)
    clean = qmm.i8_gemm(dev(w), dev(ws), x)
    ws[7], ws[80] = np.nan, np.inf
    y = qmm.i8_gemm(dev(w), dev(ws), x)
    keep = [c for c in range(90) if c not in (7, 80)]
    assert torch.equal(y[:, keep], clean[:, keep]) and y[:, 7].isnan().all() and not y[:, 80].isfinite().any()


# ------------------------------------------------------- offsets past 32 bits

def codes(*shape):
    return torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda")


def exact_rows(x, xs, w, ws, rows):
    """The fp32 results of given rows, by float64 sums (whole numbers) on the CPU."""
    q = x[rows].double().cpu().numpy()
    return ref.product_f64(q, xs[rows].cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy())


def test_more_than_4_gib_of_rows():
    say("i8 long x")
    m, k, n = 530000, 8192, 12
    x, w = codes(m, k), codes(n, k)
    xs, ws = torch.rand(m, device="cuda"), torch.rand(n, device="cuda")
    y = qmm.i8_gemm(w, ws, x, xs)
    rows = torch.tensor([0, 1, 262143, 262144, 262145, 524287, 524288, 524289, m - 2, m - 1], device="cuda")
    ref.check(f64(y[rows]), exact_rows(x, xs, w, ws, rows), F32)
    part = qmm.i8_gemm(w, ws, x[524000:524600].contiguous(), xs[524000:524600].contiguous())
    assert torch.equal(part, y[524000:524600])


@pytest.mark.parametrize("m", [2, 20, 200])
def test_more_than_4_gib_of_weights(m):
    say("i8 long w", m)
    n, k = 530000, 8192
    w, ws = codes(n, k), torch.rand(n, device="cuda")
    x, xs = codes(m, k), torch.rand(m, device="cuda")
    y = qmm.i8_gemm(w, ws, x, xs)
    at = torch.tensor([0, 262144, 524287, 524288, 524289, n - 1], device="cuda")
    ref.check(f64(y[:, at]), ref.product_f64(x.cpu().numpy(), xs.cpu().numpy(), w[at].cpu().numpy(), ws[at].cpu().numpy()), F32)


def test_more_than_2_32_outputs():
    say("i8 long y")
    m, n, k = 1100000, 4000, 16
    x, w = codes(m, k), codes(n, k)
    xs, ws = torch.rand(m, device="cuda"), torch.rand(n, device="cuda")
    y = qmm.i8_gemm(w, ws, x, xs, dtype=BF16)
    rows = torch.tensor([0, 536870, 536871, 1073741, 1073742, m - 1], device="cuda")
    ref.check(f64(y[rows]), exact_rows(x, xs, w, ws, rows), BF16)


def test_rows_and_experts_far_apart():
    """Gathered rows up to 2^32 bytes from the first, weights of experts past it."""
    say("i8 routed far")
    t, k, n, e = 2 ** 32 // 8192 - 1, 8192, 8, 3
    x, xs = codes(t, k), torch.rand(t, device="cuda")
    w, ws = codes(e, n, k), torch.rand(e, n, device="cuda")
    I = torch.randint(0, e, (t, 1), dtype=torch.int32, device="cuda")
    y = qmm.i8_gemm_grouped(w, ws, x, I, qmm.moe_route(I, e), False, a_scales=xs)
    for row in (0, 262143, 262144, t - 2, t - 1):
        i = int(I[row])
        ref.check(f64(y[row:row + 1]), exact_rows(x, xs, w[i], ws[i], [row]), F32, row)
    del x, y
    for t in (2, 50, 400):
        e, n, k = 600, 1024, 7168
        w, ws = codes(e, n, k), torch.rand(e, n, device="cuda")
        x, xs = codes(t, k), torch.rand(t, device="cuda")
        I = torch.randint(e - 20, e, (t, 2), dtype=torch.int32, device="cuda")
        I[0, 0] = 0
        y = qmm.i8_gemm_grouped(w, ws, x, I, qmm.moe_route(I, e), False, a_scales=xs)
        for p in (0, 1, 2 * t - 1):
            i = int(I.view(-1)[p])
            ref.check(f64(y[p:p + 1]), exact_rows(x, xs, w[i], ws[i], [p // 2]), F32, (t, p))
        del w


def test_the_most_rows_that_are_rounded():
    say("i8 most rows")
    m, k = (1 << 24) - 1, 16
    x = torch.randn(m, k, device="cuda", dtype=F16)
    q, s = qmm.i8_quantize(x)
    for a in (0, 1 << 23, m - 1000):
        wq, wsc = ref.rows_f64(f64(x[a:a + 1000]))
        assert np.array_equal(q[a:a + 1000].cpu().numpy(), wq) and np.array_equal(s[a:a + 1000].cpu().numpy(), wsc)
    w, ws = codes(3, k), torch.rand(3, device="cuda")
    y = qmm.i8_gemm(w, ws, x)
    rows = torch.tensor([0, 12345, m - 1], device="cuda")
    ref.check(f64(y[rows]), exact_rows(q, s, w, ws, rows), F32)


# ---------------------------------------------------------- the chain in use

def test_a_layer_in_8_bits_from_weights_to_outputs():
    """Weights rounded at load time, q, k and v and the way back, for one token and
    for a prompt: near the layer in float64 as far as 8 bits go."""
    say("i8 layer")
    r = np.random.default_rng(40)
    hidden, wide, kv = 512, 768, 256
    W = [torch.from_numpy((r.standard_normal((n, hidden)) * 0.02).astype(np.float32)).cuda() for n in (wide, kv, kv)]
    O = torch.from_numpy((r.standard_normal((hidden, wide)) * 0.02).astype(np.float32)).cuda()
    Q = [qmm.i8_quantize(w) for w in W]
    Oq = qmm.i8_quantize(O)
    for m in (1, 50, 700):
        x = activations(r, m, hidden, F16)
        q, k, v = qmm.i8_gemm_batched([(w, s, x, None, None, None) for w, s in Q], dtype=F16)
        y = qmm.i8_gemm(*Oq, q, dtype=F16)
        xd = f64(x)
        for got, w in zip((q, k, v), W):
            want = xd @ f64(w).T
            # each value is off by up to half a code of its row: 1/254 of the row's largest, as
            # noise of 1/sqrt(3) of that; the largest of a row is at most 5 of its rms here
            assert np.linalg.norm(f64(got) - want) <= 2 ** 0.5 * 5 / 254 / 3 ** 0.5 * 1.1 * np.linalg.norm(want)
        ref.check(f64(y), ref.product_f64(*ref.rows_f64(f64(q)), Oq[0].cpu().numpy(), Oq[1].cpu().numpy()), F16, m)
