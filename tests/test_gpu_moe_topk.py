"""Routing to experts against the plain formulas in 64 bits: the choice has to
be equal, number by number; the weights are formed in 64 bits and rounded
once, so they are off by half a step of fp32 (2^-24 of the value), plus the
64-bit arithmetic's own 1e-14 and the half step 2^-150 of subnormals."""
import numpy as np
import pytest

from qmm_testlib import Guarded, dev, host, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import quantized_matmul_qgemv_amd as qmm  # noqa: E402

INF = np.float32(np.inf)


def want(logits, top_k, bias=None, score="softmax", groups=1, group_keep=1, group_top=1, renormalize=True,
         scale=1.0):
    """The formulas, row by row, in float64."""
    t, e = logits.shape
    ids, weights = np.empty((t, top_k), np.int64), np.empty((t, top_k))
    size = e // groups
    for r in range(t):
        z = logits[r].astype(np.float64)
        with np.errstate(all="ignore"):
            if score == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-z))
            elif np.max(z) == -np.inf:
                s = np.zeros(e)
            else:
                s = np.exp(z - np.max(z))
                s = s / np.sum(s)
            c = s if bias is None else s + bias.astype(np.float64)
            by = z if bias is None and (groups == 1 or group_top == 1) else c
            g = np.sort(by.reshape(groups, size), axis=1)[:, size - group_top:].sum(axis=1)
        if np.isnan(s).any() or np.isnan(c).any() or (groups > 1 and np.isnan(g).any()):
            ids[r], weights[r] = np.arange(top_k), np.nan
            continue
        kept = sorted(range(groups), key=lambda i: (-g[i], i))[:group_keep]
        able = [i for i in range(e) if i // size in kept]
        ids[r] = sorted(able, key=lambda i: (-by[i], i))[:top_k]
        w = s[ids[r]]
        if renormalize:
            if score == "softmax" and np.max(z[ids[r]]) > -np.inf:
                w = np.exp(z[ids[r]] - np.max(z[ids[r]]))
            w = w / w.sum() if w.sum() > 0 else np.zeros(top_k)
        weights[r] = w * float(np.float32(scale))
    return ids, weights


def compare(logits, top_k, bias=None, **kw):
    t = len(logits)
    ids, weights = Guarded((t, top_k), torch.int32), Guarded((t, top_k), torch.float32)
    qmm.moe_topk(dev(logits), top_k, bias=None if bias is None else dev(bias), expert_ids=ids.t, weights=weights.t, **kw)
    torch.cuda.synchronize()
    ids.check("expert_ids")
    weights.check("weights")
    wi, ww = want(logits, top_k, bias, **kw)
    gi, gw = host(ids.t), host(weights.t).astype(np.float64)
    assert np.array_equal(gi, wi), f"{np.mean(np.any(gi != wi, axis=1)):.3g} of the rows choose otherwise"
    assert np.array_equal(np.isnan(gw), np.isnan(ww))
    off = np.abs(gw - ww) - (2.0 ** -24 + 1e-14) * np.abs(ww) - 2.0 ** -149
    assert np.all(np.isnan(ww) | (off <= 0)), float(np.nanmax(off))


CASES = [
    (1, 1, 1, {}),
    (1, 128, 8, {}),
    (3, 8, 2, {}),
    (5, 60, 4, dict(renormalize=False)),
    (17, 64, 6, dict(renormalize=False, scale=2.5)),
    (33, 65, 9, dict(score="sigmoid")),
    (64, 256, 8, dict(score="sigmoid", groups=8, group_keep=4, group_top=2, bias=True, scale=2.5)),
    (257, 128, 8, dict(bias=True)),
    (19, 160, 6, dict(groups=8, group_keep=3, renormalize=False, scale=16.0)),
    (19, 160, 6, dict(groups=8, group_keep=3, group_top=2)),
    (7, 1024, 64, dict(score="sigmoid", bias=True)),
    (7, 1024, 64, {}),
    (9, 999, 10, dict(groups=27, group_keep=5, score="sigmoid", group_top=2)),
    (21, 64, 3, dict(groups=64, group_keep=5)),
    (11, 512, 22, dict(score="sigmoid", renormalize=False, bias=True)),
    (13, 384, 8, dict(score="sigmoid", bias=True, scale=2.827)),
    (6, 16, 16, dict(score="sigmoid", groups=2, group_keep=2, group_top=2)),
    (1009, 72, 6, dict(groups=4, group_keep=2, bias=True)),
    # every list length with every number of experts a lane holds, by logit and by score
    (31, 50, 12, {}),
    (31, 50, 12, dict(bias=True)),
    (18, 120, 16, {}),
    (18, 120, 11, dict(score="sigmoid", bias=True)),
    (15, 200, 16, {}),
    (15, 256, 16, dict(bias=True)),
    (15, 300, 12, dict(renormalize=False)),
    (15, 500, 16, dict(score="sigmoid", bias=True)),
    (15, 400, 8, dict(bias=True)),
    (15, 512, 8, dict(groups=16, group_keep=3)),
    (15, 512, 8, dict(groups=2, group_keep=1, group_top=2, score="sigmoid")),
    (4, 513, 8, dict(bias=True)),
    (4, 100, 17, dict(score="sigmoid", bias=True)),
]


@pytest.mark.parametrize("t, e, top_k, kw", CASES, ids=lambda v: str(v).replace(" ", "") if not isinstance(v, dict) else "-".join(f"{k}{x}" for k, x in v.items()) or "plain")
def test_parity(t, e, top_k, kw):
    say("moe_topk", t, e, top_k, kw)
    r = np.random.default_rng([71, t, e, top_k])
    kw = dict(kw)
    bias = (r.standard_normal(e) * 0.1).astype(np.float32) if kw.pop("bias", False) else None
    compare((r.standard_normal((t, e)) * 2).astype(np.float32), top_k, bias, **kw)


@pytest.mark.parametrize("kw", [{}, dict(score="sigmoid"), dict(score="sigmoid", bias=True), dict(bias=True),
                                dict(groups=8, group_keep=3), dict(groups=8, group_keep=3, group_top=2, score="sigmoid"),
                                dict(groups=8, group_keep=3, group_top=2, bias=True)], ids=str)
def test_ties_go_to_the_lower_index(kw):
    say("moe_topk ties", kw)
    r = np.random.default_rng(72)
    kw = dict(kw)
    logits = r.integers(-2, 3, (200, 96)).astype(np.float32)
    logits[logits == 0] *= np.where(r.random(int((logits == 0).sum())) < 0.5, -1, 1)  # zeros of both signs are equal
    bias = (r.integers(0, 2, 96) * 0.25).astype(np.float32) if kw.pop("bias", False) else None
    compare(logits, 7, bias, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_masks_infinities_and_nan(score, biased, groups):
    say("moe_topk masks", score, biased, groups)
    r = np.random.default_rng(73)
    e = 40
    l = (r.standard_normal((24, e)) * 2).astype(np.float32)
    l[0] = -INF                       # every expert switched off
    l[1, 3:] = -INF                   # fewer left than are chosen
    l[2, :37] = -INF
    l[3, ::2] = -INF
    l[4] = np.finfo(np.float32).min   # a mask of the lowest value, everywhere
    l[5, 1:] = np.finfo(np.float32).min
    l[6, 7] = np.nan
    l[7] = np.nan
    l[8, 5] = INF
    l[9, [5, 30]] = INF
    l[10] = 1e4 * r.standard_normal(e)
    l[11] = 3e38
    l[12] = -3e38
    l[13] = 0
    l[14] = np.float32(1e-45) * r.integers(0, 5, e)  # smallest subnormals, apart
    l[15, 9] = -np.float32(0)
    l[16] = -200 - np.arange(e)       # scores below the smallest fp32
    l[17] = 100 + np.arange(e)
    bias = (r.standard_normal(e) * 0.1).astype(np.float32) if biased else None
    for renorm in (True, False):
        for top in ((1,) if groups == 1 else (1, 2)):
            compare(l, 6, bias, score=score, groups=groups, group_keep=max(1, groups - 1), group_top=top, renormalize=renorm)


@pytest.mark.parametrize("groups, top", [(1, 1), (4, 1), (4, 2)])
def test_bias_infinities(groups, top):
    """-inf takes an expert out, +inf forces it in; a group of both has no sum."""
    say("moe_topk bias infinities", groups, top)
    r = np.random.default_rng(74)
    l = r.standard_normal((16, 32)).astype(np.float32)
    b = np.zeros(32, np.float32)
    b[:6] = -INF
    compare(l, 5, b, score="sigmoid", groups=groups, group_keep=max(1, groups - 1), group_top=top)
    b[30] = INF
    compare(l, 5, b, score="sigmoid", groups=groups, group_keep=max(1, groups - 1), group_top=top)
    b[:] = -INF
    compare(l, 5, b, groups=groups, group_keep=max(1, groups - 1), group_top=top)
    b[2] = INF
    compare(l, 5, b, groups=groups, group_keep=max(1, groups - 1), group_top=top)
    b[3] = np.nan
    compare(l, 5, b, groups=groups, group_keep=max(1, groups - 1), group_top=top)


@pytest.mark.parametrize("groups, top", [(1, 1), (4, 2), (8, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_between_neighbours(score, groups, top):
    """Scores closer than fp32 can tell apart: the choice is that of 64 bits."""
    say("moe_topk neighbours", score, groups, top)
    r = np.random.default_rng(75)
    t, e = 96, 64
    l = np.full((t, e), 6.0, np.float32)
    for _ in range(40):
        l = np.where(r.random((t, e)) < 0.5, np.nextafter(l, INF, dtype=np.float32), l)
    compare(l, 8, np.zeros(e, np.float32), score=score, groups=groups, group_keep=max(1, groups // 2), group_top=top)
    # a bias that makes up for the difference of two logits to about fp32's last bit
    l2 = (r.standard_normal((t, e))).astype(np.float32)
    s0 = 1.0 / (1.0 + np.exp(-l2[0].astype(np.float64)))
    b = (0.75 - s0).astype(np.float32)
    l2[1:] = l2[0]
    compare(l2, 8, b, score="sigmoid", groups=groups, group_keep=max(1, groups // 2), group_top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e, top_k, groups, top", [(64, 8, 1, 1), (64, 5, 1, 1), (128, 16, 1, 1), (256, 8, 8, 2), (48, 3, 4, 1),
                                                   (500, 6, 1, 1)])
def test_some_neighbours(score, e, top_k, groups, top):
    """A handful of experts, fewer and more than are chosen, nearer to each
    other than fp32 scores tell apart, the others far; and groups of them."""
    say("moe_topk some neighbours", score, e, top_k, groups, top)
    r = np.random.default_rng([79, e, top_k])
    rows, biases = [], (r.standard_normal(e) * 0.01).astype(np.float32)
    for n in list(range(1, 19)) * 4:
        l = np.clip(r.standard_normal(e), -2, 2) - 4.0
        at = r.permutation(e)[:n]
        high = r.permutation(e)[:max(0, top_k - 1 - n // 2)]
        l[high] = 3 + r.random(len(high))
        l = l.astype(np.float32)
        # in the sum with the bias they meet at one value, apart by a few steps of fp32
        s = 0.4 - biases[at].astype(np.float64) + r.integers(-3, 4, n) * 2.0 ** -26
        l[at] = np.log(s / (1 - s)).astype(np.float32) if score == "sigmoid" else np.float32(2.0) + r.integers(-2, 3, n).astype(np.float32) * np.float32(2.0 ** -22)
        rows.append(l)
    bias = biases if score == "sigmoid" else np.zeros(e, np.float32)
    compare(np.stack(rows), top_k, bias, score=score, groups=groups, group_keep=max(1, groups // 2), group_top=top)
    if groups > 1:  # groups alike but for a step or two of one expert
        part = r.standard_normal(e // groups).astype(np.float32)
        l = np.tile(part, (64, groups)).reshape(64, groups, -1)
        best = int(part.argmax())
        for i in range(64):
            for g in range(groups):
                l[i, g, best] += np.float32(r.integers(-2, 3)) * np.spacing(l[i, g, best])
        compare(l.reshape(64, e), min(top_k, e // groups), np.zeros(e, np.float32), score=score, groups=groups,
                group_keep=max(1, groups // 2), group_top=top)


def test_other_stream_and_repeat():
    say("moe_topk stream")
    r = np.random.default_rng(76)
    l, b = dev(r.standard_normal((300, 256)).astype(np.float32)), dev((r.standard_normal(256) * 0.1).astype(np.float32))
    kw = dict(score="sigmoid", groups=8, group_keep=4, group_top=2)
    first = qmm.moe_topk(l, 8, bias=b, **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    given = qmm.moe_topk(l, 8, bias=b, stream=st, **kw)
    with torch.cuda.stream(st):
        current = qmm.moe_topk(l, 8, bias=b, **kw)
    torch.cuda.synchronize()
    for other in (given, current):
        assert all(torch.equal(x, y) for x, y in zip(first, other))


def test_in_a_graph():
    say("moe_topk graph")
    l = torch.randn(130, 128, device="cuda")
    ids, w = qmm.moe_topk(l, 8)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.moe_topk(l, 8, expert_ids=ids, weights=w)
    for _ in range(3):
        l.copy_(torch.randn(130, 128, device="cuda"))
        eager = qmm.moe_topk(l, 8)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, eager[0]) and torch.equal(w, eager[1])


def test_refusals_on_the_device():
    l = torch.zeros(4, 32, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        qmm.moe_topk(torch.zeros(32, 4, device="cuda").t(), 2)
    with pytest.raises(TypeError, match="dtype"):
        qmm.moe_topk(l.half(), 2)
    with pytest.raises(qmm.QmmError, match="top_k=33"):
        qmm.moe_topk(l, 33)
    ids, w = qmm.moe_topk(torch.zeros(0, 32, device="cuda"), 2)
    assert ids.shape == w.shape == (0, 2)


def test_routed_layer_end_to_end():
    """Logits from the router's product, the choice, the bucketing, the experts'
    products and the weighted sum, against the same chain in 64 bits."""
    say("moe_topk chain")
    import oracle
    import synth
    from qmm_testlib import assert_close, quantized
    t, e, top_k, n, k, bits = 37, 16, 4, 96, 128, 4
    x = synth.draw_act((77, 0), t, k)
    router = synth.draw_weight((77, 1), e, k).astype(np.float16)
    qs = [quantized((77, 2, i), n, k, bits) for i in range(e)]
    words, s, b = (np.stack([q[j] for q in qs]) for j in (2, 3, 4))
    logits = qmm.qgemm(dev(router.view(np.int32)), None, None, dev(x), 16)
    ids, w = qmm.moe_topk(logits, top_k)
    plan = qmm.moe_route(ids, e)
    y = qmm.qgemm_grouped(dev(words), dev(s), dev(b), dev(x), ids, bits, False, plan=plan)
    out = qmm.moe_combine(y, w)
    torch.cuda.synchronize()
    wi, ww = want(host(logits), top_k)
    assert np.array_equal(host(ids), wi)
    pairs = oracle.grouped_f64(words, s, b, x, wi.astype(np.int32), bits, False)
    assert_close(host(out), oracle.moe_combine_f64(pairs, ww), "routed layer")
