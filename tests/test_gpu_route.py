"""moe_ffn_route against its definition in 64 bits (numpy): ids equal, weights within the roundings counted here."""

import math

import numpy as np
import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FLT_MAX = float(np.finfo(np.float32).max)


def reference(logits, k, bias, sigmoid, groups, top_groups, top2, renorm, scale):
    """ids [T, k], weights in 64 bits, and the relative error an fp32 evaluation of each weight may have."""
    l = np.minimum(logits.astype(np.float64), FLT_MAX)
    l[np.isnan(l)] = -np.inf
    T, E = l.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    rel = np.zeros((T, k))
    b = np.zeros(E) if bias is None else np.minimum(bias.astype(np.float64), FLT_MAX)
    for t in range(T):
        live = l[t] > -np.inf
        s = np.zeros(E)
        if live.any():
            if sigmoid:
                with np.errstate(over="ignore"):
                    s[live] = 1.0 / (1.0 + np.exp(-l[t][live]))
            else:
                s[live] = np.exp(l[t][live] - l[t].max())
                s /= s.sum()
        ok = live & ~np.isnan(b) & (b > -np.inf)
        c = np.where(ok, s + np.where(ok, b, 0.0), -np.inf)
        if groups > 1:
            gs = E // groups
            vals = []
            for g in range(groups):
                m = sorted((v for v in c[g * gs:(g + 1) * gs] if v > -np.inf), reverse=True)
                vals.append(-np.inf if not m else sum(m[:2]) if top2 else m[0])
            keep = sorted(range(groups), key=lambda g: (-vals[g], g))[:top_groups]
            for g in range(groups):
                if g not in keep:
                    c[g * gs:(g + 1) * gs] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-c[e], -l[t][e], e)) if c[e] > -np.inf][:k]
        if not order:
            continue
        ids[t, :len(order)] = order
        lo = l[t][order]
        if renorm:
            if sigmoid:
                logs = np.where(lo < -30, lo, -np.log1p(np.exp(np.minimum(-lo, 700.0))))
                z = np.exp(logs - logs.max())
            else:
                z = np.exp(lo - lo.max())
            v = z / z.sum()
            span = lo.max() - lo
        else:
            v = s[order]
            span = np.zeros(len(order)) if sigmoid else l[t].max() - lo
        w[t, :len(order)] = v * scale
        # fp32: the exponent's argument rounds once (span half-ulps of the result), exp, sum, quotient, scale: 16 more
        rel[t, :len(order)] = (np.minimum(span, 200.0) + 16) * 2.0**-24
    return ids, w, rel


def check(logits, k, bias=None, score=fb.SCORE_SOFTMAX, groups=1, top_groups=1, group_score=fb.GROUP_MAX, renorm=True,
          scale=1.0):
    ids, w = fb.moe_ffn_route(logits, k, bias=bias, score=score, groups=groups, top_groups=top_groups,
                              group_score=group_score, renorm=renorm, scale=scale)
    want_ids, want_w, rel = reference(logits.double().cpu().numpy(), k, None if bias is None else bias.cpu().numpy(),
                                      score == fb.SCORE_SIGMOID, groups, top_groups, group_score == fb.GROUP_TOP2,
                                      renorm, scale)
    got = ids.cpu().numpy()
    assert np.array_equal(got, want_ids), np.argwhere(got != want_ids)[:4]
    err = np.abs(w.cpu().numpy().astype(np.float64) - want_w)
    assert (err <= np.abs(want_w) * rel + 2.0**-126).all(), float((err / np.maximum(np.abs(want_w), 1e-30)).max())
    return got, w


def make(T, E, dtype=torch.float32, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, E + pad, generator=g, device="cuda") * 2).to(dtype)[:, :E]


def make_bias(E, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(E, generator=g, device="cuda") * 0.1


@pytest.mark.parametrize("score", [fb.SCORE_SOFTMAX, fb.SCORE_SIGMOID])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,k,groups,top_groups", [
    (1, 1, 1, 1, 1), (1, 128, 8, 1, 1), (3, 5, 5, 1, 1), (33, 33, 7, 1, 1), (130, 256, 8, 8, 4), (17, 200, 6, 8, 3),
    (9, 1024, 32, 1, 1), (5, 1020, 9, 17, 2), (64, 96, 4, 32, 5), (31, 60, 2, 4, 4), (7, 512, 8, 16, 1),
])
def test_shapes(T, E, k, groups, top_groups, dtype, score):
    lg = make(T, E, dtype, seed=T * E)
    for bias in (None, make_bias(E)):
        for gscore in (fb.GROUP_MAX, fb.GROUP_TOP2):
            check(lg, k, bias, score, groups, top_groups, gscore, renorm=gscore == fb.GROUP_MAX, scale=2.5)


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_rows(pad, dtype):
    check(make(41, 128, dtype, 3, pad), 8, make_bias(128), fb.SCORE_SIGMOID, 8, 4, fb.GROUP_TOP2)
    # a view that starts between two 16-byte boundaries
    check(make(12, 131, dtype, 4, pad)[:, 1:130], 3)


@pytest.mark.parametrize("score", [fb.SCORE_SOFTMAX, fb.SCORE_SIGMOID])
@pytest.mark.parametrize("groups", [1, 4])
def test_masks(score, groups):
    lg = make(8, 32, seed=5)
    lg[0] = -math.inf                      # nothing left
    lg[1, 1:] = -math.inf                  # one expert
    lg[2] = torch.finfo(torch.float32).min  # the lowest value is a number, not a mask
    lg[3, ::2] = math.nan
    lg[4, 5] = math.inf
    lg[4, 9] = math.inf
    lg[5] = math.nan
    lg[6, 8:] = -math.inf
    for bias in (None, torch.zeros(32, device="cuda"), make_bias(32)):
        for gscore in (fb.GROUP_MAX, fb.GROUP_TOP2):
            for renorm in (True, False):
                check(lg, 6, bias, score, groups, min(groups, 2), gscore, renorm)
    bias = make_bias(32)
    bias[::3] = -math.inf
    bias[1] = math.nan
    bias[2] = math.inf
    check(lg, 6, bias, score, groups, min(groups, 2))


@pytest.mark.parametrize("score", [fb.SCORE_SOFTMAX, fb.SCORE_SIGMOID])
def test_ties_go_to_the_lower_index(score):
    lg = torch.zeros(4, 64, device="cuda")
    lg[1, 40:] = 1.0
    lg[2] = (torch.arange(64, device="cuda") % 3).float()
    lg[3] = -30.0
    for bias in (None, torch.zeros(64, device="cuda"), torch.full((64,), 0.25, device="cuda")):
        got, _ = check(lg, 8, bias, score)
        assert got[0].tolist() == list(range(8))
        check(lg, 8, bias, score, 8, 3, fb.GROUP_TOP2)


@pytest.mark.parametrize("score", [fb.SCORE_SOFTMAX, fb.SCORE_SIGMOID])
def test_scores_that_fp32_cannot_tell_apart(score):
    """Biases chosen so that c of neighbours differs by far less than an fp32 step of c, either way round."""
    g = torch.Generator().manual_seed(11)
    for seed in range(8):
        l = torch.randn(1, 64, generator=g)
        s = torch.sigmoid(l.double()) if score == fb.SCORE_SIGMOID else torch.softmax(l.double(), 1)
        # the fp32 bias next to 0.75 - s: c is 0.75 to within half a step of the bias for every expert
        bias = (0.75 - s[0]).float()
        check(l.cuda(), 8, bias.cuda(), score)
        check(l.cuda(), 4, bias.cuda(), score, 8, 3, fb.GROUP_TOP2)
        check(l.cuda(), 4, bias.cuda(), score, 8, 3, fb.GROUP_MAX)


def test_far_logits_keep_their_ratios():
    lg = torch.tensor([[-200.0, -201.0, -203.0, -900.0], [90.0, 89.0, 60.0, -5.0], [1e30, 3e30, -1e30, 0.0]],
                      device="cuda")
    for score in (fb.SCORE_SIGMOID, fb.SCORE_SOFTMAX):
        check(lg, 2, None, score)
    _, w = check(lg[:1], 2, None, fb.SCORE_SIGMOID)
    assert abs(float(w[0, 0]) - 1 / (1 + math.exp(-1))) < 1e-6


def test_repeats_and_streams_and_graph():
    lg, bias = make(3000, 256, torch.bfloat16, 9), make_bias(256)
    kw = dict(bias=bias, score=fb.SCORE_SIGMOID, groups=8, top_groups=4, group_score=fb.GROUP_TOP2)
    ids, w = fb.moe_ffn_route(lg, 8, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids2, w2 = fb.moe_ffn_route(lg, 8, stream=side, **kw)
    side.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    ids3, w3 = torch.zeros_like(ids), torch.zeros_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.moe_ffn_route(lg, 8, ids=ids3, weights=w3, **kw)
    lg.copy_(make(3000, 256, torch.bfloat16, 10))
    graph.replay()
    ids, w = fb.moe_ffn_route(lg, 8, **kw)
    torch.cuda.synchronize()
    assert torch.equal(ids, ids3) and torch.equal(w, w3)


def test_no_tokens():
    ids, w = fb.moe_ffn_route(torch.zeros(0, 16, device="cuda"), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


@pytest.mark.parametrize("T,E,k,groups,top_groups,dtype", [
    (6000, 64, 6, 1, 1, torch.float32), (5000, 64, 4, 8, 4, torch.bfloat16), (4000, 50, 8, 1, 1, torch.float16),
])
def test_many_tokens(T, E, k, groups, top_groups, dtype):
    """More tokens than the GPU has warps for at once."""
    lg = make(T, E, dtype, seed=T)
    for score in (fb.SCORE_SOFTMAX, fb.SCORE_SIGMOID):
        check(lg, k, make_bias(E), score, groups, top_groups, fb.GROUP_TOP2)
    check(lg, k, None, fb.SCORE_SOFTMAX, groups, top_groups)


@pytest.mark.parametrize("k", [8, 20, 32])
def test_more_candidates_than_lanes(k):
    """Long runs of scores next to the cut, equal and almost equal."""
    g = torch.Generator(device="cuda").manual_seed(k)
    lg = (torch.randn(6, 256, generator=g, device="cuda") * 1e-7).float()
    lg[1] = 0.5
    lg[2, ::2] = 0.5
    lg[3] = (torch.randn(256, generator=g, device="cuda") * 2).bfloat16().float()
    for bias in (None, torch.zeros(256, device="cuda"), make_bias(256) * 1e-7):
        for score in (fb.SCORE_SOFTMAX, fb.SCORE_SIGMOID):
            check(lg, k, bias, score)
            check(lg, k, bias, score, 8, 4, fb.GROUP_TOP2)
            check(lg, k, bias, score, 4, 2, fb.GROUP_MAX)
