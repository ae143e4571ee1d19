"""qmm_moe_route on the GPU against the definition in Python floats (f64).

The ids must be equal.  The weights are rounded to f32 once from f64 values
that a few f64 operations lead to: half an f32 step (2^-24 of the value) plus
1e-13.
"""
import math

import numpy as np
import pytest
import torch

import gguf_block_quant_qmm_amd as q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def reference(logits, bias, k, scoring, groups, keep, top, renorm, scale):
    N, E = logits.shape
    ids, ws = np.zeros((N, k), np.int32), np.zeros((N, k))
    fmax = float(np.finfo(np.float32).max)
    for n in range(N):
        l = [(-math.inf if math.isnan(v) else min(v, fmax)) for v in logits[n].tolist()]
        if scoring == q.QMM_ROUTE_SIGMOID:
            with np.errstate(over="ignore"):
                s = [float(1.0 / (1.0 + np.exp(np.float64(-v)))) for v in l]
        else:
            m = max(l)
            e = [0.0 if m == -math.inf else math.exp(v - m) for v in l]
            t = math.fsum(e)
            s = [v / t if t > 0 else 0.0 for v in e]
        c = [v + (0.0 if bias is None else float(bias[i])) for i, v in enumerate(s)]
        c = [-math.inf if math.isnan(v) else v for v in c]
        gs = E // groups
        score = []
        for g in range(groups):
            v = sum(sorted(c[g * gs:(g + 1) * gs])[-top:])
            score.append(-math.inf if math.isnan(v) else v)
        open_ = sorted(range(groups), key=lambda g: (-score[g], g))[:keep]
        some = [e for g in open_ for e in range(g * gs, (g + 1) * gs)]
        pick = sorted(some, key=lambda e: (-c[e], e))[:k]
        w = [s[e] for e in pick]
        if renorm:
            t = math.fsum(w)
            w = [v / t if t > 0 else 0.0 for v in w]
        ids[n], ws[n] = pick, [v * scale for v in w]
    return ids, ws


def check(logits, k, bias=None, scoring=q.QMM_ROUTE_SOFTMAX, groups=1, keep=1, top=1, renorm=True, scale=1.0):
    N, E = logits.shape
    ids = torch.full((N + 1, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((N + 1, k), -9.0, device="cuda")
    q.qmm_moe_route(torch.from_numpy(logits).cuda(), N, E, k, ids[:N], w[:N],
                    bias=None if bias is None else torch.from_numpy(bias).cuda(), scoring=scoring, groups=groups,
                    topk_groups=keep, group_top=top, renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    want_i, want_w = reference(logits, bias, k, scoring, groups, keep, top, renorm, scale)
    assert torch.all(ids[N] == -9) and torch.all(w[N] == -9.0)  # rows behind the last token
    assert np.array_equal(ids[:N].cpu().numpy(), want_i)
    got = w[:N].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want_w) <= 2.0 ** -24 * np.abs(want_w) * (1 + 2.0 ** -20) + 1e-13)


def logits_of(N, E, seed):
    return (2.0 * np.random.default_rng([11, N, E, seed]).standard_normal((N, E))).astype(np.float32)


@pytest.mark.parametrize("E", [1, 2, 3, 8, 60, 63, 64, 65, 128, 160, 255, 256, 257, 384, 512, 513, 1000, 1024])
@pytest.mark.parametrize("scoring", [q.QMM_ROUTE_SOFTMAX, q.QMM_ROUTE_SIGMOID])
def test_experts_and_scorings(E, scoring):
    for N in (1, 2, 5, 37):
        for k in sorted({1, min(2, E), min(8, E), min(32, E)}):
            check(logits_of(N, E, k), k, scoring=scoring, renorm=k % 2 == 0, scale=1.0 if k == 1 else 2.5)


@pytest.mark.parametrize("E,groups,keep,top,k", [(256, 8, 4, 2, 8), (256, 8, 4, 1, 8), (64, 8, 1, 2, 8), (160, 8, 3, 1, 6),
                                                 (12, 4, 2, 2, 5), (1024, 16, 5, 2, 32), (1024, 128, 7, 2, 32), (30, 10, 9, 1, 27),
                                                 (8, 8, 3, 1, 3), (72, 8, 8, 2, 9), (1000, 500, 20, 2, 32)])
@pytest.mark.parametrize("scoring", [q.QMM_ROUTE_SOFTMAX, q.QMM_ROUTE_SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
def test_groups_and_bias(E, groups, keep, top, k, scoring, biased):
    bias = (0.1 * np.random.default_rng(E).standard_normal(E)).astype(np.float32) if biased else None
    for N in (1, 33):
        check(logits_of(N, E, 1), k, bias=bias, scoring=scoring, groups=groups, keep=keep, top=top, scale=1.7)


@pytest.mark.parametrize("scoring", [q.QMM_ROUTE_SOFTMAX, q.QMM_ROUTE_SIGMOID])
def test_ties_go_to_the_lower_index(scoring):
    l = np.round(logits_of(40, 130, 2))          # many equal logits
    check(l, 16, scoring=scoring)
    check(np.zeros((3, 64), np.float32), 8, scoring=scoring)
    check(np.zeros((3, 64), np.float32), 8, scoring=scoring, groups=8, keep=2, top=2)
    check(np.round(logits_of(20, 256, 3)), 8, scoring=scoring, groups=8, keep=4, top=2)
    check(l, 16, scoring=scoring, bias=np.where(np.arange(130) % 3, 0.0, 0.25).astype(np.float32))


@pytest.mark.parametrize("scoring", [q.QMM_ROUTE_SOFTMAX, q.QMM_ROUTE_SIGMOID])
def test_masked_experts(scoring):
    l = logits_of(12, 64, 4)
    l[0] = -np.inf                               # nothing left
    l[1] = np.nan
    l[2, 5:] = -np.inf                           # fewer left than chosen
    l[3, ::2] = -np.inf
    l[4, 3] = np.inf
    l[5, 3], l[5, 9] = np.inf, np.inf
    l[6, 7] = np.nan
    l[7] = np.finfo(np.float32).min              # the type's lowest value everywhere
    l[8, :60] = np.finfo(np.float32).min
    l[9] *= 1e30
    for renorm in (False, True):
        check(l, 8, scoring=scoring, renorm=renorm)
        check(l, 8, scoring=scoring, renorm=renorm, groups=8, keep=3, top=2)
        b = np.zeros(64, np.float32)
        b[10:20] = -np.inf                       # experts switched off through the bias
        check(l, 8, scoring=scoring, renorm=renorm, bias=b)
        check(l, 8, scoring=scoring, renorm=renorm, bias=b, groups=4, keep=2, top=2)


def test_large_batch_and_graph_replays():
    check(logits_of(4099, 64, 5), 4)
    N, E, k = 70, 256, 8
    l = torch.randn(N, E, device="cuda")
    b = 0.1 * torch.randn(E, device="cuda")
    ids, w = torch.empty((N, k), dtype=torch.int32, device="cuda"), torch.empty((N, k), device="cuda")
    call = lambda: q.qmm_moe_route(l, N, E, k, ids, w, bias=b, scoring=q.QMM_ROUTE_SIGMOID, groups=8, topk_groups=4, group_top=2)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(4):
        l.normal_()
        ids.zero_(), w.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = (ids.clone(), w.clone())
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], ids) and torch.equal(got[1], w), f"replay {i}"
