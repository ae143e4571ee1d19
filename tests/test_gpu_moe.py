"""qmm_moe_swiglu and qmm_moe_down on the GPU against the f64 oracle.

Tolerances, from the documented bounds.  With S the sum of |w x| of a
projection the f32-class products are within tau = 1e-5 of S.  SwiGLU:
    |out - exact| <= tau (1.1 S_g (|u| + tau S_u) + |silu(g)| S_u) + 4 2^-24 |out|
(|silu'| < 1.1; silu and the product add four f32 roundings).  Down: each
slot's product within tau S, one rounding per multiply-add of the T slots and
the residual: sum_t |w_t| tau S_t + (T + 1) 2^-24 (sum_t |w_t y_t| + |res|).
"""
import numpy as np
import pytest
import torch

import gguf_block_quant_qmm_amd as q
import oracle
from qmm_inputs import GEOMETRY, NAMES, make_blob, make_x, rng_for

pytestmark = pytest.mark.gpu

TAU = 1e-5
DTYPES = sorted(NAMES)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def experts(dt, E, M, K, seed):
    return np.concatenate([make_blob(dt, M, K, rng_for(2100 + seed, e)) for e in range(E)])


def slot_products(dt, blob, E, M, K, ids, rows):
    """(Y64, bound sums) of every slot's product; zeros where the id is no expert."""
    nb = M * (K // GEOMETRY[dt][0]) * GEOMETRY[dt][1]
    y, S = np.zeros((len(ids), M)), np.zeros((len(ids), M))
    for e in range(E):
        at = np.nonzero(ids == e)[0]
        if at.size:
            _, y[at], S[at] = oracle.matmul(dt, blob[e * nb:(e + 1) * nb], M, K, np.ascontiguousarray(rows[at]))
    return y, S


def silu(v):
    return v * np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))


def work_of(n, fill=0xA5):
    return torch.full((n,), fill, dtype=torch.uint8, device="cuda") if n else None


def run_swiglu(dt, E, M, K, N, T, ids, gate, up, X, stream=None):
    out = torch.full((N * T + 1, M), 7.0, device="cuda")
    q.qmm_moe_swiglu(gate, up, dt, E, M, K, N, T, ids, X, out[:N * T], work=work_of(q.moe_swiglu_work_bytes(dt, E, M, K, N, T)),
                     stream=stream)
    torch.cuda.synchronize()
    assert torch.all(out[N * T] == 7.0)
    return out[:N * T]


def check_swiglu(dt, E, M, K, N, T, ids=None, seed=0, X=None, S_of=None):
    g = np.random.default_rng([21, dt, E, M, K, N, T, seed])
    ids = g.integers(0, E, (N, T), dtype=np.int32) if ids is None else np.asarray(ids, np.int32).reshape(N, T)
    G, U = experts(dt, E, M, K, seed), experts(dt, E, M, K, seed + 1)
    X = make_x(N, K, g) if X is None else X
    out = run_swiglu(dt, E, M, K, N, T, dev(ids), dev(G), dev(U), dev(X)).cpu().numpy().astype(np.float64)
    rows = np.repeat(X, T, axis=0)
    gv, Sg = slot_products(dt, G, E, M, K, ids.reshape(-1), rows)
    uv, Su = slot_products(dt, U, E, M, K, ids.reshape(-1), rows)
    want = silu(gv) * uv
    tol = TAU * (1.1 * Sg * (np.abs(uv) + TAU * Su) + np.abs(silu(gv)) * Su) + 4 * 2.0 ** -24 * np.abs(want)
    bad = np.abs(out - want) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.max(np.abs(out - want) / np.maximum(tol, 1e-300)):.3g} of the bound"
    none = (ids.reshape(-1) < 0) | (ids.reshape(-1) >= E)
    assert np.all(out[none] == 0.0)


def check_down(dt, E, M, K, N, T, ids=None, seed=0, residual=True, in_place=False, H=None):
    g = np.random.default_rng([22, dt, E, M, K, N, T, seed])
    ids = g.integers(0, E, (N, T), dtype=np.int32) if ids is None else np.asarray(ids, np.int32).reshape(N, T)
    W = experts(dt, E, M, K, seed)
    H = make_x(N * T, K, g) if H is None else H
    wt = g.standard_normal((N, T)).astype(np.float32)
    none = (ids < 0) | (ids >= E)
    wt[none] = np.nan                              # a skipped slot's weight and row are not looked at
    H = H.copy()
    H[none.reshape(-1)] = np.nan
    R = g.standard_normal((N, M)).astype(np.float32) if residual else None
    Y = torch.full((N + 1, M), 7.0, device="cuda")
    Rd = dev(R)
    if in_place:
        Y[:N] = Rd
        Rd = Y[:N]
    q.qmm_moe_down(dev(W), dt, E, M, K, N, T, dev(ids), dev(wt), dev(H), Y[:N], residual=Rd,
                   work=work_of(q.moe_down_work_bytes(dt, E, M, K, N, T)))
    torch.cuda.synchronize()
    assert torch.all(Y[N] == 7.0)
    y, S = slot_products(dt, W, E, M, K, ids.reshape(-1), np.nan_to_num(H))
    w = np.where(none, 0.0, np.nan_to_num(wt)).astype(np.float64)[:, :, None]
    y, S = y.reshape(N, T, M), S.reshape(N, T, M)
    res = R.astype(np.float64) if residual else 0.0
    want = (w * y).sum(1) + res
    tol = (np.abs(w) * TAU * S).sum(1) + (T + 1) * 2.0 ** -24 * (np.abs(w * y).sum(1) + np.abs(res))
    err = np.abs(Y[:N].cpu().numpy().astype(np.float64) - want)
    assert np.all(err <= tol), f"worst {np.max(err / np.maximum(tol, 1e-300)):.3g} of the bound"


# block counts per row: one, odd, even; more units than a wavefront has lanes
KS = {32: [32, 64, 96, 160, 1024, 2080, 4096, 4160], 256: [256, 512, 768, 1280, 4096, 4352]}


@pytest.mark.parametrize("dt", DTYPES, ids=lambda d: NAMES[d])
@pytest.mark.parametrize("M", [1, 3, 64, 130])
def test_one_token(dt, M):
    for K in KS[GEOMETRY[dt][0]]:
        check_swiglu(dt, 4, M, K, 1, 2)
        check_down(dt, 4, M, K, 1, 2)


@pytest.mark.parametrize("dt", DTYPES, ids=lambda d: NAMES[d])
@pytest.mark.parametrize("N,T,E", [(2, 1, 1), (5, 3, 7), (7, 8, 16), (33, 4, 5), (150, 2, 3), (260, 1, 2)])
def test_batches(dt, N, T, E):
    bs = GEOMETRY[dt][0]
    for K in (bs, 3 * bs, 2 * bs, 512):
        for M in (5, 96):
            check_swiglu(dt, E, M, K, N, T)
            check_down(dt, E, M, K, N, T, residual=M == 96)


@pytest.mark.parametrize("dt", DTYPES, ids=lambda d: NAMES[d])
def test_long_rows(dt):
    for K in (8448, 14336, 16640):
        check_swiglu(dt, 2, 9, K, 1, 2)
        check_down(dt, 2, 9, K, 1, 2)
        check_down(dt, 2, 33, K, 40, 2)
        check_swiglu(dt, 2, 33, K, 40, 2)


def tokens_on_matrix_cores(need, dt, E, M, K, T, start=1):
    """The fewest tokens (from `start`) that run the matrix-core form: the one with a workspace."""
    lo, hi = start - 1, start
    while need(dt, E, M, K, hi, T) == 0:
        lo, hi = hi, 2 * hi
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (lo, mid) if need(dt, E, M, K, mid, T) else (mid, hi)
    return hi


# (E, T, M, K in blocks of 32 or 256): one weight block per row, odd block counts,
# rows that are not a multiple of a fragment or a workgroup, K that the workgroups share
MANY = [(1, 1, 1, 1), (3, 2, 5, 3), (2, 1, 33, 2), (5, 3, 70, 5), (4, 2, 257, 4), (2, 2, 130, 17)]


@pytest.mark.parametrize("dt", DTYPES, ids=lambda d: NAMES[d])
@pytest.mark.parametrize("E,T,M,blocks", MANY)
def test_many_tokens(dt, E, T, M, blocks):
    K = blocks * GEOMETRY[dt][0]
    N = tokens_on_matrix_cores(q.moe_swiglu_work_bytes, dt, E, M, K, T)
    g = np.random.default_rng(N)
    ids = g.integers(-1, E + 1, (N, T), dtype=np.int32)   # some slots without an expert
    check_swiglu(dt, E, M, K, N, T, ids=ids)
    N = tokens_on_matrix_cores(q.moe_down_work_bytes, dt, E, M, K, T)
    check_down(dt, E, M, K, N, T, ids=g.integers(-1, E + 1, (N, T), dtype=np.int32), in_place=M % 2 == 0)
    check_down(dt, E, M, K, N + 1, T, residual=False)


@pytest.mark.parametrize("dt", DTYPES, ids=lambda d: NAMES[d])
def test_few_slots_per_expert_on_matrix_cores(dt):
    """Tiles of 32 slots, most of them partly filled; experts with none, one, 32 and 33 slots."""
    E, T, M, K = 16, 2, 500, 2048
    for need, check in ((q.moe_swiglu_work_bytes, check_swiglu), (q.moe_down_work_bytes, check_down)):
        N = tokens_on_matrix_cores(need, dt, E, M, K, T, start=70)
        ids = np.full(N * T, -1, np.int32)
        ids[:33], ids[33:65], ids[65], ids[66:N * T - 5] = 3, 9, 15, 0
        g = np.random.default_rng(2)
        check(dt, E, M, K, N, T, ids=g.permutation(ids))
        check(dt, E, M, K, N, T)


@pytest.mark.parametrize("dt", DTYPES, ids=lambda d: NAMES[d])
def test_shared_k_on_matrix_cores(dt):
    """Long rows and few of them: workgroups share a row's k-tiles."""
    for M, K in ((300, 14336), (40, 16640)):
        N = tokens_on_matrix_cores(q.moe_swiglu_work_bytes, dt, 2, M, K, 2)
        check_swiglu(dt, 2, M, K, N, 2)
        N = tokens_on_matrix_cores(q.moe_down_work_bytes, dt, 2, M, K, 2)
        check_down(dt, 2, M, K, N, 2)


@pytest.mark.parametrize("E", [65, 200, 1024])
@pytest.mark.parametrize("dt", [q.QMM_Q4_0, q.QMM_Q4_K], ids=lambda d: NAMES[d])
def test_many_experts(dt, E):
    """More experts than a wavefront has lanes, in both forms; the last expert has slots."""
    M, K, T = 40, 256, 8
    for need, check in ((q.moe_swiglu_work_bytes, check_swiglu), (q.moe_down_work_bytes, check_down)):
        for N in (1, 3, tokens_on_matrix_cores(need, dt, E, M, K, T)):
            g = np.random.default_rng([E, N])
            ids = g.integers(0, E, (N, T), dtype=np.int32)
            ids[0, 0], ids[-1, -1] = E - 1, -1
            check(dt, E, M, K, N, T, ids=ids)


@pytest.mark.parametrize("T", [1, 2, 3, 8, 9, 31, 32])
def test_slots_per_token(T):
    for N in (1, 2, 40):
        check_swiglu(q.QMM_Q4_0, 6, 70, 256, N, T)
        check_down(q.QMM_Q6_K, 6, 70, 512, N, T)


@pytest.mark.parametrize("N", [1, 6, 80])
@pytest.mark.parametrize("dt", [q.QMM_Q4_0, q.QMM_Q6_K, q.QMM_Q5_K], ids=lambda d: NAMES[d])
def test_padding_and_uneven_experts(dt, N):
    E, M, K, T = 9, 75, 512, 3
    g = np.random.default_rng(N)
    ids = g.integers(0, E, (N, T), dtype=np.int32)
    ids[0] = -1                                    # a token with no expert at all
    ids[N // 2, 0] = E                             # just outside
    ids[N - 1, T - 1] = np.int32(2 ** 31 - 1)
    ids[N // 3, 1] = np.int32(-2 ** 31)
    for I in (ids, np.full((N, T), -1), np.full((N, T), E - 1), np.zeros((N, T))):  # last: one expert, thrice per token
        check_swiglu(dt, E, M, K, N, T, ids=I)
        check_down(dt, E, M, K, N, T, ids=I)
        check_down(dt, E, M, K, N, T, ids=I, in_place=True)


@pytest.mark.parametrize("dt", DTYPES, ids=lambda d: NAMES[d])
@pytest.mark.parametrize("many", [False, True])
def test_scales_of_activations(dt, many):
    """Rows of very different magnitudes beside each other, and within a row."""
    E, M, K, T = 3, 40, 512, 2
    N = tokens_on_matrix_cores(q.moe_swiglu_work_bytes, dt, E, M, K, T) * 2 if many else 48
    g = np.random.default_rng(5)
    X = make_x(N * T, K, g)
    X *= (10.0 ** g.uniform(-12, 12, (N * T, 1))).astype(np.float32)
    X[:, ::7] *= 1e-3
    X[0, :] = 0.0
    check_down(dt, E, M, K, N, T, H=X)
    check_swiglu(dt, E, M, K, N, T, X=np.ascontiguousarray(X[:N]))


def test_non_finite_rows_stay_in_their_token():
    dt, E, M, K, T = q.QMM_Q4_K, 3, 64, 512, 2
    for N in (4, 64, tokens_on_matrix_cores(q.moe_swiglu_work_bytes, dt, E, M, K, T)):
        g = np.random.default_rng(6)
        ids = g.integers(0, E, (N, T), dtype=np.int32)
        G, U, X = experts(dt, E, M, K, 0), experts(dt, E, M, K, 1), make_x(N, K, g)
        clean = run_swiglu(dt, E, M, K, N, T, dev(ids), dev(G), dev(U), dev(X)).clone()
        X[1, 5], X[2, 9] = np.nan, np.inf
        got = run_swiglu(dt, E, M, K, N, T, dev(ids), dev(G), dev(U), dev(X))
        same = [s for s in range(N * T) if s // T not in (1, 2)]
        assert torch.equal(got[same], clean[same])
        assert torch.all(torch.isnan(got[T:2 * T]))
        assert not torch.any(torch.isfinite(got[2 * T:3 * T]) & (got[2 * T:3 * T] != 0))


@pytest.mark.parametrize("dt", DTYPES, ids=lambda d: NAMES[d])
def test_results_repeat_and_do_not_hang_on_neighbours(dt):
    """Bitwise: run to run, and for a token moved elsewhere among the same tokens."""
    E, M, K, T = 5, 96, 1024, 3
    for N in (70, tokens_on_matrix_cores(q.moe_swiglu_work_bytes, dt, E, M, K, T)):
        g = np.random.default_rng(8)
        ids, X = g.integers(0, E, (N, T), dtype=np.int32), make_x(N, K, g)
        G, U = dev(experts(dt, E, M, K, 0)), dev(experts(dt, E, M, K, 1))
        a = run_swiglu(dt, E, M, K, N, T, dev(ids), G, U, dev(X)).clone()
        b = run_swiglu(dt, E, M, K, N, T, dev(ids), G, U, dev(X)).clone()
        p = g.permutation(N)
        c = run_swiglu(dt, E, M, K, N, T, dev(ids[p]), G, U, dev(X[p]))
        assert torch.equal(a, b)
        assert torch.equal(a.view(N, T, M)[torch.from_numpy(p).cuda()], c.view(N, T, M))


@pytest.mark.parametrize("N", [1, 9, 96, 640])
def test_block_together(N):
    """norm -> router product -> routing -> experts -> sum with the residual ->
    next norm as Q8_0 -> the int8 product, eager on a side stream, then
    captured and replayed on new inputs against eager runs."""
    dt, E, T, K, M = q.QMM_Q4_K, 16, 4, 1024, 512
    g = np.random.default_rng(N)
    Wr = dev(make_blob(q.QMM_Q8_0, E, K, rng_for(2200, 0)))
    G, U = dev(experts(dt, E, M, K, 0)), dev(experts(dt, E, M, K, 1))
    D = dev(experts(q.QMM_Q6_K, E, K, M, 2))
    Wq = dev(make_blob(q.QMM_Q8_0, 64, K, rng_for(2200, 1)))
    w1, w2 = (dev((1 + 0.1 * g.standard_normal(K)).astype(np.float32)) for _ in range(2))
    attn, x0 = dev(make_x(N, K, g)), dev(make_x(N, K, g))
    e = lambda *s, dtype=torch.float32: torch.empty(s, device="cuda", dtype=dtype)
    x1, h, lg, ids, wt = e(N, K), e(N, K), e(N, E), e(N, T, dtype=torch.int32), e(N, T)
    act, x2, sc, qq, y = e(N, T, M), e(N, K), e(N, K // 32), e(N, K, dtype=torch.int8), e(N, 64)
    assert (q.moe_swiglu_work_bytes(dt, E, M, K, N, T) > 0) == (N >= 96)  # both forms
    ws = work_of(q.moe_swiglu_work_bytes(dt, E, M, K, N, T))
    wd = work_of(q.moe_down_work_bytes(q.QMM_Q6_K, E, K, M, N, T))
    outs = (x1, h, lg, ids, wt, act, x2, sc, qq, y)

    def block():
        q.qmm_block_norm(x0, N, K, residual_out=x1, block=attn, w_pre=w1, H=h)
        q.qmm_gemm(Wr, q.QMM_Q8_0, E, K, N, h, lg)
        q.qmm_moe_route(lg, N, E, T, ids, wt)
        q.qmm_moe_swiglu(G, U, dt, E, M, K, N, T, ids, h, act, work=ws)
        q.qmm_moe_down(D, q.QMM_Q6_K, E, K, M, N, T, ids, wt, act, x2, residual=x1, work=wd)
        q.qmm_block_norm(x2, N, K, w_pre=w2, scales=sc, quants=qq)
        q.qmm_gemm_q8act(Wq, q.QMM_Q8_0, 64, K, N, sc, qq, y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    torch.cuda.synchronize()
    # every step against f64 on the step's own inputs
    n64 = lambda t: t.cpu().numpy().astype(np.float64)
    assert np.allclose(n64(x1), n64(x0) + n64(attn), rtol=2.0 ** -23, atol=1e-12)
    want = n64(x1) / np.sqrt((n64(x1) ** 2).mean(1, keepdims=True) + 1e-5) * n64(w1)
    assert np.allclose(n64(h), want, rtol=2.0 ** -23, atol=0)
    order = np.argsort(-n64(lg), axis=1, kind="stable")[:, :T]
    assert np.array_equal(ids.cpu().numpy(), order)
    s = np.exp(np.take_along_axis(n64(lg), order, 1))
    # subnormal weights: the f32 step is 2^-149 whatever the value, half of it the rounding
    assert np.allclose(n64(wt), s / s.sum(1, keepdims=True), rtol=2.0 ** -23, atol=2.0 ** -149)
    idf, rows = ids.cpu().numpy().reshape(-1), np.repeat(h.cpu().numpy(), T, 0)
    gv, Sg = slot_products(dt, G.cpu().numpy(), E, M, K, idf, rows)
    uv, Su = slot_products(dt, U.cpu().numpy(), E, M, K, idf, rows)
    tol = TAU * (1.1 * Sg * (np.abs(uv) + TAU * Su) + np.abs(silu(gv)) * Su) + 4 * 2.0 ** -24 * np.abs(silu(gv) * uv)
    assert np.all(np.abs(n64(act).reshape(N * T, M) - silu(gv) * uv) <= tol)
    yv, S = slot_products(q.QMM_Q6_K, D.cpu().numpy(), E, K, M, idf, act.cpu().numpy().reshape(N * T, M))
    w = n64(wt)[:, :, None]
    want, tol = (w * yv.reshape(N, T, K)).sum(1) + n64(x1), (w * TAU * S.reshape(N, T, K)).sum(1)
    tol += (T + 1) * 2.0 ** -24 * ((w * np.abs(yv.reshape(N, T, K))).sum(1) + np.abs(n64(x1)))
    assert np.all(np.abs(n64(x2) - want) <= tol)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    for i in range(4):
        attn.normal_(), x0.normal_()
        for t in outs:
            t.zero_()
        for t in (ws, wd):
            if t is not None:
                t.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        block()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs)), f"replay {i}"


@pytest.mark.parametrize("many", [False, True])
def test_two_graphs_share_a_workspace_and_two_streams_do_not(many):
    """Two captured calls with one workspace, replayed in turn on new inputs; then
    two calls at once on two streams with a workspace each.  Bitwise against
    calls by themselves."""
    dt, E, M, K, T = q.QMM_Q5_K, 4, 130, 768, 2
    N = tokens_on_matrix_cores(q.moe_down_work_bytes, dt, E, M, K, T) if many else 5
    g = np.random.default_rng(4)
    W = [dev(experts(dt, E, M, K, s)) for s in (0, 1)]
    ids = [dev(g.integers(-1, E, (N, T), dtype=np.int32)) for _ in range(2)]
    wt, H, R = (torch.randn(*s, device="cuda") for s in ((N, T), (N * T, K), (N, M)))
    Y = [torch.empty(N, M, device="cuda") for _ in range(2)]
    n = q.moe_down_work_bytes(dt, E, M, K, N, T)
    assert (n > 0) == many
    shared = work_of(n)
    call = lambda i, out, work: q.qmm_moe_down(W[i], dt, E, M, K, N, T, ids[i], wt, H, out, residual=R, work=work)
    call(0, Y[0], shared)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i, Y[i], shared)
    for rep in range(4):
        H.normal_(), wt.normal_()
        for i in (0, 1):
            graphs[(i + rep) % 2].replay()
        torch.cuda.synchronize()
        for i in range(2):
            alone = torch.empty_like(Y[i])
            call(i, alone, work_of(n))
            torch.cuda.synchronize()
            assert torch.equal(alone, Y[i]), f"replay {rep}, graph {i}"
    streams, works = [torch.cuda.Stream() for _ in range(2)], [work_of(n) for _ in range(2)]
    want = [y.clone() for y in Y]
    torch.cuda.synchronize()
    for rep in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                Y[i].zero_()
                call(i, Y[i], works[i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(Y, want)), f"round {rep}"


def test_long_inputs_run_in_passes():
    """More slots than one pass of the workspace holds (2^22 over T): rows on both sides of a pass's end."""
    dt, E, M, K, T = q.QMM_Q4_0, 2, 3, 32, 2
    N = (1 << 21) + 5
    work = work_of(q.moe_down_work_bytes(dt, E, M, K, N, T))
    assert work is not None and work.numel() < 2 * q.moe_down_work_bytes(dt, E, M, K, 1 << 21, T)
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(-1, E, (N, T), device="cuda", dtype=torch.int32, generator=g)
    H = torch.randn(N * T, K, device="cuda", generator=g)
    wt = torch.randn(N, T, device="cuda", generator=g)
    blob = experts(dt, E, M, K, 0)
    Y = torch.full((N + 1, M), 7.0, device="cuda")
    q.qmm_moe_down(dev(blob), dt, E, M, K, N, T, ids, wt, H, Y[:N], work=work)
    torch.cuda.synchronize()
    assert torch.all(Y[N] == 7.0)
    W = torch.from_numpy(oracle.dequant(dt, blob, E * M, K)).cuda().view(E, M, K)
    for lo, hi in ((0, 500), ((1 << 21) - 300, N)):
        h, i, w = H.view(N, T, K)[lo:hi].double(), ids[lo:hi], wt[lo:hi].double()
        Wi = torch.where((i >= 0)[..., None, None], W[i.clamp(min=0).long()], torch.zeros((), device="cuda", dtype=torch.float64))
        y, S = (Wi * h[:, :, None]).sum(3), (Wi * h[:, :, None]).abs().sum(3)
        want = (w[..., None] * y).sum(1)
        tol = (w.abs()[..., None] * TAU * S).sum(1) + (T + 1) * 2.0 ** -24 * (w[..., None] * y).abs().sum(1)
        assert torch.all((Y[lo:hi].double() - want).abs() <= tol)


def test_long_gate_up_inputs_run_in_passes():
    """The same for gate/up, whose passes write their slots' rows at once."""
    dt, E, M, K, T = q.QMM_Q8_0, 2, 3, 32, 2
    N = (1 << 21) + 5
    work = work_of(q.moe_swiglu_work_bytes(dt, E, M, K, N, T))
    assert work is not None and work.numel() < 2 * q.moe_swiglu_work_bytes(dt, E, M, K, 1 << 21, T)
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(-1, E, (N, T), device="cuda", dtype=torch.int32, generator=g)
    X = torch.randn(N, K, device="cuda", generator=g)
    blobs = [experts(dt, E, M, K, s) for s in (0, 1)]
    out = torch.full((N * T + 1, M), 7.0, device="cuda")
    q.qmm_moe_swiglu(dev(blobs[0]), dev(blobs[1]), dt, E, M, K, N, T, ids, X, out[:N * T], work=work)
    torch.cuda.synchronize()
    assert torch.all(out[N * T] == 7.0)
    W = [torch.from_numpy(oracle.dequant(dt, b, E * M, K)).cuda().view(E, M, K) for b in blobs]
    for lo, hi in ((0, 500), ((1 << 21) - 300, N)):
        i, x = ids[lo:hi], X[lo:hi, None, None].double()
        live = (i >= 0)[..., None, None]
        (gv, Sg), (uv, Su) = (((w * x).sum(3), (w * x).abs().sum(3)) for w in (torch.where(live, w[i.clamp(min=0).long()], 0.0) for w in W))
        want = gv * torch.sigmoid(gv) * uv
        tol = TAU * (1.1 * Sg * (uv.abs() + TAU * Su) + (gv * torch.sigmoid(gv)).abs() * Su) + 4 * 2.0 ** -24 * want.abs()
        got = out[lo * T:hi * T].view(hi - lo, T, M).double()
        assert torch.all((got - want).abs() <= tol)
