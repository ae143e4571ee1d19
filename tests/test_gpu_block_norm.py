"""qmm_block_norm on the GPU against f64.

Tolerances: the kernel computes in f64 and rounds every stored value to f32
once, so r and h differ from the f64 formula by at most half an f32 step
(2^-24 of the value) and the f64 sums' own error: 1e-13 of the terms, far
below it; 2^-149 covers half a step of subnormals.  h is compared with the
formula on the r that the kernel stored.  The Q8_0 blocks must be the oracle's
quantization of the stored h, bit for bit.
"""
import numpy as np
import pytest
import torch

import gguf_block_quant_qmm_amd as q
import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def unit(v, w, eps):
    with np.errstate(invalid="ignore"):
        h = v / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return h if w is None else h * w.astype(np.float64)


def close(got, want, terms):
    """got against f64; from 2^128 - 2^103 on the rounding to f32 is infinite, and
    what follows from an infinite r (inf / inf, finite / inf) is NaN or 0."""
    got = got.cpu().numpy().astype(np.float64)
    over = np.abs(want) >= 2.0 ** 128 - 2.0 ** 103
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[over], np.copysign(np.inf, want[over]))
    fine = ~over & ~np.isnan(want)
    got, want, terms = got[fine], want[fine], terms[fine]
    assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) * (1 + 2.0 ** -20) + 1e-13 * terms + 2.0 ** -149)


def check(N, K, post=True, gate="row", pre=True, block=True, h=True, q8=False, scale=0.5, eps=1e-5, seed=0, in_place=False,
          mag=1.0, stream=None):
    g = np.random.default_rng([7, N, K, seed])
    f = lambda *s: (mag * g.standard_normal(s)).astype(np.float32)
    B = f(N, K) if block else None
    R, wp, wn = f(N, K), (1 + 0.1 * f(K)).astype(np.float32) if post else None, f(K) if pre else None
    gt = {"none": None, "row": f(K), "token": f(N, K)}[gate]
    Rd = dev(R)
    guard = torch.full((N + 1, K), 7.0, device="cuda")
    r = Rd if in_place else (torch.full_like(guard, 7.0)[:N] if block else None)
    H = guard[:N] if h else None
    sc = torch.full((N + 1, max(K // 32, 1)), 7.0, device="cuda") if q8 else None
    qq = torch.full((N + 1, K), 7, dtype=torch.int8, device="cuda") if q8 else None
    q.qmm_block_norm(Rd, N, K, residual_out=r, block=dev(B), w_post=dev(wp), gate=dev(gt), gate_stride=K if gate == "token" else 0,
                     scale=scale, w_pre=dev(wn), eps=eps, H=H, scales=sc[:N] if q8 else None, quants=qq[:N] if q8 else None,
                     stream=stream)
    torch.cuda.synchronize()
    want, terms = R.astype(np.float64), np.abs(R.astype(np.float64))
    if block:
        p = unit(B.astype(np.float64), wp, eps) if post else B.astype(np.float64)
        p = scale * p * (1.0 if gt is None else gt.astype(np.float64))
        want, terms = want + p, terms + np.abs(p)
        close(r, want, terms)
        rk = r.cpu().numpy()
    else:
        rk = R
    hk = unit(rk.astype(np.float64), wn, eps)
    if h:
        close(H, hk, np.abs(hk))
        assert torch.all(guard[N] == 7.0)
    if q8:
        assert torch.all(sc[N] == 7.0) and torch.all(qq[N] == 7)
        # the quantizer's bits on the f32 h (from a call that stores it)
        H2 = torch.empty((N, K), device="cuda")
        q.qmm_block_norm(dev(rk), N, K, w_pre=dev(wn), eps=eps, H=H2)
        s_o, q_o = oracle.quantize_q8_0(H2.cpu().numpy())
        assert np.array_equal(sc[:N].cpu().numpy(), s_o) and np.array_equal(qq[:N].cpu().numpy(), q_o)


@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 63, 64, 65, 96, 255, 256, 257, 511, 512, 1000, 1023, 1024, 1025, 1028, 2049,
                               4092, 4096, 4099, 8191, 8196, 16380, 16383, 16384])
@pytest.mark.parametrize("N", [1, 2, 3, 5])
def test_widths(N, K):
    check(N, K)


@pytest.mark.parametrize("K", [16385, 16388, 20000, 32769])
def test_rows_beyond_the_registers(K):
    check(3, K)
    check(2, K, gate="token", in_place=True)
    check(2, K, block=False)


@pytest.mark.parametrize("K", [32, 64, 96, 992, 1024, 1056, 4096, 8224, 16384, 16416, 40000])
def test_q8_blocks(K):
    check(3, K, q8=True)
    check(1, K, q8=True, h=False, gate="none", post=False)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "row", "token"])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("block", [False, True])
def test_forms(post, gate, pre, block):
    for K in (96, 1031, 4096):
        check(6, K, post=post, gate=gate, pre=pre, block=block, q8=K % 32 == 0)
        if block:
            check(6, K, post=post, gate=gate, pre=pre, h=False)      # the residual alone
            check(6, K, post=post, gate=gate, pre=pre, in_place=True)


def test_large_and_small_values():
    check(4, 4096, mag=1e30)     # squares beyond f32, and a gate of 1e30: r itself overflows
    check(4, 4096, mag=1e30, gate="none")
    check(4, 100, mag=1e37, gate="none", post=False)
    check(4, 4096, mag=1e-30, eps=0.0)
    check(4, 257, mag=1e19, q8=False)
    check(300, 4096, seed=3)
    check(64, 4096, seed=5, scale=0.22, q8=True)  # a scale that f32 does not hold
    check(1025, 40, seed=4)


@pytest.mark.parametrize("K", [96, 4096, 20000])
def test_scale_and_norm_beyond_f64_together(K):
    """A scale of 1e300 on a block of 1e-30: scale / norm is beyond f64, the products with the block's zeros are 0."""
    B = np.full((2, K), 1e-30, np.float32)
    B[:, ::3] = 0.0
    R = np.random.default_rng(9).standard_normal((2, K)).astype(np.float32)
    for scale, want in ((1e300, np.where(B == 0.0, R, np.float32(np.inf))), (-1e300, np.where(B == 0.0, R, np.float32(-np.inf)))):
        r = torch.empty((2, K), device="cuda")
        q.qmm_block_norm(dev(R), 2, K, residual_out=r, block=dev(B), w_post=dev(np.ones(K, np.float32)), scale=scale, eps=0.0)
        torch.cuda.synchronize()
        assert np.array_equal(r.cpu().numpy(), want)


def test_zero_rows_and_non_finite_values_stay_in_their_row():
    N, K = 5, 4096
    R = np.random.default_rng(3).standard_normal((N, K)).astype(np.float32)
    R[1] = 0.0
    R[2, 7] = np.nan
    R[3, 9] = np.inf
    H = torch.empty((N, K), device="cuda")
    q.qmm_block_norm(dev(R), N, K, eps=1e-6, H=H)
    torch.cuda.synchronize()
    h = H.cpu().numpy()
    assert np.all(h[1] == 0.0) and np.all(np.isnan(h[2]))
    assert np.isnan(h[3, 9]) and np.all(h[3, :9] == 0.0)  # finite / inf = 0, inf / inf = NaN
    for n in (0, 4):
        close(H[n:n + 1], unit(R[n:n + 1].astype(np.float64), None, 1e-6), np.abs(h[n:n + 1]).astype(np.float64))


def test_stream_and_graph_replays():
    N, K = 33, 4096
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        check(N, K, q8=True)
    B, R, w = (torch.randn(N, K, device="cuda") for _ in range(3))
    w = w[0].contiguous()
    r, H = torch.empty_like(R), torch.empty_like(R)
    call = lambda: q.qmm_block_norm(R, N, K, residual_out=r, block=B, w_post=w, w_pre=w, H=H)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(4):
        B.normal_()
        R.normal_()
        r.zero_(), H.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = (r.clone(), H.clone())
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], r) and torch.equal(got[1], H), f"replay {i}"


def test_more_rows_than_one_launch():
    """2^21 rows go per launch: rows on both sides of the border, against f64 on the GPU."""
    N, K = (1 << 21) + 3, 40
    B, R = torch.randn(N, K, device="cuda"), torch.randn(N, K, device="cuda")
    gt, w = torch.rand(N, K, device="cuda"), torch.rand(K, device="cuda")
    r, H = torch.empty_like(R), torch.empty_like(R)
    q.qmm_block_norm(R, N, K, residual_out=r, block=B, w_post=w, gate=gt, gate_stride=K, scale=0.5, w_pre=w, H=H)
    torch.cuda.synchronize()
    p = B.double()
    p = 0.5 * gt.double() * p / torch.sqrt(p.square().mean(1, keepdim=True) + 1e-5) * w.double()
    want = R.double() + p
    assert torch.all((r.double() - want).abs() <= 2.0 ** -24 * want.abs() * (1 + 2.0 ** -20) + 1e-13 * (R.double().abs() + p.abs()))
    h = r.double()
    h = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-5) * w.double()
    assert torch.all((H.double() - h).abs() <= 2.0 ** -24 * h.abs() * (1 + 2.0 ** -20) + 1e-13 * h.abs())
