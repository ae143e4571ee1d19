"""Rotary positions against the formula in f64, and the frequency tables.

A result is the f64 formula rounded to f32 once: within 2^-24 of the value, a
few f64 steps more (the angle is the same f64 product on both sides; sine and
cosine may differ by a few units of 2^-53, times |u| + |w|).
"""
import numpy as np
import pytest
import torch

import gguf_block_quant_qmm_amd as q
from tests import kv_ref as ref

pytestmark = pytest.mark.gpu
ONE = 2.0 ** -24 * (1 + 2.0 ** -20)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def freqs_of(rot, base=10000.0):
    return (base ** (-2.0 * np.arange(rot // 2) / rot)).astype(np.float32)


def bound(x, want, rot, layout, mscale):
    """2^-24 of the value plus 2^-50 of the pair's size."""
    i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == ref.HALF else (slice(0, rot, 2), slice(1, rot, 2))
    size = np.zeros_like(want)
    size[..., i] = size[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    return ONE * np.abs(want) + 2.0 ** -50 * size * abs(mscale) + 2.0 ** -149


@pytest.mark.parametrize("N,H,D,rot,layout,mscale,pad,far", [
    (1, 32, 128, 128, ref.HALF, 1.0, 0, 8192),
    (1, 1, 64, 64, ref.INTERLEAVED, 1.0, 0, 1),
    (37, 9, 96, 64, ref.INTERLEAVED, 1.2079, 0, 131072),
    (5, 3, 80, 32, ref.HALF, 1.0, 4, 1 << 31),
    (7, 40, 128, 128, ref.HALF, 0.5, 64, 4096),
    (3, 17, 256, 128, ref.HALF, 1.0, 0, 100000),
    (2, 2, 1024, 1024, ref.INTERLEAVED, 1.0, 8, 5000),
    (300, 5, 8, 8, ref.INTERLEAVED, 1.0, 0, 5000),
    (64, 33, 192, 24, ref.HALF, -1.5, 0, 1000),
])
def test_rope_matches_formula(N, H, D, rot, layout, mscale, pad, far):
    r = np.random.default_rng([N, H, D, rot])
    width = H * D + pad
    x = r.standard_normal((N, width)).astype(np.float32)
    pos = r.integers(-(far - 1) if N % 2 else 0, far, N).astype(np.int32)
    f = freqs_of(rot)
    xd = torch.from_numpy(x).cuda()
    y = torch.full((N, H * D), 7.5, device="cuda")
    q.qmm_rope(xd, N, H, D, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(), rot, y, layout=layout,
               mscale=mscale, x_stride=width)
    torch.cuda.synchronize()
    got = y.cpu().numpy().reshape(N, H, D)
    for n in range(N):
        v = x[n, :H * D].reshape(H, D).astype(np.float64)
        want = ref.rotate(v, pos[n], f, rot, layout, mscale)
        assert np.all(np.abs(got[n] - want) <= bound(v, want, rot, layout, mscale)), n
        assert np.array_equal(got[n][:, rot:], x[n, :H * D].reshape(H, D)[:, rot:])
    # in place, strided, on another stream; what lies between the rows stays
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        st.wait_stream(torch.cuda.default_stream())
        q.qmm_rope(xd, N, H, D, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(), rot, xd, layout=layout,
                   mscale=mscale, x_stride=width, y_stride=width)
    st.synchronize()
    assert torch.equal(xd[:, :H * D], y) and np.array_equal(xd[:, H * D:].cpu().numpy(), x[:, H * D:])


@pytest.mark.parametrize("layout", [ref.HALF, ref.INTERLEAVED])
def test_negative_positions_are_the_gradient(layout):
    """y = R x is linear: the gradient of <g, y> is R^T g, the turn by -pos; and
    <g, (R(x + h e) - R(x - h e)) / 2h> for single values says the same."""
    N, H, D, rot = 4, 3, 64, 48
    r = np.random.default_rng(5)
    x, g = (torch.from_numpy(r.standard_normal((N, H * D)).astype(np.float32)).cuda() for _ in range(2))
    pos = torch.tensor([0, 1, 77, 30011], dtype=torch.int32, device="cuda")
    f = torch.from_numpy(freqs_of(rot)).cuda()

    def turn(v, p):
        y = torch.empty_like(v)
        q.qmm_rope(v, N, H, D, p, f, rot, y, layout=layout)
        return y.double()

    grad = turn(g, -pos)
    dot = (turn(x, pos) * g.double()).sum()
    # every product carries three roundings of 2^-24: x's turn, g's turn
    size = (turn(x, pos).abs() * g.double().abs()).sum() + (x.double().abs() * grad.abs()).sum()
    assert abs(dot - (x.double() * grad).sum()) <= 2.0 ** -24 * 1.01 * size
    for at in ((0, 0), (1, 5), (2, 70), (3, 191), (2, 23)):
        e = torch.zeros_like(x)
        e[at] = 1.0
        up, down = turn(x + e, pos), turn(x - e, pos)
        diff = ((up - down) / 2 * g.double())[at[0]].sum()
        # x +- 1 rounds by 2^-24 (|x| + 1) once, each result once more
        tol = 2.0 ** -24 * 1.01 * ((up.abs() + down.abs()) * g.double().abs())[at[0]].sum() + 2.0 ** -22 * (1 + x[at].abs()) * g.abs().max()
        assert abs(diff - grad[at]) <= tol


def test_frequencies():
    def make(rot, base, **kw):
        out = torch.full((rot // 2 + 1,), -1.0, device="cuda")
        kw = {k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v for k, v in kw.items()}
        q.qmm_rope_freqs(rot, base, out, **kw)
        torch.cuda.synchronize()
        assert out[-1].item() == -1.0
        return out[:-1].cpu().numpy().astype(np.float64)

    def near(got, want):
        assert np.all(np.abs(got - want) <= ONE * want)

    for rot, base in ((2, 10.0), (64, 10000.0), (128, 500000.0), (1024, 1e6)):
        i = np.arange(rot // 2)
        plain = base ** (-2.0 * i / rot)
        near(make(rot, base), plain)
        near(make(rot, base, factor=4.0), plain / 4.0)
        extra = (1.0 + np.arange(rot // 2) % 7).astype(np.float32)
        near(make(rot, base, factors=extra), plain / extra)
        for factor, context in ((8.0, 4096.0), (2.0, 131072.0), (16.0, 20.0)):
            r = [rot * np.log(context / (2 * np.pi * b)) / (2 * np.log(base)) for b in (32.0, 1.0)]
            low, high = max(np.floor(r[0]), 0.0), min(np.ceil(r[1]), rot - 1.0)
            g = np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
            near(make(rot, base, factor=factor, context=context), plain * (1 - g) + plain / factor * g)


def test_rope_of_nonfinite_stays_in_its_pair():
    N, H, D, rot = 2, 2, 64, 64
    x = torch.randn(N, H * D, generator=torch.Generator().manual_seed(1)).cuda()
    pos, f = torch.tensor([3, 9], dtype=torch.int32, device="cuda"), torch.from_numpy(freqs_of(rot)).cuda()
    want, bad, y = torch.empty_like(x), x.clone(), torch.empty_like(x)
    q.qmm_rope(x, N, H, D, pos, f, rot, want)
    bad[1, 64 + 5] = float("nan")
    bad[0, 7] = float("inf")
    q.qmm_rope(bad, N, H, D, pos, f, rot, y)
    torch.cuda.synchronize()
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[1, 64 + 5] = hit[1, 64 + 37] = hit[0, 7] = hit[0, 39] = True
    assert torch.equal(y[~hit], want[~hit]) and not torch.isfinite(y[hit]).any()
