"""The attention half of a decoder layer run as a program runs it: norm, the Q/K/V
projection of GGUF weights, head norms and rotation into the cache, attention,
output projection with the residual in the next block norm; a prompt in one
call, then decoded and drafted tokens, two sequences on one set of pages.

Every step is held against f64 on its own inputs (the bounds of include/qmm.h),
and the cache must not depend on how its tokens came in: one prompt call or one
token at a time, the same bytes.
"""
import numpy as np
import pytest
import torch

import gguf_block_quant_qmm_amd as q
import oracle
from qmm_inputs import make_blob, rng_for
from tests import kv_ref as ref

pytestmark = pytest.mark.gpu
HQ, HK, D, KX, PAGE, PAGES, EPS = 4, 2, 64, 256, 16, 16, 1e-5
WIDE = (HQ + 2 * HK) * D


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Layer:
    def __init__(self, kv, wtype=q.QMM_Q8_0):
        r = np.random.default_rng(7)
        self.kv, self.wtype = kv, wtype
        self.wqkv, self.wo = make_blob(wtype, WIDE, KX, rng_for(8, 1)), make_blob(wtype, KX, HQ * D, rng_for(8, 2))
        self.d_wqkv, self.d_wo = dev(self.wqkv), dev(self.wo)
        self.norms = [(1 + 0.1 * r.standard_normal(D)).astype(np.float32) for _ in range(2)]
        self.freqs = torch.empty(D // 2, device="cuda")
        q.qmm_rope_freqs(D, 10000.0, self.freqs, factor=4.0, context=64.0)
        size = q.kv_pool_bytes(kv, PAGES, PAGE, HK, D)
        self.k, self.v = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.cache = q.KvCache(self.k, self.v, kv, PAGES, PAGE, HK, D)
        # two sequences whose pages interleave
        self.table = np.array([[2 * i, 2 * i + 1] for i in range(PAGES // 2)], np.int32).T.copy()

    def step(self, x, lens, new):
        """x [rows][KX] (f32 on the device) of `new` tokens for each sequence, the last of lens."""
        rows = x.shape[0]
        h, qkv = torch.empty_like(x), torch.empty(rows, WIDE, device="cuda")
        qr, o = torch.empty(rows, HQ * D, device="cuda"), torch.empty(rows, HQ * D, device="cuda")
        p, res = torch.empty(rows, KX, device="cuda"), torch.empty(rows, KX, device="cuda")
        batch = q.KvBatch(dev(self.table), dev(np.asarray(lens, np.int32)), len(lens), self.table.shape[1], new, rows)
        q.qmm_block_norm(x, rows, KX, H=h, eps=EPS)
        for n in range(rows):  # the decode product for every row: a token's bits are the same in every batch
            q.qmm_gemv(self.d_wqkv, self.wtype, WIDE, KX, h[n], qkv[n])
        q.qmm_kv_append(self.cache, batch, qkv[:, HQ * D:], qkv[:, (HQ + HK) * D:], freqs=self.freqs, rot=D,
                        layout=q.QMM_ROPE_INTERLEAVED, Q=qkv, q_heads=HQ, q_out=qr, q_norm=dev(self.norms[0]),
                        k_norm=dev(self.norms[1]), eps=EPS, q_stride=WIDE, k_stride=WIDE, v_stride=WIDE)
        work = torch.empty(q.attention_work_bytes(self.cache, batch, HQ), dtype=torch.uint8, device="cuda")
        q.qmm_attention(self.cache, batch, qr, HQ, o, work=work)
        q.qmm_gemm(self.d_wo, self.wtype, KX, HQ * D, rows, o, p)
        q.qmm_block_norm(x, rows, KX, block=p, residual_out=res)
        torch.cuda.synchronize()
        self.check(x, h, qkv, qr, o, p, res, lens, new)
        return o, res

    def check(self, x, h, qkv, qr, o, p, res, lens, new):
        x, h, qkv, qr, o, p, res = (t.cpu().numpy() for t in (x, h, qkv, qr, o, p, res))
        rows, freqs, one = len(x), self.freqs.cpu().numpy(), 2.0 ** -24 * (1 + 2.0 ** -20)
        _, Y, S = oracle.matmul(self.wtype, self.wqkv, WIDE, KX, h)
        assert np.all(np.abs(qkv - Y) <= 1e-5 * S)
        where = ref.places(self.table, lens, None, new, PAGE, PAGES, rows, self.table.shape[1])
        K, V = (ref.decoded(t.cpu().numpy(), self.kv, PAGE, HK, D, val) for t, val in ((self.k, False), (self.v, True)))
        for n, (s, i, _) in enumerate(where):
            y = ref.rotate(ref.unit(qkv[n, :HQ * D].reshape(HQ, D).astype(np.float64), self.norms[0].astype(np.float64), EPS),
                           i, freqs, D, ref.INTERLEAVED)
            assert np.all(np.abs(qr[n].reshape(HQ, D) - y) <= one * np.abs(y) + 2.0 ** -47)
            j = np.arange(i + 1)
            for hq in range(HQ):
                k, v = (a[self.table[s][j // PAGE], hq * HK // HQ, j % PAGE] for a in (K, V))
                qq = qr[n, hq * D:(hq + 1) * D].astype(np.float64)
                want, pr, _ = ref.attend(qq, k, v, D ** -0.5)
                e = D ** -0.5 * (2.0 ** -17 * (np.abs(k) @ np.abs(qq)) + 2.0 ** -36 * np.abs(qq).max() * np.abs(k).sum(1)).max()
                tol = (2 * e + 2.0 ** -17 + len(j) * 2.0 ** -26) * (pr @ np.abs(v) + np.abs(want)) + len(j) * 2.0 ** -32 * np.abs(v).max()
                assert np.all(np.abs(o[n, hq * D:(hq + 1) * D] - want) <= tol)
        _, Y, S = oracle.matmul(self.wtype, self.wo, KX, HQ * D, o)
        assert np.all(np.abs(p - Y) <= q.tolerance(self.wtype, KX, HQ * D, rows) * S)
        want = x.astype(np.float64) + p
        assert np.all(np.abs(res - want) <= one * np.abs(want))


@pytest.mark.parametrize("kv", [q.QMM_F16, q.QMM_Q8_0])
def test_prompt_then_decode_then_drafts(kv):
    r = np.random.default_rng(9)
    n = 37
    x = r.standard_normal((2, n + 1 + 3, KX)).astype(np.float32)
    a = Layer(kv)
    o_prompt, _ = a.step(dev(x[:, :n].reshape(-1, KX)), [n, n], n)      # one call: the form for many rows
    b = Layer(kv)
    for t in range(n):                                                    # one token at a time
        o_one, _ = b.step(dev(x[:, t]), [t + 1, t + 1], 1)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    # the last prompt token of either way: within both bounds of the same exact value
    last = o_prompt.view(2, n, -1)[:, -1]
    assert torch.allclose(last, o_one, rtol=0, atol=1e-4)
    a.step(dev(x[:, n]), [n + 1, n + 1], 1)                               # a decoded token
    a.step(dev(x[:, n + 1:].reshape(-1, KX)), [n + 4, n + 4], 3)          # three drafted ones
    for t in range(n, n + 4):
        b.step(dev(x[:, t]), [t + 1, t + 1], 1)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


def test_cross_attention_to_states_of_another_length():
    """The states' keys and values go in without a rotation, once; queries of another
    length look at all of them."""
    a = Layer(q.QMM_F16)
    r = np.random.default_rng(11)
    states, rows = [29, 50], 7
    starts = np.array([0, 29, 79], np.int32)
    kvx = r.standard_normal((79, 2 * HK * D)).astype(np.float32)
    x = dev(kvx)
    put = q.KvBatch(dev(a.table), dev(np.asarray(states, np.int32)), 2, 8, 50, 79, starts=dev(starts))
    q.qmm_kv_append(a.cache, put, x, x[:, HK * D:], k_stride=2 * HK * D, v_stride=2 * HK * D)
    look = q.KvBatch(dev(a.table), dev(np.asarray(states, np.int32)), 2, 8, rows, 2 * rows)
    qs = r.standard_normal((2 * rows, HQ * D)).astype(np.float32)
    out = torch.empty(2 * rows, HQ * D, device="cuda")
    work = torch.empty(q.attention_work_bytes(a.cache, look, HQ), dtype=torch.uint8, device="cuda")
    q.qmm_attention(a.cache, look, dev(qs), HQ, out, causal=False, work=work)
    torch.cuda.synchronize()
    got = out.cpu().numpy()
    for n in range(2 * rows):
        s = n // rows
        kk = kvx[starts[s]:starts[s + 1]].astype(np.float16).astype(np.float64).reshape(-1, 2, HK, D)
        for hq in range(HQ):
            qq, k, v = qs[n, hq * D:(hq + 1) * D].astype(np.float64), kk[:, 0, hq * HK // HQ], kk[:, 1, hq * HK // HQ]
            want, pr, _ = ref.attend(qq, k, v, D ** -0.5)
            e = D ** -0.5 * 2.0 ** -17 * (np.abs(k) @ np.abs(qq)).max() + 2.0 ** -30
            tol = (2 * e + 2.0 ** -17 + len(k) * 2.0 ** -26) * (pr @ np.abs(v) + np.abs(want)) + 2.0 ** -25 * np.abs(v).max()
            assert np.all(np.abs(got[n, hq * D:(hq + 1) * D] - want) <= tol)
