"""Attention over the paged cache against the softmax in f64.

Every place of the pools that no token holds is NaN or infinite, so a result that
looks at one shows.  The bound is include/qmm.h's, which counts every rounding at
its worst.  A second check is for what the bound is too wide to see (a dropped
f16 part costs 2^-12 of a score): over a whole call the error's root mean square
stays within 2^-17 of the output's, eight times what an f32 computation of these
sizes loses at random (its scores carry about sqrt(dim) 2^-24 S, at most 2^-20).
"""
import numpy as np
import pytest
import torch

import gguf_block_quant_qmm_amd as q
from tests import kv_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """A filled cache; what no token holds is NaN."""

    def __init__(self, dtype, Hq, Hk, D, page, lens, new, starts=None, rows=None, max_pages=None, causal=True, window=0,
                 cap=0.0, scale=None, q_scale=1.5, seed=0, pad=0, spare=2):
        self.__dict__.update(locals())
        self.scale = D ** -0.5 if scale is None else scale
        r = self.r = np.random.default_rng([dtype, Hq, Hk, D, page, new, len(lens), seed])
        need = [max(1, -(-max(n, 1) // page)) for n in lens]
        self.max_pages = max_pages or max(need)
        need = [min(n, self.max_pages) for n in need]
        self.pages = sum(need) + spare
        order, at = r.permutation(self.pages), 0
        self.table = np.full((len(lens), self.max_pages), -1, np.int32)
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.rows = rows or (starts[-1] if starts else len(lens) * new)
        self.Q = (q_scale * r.standard_normal((self.rows, Hq * D + pad))).astype(np.float32)
        size = self.pages * Hk * ref.record(dtype, page, D)
        held = np.zeros((self.pages, page), bool)
        for s, n in enumerate(lens):
            for i in range(max(0, min(n, self.max_pages * page))):
                held[self.table[s, i // page], i % page] = True
        self.k_pool, self.v_pool = (np.zeros(size, np.uint8) for _ in range(2))
        n = page * D
        for pool, values in ((self.k_pool, False), (self.v_pool, True)):
            rec = pool.reshape(self.pages, Hk, -1)
            inside = held[:, None, None, :] if values else held[:, None, :, None]
            shape = (self.pages, Hk, D, page) if values else (self.pages, Hk, page, D)
            if dtype == ref.F16:
                x = r.standard_normal(shape).astype(np.float16)
                bad = np.where(r.random(shape) < 0.5, np.float16(np.nan), np.float16(-np.inf))
                rec[...] = np.ascontiguousarray(np.where(inside, x, bad)).reshape(self.pages, Hk, -1).view(np.uint8)
            else:
                codes = r.integers(-127, 128, shape).astype(np.int8)
                sc = (0.005 + 0.02 * r.random((self.pages, Hk, D // 32, page))).astype(np.float16)
                sc = np.where(held[:, None, None, :], sc, np.float16(np.nan))
                rec[..., :n] = codes.reshape(self.pages, Hk, -1).view(np.uint8)
                rec[..., n:] = np.ascontiguousarray(sc).reshape(self.pages, Hk, -1).view(np.uint8)

    def buffers(self):
        self.k, self.v = dev(self.k_pool), dev(self.v_pool)
        self.out = torch.full((self.rows, self.Hq * self.D), 7.5, device="cuda")
        self.cache = q.KvCache(self.k, self.v, self.dtype, self.pages, self.page, self.Hk, self.D)
        self.d_lens = dev(np.asarray(self.lens, np.int32))
        self.batch = q.KvBatch(dev(self.table), self.d_lens, len(self.lens), self.max_pages, self.new, self.rows,
                               starts=dev(np.asarray(self.starts, np.int32)) if self.starts else None)
        self.d_q = dev(self.Q)
        self.need = q.attention_work_bytes(self.cache, self.batch, self.Hq)
        # fill: NaN bits, so that a part that no workgroup wrote shows
        self.work = torch.full((self.need,), 255, dtype=torch.uint8, device="cuda")
        return self

    def call(self, **kw):
        kw = {**dict(scale=self.scale, causal=self.causal, window=self.window, softcap=self.cap, work=self.work,
                     q_stride=self.Q.shape[1] if self.pad else 0), **kw}
        q.qmm_attention(self.cache, self.batch, self.d_q, self.Hq, kw.pop("out", self.out), **kw)

    def check(self, lens=None, rows=None):
        """Every row (or the named ones) within the bound; padding untouched."""
        D, G, page, Hk = self.D, self.Hq // self.Hk, self.page, self.Hk
        lens = self.lens if lens is None else lens
        got = self.out.cpu().numpy().astype(np.float64).reshape(self.rows, self.Hq, D)
        K, V = (ref.decoded(p, self.dtype, page, Hk, D, val) for p, val in ((self.k_pool, False), (self.v_pool, True)))
        where = ref.places(self.table, lens, self.starts, self.new, page, self.pages, self.rows, self.max_pages)
        err2 = ref2 = 0.0
        kv = {}
        for n, w in enumerate(where):
            if w is None:
                assert np.all(got[n] == 7.5), f"padding row {n} was written"
                continue
            if rows is not None and n not in rows:
                continue
            s, i, _ = w
            j = ref.visible(s, i, self.table, lens, page, self.pages, self.max_pages, self.causal, self.window)
            if s not in kv:
                kv.clear()
                every = np.arange(max(0, min(int(lens[s]), self.max_pages * page)))
                at = self.table[s][every // page]
                at = np.where((at >= 0) & (at < self.pages), at, 0)
                kv[s] = K[at, :, every % page], V[at, :, every % page]
            for h in range(Hk):
                k, v = kv[s][0][j, h], kv[s][1][j, h]
                for hq in range(h * G, h * G + G):
                    x = self.Q[n, hq * D:(hq + 1) * D].astype(np.float64)
                    want, p, _ = ref.attend(x, k, v, self.scale, self.cap)
                    if len(j) == 0:
                        assert np.all(got[n, hq] == 0.0), f"row {n} head {hq} sees nothing"
                        continue
                    e = (2.0 ** -17 * abs(self.scale) * (np.abs(k) @ np.abs(x))
                         + 2.0 ** -36 * abs(self.scale) * np.abs(x).max() * np.abs(k).sum(1)).max() + 2.0 ** -21 * self.cap
                    tol = ((2 * e + 2.0 ** -17 + len(j) * 2.0 ** -26) * (p @ np.abs(v) + np.abs(want))
                           + len(j) * 2.0 ** -32 * np.abs(v).max())
                    err = np.abs(got[n, hq] - want)
                    assert np.all(err <= tol), f"row {n} (sequence {s}, index {i}) head {hq}: {(err / tol).max():.3g} of the bound"
                    err2, ref2 = err2 + (err ** 2).sum(), ref2 + (want ** 2).sum()
        assert err2 <= 2.0 ** -34 * ref2, f"rms error {np.sqrt(err2 / max(ref2, 1e-300)):.3g} of the output's"


def name(c):
    return f"{'f16' if c['dtype'] == 1 else 'q8'}-{c['Hq']}x{c['Hk']}x{c['D']}-p{c['page']}-s{len(c['lens'])}-n{c['new']}" + \
        ("" if c.get("causal", True) else "-all") + (f"-w{c['window']}" if c.get("window") else "")


FEW = [dict(dtype=dt, Hq=G * Hk, Hk=Hk, D=D, page=page, lens=lens, new=new)
       for dt in (1, 8)
       for D, Hk, G, page, lens, new in (
           (128, 8, 4, 64, [513], 1), (128, 2, 8, 16, [1, 33, 700], 1), (64, 3, 1, 32, [95, 64, 2], 1),
           (64, 2, 4, 16, [70, 300], 4), (96, 2, 3, 16, [31, 257], 3), (96, 1, 7, 128, [400], 5),
           (128, 2, 4, 32, [900, 45], 7), (192, 2, 2, 64, [130, 65], 2), (192, 1, 5, 16, [99], 3),
           (192, 1, 4, 16, [300], 7), (256, 1, 8, 256, [257], 1), (256, 2, 4, 16, [64, 310], 4), (256, 1, 8, 32, [200], 4),
           (64, 1, 71, 64, [333], 1))]
MORE = [
    dict(dtype=1, Hq=4, Hk=2, D=64, page=16, lens=[300, 40, 1], new=3, starts=[1, 4, 4, 6], rows=9),
    dict(dtype=8, Hq=4, Hk=2, D=64, page=16, lens=[300, 40, 9], new=6, starts=[0, 6, 7, 12], rows=14),
    dict(dtype=1, Hq=8, Hk=2, D=128, page=64, lens=[700, 300], new=2, window=100),
    dict(dtype=8, Hq=8, Hk=2, D=128, page=16, lens=[700, 300], new=5, window=33),
    dict(dtype=1, Hq=8, Hk=8, D=64, page=32, lens=[1], new=1, window=1),
    dict(dtype=1, Hq=6, Hk=2, D=96, page=16, lens=[77, 200, 5], new=4, causal=False),
    dict(dtype=8, Hq=4, Hk=4, D=64, page=128, lens=[5, 200], new=9, causal=False),
    dict(dtype=1, Hq=8, Hk=1, D=128, page=64, lens=[600], new=1, cap=20.0),
    dict(dtype=8, Hq=8, Hk=2, D=256, page=64, lens=[100], new=3, cap=5.0, scale=-0.3),
    dict(dtype=1, Hq=2, Hk=1, D=64, page=64, lens=[500], new=1, scale=0.0),
    dict(dtype=1, Hq=2, Hk=1, D=64, page=64, lens=[500], new=1, q_scale=1e-30),
    dict(dtype=1, Hq=2, Hk=1, D=64, page=64, lens=[200], new=1, q_scale=1e25, scale=1e-26),
    dict(dtype=8, Hq=2, Hk=1, D=64, page=64, lens=[500], new=4, q_scale=30.0),
    dict(dtype=1, Hq=8, Hk=2, D=128, page=64, lens=[20000], new=1, pad=64),
    dict(dtype=8, Hq=4, Hk=1, D=128, page=32, lens=[17001, 5], new=3),
    dict(dtype=1, Hq=4, Hk=1, D=64, page=1024, lens=[40, 3000], new=1, max_pages=40),
]


MANY = [dict(dtype=dt, Hq=G * Hk, Hk=Hk, D=D, page=page, lens=lens, new=new, **kw)
        for dt in (1, 8)
        for D, Hk, G, page, lens, new, kw in (
            (128, 2, 4, 64, [200], 200, {}), (64, 1, 3, 16, [133, 75], 75, {}), (96, 2, 1, 32, [97, 400], 97, {}),
            (192, 1, 2, 128, [150], 150, {}), (256, 1, 2, 16, [90, 300], 41, {}), (128, 1, 4, 32, [1500], 40, {}),
            (64, 2, 1, 16, [300, 170, 41], 160, dict(starts=[2, 162, 162, 203], rows=210)),
            (64, 2, 4, 64, [600], 100, dict(window=70)), (128, 1, 1, 16, [260, 33], 60, dict(window=1)),
            (96, 1, 40, 16, [77, 200, 5], 2, dict(causal=False)), (64, 1, 4, 256, [70, 900], 50, dict(causal=False)),
            (64, 1, 2, 16, [100], 70, dict(cap=10.0)), (128, 1, 2, 16, [100], 70, dict(scale=-0.2)),
            (64, 1, 2, 16, [100], 70, dict(scale=0.0)), (64, 1, 2, 64, [100], 70, dict(scale=-0.1, cap=4.0)),
            (128, 2, 1, 64, [20, 64, 1], 64, {}), (64, 1, 2, 32, [150], 60, dict(q_scale=40.0)),
            (128, 1, 2, 64, [333], 333, dict(pad=32)))]


@pytest.mark.parametrize("kw", FEW + MORE + MANY, ids=name)
def test_attention_matches_the_softmax(kw):
    c = Case(**kw).buffers()
    c.call()
    torch.cuda.synchronize()
    c.check()
    first = c.out.clone()
    c.out.fill_(7.5)
    c.work.fill_(1)
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)  # the same bits again


@pytest.mark.parametrize("dtype", [1, 8])
@pytest.mark.parametrize("new", [1, 6, 40])
def test_rows_that_see_nothing(dtype, new):
    """Empty and negative lengths, fewer tokens than rows, pages that are none."""
    c = Case(dtype, 4, 2, 64, 16, [0, -7, 3, 50, 90, 2000], new, max_pages=8, seed=1)
    c.table[3] = -1
    c.table[4, 1:4] = [c.pages, 2 ** 31 - 1, -(2 ** 31)]
    c.buffers().call()
    torch.cuda.synchronize()
    c.check()


def test_window_without_pages_sees_nothing():
    c = Case(1, 2, 1, 64, 16, [200], 2, window=20, seed=2)
    c.table[0, 11:] = -1
    c.buffers().call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("dtype", [1, 8])
@pytest.mark.parametrize("new,window", [(4, 0), (4, 3), (8, 0), (37, 0), (37, 20)])
def test_what_a_row_does_not_see_does_not_reach_it(dtype, new, window):
    """A NaN or infinity in the key and value of one new token: rows that see it are
    what the formula says, not finite; rows that do not are what they were."""
    clean = Case(dtype, 4, 1, 64, 16, [61], new, window=window, seed=3).buffers()
    clean.call()
    for which in ("k", "v"):
        for bad in (np.nan, np.inf):
            c = Case(dtype, 4, 1, 64, 16, [61], new, window=window, seed=3)
            i = 61 - new + new // 2  # the new token in the middle
            pool = c.k_pool if which == "k" else c.v_pool
            a, sc = ref.fields(pool, dtype, 16, 1, 64, which == "v")
            pg, off = c.table[0, i // 16], i % 16
            if dtype == 1:
                a[(pg, 0, slice(5, 7), off) if which == "v" else (pg, 0, off, slice(5, 7))] = bad
            else:
                rec = pool.reshape(c.pages, 1, -1)[pg, 0, 16 * 64:].view(np.float16).reshape(2, 16)
                rec[0, off] = bad
            c.buffers().call()
            torch.cuda.synchronize()
            for n in range(new):
                at = 61 - new + n
                sees = at >= i and (not window or i > at - window)
                if not sees:
                    assert torch.equal(c.out[n], clean.out[n]), (which, bad, n)
                elif which == "v" and dtype == 1:
                    o = c.out[n].view(4, 64)
                    assert not torch.isfinite(o[:, 5:7]).any()
                    rest = torch.cat([o[:, :5], o[:, 7:]], 1), torch.cat([clean.out[n].view(4, 64)[:, :5], clean.out[n].view(4, 64)[:, 7:]], 1)
                    assert torch.equal(*rest)
                elif which == "v":
                    o = c.out[n].view(4, 64)
                    assert not torch.isfinite(o[:, :32]).all() and torch.equal(o[:, 32:], clean.out[n].view(4, 64)[:, 32:])
                else:
                    # a NaN score leaves nothing finite; an infinite key's may be of either
                    # sign (no share, or NaN), or NaN itself where its terms differ in sign
                    o = torch.isnan(c.out[n].view(4, 64))
                    assert o.all() if np.isnan(bad) else (o.all(1) | torch.isfinite(c.out[n].view(4, 64)).all(1)).all()


@pytest.mark.parametrize("dtype", [1, 8])
@pytest.mark.parametrize("new", [2, 30])
def test_nan_query_stays_in_its_row(dtype, new):
    c = Case(dtype, 8, 2, 128, 32, [300, 90], new, seed=4).buffers()
    c.call()
    want = c.out.clone()
    c.d_q[1, 130] = float("nan")
    c.d_q[2, 5] = float("inf")
    c.call()
    torch.cuda.synchronize()
    got, want = c.out.view(2 * new, 8, 128), want.view(2 * new, 8, 128)
    hit = torch.zeros(2 * new, 8, dtype=torch.bool)
    hit[1, 1] = hit[2, 0] = True
    assert torch.isnan(got[hit.cuda()]).all() and torch.equal(got[~hit.cuda()], want[~hit.cuda()])


@pytest.mark.parametrize("dtype", [1, 8])
def test_large_offsets(dtype):
    """A pool beyond 2^32 bytes: the sequence's pages lie at its end."""
    D, Hk, page = 256, 64, 256
    rec = ref.record(dtype, page, D)
    pages = (2 ** 32 + 2 ** 28) // (Hk * rec) + 3
    c = Case(dtype, Hk, Hk, D, page, [300], 1, seed=5, spare=0)
    assert c.pages == 2
    big = []
    for pool in (c.k_pool, c.v_pool):
        t = torch.zeros(pages * Hk * rec, dtype=torch.uint8, device="cuda")
        t.view(pages, -1)[pages - 2:] = dev(pool).view(2, -1)
        big.append(t)
    c.buffers().call()
    want = c.out.clone()
    c.cache = q.KvCache(*big, dtype, pages, page, Hk, D)
    moved = dev(c.table + (pages - 2))
    c.batch = q.KvBatch(moved, c.d_lens, 1, c.max_pages, 1, 1)
    c.out.fill_(0)
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)
    c.check()


@pytest.mark.parametrize("new", [1, 5, 20])
def test_captured_call_follows_the_lengths(new):
    """Two captured calls, each with its own work, replayed together on two
    streams while lengths change between replays."""
    cs = [Case(dt, 8, 2, 128, 32, [900, 900, 900], new, seed=6 + dt).buffers() for dt in (1, 8)]
    for c in cs:
        c.call()
    torch.cuda.synchronize()
    graphs = []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cs]
    for lens in ([900, 1, 33], [5, 899, 640], [0, 31, 900]):
        for c in cs:
            c.d_lens.copy_(dev(np.asarray(lens, np.int32)))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for c in cs:
            c.check(lens)


def test_a_sequence_does_not_depend_on_the_others():
    kw = dict(dtype=1, Hq=8, Hk=2, D=64, page=16, new=2, max_pages=30)
    a = Case(lens=[400, 90, 33], seed=9, **kw).buffers()
    a.call()
    want = a.out.clone()
    a.d_lens.copy_(torch.tensor([17, 90, 2], dtype=torch.int32))
    a.call()
    torch.cuda.synchronize()
    assert torch.equal(a.out[2:4], want[2:4]) and not torch.equal(a.out[:2], want[:2])


def test_work_is_checked():
    c = Case(1, 8, 2, 64, 64, [5000], 1).buffers()
    assert c.need > 0
    with pytest.raises(q.QmmError) as e:
        c.call(work=c.work[:c.need - 16])
    assert e.value.code == q.QMM_ERR_SCRATCH
    with pytest.raises(q.QmmError) as e:
        c.call(work=None)
    assert e.value.code == q.QMM_ERR_NULL
