"""Appending keys and values to a paged cache, keys and queries normed and turned
on the way, against the f64 formula of each row.

Queries: the formula rounded to f32 once.  f16 places: that f32 value rounded to
f16 (2^-11 of the value, half of the smallest step below 2^-14), so within both
roundings of the formula.  Q8_0 places: the codes and scales of the f32 value,
where a code may differ by one only if the f64 formula lies within 2^-40 of the
rounding border.  Whatever no token goes to keeps its bytes.
"""
import numpy as np
import pytest
import torch

import gguf_block_quant_qmm_amd as q
import oracle
from tests import kv_ref as ref

pytestmark = pytest.mark.gpu
ONE = 2.0 ** -24 * (1 + 2.0 ** -20)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    def __init__(self, dtype, Hq, Hk, D, page, lens, new, starts=None, rows=None, rot=None, layout=ref.HALF, norm=False,
                 pos=False, spare=3, seed=0, fused=True, with_q=True):
        self.__dict__.update(locals())
        r = self.r = np.random.default_rng([dtype, Hq, Hk, D, page, new, seed])
        self.rot = D if rot is None else rot
        self.need = [max(1, -(-max(n, 1) // page)) for n in lens]
        self.pages, self.max_pages = sum(self.need) + spare, max(self.need)
        order = r.permutation(self.pages)
        self.table, at = np.full((len(lens), self.max_pages + 2), -5, np.int32), 0
        for s, n in enumerate(self.need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.rows = rows or (starts[-1] if starts else len(lens) * new)
        self.qkv = r.standard_normal((self.rows, (Hq + 2 * Hk) * D)).astype(np.float32)
        self.freqs = (10000.0 ** (-2.0 * np.arange(self.rot // 2) / self.rot)).astype(np.float32) if self.rot else None
        self.positions = r.integers(0, 5000, self.rows).astype(np.int32) if pos else None
        self.wq, self.wk = ((1 + 0.1 * r.standard_normal(D)).astype(np.float32) for _ in range(2)) if norm else (None, None)
        size = q.kv_pool_bytes(dtype, self.pages, page, Hk, D)
        assert size == self.pages * Hk * ref.record(dtype, page, D)
        self.k0, self.v0 = (r.integers(0, 256, size).astype(np.uint8) for _ in range(2))

    def buffers(self):
        self.k, self.v = dev(self.k0), dev(self.v0)
        self.q_out = torch.full((self.rows, self.Hq * self.D), 7.5, device="cuda")
        self.cache = q.KvCache(self.k, self.v, self.dtype, self.pages, self.page, self.Hk, self.D)
        self.d_table, self.d_lens = dev(self.table), dev(np.asarray(self.lens, np.int32))
        self.d_starts = dev(np.asarray(self.starts, np.int32)) if self.starts else None
        self.batch = q.KvBatch(self.d_table, self.d_lens, len(self.lens), self.max_pages, self.new, self.rows,
                               starts=self.d_starts, table_stride=self.table.shape[1])
        x, (Hq, Hk, D) = dev(self.qkv), (self.Hq, self.Hk, self.D)
        parts = [x[:, :Hq * D], x[:, Hq * D:(Hq + Hk) * D], x[:, (Hq + Hk) * D:]]
        wide = x.shape[1] if self.fused else 0
        self.parts = [p if self.fused else p.contiguous() for p in parts]
        self.kw = dict(freqs=None if self.freqs is None else dev(self.freqs), rot=self.rot, layout=self.layout,
                       pos=None if self.positions is None else dev(self.positions), q_stride=wide, k_stride=wide,
                       v_stride=wide, eps=1e-6)
        if self.norm:
            self.kw.update(q_norm=dev(self.wq), k_norm=dev(self.wk))
        if self.with_q:
            self.kw.update(Q=self.parts[0], q_heads=Hq, q_out=self.q_out)

    def call(self, **kw):
        q.qmm_kv_append(self.cache, self.batch, self.parts[1], self.parts[2], **{**self.kw, **kw})

    def check(self, lens=None):
        c, D, page = self, self.D, self.page
        lens = self.lens if lens is None else lens
        where = ref.places(c.table, lens, c.starts, c.new, page, c.pages, c.rows, c.max_pages)
        got_q, x = c.q_out.cpu().numpy(), c.qkv.reshape(c.rows, -1, D).astype(np.float64)
        k, v = c.k.cpu().numpy(), c.v.cpu().numpy()
        touched = np.zeros((c.pages, page), bool)
        a = [ref.fields(p, c.dtype, page, c.Hk, D, val) for p, val in ((k, False), (v, True))]
        for n, w in enumerate(where):
            if w is None or not c.with_q:
                assert np.all(got_q[n] == 7.5)
            if w is None:
                continue
            _, i, pg = w
            at = i if c.positions is None else c.positions[n]
            parts = [x[n, :c.Hq], x[n, c.Hq:c.Hq + c.Hk]]
            if c.norm:
                parts = [ref.unit(p, wt.astype(np.float64), 1e-6) for p, wt in zip(parts, (c.wq, c.wk))]
            if c.rot:
                parts = [ref.rotate(p, at, c.freqs, c.rot, c.layout) for p in parts]
            if c.with_q:
                err = np.abs(got_q[n].reshape(c.Hq, D) - parts[0])
                assert np.all(err <= ONE * np.abs(parts[0]) + 2.0 ** -47), f"row {n}: query"
            if pg < 0:
                continue
            off = i % page
            assert not touched[pg, off]
            touched[pg, off] = True
            for (codes, scales), y, values in ((a[0], parts[1], False), (a[1], x[n, c.Hq + c.Hk:], True)):
                got = codes[pg, :, :, off] if values else codes[pg, :, off]
                if c.dtype == ref.F16:
                    tol = (2.0 ** -11 + 2 * ONE) * np.abs(y) + 2.0 ** -25 * (1 + 2.0 ** -10)
                    assert np.all(np.abs(got.astype(np.float64) - y) <= tol), f"row {n} values {values}"
                    if values:
                        assert np.array_equal(got.view(np.uint16), y.astype(np.float16).view(np.uint16))
                    continue
                want_s, want_q = oracle.quantize_q8_0(y.astype(np.float32))
                assert np.array_equal(scales[pg, :, :, off].astype(np.float32), want_s.reshape(c.Hk, -1)), f"row {n}"
                off_by = np.abs(got.astype(np.int32) - want_q.reshape(c.Hk, D))
                if values:
                    assert np.all(off_by == 0)
                else:
                    d = np.repeat(np.abs(y.reshape(c.Hk, -1, 32)).max(2) / 127, 32, axis=1)
                    edge = np.abs(np.abs(y / d) % 1.0 - 0.5)
                    assert np.all((off_by == 0) | ((off_by == 1) & (edge < 2.0 ** -17)))
                    assert (off_by != 0).mean() <= 1e-4
        # every other byte is as it was
        for pool, before, values in ((k, c.k0, False), (v, c.v0, True)):
            now, was = (ref.fields(p, c.dtype, page, c.Hk, D, values) for p in (pool, before))
            by_place = touched[:, None, None, :]  # [..][page] last
            for m, o, inside in zip(now, was, (by_place if values else touched[:, None, :, None], by_place)):
                if m is not None:
                    bits = np.uint8 if m.dtype == np.int8 else np.uint16
                    assert ((m.view(bits) == o.view(bits)) | inside).all()


CASES = [
    dict(dtype=1, Hq=32, Hk=8, D=128, page=64, lens=[2000], new=1),
    dict(dtype=8, Hq=32, Hk=8, D=64, page=32, lens=[335, 599, 172, 436, 700], new=7, starts=[0, 4, 10, 12, 17, 24], norm=True),
    dict(dtype=1, Hq=4, Hk=2, D=96, page=16, lens=[70, 31, 16], new=37, starts=[2, 39, 39, 50], rows=55, layout=ref.INTERLEAVED, rot=64),
    dict(dtype=8, Hq=6, Hk=3, D=192, page=16, lens=[100, 3], new=70, starts=[0, 70, 73], layout=ref.INTERLEAVED),
    dict(dtype=8, Hq=2, Hk=2, D=256, page=256, lens=[90, 300], new=90, rot=128, pos=True),
    dict(dtype=1, Hq=8, Hk=1, D=256, page=128, lens=[130, 200], new=129, norm=True, fused=False),
    dict(dtype=1, Hq=3, Hk=3, D=64, page=1024, lens=[1025, 2048, 1], new=1, rot=16, pos=True),
    dict(dtype=8, Hq=1, Hk=1, D=96, page=32, lens=[33], new=33, rot=0, fused=False),
    dict(dtype=1, Hq=5, Hk=5, D=128, page=64, lens=[200, 129], new=65, with_q=False, fused=False),
    dict(dtype=1, Hq=16, Hk=4, D=192, page=32, lens=[5] * 70, new=5, norm=True, rot=48),
    # from 2048 tokens on: tiles of 64 places
    dict(dtype=1, Hq=1, Hk=2, D=96, page=16, lens=[1500, 1024], new=1024, starts=[3, 1010, 2034], rows=2040),
    dict(dtype=8, Hq=1, Hk=1, D=192, page=64, lens=[777, 2050], new=1100, starts=[0, 500, 1600]),
    dict(dtype=8, Hq=1, Hk=1, D=64, page=32, lens=[5, 1031, 90], new=1031, starts=[0, 5, 1036, 1099]),
    dict(dtype=8, Hq=7, Hk=1, D=128, page=64, lens=[64] * 130, new=2, starts=list(range(0, 131)), rows=140),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda c: f"{c['dtype']}-{c['Hq']}x{c['Hk']}x{c['D']}-p{c['page']}-n{c['new']}")
def test_append_matches_formula(kw):
    c = Case(**kw)
    c.buffers()
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("dtype", [1, 8])
def test_tokens_without_a_page_are_dropped(dtype):
    """Page ids outside the pool, lengths beyond the table or below the new tokens."""
    c = Case(dtype, 2, 2, 64, 16, [40, 40, 3, 0, 200, -4], 9, seed=3)
    c.table[0, :] = c.pages
    c.table[1, :] = -1
    c.table[4, :3] = 2 ** 31 - 1
    c.buffers()
    c.call()
    torch.cuda.synchronize()
    c.check()


def test_more_new_rows_than_max_new_and_rows_cut():
    """Rows beyond max_new, and beyond the arrays, are left alone."""
    c = Case(1, 2, 2, 64, 32, [50, 60], 8, starts=[0, 12, 24], rows=20, seed=4)
    c.buffers()
    c.call()
    torch.cuda.synchronize()
    c.check()


def test_nonfinite_and_large_values():
    for dtype in (1, 8):
        c = Case(dtype, 1, 2, 64, 16, [20], 4, rot=0, seed=5, norm=False)
        c.qkv[1, 64] = np.inf
        c.qkv[2, 70] = np.nan
        c.qkv[0, 64 + 128 + 3] = 1e6
        c.qkv[3, 64 + 128 + 9] = -np.inf
        c.buffers()
        c.call()
        torch.cuda.synchronize()
        k, v = (ref.fields(p.cpu().numpy(), dtype, 16, 2, 64, val) for p, val in ((c.k, False), (c.v, True)))
        for n in range(4):
            i = 16 + n
            pg, off = c.table[0, i // 16], i % 16
            for (codes, scales), src, val in ((k, c.qkv[n, 64:192], False), (v, c.qkv[n, 192:], True)):
                got = codes[pg, :, :, off] if val else codes[pg, :, off]
                if dtype == 1:
                    with np.errstate(over="ignore"):
                        assert np.array_equal(got, src.reshape(2, 64).astype(np.float16), equal_nan=True)
                else:
                    with np.errstate(all="ignore"):
                        s, cd = oracle.quantize_q8_0(src.reshape(1, 128))
                    assert np.array_equal(got.reshape(-1), cd.reshape(-1))
                    assert np.array_equal(scales[pg, :, :, off].reshape(-1).astype(np.float32), s.reshape(-1))


def test_queries_in_place():
    c = Case(1, 4, 2, 128, 16, [30], 5, seed=6, fused=False)
    c.buffers()
    c.call()
    x = c.parts[0].clone()
    c.call(Q=x, q_out=x)
    torch.cuda.synchronize()
    assert torch.equal(x, c.q_out)


@pytest.mark.parametrize("dtype", [1, 8])
def test_captured_call_follows_the_lengths(dtype):
    """One capture, replayed as the sequence grows: every step's token lands in its place."""
    c = Case(dtype, 4, 2, 64, 16, [1, 14], 1, seed=7, spare=6)
    c.max_pages = 3
    c.table[:, :3] = np.arange(6).reshape(2, 3)
    c.buffers()
    c.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    c.k.copy_(dev(c.k0))
    c.v.copy_(dev(c.v0))
    for lens in ([1, 14], [2, 15], [16, 33], [47, 48]):
        c.d_lens.copy_(dev(np.asarray(lens, np.int32)))
        c.k.copy_(dev(c.k0))
        c.v.copy_(dev(c.v0))
        g.replay()
        torch.cuda.synchronize()
        c.check(lens)
