"""Attention over a Q8_0 cache whose block scales span what f16 holds, against the
softmax in f64 under the bound and the root mean square limit of test_gpu_attention:
2^-24 (the smallest step) to 65504, zeros, scales that grow and shrink along the
sequence, one block or token far above the others.  Both forms of the kernels, with
the tokens of a row in one workgroup and shared out.
"""
import numpy as np
import pytest
import torch

from tests import kv_ref as ref
from tests.test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def each(r, n, blocks):
    """Uniform in the logarithm over 2^-24 .. 1, each block its own."""
    return 2.0 ** r.uniform(-24, 0, (n, blocks))


def smallest(r, n, blocks):
    return np.full((n, blocks), 2.0 ** -24)


def tiny(r, n, blocks):
    return 2.0 ** r.uniform(-24, -21, (n, blocks))


def small(r, n, blocks):
    """Values about 2^-18 to 2^-7: where the two f16 parts of a value trade places."""
    return 2.0 ** r.uniform(-21, -14, (n, blocks))


def growing(r, n, blocks):
    return np.repeat(2.0 ** np.linspace(-24, 2, n), blocks).reshape(n, blocks)


def shrinking(r, n, blocks):
    return growing(r, n, blocks)[::-1]


def some_zero(r, n, blocks):
    return np.where(r.random((n, blocks)) < 0.6, 0.0, 2.0 ** r.uniform(-20, -4, (n, blocks)))


def all_zero(r, n, blocks):
    return np.zeros((n, blocks))


def one_block(r, n, blocks):
    s = 2.0 ** r.uniform(-20, -16, (n, blocks))
    s[:, blocks - 1] *= 2.0 ** 16
    return s


def one_token(r, n, blocks):
    s = 2.0 ** r.uniform(-24, -20, (n, blocks))
    s[n // 3] = 60000.0
    return s


def large(r, n, blocks):
    return 2.0 ** r.uniform(1, 12, (n, blocks))


def largest(r, n, blocks):
    return np.where(r.random((n, blocks)) < 0.5, 65504.0, -65504.0)


def some_large(r, n, blocks):
    """From the usual to far above it, token by token."""
    return np.repeat(2.0 ** np.where(r.random(n) < 0.1, r.uniform(2, 15, n), r.uniform(-8, 2, n)), blocks).reshape(n, blocks)


SPREADS = [each, smallest, tiny, small, growing, shrinking, some_zero, all_zero, one_block, one_token, large, some_large, largest]
# query heads, key-value heads, dim, page, tokens, new tokens: one tile of 8, 16 and 32
# rows, and many rows
SIZES = [(4, 1, 64, 16, 300, 1), (4, 1, 96, 16, 90, 4), (8, 2, 128, 32, 260, 7), (2, 1, 256, 64, 1500, 3),
         (4, 1, 64, 16, 130, 40), (2, 1, 96, 32, 260, 70), (8, 2, 128, 64, 900, 50), (2, 1, 192, 16, 200, 30),
         (1, 1, 256, 64, 700, 130)]


def rescale(c, values, spread, r, s=0):
    """Gives the tokens of sequence s the scales of `spread`, in order."""
    n, blocks, page = c.lens[s], c.D // 32, c.page
    size = page * c.D
    rec = (c.v_pool if values else c.k_pool).reshape(c.pages, c.Hk, -1)
    for h in range(c.Hk):
        sc = spread(r, n, blocks).astype(np.float16)
        for i in range(n):
            rec[c.table[s, i // page], h, size:].view(np.float16).reshape(blocks, page)[:, i % page] = sc[i]


@pytest.mark.parametrize("spread", SPREADS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_value_scales(size, spread):
    Hq, Hk, D, page, n, new = size
    for keys in (1.0, 0.01):  # 0.01: small scores, so that a value's error is not behind theirs
        c = Case(8, Hq, Hk, D, page, [n], new, seed=31, q_scale=1.5 * keys)
        rescale(c, True, spread, np.random.default_rng([9, n]))
        c.buffers().call()
        torch.cuda.synchronize()
        c.check()


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("scale", [2.0 ** -24, 2.0 ** -21, 3.99, 4.0, 511.5, 65504.0])
def test_small_codes(size, scale):
    """Codes of -2 .. 2: values of a bit or two, at scales on both sides of every border."""
    Hq, Hk, D, page, n, new = size
    c = Case(8, Hq, Hk, D, page, [n], new, seed=34)
    rescale(c, True, lambda r, n, b: np.full((n, b), scale), None)
    codes = c.v_pool.reshape(c.pages, Hk, -1)[..., :page * D].view(np.int8)
    codes[...] = np.random.default_rng(11).integers(-2, 3, codes.shape)
    c.buffers().call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("spread", [each, growing, shrinking, some_zero, one_block], ids=lambda f: f.__name__)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_key_scales(size, spread):
    Hq, Hk, D, page, n, new = size
    c = Case(8, Hq, Hk, D, page, [n], new, seed=32, q_scale=0.1)
    rescale(c, False, lambda r, n, b: np.minimum(spread(r, n, b), 0.25), np.random.default_rng([10, n]))
    c.buffers().call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("new", [3, 8, 40])
@pytest.mark.parametrize("scale", [2.0 ** -24, 60000.0, -65504.0, 0.0])
def test_a_scale_that_a_row_does_not_see_does_not_reach_it(new, scale):
    """The value scales of a new token in the middle: rows before it keep their bits."""
    outs = []
    for at in (None, scale):
        c = Case(8, 4, 1, 64, 16, [61], new, seed=33)
        if at is not None:
            i = 61 - new + new // 2
            rec = c.v_pool.reshape(c.pages, 1, -1)[c.table[0, i // 16], 0]
            rec[16 * 64:].view(np.float16).reshape(2, 16)[:, i % 16] = at
        c.buffers().call()
        torch.cuda.synchronize()
        c.check()
        outs.append(c.out.clone())
    assert torch.equal(outs[0][:new // 2], outs[1][:new // 2])
    assert not torch.equal(outs[0][new // 2:], outs[1][new // 2:])


@pytest.mark.parametrize("seed", range(24))
def test_random_scales_masks_and_pages(seed):
    """Scales of every size beside windows, ragged rows, other sequences and pages that are none."""
    r = np.random.default_rng([78, seed])
    D, Hk, G = int(r.choice([64, 96, 128, 192, 256])), int(r.choice([1, 2])), int(r.choice([1, 2, 4]))
    page, seqs, new = int(r.choice([16, 32, 64])), int(r.integers(1, 4)), int(r.choice([1, 7, 40, 90]))
    lens = [int(r.integers(1, 400)) for _ in range(seqs)]
    kw = {}
    if r.random() < 0.5:
        n = [int(r.integers(0, new + 1)) for _ in range(seqs)]
        kw["starts"] = [int(v) for v in np.cumsum([r.integers(0, 3)] + n)]
        kw["rows"] = max(1, kw["starts"][-1] + int(r.integers(0, 4)))
    if r.random() < 0.3:
        kw["causal"] = False
    elif r.random() < 0.5:
        kw["window"] = int(r.choice([3, 31, 100]))
    c = Case(8, G * Hk, Hk, D, page, lens, new, seed=seed, cap=float(r.choice([0.0, 0.0, 15.0])), **kw)
    for s in range(seqs):
        rescale(c, True, SPREADS[int(r.integers(len(SPREADS)))], r, s)
    if r.random() < 0.4:
        hit = r.random(c.table.shape) < 0.25
        c.table[hit] = r.choice([-1, c.pages, 2 ** 31 - 1, -2 ** 31], hit.sum()).astype(np.int32)
    c.buffers().call()
    torch.cuda.synchronize()
    c.check()
