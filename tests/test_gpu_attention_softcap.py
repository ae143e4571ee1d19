"""How exactly attention caps its scores: c tanh(x / c) relative to the score, for
caps from below the scores to far above them.

Two tokens, one with a key of zeros: the output is p = 1 / (1 + exp(-c tanh(s / c)))
for a score s that the query gives exactly but for its f16 parts.  A capped score off by r
of itself moves p by r |x| p (1 - p).  The score's own roundings (parts 2^-23, multiplier 3 of
2^-24) and those of the capping (2^-21) are below 2^-20 of it; the exponentials' arguments (up to
16 + 2 |x| in base 2, so 2^-20 and what the |x| term holds), the exponentials, parts, sums and the quotient
(2^-23 each) below 2^-19 of p.  What two f16 parts cannot hold of a probability is half their smallest
step, 2^-25, where the largest probability stands as 2^7 at least: 2^-32 more.
"""
import numpy as np
import pytest
import torch

import gguf_block_quant_qmm_amd as q
from tests import kv_ref as ref
from tests.test_gpu_attention import Case, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("cap", [0.5, 5.0, 30.0, 50.0, 1000.0, 1e6, 1e30, 3e38])
@pytest.mark.parametrize("dtype", [1, 8])
@pytest.mark.parametrize("rows", [7, 16, 32, 500])
def test_capped_scores(dtype, rows, cap):
    D, page = 64, 16
    s = 2.0 ** np.linspace(-8, 4.5, rows)
    s = np.where(np.arange(rows) % 3 == 1, -s, s).astype(np.float32)
    size = ref.record(dtype, page, D)
    k, v = np.zeros(size, np.uint8), np.zeros(size, np.uint8)
    if dtype == 1:
        k.view(np.float16).reshape(page, D)[1, 0] = 1.0
        v.view(np.float16).reshape(D, page)[:, 1] = 1.0
    else:
        k[:page * D].reshape(page, D)[1, 0] = 64
        k[page * D:].view(np.float16).reshape(D // 32, page)[0, 1] = 1 / 64
        v[:page * D].reshape(D, page)[:, 1] = 64
        v[page * D:].view(np.float16).reshape(D // 32, page)[:, 1] = 1 / 64
    Q = np.zeros((rows, D), np.float32)
    Q[:, 0] = s
    out = torch.empty(rows, D, device="cuda")
    cache = q.KvCache(dev(k), dev(v), dtype, 1, page, 1, D)
    batch = q.KvBatch(dev(np.zeros(1, np.int32)), dev(np.array([2], np.int32)), 1, 1, rows, rows)
    work = torch.empty(q.attention_work_bytes(cache, batch, 1), dtype=torch.uint8, device="cuda")
    q.qmm_attention(cache, batch, dev(Q), 1, out, scale=1.0, causal=False, softcap=cap, work=work)
    torch.cuda.synchronize()
    x = cap * np.tanh(s.astype(np.float64) / cap)
    p = 1 / (1 + np.exp(-x))
    err = np.abs(out.cpu().numpy().astype(np.float64) - p[:, None]).max(1)
    tol = 2.0 ** -20 * p * (1 - p) * np.abs(x) + 2.0 ** -19 * p + 2.0 ** -32
    assert np.all(err <= tol), f"score {s[(err / tol).argmax()]}: {(err / tol).max():.3g} of the bound"


@pytest.mark.parametrize("cap", [30.0, 1e3, 1e5, 1e20, 1e38])
@pytest.mark.parametrize("dtype", [1, 8])
@pytest.mark.parametrize("new", [1, 4, 9, 60])
def test_caps_above_the_scores(dtype, new, cap):
    c = Case(dtype, 4, 1, 64, 16, [400], new, cap=cap, seed=41).buffers()
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("dtype", [1, 8])
@pytest.mark.parametrize("new", [1, 9, 60])
def test_a_row_does_not_depend_on_how_far_others_are_capped(dtype, new):
    """Rows with scores far below the cap keep their bits beside rows that reach it."""
    c = Case(dtype, 4, 1, 64, 16, [200], new, cap=4.0, q_scale=0.05, causal=False, seed=42).buffers()
    c.call()
    want = c.out.clone()
    c.d_q[:, :64] *= 400.0  # head 0 of each row
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(c.out[:, 64:], want[:, 64:]) and not torch.equal(c.out[:, :64], want[:, :64])
