"""Attention over f16 keys or values that are all below 2^-14.  The matrix cores align a
product as if such a factor were 2^-14: a step then keeps its sum to 2^-23 of 2^-14 times
the other factor's largest value, for either f16 part.  Over the probabilities, of which the
largest of a step and all steps come to their sum at most, that is 2^-36 of an output; over
queries that stand as 2^14 at least, up to 16 steps, 2^-32 |scale| max |q| of a score.
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


@pytest.mark.parametrize("most", [1, 3, 100, 1023])
@pytest.mark.parametrize("keys", [False, True])
@pytest.mark.parametrize("size", [(4, 1, 64, 16, 300, 1), (8, 2, 128, 32, 260, 7), (4, 1, 64, 16, 130, 40),
                                  (1, 1, 256, 64, 700, 60)], ids=lambda s: "x".join(map(str, s)))
def test_subnormal_keys_and_values(size, keys, most):
    Hq, Hk, D, page, n, new = size
    c = Case(1, Hq, Hk, D, page, [n], new, seed=61, q_scale=2.0 ** 24 / most if keys else 1.5)
    h = (c.k_pool if keys else c.v_pool).view(np.float16)
    held = np.isfinite(h)
    r = np.random.default_rng(62)
    h[held] = (r.integers(1, most + 1, held.sum()) * r.choice([-1, 1], held.sum()) * 2.0 ** -24).astype(np.float16)
    c.buffers().call()
    torch.cuda.synchronize()
    K, V = (ref.decoded(p, 1, page, Hk, D, v) for p, v in ((c.k_pool, False), (c.v_pool, True)))
    j = np.arange(n)
    at = c.table[0][j // page]
    K, V = K[at, :, j % page], V[at, :, j % page]
    got = c.out.cpu().numpy().astype(np.float64).reshape(new, Hq, D)
    for row in range(new):
        m = n - new + row + 1
        for hq in range(Hq):
            x, k, v = c.Q[row, hq * D:(hq + 1) * D].astype(np.float64), K[:m, hq * Hk // Hq], V[:m, hq * Hk // Hq]
            want, p, _ = ref.attend(x, k, v, c.scale)
            e = c.scale * (2.0 ** -17 * (np.abs(k) @ np.abs(x)).max() + 2.0 ** -36 * np.abs(x).max() * np.abs(k).sum(1).max()
                           + 2.0 ** -32 * np.abs(x).max())
            tol = ((2 * e + 2.0 ** -17 + m * 2.0 ** -26) * (p @ np.abs(v) + np.abs(want)) + m * 2.0 ** -32 * np.abs(v).max()
                   + 2.0 ** -36)
            assert np.all(np.abs(got[row, hq] - want) <= tol), f"row {row} head {hq}"
