"""The routed experts' products of activations close to f32's smallest, in both
forms, against the f64 oracle.

The bound of a slot's product (include/qmm.h): 1e-5 S and, for either form,
2^-125 sum |w| + K 2^-149, what products below f32's normal range lose.  The
few-slot form multiplies x by codes that stand for themselves times 2^-24
(Q4_0's, Q6_K's): a subnormal product is off by 2^-150, which the block's scale
2^24 d makes 2^-126 d, at most 2^-126 |w| for a code that is not zero; the
others lose 2^-150 a product.  The matrix-core form scales a row by at most
2^126 before it is split, whose last step is then 2^-24 2^-126 (times 16 for a
high nibble's activations).
"""
import numpy as np
import pytest
import torch

import gguf_block_quant_qmm_amd as q
import oracle
import test_gpu_moe as moe
from qmm_inputs import NAMES

pytestmark = pytest.mark.gpu

DTYPES = sorted(NAMES)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dt", DTYPES, ids=lambda d: NAMES[d])
@pytest.mark.parametrize("many", [False, True])
def test_activations_near_the_smallest(dt, many):
    E, M, K, T = 3, 40, 512, 2
    N = moe.tokens_on_matrix_cores(q.moe_down_work_bytes, dt, E, M, K, T) * 2 if many else 48
    assert (q.moe_down_work_bytes(dt, E, M, K, N, T) > 0) == many
    g = np.random.default_rng([31, dt])
    ids = g.integers(0, E, (N, T), dtype=np.int32)
    # rows from 2^-90 down to the smallest subnormal, and rows that mix both ends
    H = np.ldexp(g.uniform(1.0, 2.0, (N * T, K)), -g.integers(90, 150, (N * T, 1))) * g.choice([-1.0, 1.0], (N * T, K))
    H[::5, ::3] = np.ldexp(1.0, -149)
    H = H.astype(np.float32)
    W = moe.experts(dt, E, M, K, 0)
    wt = np.ones((N, T), np.float32)
    Y = torch.empty((N, M), device="cuda")
    q.qmm_moe_down(moe.dev(W), dt, E, M, K, N, T, moe.dev(ids), moe.dev(wt), moe.dev(H), Y,
                   work=moe.work_of(q.moe_down_work_bytes(dt, E, M, K, N, T)))
    torch.cuda.synchronize()
    y, S = moe.slot_products(dt, W, E, M, K, ids.reshape(-1), H)
    w1 = np.abs(oracle.dequant(dt, W, E * M, K)).sum(1).reshape(E, M)[ids.reshape(-1)]
    tol = moe.TAU * S + 2.0 ** -125 * w1 + K * 2.0 ** -149
    y, S, tol = y.reshape(N, T, M), S.reshape(N, T, M), tol.reshape(N, T, M)
    want = y.sum(1)
    # the sum over the slots: a rounding each, of the value or of the smallest step
    tol = tol.sum(1) + (T + 1) * (2.0 ** -24 * np.abs(y).sum(1) + 2.0 ** -150)
    err = np.abs(Y.cpu().numpy().astype(np.float64) - want)
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3g} of the bound"
