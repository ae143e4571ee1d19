"""The routed experts' products on rows so long that the few-slot form takes
several rounds over a row, and in its largest workgroups, against the f64
oracle (the bounds of test_gpu_moe.py)."""
import numpy as np
import pytest
import torch

import gguf_block_quant_qmm_amd as q
import oracle
import test_gpu_moe as moe
from qmm_inputs import GEOMETRY, NAMES, make_blob, make_x, rng_for

pytestmark = pytest.mark.gpu

DTYPES = sorted(NAMES)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


# A wavefront takes 4096 weights of a row, eight of them a round: a full round, one
# chunk more, two rounds and part of a third; odd numbers of 32-weight blocks too
LONG = {32: [32768, 32800, 36864, 36896, 66016], 256: [32768, 33024, 36864, 66048]}


@pytest.mark.parametrize("dt", DTYPES, ids=lambda d: NAMES[d])
@pytest.mark.parametrize("M", [1, 7])
def test_rows_of_several_rounds(dt, M):
    for K in LONG[GEOMETRY[dt][0]]:
        assert q.moe_swiglu_work_bytes(dt, 3, M, K, 1, 2) == 0 and q.moe_down_work_bytes(dt, 3, M, K, 1, 2) == 0
        moe.check_swiglu(dt, 3, M, K, 1, 2)
        moe.check_swiglu(dt, 3, M, K, 2, 1, ids=[2, -1])
        moe.check_down(dt, 3, M, K, 1, 2)
        moe.check_down(dt, 3, M, K, 1, 2, ids=[-1, 1], in_place=True)


def test_largest_workgroup():
    """Many slots of many experts on rows of nine chunks: 256 rows and eight
    items per workgroup, 152 KB of LDS.  Every expert holds the same matrix."""
    dt, E, M, K, N, T = q.QMM_Q4_0, 160, 256, 36864, 256, 1
    assert q.moe_swiglu_work_bytes(dt, E, M, K, N, T) == 0 and q.moe_down_work_bytes(dt, E, M, K, N, T) == 0
    one = [make_blob(dt, M, K, rng_for(2300, i)) for i in range(2)]
    G, U = (torch.from_numpy(b).cuda().repeat(E) for b in one)
    g = np.random.default_rng(12)
    X = make_x(N, K, g)
    ids = g.integers(0, E, (N, T), dtype=np.int32)
    out = moe.run_swiglu(dt, E, M, K, N, T, moe.dev(ids), G, U, moe.dev(X)).cpu().numpy().astype(np.float64)
    Y = torch.empty((N, M), device="cuda")
    q.qmm_moe_down(U, dt, E, M, K, N, T, moe.dev(ids), torch.ones((N, T), device="cuda"), moe.dev(X), Y)
    torch.cuda.synchronize()
    at = np.array([0, 1, 100, N - 1])
    gv, Sg = oracle.matmul(dt, one[0], M, K, X[at])[1:]
    uv, Su = oracle.matmul(dt, one[1], M, K, X[at])[1:]
    want = moe.silu(gv) * uv
    tol = moe.TAU * (1.1 * Sg * (np.abs(uv) + moe.TAU * Su) + np.abs(moe.silu(gv)) * Su) + 4 * 2.0 ** -24 * np.abs(want)
    assert np.all(np.abs(out[at] - want) <= tol)
    assert np.all(np.abs(Y.cpu().numpy()[at] - uv) <= moe.TAU * Su + 2.0 ** -23 * np.abs(uv))
