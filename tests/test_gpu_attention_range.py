"""Attention at the ends of what scale and softcap may be: any finite f32 scale, any
softcap that is one or rounds to 0; queries as far the other way; scores that are 0
under multipliers beyond f32.  Against the softmax in f64 under test_gpu_attention's bound.
"""
import pytest
import torch

from tests.test_gpu_attention import Case

pytestmark = pytest.mark.gpu
ROWS = [1, 4, 9, 60]  # one tile of 8, 16 and 32 rows (4 heads), many rows


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("cap", [1e-20, 1e-38, 1e-40, 1e-45, 1e-50, 1e-300])
@pytest.mark.parametrize("scale", [None, -1.0, 0.0])
@pytest.mark.parametrize("dtype", [1, 8])
@pytest.mark.parametrize("new", ROWS)
def test_smallest_caps(dtype, new, scale, cap):
    """All scores within the cap of 0: equal shares; a query of zeros has scores of exactly 0."""
    c = Case(dtype, 4, 1, 64, 16, [150], new, cap=cap, scale=scale, seed=51)
    c.Q[0] = 0
    c.buffers().call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("scale,q_scale", [(3e38, 1e-37), (-3.4e38, 3e-38), (1e-40, 3e37), (1e-44, 1e37), (1e-300, 1.0), (5e-324, 3e37)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("dtype", [1, 8])
@pytest.mark.parametrize("new", ROWS)
def test_far_scales(dtype, new, cap, scale, q_scale):
    c = Case(dtype, 4, 1, 64, 16, [150], new, cap=cap, scale=scale, q_scale=q_scale, seed=52)
    c.Q[0] = 0
    c.buffers().call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("scale,cap", [(1e6, 0.0), (-3e38, 0.0), (3e38, 1.0), (1.0, 1e-39)])
@pytest.mark.parametrize("dtype", [1, 8])
@pytest.mark.parametrize("new", ROWS)
def test_keys_of_zeros(dtype, new, scale, cap):
    """Scores of exactly 0, however large the queries: equal shares."""
    c = Case(dtype, 4, 1, 64, 16, [150], new, cap=cap, scale=scale, q_scale=3e37, seed=53)
    c.k_pool[:] = 0
    c.buffers().call()
    torch.cuda.synchronize()
    c.check()
