"""The routed experts' products on rows so long that the few-slot form takes
several rounds over a row, against the f64 oracle (the bounds of
test_gpu_moe.py)."""
import pytest
import torch

import gguf_block_quant_qmm_amd as q
import test_gpu_moe as moe
from qmm_inputs import GEOMETRY, NAMES

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
