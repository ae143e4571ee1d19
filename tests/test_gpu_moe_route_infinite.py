"""qmm_moe_route with biases of both infinities: the choices are the definition's
(include/qmm.h), a group's score that is NaN counting as -inf."""
import numpy as np
import pytest
import torch

import gguf_block_quant_qmm_amd as q
import test_gpu_moe_route as route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def run(logits, bias, **kw):
    N, E = logits.shape
    k = kw.pop("topk")
    ids, w = torch.empty((N, k), dtype=torch.int32, device="cuda"), torch.empty((N, k), device="cuda")
    q.qmm_moe_route(torch.from_numpy(logits).cuda(), N, E, k, ids, w, bias=torch.from_numpy(bias).cuda(), **kw)
    torch.cuda.synchronize()
    return ids.cpu().numpy()


@pytest.mark.parametrize("scoring", [q.QMM_ROUTE_SOFTMAX, q.QMM_ROUTE_SIGMOID])
def test_infinite_biases_in_one_group(scoring):
    l, b = route.logits_of(9, 32, 1), np.zeros(32, np.float32)
    b[8:16] = -np.inf
    b[11] = np.inf                                # group 1 of 4: +inf beside -inf alone
    # by its two largest the group's score is NaN: behind every other group
    got = run(l, b, topk=16, scoring=scoring, groups=4, topk_groups=2, group_top=2)
    assert not np.any((got >= 8) & (got < 16))
    # by its largest alone it comes first, and with every group open too
    for kw in (dict(groups=4, topk_groups=2, group_top=1), dict(groups=4, topk_groups=4, group_top=2), dict()):
        assert np.all(run(l, b, topk=8, scoring=scoring, **kw)[:, 0] == 11)
    for keep, top in ((1, 2), (2, 2), (3, 2), (4, 2), (2, 1)):
        route.check(l, 8, bias=b, scoring=scoring, groups=4, keep=keep, top=top)
    b[12] = np.inf                                # two of them: the sum is +inf
    assert np.all(run(l, b, topk=8, scoring=scoring, groups=4, topk_groups=2, group_top=2)[:, :2] == [11, 12])
    route.check(l, 8, bias=b, scoring=scoring, groups=4, keep=2, top=2)
