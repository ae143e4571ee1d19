"""Random sizes, masks, page tables and lengths through qmm_attention, against the
softmax in f64 (the bound and the poisoned places of test_gpu_attention)."""
import numpy as np
import pytest
import torch

from tests.test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(seed):
    r = np.random.default_rng([77, seed])
    D, Hk = int(r.choice([64, 96, 128, 192, 256])), int(r.choice([1, 1, 2, 3]))
    G = int(r.choice([1, 2, 3, 4, 7, 8, 9, 16]))
    page = int(r.choice([16, 32, 64, 128]))
    seqs = int(r.integers(1, 5))
    new = int(r.choice([1, 1, 2, 3, 5, 8, 17, 33, 70]))
    lens = [int(r.choice([r.integers(0, 70), r.integers(1, 700), page * r.integers(0, 6), new])) for _ in range(seqs)]
    kw = dict(dtype=int(r.choice([1, 8])), Hq=G * Hk, Hk=Hk, D=D, page=page, lens=lens, new=new, seed=seed, pad=int(r.choice([0, 4, 64])))
    if r.random() < 0.4:  # ragged, with padding rows before, between nothing and after
        n = [int(r.integers(0, new + 1)) for _ in range(seqs)]
        kw["starts"] = [int(v) for v in np.cumsum([r.integers(0, 3)] + n)]
        kw["rows"] = max(1, kw["starts"][-1] + int(r.integers(0, 4)))
    if r.random() < 0.3:
        kw["causal"] = False
    elif r.random() < 0.4:
        kw["window"] = int(r.choice([1, 5, 31, 64, 200]))
    if r.random() < 0.2:
        kw["cap"] = 15.0
    c = Case(**kw)
    if r.random() < 0.3:  # some pages are none
        hit = r.random(c.table.shape) < 0.25
        c.table[hit] = r.choice([-1, c.pages, 2 ** 31 - 1, -2 ** 31], hit.sum()).astype(np.int32)
    c.buffers().call()
    torch.cuda.synchronize()
    c.check()
