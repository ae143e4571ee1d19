"""The smoke check of the sparse feed-forward block refuses every step's wrong
output (CPU only: the outputs are the oracle's, the mistakes planted here)."""
import numpy as np
import pytest

import oracle
from __graft_entry__ import check_sparse_block
from qmm_inputs import Q4_K, make_blob, make_x, rng_for

DT, E, T, N, K, M = Q4_K, 4, 2, 3, 256, 256


def block():
    """Right outputs of every step, each rounded to f32 once."""
    blobs = [np.concatenate([make_blob(DT, m, k, rng_for(3, 10 * i + e)) for e in range(E)])
             for i, (m, k) in enumerate(((M, K), (M, K), (K, M)))]
    x, logits = make_x(N, K, rng_for(3, 100)), make_x(N, E, rng_for(3, 101))
    x64 = x.astype(np.float64)
    h = (x64 / np.sqrt((x64 * x64).mean(1, keepdims=True) + 1e-5)).astype(np.float32)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :T].astype(np.int32)
    s = np.exp(np.take_along_axis(logits.astype(np.float64), ids, 1))
    wt = (s / s.sum(1, keepdims=True)).astype(np.float32)
    o = dict(dtype=DT, E=E, blobs=blobs, x=x, logits=logits, h=h, ids=ids, wt=wt, act=None, y=None)
    o["act"] = swiglu(o)
    o["y"] = down(o)
    return o


def swiglu(o):
    g, u = (b.reshape(E, -1) for b in o["blobs"][:2])
    return np.stack([[oracle.swiglu(DT, g[e], u[e], M, K, o["h"][n])["out64"][0] for e in o["ids"][n]]
                     for n in range(N)]).astype(np.float32)


def down(o):
    d = o["blobs"][2].reshape(E, -1)
    return (o["x"] + np.stack([sum(np.float64(o["wt"][n, t]) * oracle.matmul(DT, d[o["ids"][n, t]], K, M, o["act"][n, t])[1][0]
                                   for t in range(T)) for n in range(N)])).astype(np.float32)


def test_right_outputs_pass():
    assert set(check_sparse_block(**block())) == {"norm", "routing", "gate/up", "down"}


def zero_act(o):
    o["act"] = np.zeros_like(o["act"])


def no_gate(o):
    u = o["blobs"][1].reshape(E, -1)
    o["act"] = np.stack([[oracle.matmul(DT, u[e], M, K, o["h"][n])[0][0] for e in o["ids"][n]] for n in range(N)])


def other_slot(o):
    o["act"] = np.ascontiguousarray(o["act"][:, ::-1])


def scaled_norm(o):
    o["h"] = o["h"] * np.float32(1 + 1e-6)
    o["act"] = swiglu(o)


def equal_weights(o):
    o["wt"] = np.full_like(o["wt"], 1 / T)


def not_renormalised(o):
    s = np.exp(o["logits"].astype(np.float64))
    o["wt"] = np.take_along_axis(s / s.sum(1, keepdims=True), o["ids"], 1).astype(np.float32)


def second_expert_first(o):
    o["ids"], o["wt"] = np.ascontiguousarray(o["ids"][:, ::-1]), np.ascontiguousarray(o["wt"][:, ::-1])
    o["act"] = swiglu(o)


@pytest.mark.parametrize("mistake,step", [(zero_act, "gate/up"), (no_gate, "gate/up"), (other_slot, "gate/up"), (scaled_norm, "norm"),
                                          (equal_weights, "routing"), (not_renormalised, "routing"), (second_expert_first, "routing")])
def test_a_wrong_step_is_refused_though_the_rest_follows_from_it(mistake, step):
    o = block()
    mistake(o)
    o["y"] = down(o)
    with pytest.raises(AssertionError, match=step):
        check_sparse_block(**o)


@pytest.mark.parametrize("n,k", [(0, 0), (N - 1, K - 1)])
def test_a_wrong_sum_is_refused(n, k):
    o = block()
    o["y"][n, k] = o["x"][n, k]
    with pytest.raises(AssertionError, match="down"):
        check_sparse_block(**o)
