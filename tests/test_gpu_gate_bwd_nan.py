"""A NaN logit in the gate's backward: it shows in every gradient that the formula makes of it, and nowhere else."""
import numpy as np
import pytest
import torch

import oracle as O
from token_dispatch_gb300 import _lib as L
from tests.gpu_util import DEV
from tests.test_gpu_gate import REL, TINY, mode_of, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from token_dispatch_gb300 import build
    build.build()


@pytest.mark.parametrize("renorm", [False, True], ids=["plain", "renorm"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(8, 3), (30, 4), (64, 6), (257, 5), (384, 8), (1024, 16)])
def test_gate_bwd_keeps_a_nan(E, K, sigmoid, renorm):
    rng = np.random.default_rng(E)
    l = (1.7 * rng.standard_normal((40, E))).astype(np.float32)
    idx = np.stack([rng.permutation(E)[:K] for _ in range(40)]).astype(np.int32)
    l[:, (E + 1) // 2:][::3] = -np.inf
    chosen, beside = np.arange(10, 20), np.arange(20, 30)  # rows 30 to 39 and 0 to 9 have no NaN
    l[chosen, idx[chosen, 1]] = np.nan
    for t in beside:
        l[t, next(e for e in range(E) if e not in idx[t])] = np.nan
    dg = rng.standard_normal((40, K)).astype(np.float32)
    out = torch.full((40, E), 7.0, device=DEV)
    L.moe_gate_bwd(to_dev(dg), to_dev(l), to_dev(idx), 40, E, K, mode_of(sigmoid, renorm), 1.5, out)
    got = out.cpu().numpy()
    nan = np.zeros((40, E), bool)
    if not sigmoid and not renorm:  # the whole row's softmax
        nan[10:30] = True
    else:  # of the chosen scores: their sum's with RENORM, else each its own
        for t in chosen:
            nan[t, idx[t] if renorm else idx[t, 1:2]] = True
    assert np.array_equal(np.isnan(got), nan)
    clean = np.where(np.isnan(l), 0, l) if sigmoid or renorm else l
    rows = [t for t in range(40) if not nan[t].any()]
    ref = O.gate_group_bwd(dg[rows].astype(np.float64), clean[rows], idx[rows], sigmoid, renorm, 1.5)
    # each term of a difference is within REL of itself, and the scores are at most 1
    mag = 1.5 * np.abs(dg[rows]).sum(axis=1, keepdims=True)
    assert (np.abs(got[rows] - ref) <= 2 * REL * mag + TINY).all()
