"""What the header says of the accuracy of moe_orthogonalize, held against a model of its roundings.  CPU only."""
import numpy as np
import pytest

import oracle as O
from tests.test_gpu_ortho import COEF, EPS, matrices, rounded

SIZES = [(64, 96), (200, 300), (512, 768), (768, 512)]


LOW = [(*size, rank) for size in SIZES for rank in (1, 2, 4, 8, 16, 64) if rank <= min(size) / 4]


@pytest.mark.parametrize("M,N,rank", LOW, ids=["%dx%d_r%d" % s for s in LOW])
def test_noise_of_low_rank_matrices(M, N, rank):
    """A rounding to fp16 is off by 2^-11 at most and by 0.42 times that in the mean square (uniform in a step of between
    2^-11 and 2^-10 of the value); that of X before step k is grown by at most a in each step from k on.  Half as
    much again for the roundings of X X^T and of the polynomial."""
    rng = np.random.default_rng(rank)
    u = rng.standard_normal((M, rank)) @ rng.standard_normal((rank, N))
    exact = [O.orthogonalize(u[None], k, *COEF, EPS)[0] for k in range(6)]
    off = np.linalg.norm(rounded(u, 5) - exact[5])
    grown = [COEF[0] ** (5 - k) * 0.42 * 2.0 ** -11 * np.linalg.norm(exact[k]) for k in range(5)]
    assert off <= 1.5 * np.linalg.norm(grown)
    assert 0.08 < off < 0.17  # 0.1 to 0.15, whatever the rank and the size
    assert 0.6 * rank ** 0.5 < np.linalg.norm(exact[5]) < 1.25 * rank ** 0.5


@pytest.mark.parametrize("M,N", SIZES, ids=["%dx%d" % s for s in SIZES])
def test_noise_with_directions_that_stand_out(M, N):
    u = matrices(np.random.default_rng(1), 1, M, N)[0]
    exact = O.orthogonalize(u[None], 5, *COEF, EPS)[0]
    rel = np.linalg.norm(rounded(u, 5) - exact) / np.linalg.norm(exact)
    assert rel < 2e-3
