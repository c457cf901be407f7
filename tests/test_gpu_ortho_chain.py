"""Matrices past what one CTA takes, through the whole chain of kernels: coefficients and step counts, sizes of numbers,
zeros, NaN and infinities, and matrices of low rank; each against float64."""
import numpy as np
import pytest
import torch

import oracle as O
from token_dispatch_gb300 import _lib as L
from token_dispatch_gb300 import synth
from tests.gpu_util import DEV, to64
from tests.test_gpu_ortho import COEF, EPS, bound, held, matrices, muon, run

pytestmark = pytest.mark.gpu

# rows of four, odd ones, a tall matrix, sums split along K
CHAIN = [(2, 200, 300), (2, 201, 301), (3, 300, 129), (1, 900, 384)]
IDS = ["x".join(map(str, s)) for s in CHAIN]


@pytest.fixture(scope="module", autouse=True)
def built():
    from token_dispatch_gb300 import build
    build.build()


def rounded(u, steps, coef):
    """The oracle's result with the kernels' roundings to fp16: X, and X X^T and the polynomial but for their diagonals."""
    a, b, c = coef
    x = u.T if u.shape[0] > u.shape[1] else u
    x = held(x / np.sqrt((x ** 2).sum()))
    for k in range(steps):
        A = x @ x.T
        s = np.diag(A)
        D = held(A - np.diag(s))
        DD = D @ D
        P = (b + c * (s[:, None] + s)) * D + c * DD
        y = (a + b * s + c * s * s + c * np.diag(DD))[:, None] * x + held(P - np.diag(np.diag(P))) @ x
        x = held(y) if k + 1 < steps else y
    return x.T if u.shape[0] > u.shape[1] else x


@pytest.mark.parametrize("steps,coef", [(1, COEF), (3, COEF), (2, (1.5, -0.5, 0.0)), (7, (1.875, -1.25, 0.375)), (1, (1.0, 0.0, 0.0))])
@pytest.mark.parametrize("shape", CHAIN, ids=IDS)
def test_other_coefficients_and_steps(shape, steps, coef):
    u = np.float32(matrices(np.random.default_rng(5), *shape))
    got = to64(run(torch.from_numpy(u).to(DEV), "f32", steps, coef))
    assert L.moe_last_device_error() == L.MOE_OK
    exact = O.orthogonalize(u, steps, *coef, EPS)
    for e in range(shape[0]):
        # three times what the roundings make of it in another order of sums, what fp32 sums add (2^-21, grown by the
        # polynomial's slope a at most a step), and the result's own rounding
        size = np.linalg.norm(exact[e])
        off = 3 * np.linalg.norm(rounded(np.float64(u[e]), steps, coef) - exact[e]) + \
            2.0 ** -21 * max(coef[0], 1) ** steps * size + 2.0 ** -8 * size
        assert np.linalg.norm(got[e] - exact[e]) <= off, e


@pytest.mark.parametrize("shape", CHAIN, ids=IDS)
def test_sizes_of_numbers_do_not_matter(shape):
    u = np.float32(matrices(np.random.default_rng(6), *shape))
    want = run(torch.from_numpy(u).to(DEV), "f32", eps=0.0)
    assert torch.isfinite(want).all() and want.abs().max() > 0
    for k in (-120, -60, 60, 120):
        got = run(torch.from_numpy(np.ldexp(u, k)).to(DEV), "f32", eps=0.0)
        assert torch.equal(got, want), k
    tiny = run(torch.from_numpy(np.ldexp(u, -60)).to(DEV), "f32", eps=1e-7)
    assert torch.isfinite(tiny).all() and tiny.abs().max() < 1e-4  # eps holds it down, as in the formula


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [s[1:] for s in CHAIN], ids=["%dx%d" % s[1:] for s in CHAIN])
def test_zeros_nan_and_infinities_stay_in_their_matrix(M, N, dtype):
    E = 5 if (M, N) != (900, 384) else 1
    u = synth.store(matrices(np.random.default_rng(7), E, M, N), dtype).host
    want = run(u.to(DEV), dtype)
    values = [torch.zeros(M, N), float("nan"), float("-inf")]
    for value in values if E == 1 else [None]:  # sums that are split: a matrix at a time
        bad = u.clone()
        put = {0: value} if E == 1 else dict(zip((1, 2, 3), values))
        for e, v in put.items():
            if torch.is_tensor(v):
                bad[e] = 0
            else:
                bad[e, M - 1, N // 2] = v
        got = run(bad.to(DEV), dtype)
        assert L.moe_last_device_error() == L.MOE_OK
        for e in range(E):
            v = put.get(e)
            if v is None:
                assert torch.equal(got[e], want[e]), e
            elif torch.is_tensor(v):
                assert (got[e] == 0).all()
            else:
                assert got[e].isnan().all()


@pytest.mark.parametrize("M,N", [(200, 300), (301, 201)])
def test_momentum_step_with_zeros_nan_and_infinities(M, N):
    """A matrix without a gradient keeps its weights but for the decay; one with a NaN or an infinity loses its own alone."""
    rng = np.random.default_rng(8)
    w, g, m = (torch.from_numpy(np.float32(matrices(rng, 4, M, N))).to(DEV) for _ in range(3))
    want = muon(w, g, m, "f32")[0]
    g2, m2 = g.clone(), m.clone()
    g2[0], m2[0] = 0, 0
    g2[1, 3, 4] = float("nan")
    m2[2, 5, 6] = float("inf")
    got, _, m_out = muon(w, g2, m2, "f32")
    assert L.moe_last_device_error() == L.MOE_OK
    assert torch.equal(got[3], want[3])
    assert (m_out[0] == 0).all() and got[1].isnan().all() and got[2].isnan().all()
    keep = np.float32(1 - float(np.float32(0.02)) * float(np.float32(0.1)))
    assert torch.equal(got[0], w[0] * float(keep))


@pytest.mark.parametrize("rank", [1, 8, 64])
@pytest.mark.parametrize("shape", [(2, 96, 160), (2, 200, 300), (1, 333, 257), (1, 384, 900), (1, 512, 768)],
                         ids=lambda s: "x".join(map(str, s)) if isinstance(s, tuple) else str(s))
def test_matrices_of_low_rank(shape, rank):
    """What an expert's gradient is after a step in which it had few rows.  The roundings of X put noise into the
    directions that should stay empty, and the steps make it larger: the bound is the model's of those roundings."""
    rng = np.random.default_rng(rank)
    u = np.float32(rng.standard_normal(shape[:2] + (rank,)) @ rng.standard_normal((shape[0], rank, shape[2])))
    out = run(torch.from_numpy(u).to(DEV), "f32")
    assert L.moe_last_device_error() == L.MOE_OK
    got = to64(out)
    for e in range(shape[0]):
        exact, off = bound(np.float64(u[e]))
        assert np.linalg.norm(got[e] - exact) <= off + 2.0 ** -8 * np.linalg.norm(exact), e
    assert torch.equal(out, run(torch.from_numpy(u).to(DEV), "f32"))
