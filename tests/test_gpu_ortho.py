"""Orthogonalised updates on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

import oracle as O
from token_dispatch_gb300 import _lib as L
from token_dispatch_gb300 import synth
from tests.gpu_util import DEV, TDT, to64

pytestmark = pytest.mark.gpu
CDT = {"f32": L.MOE_F32, "bf16": L.MOE_BF16}
COEF = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


@pytest.fixture(scope="module", autouse=True)
def built():
    from token_dispatch_gb300 import build
    build.build()


def held(v):
    """fp16 of 2^10 v."""
    return np.float64(np.float16(v * 1024)) / 1024


def rounded(u, steps):
    """The oracle's result with the kernels' roundings to fp16: X, and A and the polynomial but
    for their diagonals."""
    a, b, c = COEF
    x = u.astype(np.float64)
    x = x.T if x.shape[0] > x.shape[1] else x
    x = held(x / (np.sqrt((x ** 2).sum()) + EPS))
    for k in range(steps):
        A = x @ x.T
        s = np.diag(A)
        D = held(A - np.diag(s))
        P = (b + c * (s[:, None] + s)) * D + c * (D @ D)
        d = a + b * s + c * s * s + np.diag(c * (D @ D))
        y = d[:, None] * x + held(P - np.diag(np.diag(P))) @ x
        x = held(y) if k + 1 < steps else y
    return x.T if u.shape[0] > u.shape[1] else x


def matrices(rng, E, M, N):
    """Noise with a few directions that stand out."""
    return rng.standard_normal((E, M, N)) + rng.standard_normal((E, M, 2)) @ rng.standard_normal((E, 2, N))


def bound(u, steps=5):
    """2-norm that the result may be off: three times what the roundings make of it in another order of
    sums, and what fp32 sums of that many terms add (2^-21, as much again for each step's factor of 3.5)."""
    exact = O.orthogonalize(u[None], steps, *COEF, EPS)[0]
    off = np.linalg.norm(rounded(u, steps) - exact)
    return exact, 3 * off + 2.0 ** -21 * 3.5 ** steps * np.linalg.norm(exact) / np.sqrt(min(u.shape))


def run(x, dtype, steps=5, coef=COEF, eps=EPS, stream=None):
    E, M, N = x.shape
    n = L.moe_workspace_bytes(L.MOE_OP_ORTHOGONALIZE, 0, M, E, 0, N)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)
    out = torch.full((E, M, N), 55, dtype=torch.bfloat16, device=DEV)
    L.moe_orthogonalize(x, E, M, N, CDT[dtype], steps, *coef, eps, out, ws, n, stream=stream)
    return out


SHAPES = [(1, 1, 1), (2, 1, 9), (3, 16, 24), (2, 40, 17), (5, 64, 64), (2, 130, 300), (1, 257, 255), (3, 300, 33),
          (2, 512, 256), (1, 384, 1000), (1, 777, 601), (70, 8, 8), (2, 128, 512), (1, 512, 97), (1, 128, 513),
          (2, 129, 140), (1, 520, 384), (3, 64, 450), (1, 300, 2500), (2, 2100, 260)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_matches_oracle(shape, dtype):
    u = synth.store(matrices(np.random.default_rng(sum(shape)), *shape) * 1e-3, dtype)
    x = u.host.to(DEV)
    out = run(x, dtype)
    assert L.moe_last_device_error() == L.MOE_OK
    got = to64(out)
    for e in range(shape[0]):
        exact, off = bound(u.ref[e])
        assert np.linalg.norm(got[e] - exact) <= off + 2.0 ** -8 * np.linalg.norm(exact), e
    assert torch.equal(out, run(x, dtype))


@pytest.mark.parametrize("shape", [(1, 100, 700), (1, 1, 600), (20, 129, 530), (40, 130, 257), (70, 257, 130), (1, 900, 384)],
                         ids=lambda s: "x".join(map(str, s)))
def test_few_and_many_tiles(shape):
    """Matrices past what one CTA takes: few tiles, which are halved (a second half may be empty), more that are
    whole, and the last with its sums split."""
    u = synth.store(matrices(np.random.default_rng(sum(shape)), *shape) * 1e-3, "f32")
    x = u.host.to(DEV)
    out = run(x, "f32")
    assert torch.equal(out, run(x, "f32"))
    assert L.moe_last_device_error() == L.MOE_OK
    got = to64(out)
    for e in range(shape[0]):
        exact, off = bound(u.ref[e])
        assert np.linalg.norm(got[e] - exact) <= off + 2.0 ** -8 * np.linalg.norm(exact), e


@pytest.mark.parametrize("steps,coef", [(1, COEF), (2, (1.5, -0.5, 0.0)), (12, (1.875, -1.25, 0.375))])
def test_other_coefficients_and_steps(steps, coef):
    u = matrices(np.random.default_rng(5), 2, 96, 160)
    got = to64(run(torch.from_numpy(u).float().to(DEV), "f32", steps, coef))
    exact = O.orthogonalize(np.float32(u), steps, *coef, EPS)
    # a rounding of 2^-11 to each of X, A and P a step, the last two times |b| + 2 |c| and c, all grown by a
    # factor of at most a a step (the polynomials' slope), and the result's own
    a, b, c = (abs(v) for v in coef)
    grown = sum(a ** k for k in range(steps))
    err = 2.0 ** -11 * (1 + b + 3 * c) * grown * 2 + 2.0 ** -8
    assert np.linalg.norm(got - exact) <= err * np.linalg.norm(exact)


def test_sizes_of_numbers_do_not_matter():
    """Squares that leave the type's range on either side, and a common power of two."""
    u = np.float32(matrices(np.random.default_rng(6), 1, 48, 80))
    want = run(torch.from_numpy(u).to(DEV), "f32", eps=0.0)
    for k in (-120, -60, 60, 120):
        got = run(torch.from_numpy(np.ldexp(u, k)).to(DEV), "f32", eps=0.0)
        assert torch.equal(got, want), k
    tiny = run(torch.from_numpy(np.ldexp(u, -60)).to(DEV), "f32", eps=1e-7)
    assert torch.isfinite(tiny).all() and tiny.abs().max() < 1e-4  # eps holds it down, as in the formula


def test_zeros_nan_and_infinities_stay_in_their_matrix():
    u = np.float32(matrices(np.random.default_rng(7), 5, 64, 72))
    want = run(torch.from_numpy(u).to(DEV), "f32")
    u[1], u[2, 3, 4], u[3, 5, 6] = 0, np.nan, -np.inf
    got = run(torch.from_numpy(u).to(DEV), "f32")
    assert (got[1] == 0).all() and got[2].isnan().all() and got[3].isnan().all()
    assert torch.equal(got[[0, 4]], want[[0, 4]])
    assert (run(torch.zeros((1, 8, 8), device=DEV), "f32", eps=0.0) == 0).all()


def muon(w, g, m, dtype, beta=0.95, nesterov=True, lr=0.02, decay=0.1, scale=1.5, in_place=False, low=False, stream=None):
    E, M, N = w.shape
    n = L.moe_workspace_bytes(L.MOE_OP_MUON_STEP, 0, M, E, 0, N)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)
    w_out, m_out = (w, m) if in_place else (torch.full_like(w, 55), torch.full_like(m, 55))
    w_low = torch.full(w.shape, 55, dtype=torch.bfloat16, device=DEV) if low else None
    L.moe_muon_step(w, g, m, E, M, N, CDT[dtype], beta, nesterov, lr, decay, scale, 5, *COEF, EPS, w_out, w_low, m_out,
                    ws, n, stream=stream)
    return w_out, w_low, m_out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("shape", [(3, 64, 40), (2, 100, 257), (1, 301, 77), (2, 5, 3), (1, 300, 520), (30, 642, 130)],
                         ids=lambda s: "x".join(map(str, s)))
def test_muon_step_matches_oracle(shape, nesterov, dtype):
    rng = np.random.default_rng(sum(shape) + nesterov)
    w = synth.store(rng.standard_normal(shape) * 0.05, dtype)
    g, m = (synth.store(matrices(rng, *shape) * 1e-3, "f32") for _ in range(2))
    dev = [t.host.to(DEV) for t in (w, g, m)]
    w_out, w_low, m_out = muon(*dev, dtype, nesterov=nesterov, low=True)
    assert L.moe_last_device_error() == L.MOE_OK
    f = lambda v: float(np.float32(v))  # noqa: E731  the call's parameters are floats
    rw, rm, ro = O.muon_step(w.ref, g.ref, m.ref, f(0.95), nesterov, f(0.02), f(0.1), 1.5, 5, *COEF, EPS)
    # one fused multiply-add
    assert (np.abs(to64(m_out) - rm) <= 2.0 ** -24 * np.abs(rm) + 1e-30).all()
    half, got, low = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype], to64(w_out), to64(w_low)
    u = g.ref + f(0.95) * rm if nesterov else rm
    for e in range(shape[0]):
        off = f(0.02) * 1.5 * bound(u[e])[1]
        # the new weight: its rounding, two of fp32 on the way, and the update's error
        size = np.linalg.norm(rw[e]) + np.linalg.norm(w.ref[e]) * 2.0 ** -22
        assert np.linalg.norm(got[e] - rw[e]) <= off + (half + 2.0 ** -22) * size
        assert np.linalg.norm(low[e] - rw[e]) <= off + (2.0 ** -8 + 2.0 ** -22) * size
    if dtype == "bf16":
        assert torch.equal(w_low, w_out)
    in_place = muon(*[t.clone() for t in dev], dtype, nesterov=nesterov, in_place=True)
    assert torch.equal(in_place[0], w_out) and torch.equal(in_place[2], m_out)
