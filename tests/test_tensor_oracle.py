"""Pins of the oracle of 4-bit weights and orthogonalised updates (CPU)."""
import numpy as np
import pytest

import oracle as O

COEF = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("axis", [0, 1])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_pack_rounds_to_the_nearest_of_fifteen_steps(axis, group):
    rng = np.random.default_rng(group + axis)
    w = (rng.standard_normal((2, 200, 136)) * np.exp(rng.standard_normal((2, 200, 1)))).astype(np.float32)
    q, s = O.w4_pack(w, axis, group)
    n = w.shape[1 + axis]
    x = O.w4_unpack(q, s, axis, group, n)
    for e in range(2):
        for o in range(0, w.shape[2 - axis], 7):
            row = w[e, :, o] if axis == 0 else w[e, o]
            back = x[e, :, o] if axis == 0 else x[e, o]
            for k in range(0, n, group):
                a, step = np.abs(row[k:k + group]).max(), s[e, o, k // group]
                assert a / 7 * (1 - 2e-7) <= step <= a / 7 * 17 / 16 * (1 + 2e-7)
                m, _ = np.frexp(step)
                assert m * 32 == np.floor(m * 32)  # 5 significant bits
                assert np.abs(row[k:k + group] - back[k:k + group]).max() <= step / 2 * (1 + 1e-6)
    bits = np.float32(x).view(np.uint32)
    assert not (bits & 0xffff).any()  # exact in bf16


def test_packed_words_hold_the_stated_places():
    w = np.zeros((1, 1, 256), np.float32)
    w[0, 0, 128 + 32 * 2 + 8 * 3 + 5] = 7.0  # block 1, run 2, word 3, input 5
    q, s = O.w4_pack(w, 1, 32)
    assert s[0, 0, 6] == 1.0
    at = 16 + 4 * 3 + 2
    assert q[0, 0, at] == 0x88888888 ^ (8 << 24) | (15 << 24)
    assert (np.delete(q[0, 0], at) == 0x88888888).all()


def test_pack_of_special_groups():
    w = np.zeros((1, 4, 128), np.float32)
    w[0, 1, 5], w[0, 2, 6], w[0, 3, 7] = np.nan, np.inf, 2.0 ** 127
    q, s = O.w4_pack(w, 1, 128)
    assert s[0, 0, 0] == 2.0 ** -126 and np.isnan(s[0, 1:, 0]).all()
    assert (q == 0x88888888).all()


@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 5, 9), (3, 12, 7)])
def test_orthogonalize_acts_on_singular_values_alone(shape):
    x = np.random.default_rng(1).standard_normal(shape)
    got = O.orthogonalize(x, 5, *COEF, 0.0)
    for u, g in zip(x, got):
        l, s, r = np.linalg.svd(u, full_matrices=False)
        s = s / np.sqrt((s ** 2).sum())
        for _ in range(5):
            s = COEF[0] * s + COEF[1] * s ** 3 + COEF[2] * s ** 5
        assert np.allclose(g, (l * s) @ r, atol=1e-9)
    assert (O.orthogonalize(np.zeros((1, 3, 4)), 5, *COEF, 0.0) == 0).all()


def test_muon_step_by_hand():
    w, g, m = np.ones((1, 1, 1)), np.full((1, 1, 1), 2.0), np.full((1, 1, 1), 4.0)
    o = 1.0
    for _ in range(2):
        o = 2 * o - o ** 3  # b = -1, c = 0
    got = O.muon_step(w, g, m, 0.5, True, 0.1, 0.5, 3.0, 2, 2.0, -1.0, 0.0, 0.0)
    assert got[1] == 4.0 and np.isclose(got[2], o) and np.isclose(got[0], 0.95 - 0.3 * o)
