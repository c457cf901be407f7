"""Values at the type's borders in every form of the 4-bit expert FFN (the warp-level one, and tensor memory with tiles of 16
to 128 rows): infinite and very large entries, and large ones that a code of 0 keeps out of the sum.  All forms have to
give what the formula gives."""
import numpy as np
import pytest
import torch

import oracle as O
from token_dispatch_gb300 import _lib as L
from token_dispatch_gb300 import synth
from tests.gpu_util import DEV, to64
from tests.test_gpu_w4 import ffn, weights

pytestmark = pytest.mark.gpu
# relative error of silu: (2 + 1.2 |g|) 2^-23 of the fast exponential, 2^-22 of the quotient, |g| < 20
SILU = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def built():
    from token_dispatch_gb300 import build
    build.build()


def packed(codes, scale, axis, group):
    """What ffn() takes of one tensor, from codes -8..7 [E, out, in] and scales [E, out, groups]."""
    E, out, n = codes.shape
    B = -(-n // 128)
    c = np.zeros((E, out, B * 128), np.int64)
    c[:, :, :n] = codes
    w = (c + 8).reshape(E, out, B, 4, 4, 8)
    shift = np.array([4 * (i // 2) + 16 * (i % 2) for i in range(8)])
    q = np.swapaxes((w << shift).sum(axis=-1).astype(np.uint32), 3, 4).reshape(E, out, B * 16)
    s = np.ones((E, out, B * 128 // group))
    s[:, :, :scale.shape[2]] = scale
    return (torch.from_numpy(q.view(np.int32)).to(DEV), torch.from_numpy(s).to(torch.bfloat16).to(DEV),
            O.w4_unpack(q, s, axis, group, n))


# rows of three experts: the warp-level form, and tiles of 16, 32, 64 and 128 rows
ROWS = [6, 24, 60, 120, 300]


def like(got, want, bound):
    """got is want where that is an infinity or NaN, and within bound elsewhere (infinite past bf16's range)."""
    got = to64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    assert (np.abs(got[fine] - want[fine]) <= bound[fine]).all()


@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_infinite_rows_give_what_the_formula_gives(T, group):
    """One infinite entry: act is infinite with the sign of up's weight, NaN where its code is 0 (0 times infinity)."""
    E, H, Hp = 3, 200, 136
    rng = np.random.default_rng(T + group)
    cu = np.arange(E + 1, dtype=np.int32) * (T // E)
    ws = weights(E, H, Hp, group, rng)
    x = synth.store(rng.standard_normal((T, H)), "bf16").host
    bad = T // E + 1  # a row of expert 1
    codes = rng.integers(-7, 8, (E, Hp, H))
    codes[:, :, 9] = rng.integers(1, 8, (E, Hp))  # gate: an infinite sum of plus sign
    ws[0] = packed(codes, np.full((E, Hp, -(-H // group)), 2.0 ** -7), 0, group)
    codes = rng.integers(-8, 8, (E, Hp, H))
    codes[:, ::5, 9] = 0
    ws[1] = packed(codes, np.full((E, Hp, -(-H // group)), 2.0 ** -7), 0, group)
    x[bad, 9] = float("inf")
    x = x.to(DEV)
    act, h = ffn(x, None, torch.from_numpy(cu).to(DEV), T, ws, E, H, Hp, group)
    assert L.moe_last_device_error() == L.MOE_OK
    with np.errstate(invalid="ignore"):
        want = np.float64("inf") * ws[1][2][1, 9]
    assert np.isnan(want[::5]).all() and np.isinf(want).any()
    like(act[bad], want, np.zeros_like(want))
    keep = [r for r in range(T) if r != bad]
    assert torch.isfinite(h[keep]).all() and not torch.isfinite(h[bad]).any()


@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_large_rows_stay_finite(T, group):
    """Entries up to bf16's largest, whose sums with the weights are far inside the range.  Gate sees one entry of
    size 1 alone (the other codes are 0), so act is silu of that times up's sum, and the sums of down's are of act's size."""
    E, H, Hp = 3, 256, 136
    rng = np.random.default_rng(T + group)
    cu = np.arange(E + 1, dtype=np.int32) * (T // E)
    size = 2.0 ** rng.integers(118, 128, (T, H)) * 1.9921875 * rng.choice([-1, 1], (T, H))
    size[:, 7] = 1
    x = torch.from_numpy(size).to(torch.bfloat16)
    gate = np.zeros((E, Hp, H))
    gate[:, :, 7] = rng.integers(1, 8, (E, Hp))
    n = -(-H // group)
    ws = [packed(gate.astype(np.int64), np.full((E, Hp, n), 0.25), 0, group),
          packed(rng.integers(-8, 8, (E, Hp, H)), np.full((E, Hp, n), 2.0 ** -20), 0, group),
          packed(rng.integers(-8, 8, (E, H, Hp)), np.full((E, H, -(-Hp // group)), 2.0 ** -10), 1, group)]
    act, h = ffn(x.to(DEV), None, torch.from_numpy(cu).to(DEV), T, ws, E, H, Hp, group)
    assert L.moe_last_device_error() == L.MOE_OK
    for e in range(E):
        r = slice(cu[e], cu[e + 1])
        xs = to64(x)[r]
        g, u = xs @ (ws[0][2][e]), xs @ ws[1][2][e]
        want = g / (1 + np.exp(-g)) * u
        assert np.isfinite(want).all() and np.abs(want).max() < 2.0 ** 127
        # a step of 2^-23 of the terms' sum for each of the H sums (any order), one rounding of the result to bf16, and
        # silu's exponential and quotient
        def bound(terms, value, K):
            return K * 2.0 ** -23 * terms + (2.0 ** -8 + SILU) * np.abs(value)
        silu = np.abs(g / (1 + np.exp(-g)))
        like(act[r], want, bound(np.abs(xs) @ np.abs(ws[1][2][e]) * silu, want, H))
        a = to64(act)[r]
        want = a @ ws[2][2][e].T
        like(h[r], want, bound(np.abs(a) @ np.abs(ws[2][2][e]).T, want, Hp))


@pytest.mark.parametrize("T", ROWS)
def test_codes_of_zero_keep_large_entries_out(T):
    """An entry of 2^20 that no output weighs leaves no trace in sums of terms near 1: the error is that of the terms."""
    E, H, Hp, group = 3, 256, 136, 128
    rng = np.random.default_rng(T)
    cu = np.arange(E + 1, dtype=np.int32) * (T // E)
    x = rng.standard_normal((T, H))
    x[:, 40:44] = 2.0 ** 20 * rng.choice([-1, 1], (T, 4))
    x = torch.from_numpy(x).to(torch.bfloat16)
    ws = []
    for out, n in ((Hp, H), (Hp, H), (H, Hp)):
        codes = rng.integers(-7, 8, (E, out, n))
        if n == H:
            codes[:, :, 40:44] = 0
        ws.append(packed(codes, np.full((E, out, -(-n // group)), 2.0 ** -5), 0 if n == H else 1, group))
    act, h = ffn(x.to(DEV), None, torch.from_numpy(cu).to(DEV), T, ws, E, H, Hp, group)
    assert L.moe_last_device_error() == L.MOE_OK
    for e in range(E):
        r = slice(cu[e], cu[e + 1])
        xs, wg, wu = to64(x)[r], ws[0][2][e], ws[1][2][e]
        g, u = xs @ wg, xs @ wu
        dg, du = (H * 2.0 ** -23 * (np.abs(xs) @ np.abs(w)) for w in (wg, wu))
        silu = g / (1 + np.exp(-g))
        want = silu * u
        # silu's slope is at most 1.1
        bound = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + (2.0 ** -8 + SILU) * np.abs(want)
        like(act[r], want, bound)
