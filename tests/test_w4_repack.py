"""Packing weights that were restored from 4 bits gives the same codes and scales: the oracle (CPU) and the kernels."""
import numpy as np
import pytest
import torch

import oracle as O
from token_dispatch_gb300 import _lib as L
from token_dispatch_gb300 import synth
from tests.gpu_util import DEV, TDT

SIZES = [(2, 200, 136), (1, 520, 264), (3, 64, 72)]


def weights(size, seed):
    """Groups with every significand of the largest magnitude that bf16 has, among others."""
    rng = np.random.default_rng(seed)
    return np.float32(rng.standard_normal(size) * np.exp2(rng.integers(-140, 100, (size[0], size[1], 1))))


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("axis", [0, 1])
def test_oracle_packs_restored_weights_to_themselves(size, group, axis):
    w = weights(size, group)
    n = size[1 + axis]
    q, s = O.w4_pack(w, axis, group)
    q2, s2 = O.w4_pack(O.w4_unpack(q, s, axis, group, n), axis, group)
    assert np.array_equal(s, s2) and np.array_equal(q, q2)


def test_a_group_that_fits_its_seventh_part():
    w = np.zeros((1, 3, 32))
    w[0, :, :3] = 10.5, -4.5, 1.5
    w[0, 1, 3] = 1.0  # no multiple of 1.5: the rounded product is 1.5 and an ulp, and its next number 1.5625
    w[0, 2] = -w[0, 0]
    q, s = O.w4_pack(w, 1, 32)
    assert list(s[0, :, 0]) == [1.5, 1.5625, 1.5]
    assert np.array_equal(O.w4_unpack(q, s, 1, 32, 32)[0, ::2], w[0, ::2])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("axis", [0, 1])
def test_kernels_pack_restored_weights_to_themselves(size, group, axis, dtype):
    from token_dispatch_gb300 import build
    build.build()
    E, rows, cols = size
    cdt = {"f32": L.MOE_F32, "bf16": L.MOE_BF16}[dtype]
    out, n = (cols, rows) if axis == 0 else (rows, cols)
    w = synth.store(weights(size, group + 1), dtype).host.to(DEV)
    seen = []
    for _ in range(3):
        q = torch.full((E, out, -(-n // 128) * 16), 99, dtype=torch.int32, device=DEV)
        s = torch.full((E, out, -(-n // 128) * 128 // group), 99, dtype=torch.bfloat16, device=DEV)
        L.moe_w4_pack(w, E, rows, cols, axis, group, cdt, q, s)
        w = torch.full(size, 7, dtype=TDT[dtype], device=DEV)
        L.moe_w4_unpack(q, s, E, rows, cols, axis, group, cdt, w)
        seen.append((q, s, w))
    for got in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got, seen[0]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("axis", [0, 1])
def test_kernels_choose_the_lower_scale_where_all_of_a_group_fits(group, axis, dtype):
    """Groups of whole multiples, every second one with one weight, in any place, that is none."""
    from tests.test_gpu_w4 import check_pack
    rng = np.random.default_rng(group)
    out, n = 72, 256
    step = np.ldexp(rng.integers(16, 32, (1, out, n // group, 1)), rng.integers(-9, 9, (1, out, n // group, 1)))
    k = rng.integers(-6, 7, (1, out, n // group, group)).astype(np.float64)
    at = rng.integers(0, group, (out, n // group))
    for o in range(out):
        for g in range(n // group):
            k[0, o, g, at[o, g]] = 7 * rng.choice([-1, 1])
            if (o + g) % 2:
                k[0, o, g, (at[o, g] + rng.integers(1, group)) % group] += 0.25
    w = (k * step).reshape(1, out, n)
    w = np.ascontiguousarray(np.swapaxes(w, 1, 2)) if axis == 0 else w
    check_pack(synth.store(w, dtype).host, axis, group, dtype)
