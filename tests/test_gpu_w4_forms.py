"""The 4-bit expert FFN in each of its forms that hold weights in tensor memory: ragged sizes with every group size,
crowded experts, NaN scales, and the sizes of real layers against products in 64 bits."""
import numpy as np
import pytest
import torch

from token_dispatch_gb300 import _lib as L
from token_dispatch_gb300 import synth
from tests.gpu_util import DEV
from tests.test_gpu_w4 import check_ffn, ffn, routed, weights

pytestmark = pytest.mark.gpu
# relative error of silu: (2 + 1.2 |g|) 2^-23 of the fast exponential, 2^-22 of the quotient, |g| < 20
SILU = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def built():
    from token_dispatch_gb300 import build
    build.build()


# T, E, K, H, Hp, group: 5 to 8 rows an expert (tiles of 16), strips of outputs that end inside, and one expert with
# more rows than a tile has; then wider tiles
CASES = [(40, 6, 1, 1000, 712, 64), (40, 6, 1, 1000, 712, 128), (24, 3, 1, 200, 136, 32), (21, 12, 3, 72, 1032, 128),
         (32, 4, 1, 136, 8, 64), (64, 8, 1, 264, 392, 32), (45, 3, 1, 328, 200, 64), (120, 3, 1, 200, 328, 32),
         (300, 3, 1, 392, 72, 64)]


@pytest.mark.parametrize("case", CASES, ids=["T%d_E%d_K%d_H%d_Hp%d_G%d" % c for c in CASES])
@pytest.mark.parametrize("crowded", [False, True])
def test_every_form_matches_oracle(case, crowded):
    T, E, K, H, Hp, group = case
    rng = np.random.default_rng(T + H)
    cu, src = routed(T, E, K, rng)
    R = T * K
    if crowded:  # all rows but one to each of the others
        cu = np.array([0] + [R - (E - 1) + e for e in range(E)], np.int32)
    assert L.moe_workspace_bytes(L.MOE_OP_EXPERT_FFN_W4, T, H, E, K, Hp) > 0  # not the warp-level form
    ws = weights(E, H, Hp, group, rng)
    x = synth.store(rng.standard_normal((T, H)), "bf16").host.to(DEV)
    act, h = ffn(x, torch.from_numpy(src).to(DEV), torch.from_numpy(cu).to(DEV), R, ws, E, H, Hp, group)
    assert L.moe_last_device_error() == L.MOE_OK
    check_ffn(x, src, cu, ws, act, h, group)


# rows of three experts: the warp-level form, and tiles of 16, 32, 64 and 128 rows
ROWS = [6, 24, 60, 120, 300]


@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_nan_scales_stay_in_their_output(T, group):
    E, H, Hp = 3, 200, 136
    rng = np.random.default_rng(T + group)
    cu = np.arange(E + 1, dtype=np.int32) * (T // E)
    ws = weights(E, H, Hp, group, rng)
    x = synth.store(rng.standard_normal((T, H)), "bf16").host.to(DEV)
    want = ffn(x, None, torch.from_numpy(cu).to(DEV), T, ws, E, H, Hp, group)
    ws[0][1][1, 5, H // group] = float("nan")  # the last group of an output of expert 1's gate
    act, h = ffn(x, None, torch.from_numpy(cu).to(DEV), T, ws, E, H, Hp, group)
    one = slice(cu[1], cu[2])
    assert act[one, 5].isnan().all() and h[one].isnan().all()
    act[one, 5], h[one] = want[0][one, 5], want[1][one]
    assert torch.equal(act, want[0]) and torch.equal(h, want[1])


@pytest.mark.parametrize("T,E,group", [(4096, 64, 128), (64, 64, 32)])
def test_large_calls_match_the_formula(T, E, group):
    """Sizes of a prompt and of a decoding step of a fine-grained layer, against products in 64 bits."""
    K, H, Hp = 6, 2048, 1408
    rng = np.random.default_rng(T)
    cu, src = routed(T, E, K, rng)
    gen = torch.Generator(device=DEV).manual_seed(T)
    ws, full = [], []
    for axis in (0, 0, 1):
        w = torch.randn((E, H, Hp), generator=gen, device=DEV) / (Hp if axis else H) ** 0.5
        out, n = (H, Hp) if axis else (Hp, H)
        B = -(-n // 128)
        q = torch.empty((E, out, B * 16), dtype=torch.int32, device=DEV)
        s = torch.empty((E, out, B * 128 // group), dtype=torch.bfloat16, device=DEV)
        L.moe_w4_pack(w, E, H, Hp, axis, group, L.MOE_F32, q, s)
        L.moe_w4_unpack(q, s, E, H, Hp, axis, group, L.MOE_F32, w)
        ws.append((q, s))
        full.append(w)
    x = torch.randn((T, H), generator=gen, device=DEV).bfloat16()
    act, h = ffn(x, torch.from_numpy(src).to(DEV), torch.from_numpy(cu).to(DEV), T * K, ws, E, H, Hp, group)
    assert L.moe_last_device_error() == L.MOE_OK
    src = torch.from_numpy(src).long().to(DEV)
    for e in range(E):
        r = slice(int(cu[e]), int(cu[e + 1]))
        xs = x[src[r]].double()
        wg, wu, wd = (w[e].double() for w in full)
        g, u = xs @ wg, xs @ wu
        # fp32 sums of n terms in any order: n 2^-23 of the terms' sum
        dg, du = (H * 2.0 ** -23 * (xs.abs() @ w.abs()) for w in (wg, wu))
        silu = g * torch.sigmoid(g)
        want = silu * u
        bound = 1.1 * dg * (u.abs() + du) + silu.abs() * du + (2.0 ** -8 + SILU) * want.abs() + 1e-30
        assert ((act[r].double() - want).abs() <= bound).all(), e
        a = act[r].double()
        want = a @ wd.T
        bound = Hp * 2.0 ** -23 * (a.abs() @ wd.abs().T) + 2.0 ** -8 * want.abs() + 1e-30
        assert ((h[r].double() - want).abs() <= bound).all(), e
