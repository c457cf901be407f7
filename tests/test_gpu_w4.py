"""Expert weights in 4 bits on the GPU: codes, scales and restored weights equal to the
oracle's bit for bit, and the expert FFN that reads them within its roundings."""
import numpy as np
import pytest
import torch

import oracle as O
from token_dispatch_gb300 import _lib as L
from token_dispatch_gb300 import synth
from tests.gpu_util import DEV, TDT, to64

pytestmark = pytest.mark.gpu
CDT = {"f32": L.MOE_F32, "bf16": L.MOE_BF16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from token_dispatch_gb300 import build
    build.build()


def pack(w, axis, group, dtype, stream=None):
    """q int32, scale bf16 of a device tensor."""
    E, rows, cols = w.shape
    out, n = (cols, rows) if axis == 0 else (rows, cols)
    B = -(-n // 128)
    q = torch.full((E, out, B * 16), 99, dtype=torch.int32, device=DEV)
    s = torch.full((E, out, B * 128 // group), 99, dtype=torch.bfloat16, device=DEV)
    L.moe_w4_pack(w, E, rows, cols, axis, group, CDT[dtype], q, s, stream=stream)
    return q, s


def check_pack(w, axis, group, dtype):
    """w: host tensor in the storage type."""
    E, rows, cols = w.shape
    d = w.to(DEV)
    q, s = pack(d, axis, group, dtype)
    rq, rs = O.w4_pack(to64(w), axis, group)
    assert np.array_equal(to64(s), rs, equal_nan=True)
    assert np.array_equal(q.cpu().numpy().view(np.uint32), rq)
    out = torch.full(w.shape, 7, dtype=w.dtype, device=DEV)
    L.moe_w4_unpack(q, s, E, rows, cols, axis, group, CDT[dtype], out)
    want = torch.from_numpy(np.ascontiguousarray(O.w4_unpack(rq, rs, axis, group, w.shape[1 + axis]))).float().to(w.dtype)
    assert np.array_equal(to64(out), to64(want), equal_nan=True)


SIZES = [(1, 8, 8), (3, 16, 136), (2, 136, 24), (1, 1000, 72), (5, 128, 256), (2, 264, 712)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("axis", [0, 1])
@pytest.mark.parametrize("size", SIZES, ids=["x".join(map(str, s)) for s in SIZES])
def test_pack_and_unpack_match_oracle(size, axis, group, dtype):
    if dtype == "f32":
        size = (size[0], size[1] - 4, size[2] + 4)
    rng = np.random.default_rng(sum(size))
    w = rng.standard_normal(size) * np.exp(2 * rng.standard_normal((size[0], size[1], 1)))
    w[rng.random(size) < 0.1] = 0
    check_pack(synth.store(w, dtype).host, axis, group, dtype)


@pytest.mark.parametrize("axis", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pack_at_the_types_borders(dtype, axis):
    """Groups at every power of two and its neighbours, zeros, halves of a step, NaN and infinities."""
    rows = []
    for e in range(-126, 128):
        for a in (1.0, 1.0625, 1.75, 1.9921875):
            v = np.zeros(32)
            v[0] = a * 2.0 ** min(e, 126 if a > 1 else 127)
            v[1:15] = -v[0] * (np.arange(14) + 0.5) / 14  # halves of a step where the scale is exact
            rows.append(v)
    for x in (np.nan, np.inf, -np.inf, 2.0 ** -133, 3.3e38):
        v = np.full(32, 2.0 ** -5)
        v[9] = x
        rows.append(v)
    rows.append(np.zeros(32))
    w = np.array(rows)
    w = np.concatenate([w, np.zeros((-len(w) % 128, 32))])
    w = np.ascontiguousarray(w.T if axis == 0 else w)[None]
    with np.errstate(over="ignore"):
        t = torch.from_numpy(w).float().to(TDT[dtype])
    check_pack(t, axis, 32, dtype)


def routed(T, E, K, rng, empty=()):
    """cu [E+1] and src_tok [T*K] of a routing that leaves the experts of `empty` without rows."""
    live = [e for e in range(E) if e not in empty]
    idx = np.array([rng.choice(live, K, replace=False) for _ in range(T)]).reshape(T, K)
    order = np.argsort(idx.reshape(-1), kind="stable")
    cu = np.concatenate([[0], np.cumsum(np.bincount(idx.reshape(-1), minlength=E))]).astype(np.int32)
    return cu, (order // K).astype(np.int32)


def weights(E, H, Hp, group, rng):
    """Packed tensors and what they stand for, as [E, H, Hp] float64."""
    out = []
    for axis in (0, 0, 1):
        w = rng.standard_normal((E, H, Hp)) / np.sqrt(Hp if axis else H)
        q, s = O.w4_pack(synth.round_bf16_bits(w).astype(np.uint32).__lshift__(16).view(np.float32), axis, group)
        ref = O.w4_unpack(q, s, axis, group, Hp if axis else H)
        out.append((torch.from_numpy(q.view(np.int32)).to(DEV), torch.from_numpy(s).to(torch.bfloat16).to(DEV), ref))
    return out


def ffn(x, src, cu, rows, ws, E, H, Hp, group, stream=None):
    act = torch.full((rows, Hp), 55, dtype=torch.bfloat16, device=DEV)
    h = torch.full((rows, H), 55, dtype=torch.bfloat16, device=DEV)
    n = L.moe_workspace_bytes(L.MOE_OP_EXPERT_FFN_W4, rows, H, E, 1, Hp)
    buf = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV) if n else None
    T = len(x)
    L.moe_expert_ffn_w4(x, src, T, cu, rows, ws[0][0], ws[0][1], ws[1][0], ws[1][1], ws[2][0], ws[2][1], E, H, Hp,
                        group, L.MOE_BF16, act, h, buf, n, stream=stream)
    return act, h


def spread(x, w, group):
    """Bound of the error of fp32 sums of (128 + code) x and of 136 x in groups, scaled: a sum of G terms of
    size v has partial sums of about sqrt(G) v, each of its steps rounds one by at most 2^-23 of that, and no more
    than G / 8 steps are rounded one after the other; groups add up as independent errors.  With 143 + 136 for the
    largest factors and 4 times that for the outliers."""
    step = np.abs(w).max() / 7 * 17 / 16
    return 4 * 2.0 ** -23 * 279 * (group / 8) * step * \
        np.sqrt((x ** 2).sum(axis=1))[:, None]


def check_ffn(x, src, cu, ws, act, h, group):
    x64, act64, h64 = to64(x), to64(act), to64(h)
    half = 2.0 ** -8
    for e in range(len(cu) - 1):
        r = slice(cu[e], cu[e + 1])
        if cu[e] == cu[e + 1]:
            continue
        xs = x64[r] if src is None else x64[src[r]]
        wg, wu, wd = (w[2][e] for w in ws)
        g, u = xs @ wg, xs @ wu
        dg, du = spread(xs, wg, group), spread(xs, wu, group)
        silu = g / (1 + np.exp(-g))
        ref = silu * u
        bound = half * np.abs(ref) + 1.1 * (dg * (np.abs(u) + du) + np.abs(silu) * du) + 1e-30
        assert (np.abs(act64[r] - ref) <= bound).all(), (e, np.max(np.abs(act64[r] - ref) / bound))
        ref = act64[r] @ wd.T  # from the act that was stored
        bound = half * np.abs(ref) + 1.1 * spread(act64[r], wd, group) + 1e-30
        assert (np.abs(h64[r] - ref) <= bound).all(), (e, np.max(np.abs(h64[r] - ref) / bound))


# T, E, K, H, Hp, group: one row to many, experts of more rows than a tile has, ragged blocks
CASES = [(1, 4, 1, 64, 32, 32), (1, 1, 1, 8, 8, 128), (2, 8, 2, 128, 64, 64), (5, 6, 3, 200, 72, 32),
         (7, 300, 8, 136, 40, 128), (33, 4, 2, 1000, 712, 64), (70, 3, 2, 264, 328, 128), (150, 2, 1, 520, 136, 32),
         (600, 5, 2, 320, 192, 64), (9, 1, 1, 2056, 1032, 32), (1000, 3, 1, 128, 640, 128)]


@pytest.mark.parametrize("case", CASES, ids=["T%d_E%d_K%d_H%d_Hp%d_G%d" % c for c in CASES])
@pytest.mark.parametrize("gather", [False, True])
def test_ffn_matches_oracle(case, gather):
    T, E, K, H, Hp, group = case
    rng = np.random.default_rng(T)
    cu, src = routed(T, E, K, rng, empty=() if E - K < 2 else (0, E - 1))
    ws = weights(E, H, Hp, group, rng)
    x = synth.store(rng.standard_normal((T, H) if gather else (T * K, H)), "bf16").host.to(DEV)
    act, h = ffn(x, torch.from_numpy(src).to(DEV) if gather else None, torch.from_numpy(cu).to(DEV), T * K, ws, E, H, Hp,
                 group)
    assert L.moe_last_device_error() == L.MOE_OK
    check_ffn(x, src if gather else None, cu, ws, act, h, group)
    again = ffn(x, torch.from_numpy(src).to(DEV) if gather else None, torch.from_numpy(cu).to(DEV), T * K, ws, E, H, Hp,
                group)
    assert torch.equal(act, again[0]) and torch.equal(h, again[1])


@pytest.mark.parametrize("T", [1, 16])
def test_few_rows_of_many_experts(T):
    """One row to each of four experts, and about one to each of 64: either side of the rule that chooses the form
    for up to four rows.  Against the restored weights (exact in fp32), in 64 bits."""
    E, K, H, Hp, group = 64, 4, 1024, 1408, 32
    rng = np.random.default_rng(50 + T)
    assert (L.moe_workspace_bytes(L.MOE_OP_EXPERT_FFN_W4, T, H, E, K, Hp) > 0) == (T > 1)
    cu, src = routed(T, E, K, rng)
    gen = torch.Generator(device=DEV).manual_seed(T)
    ws = []
    for axis in (0, 0, 1):
        w = torch.randn((E, H, Hp), generator=gen, device=DEV) / (Hp if axis else H) ** 0.5
        q, s = pack(w, axis, group, "f32")
        L.moe_w4_unpack(q, s, E, H, Hp, axis, group, L.MOE_F32, w)
        ws.append((q, s, w))
    x = torch.randn((T, H), generator=gen, device=DEV).bfloat16()
    act, h = ffn(x, torch.from_numpy(src).to(DEV), torch.from_numpy(cu).to(DEV), T * K, ws, E, H, Hp, group)
    assert L.moe_last_device_error() == L.MOE_OK
    live = [e for e in range(E) if cu[e] < cu[e + 1]]
    host = [(None, None, {e: to64(w[2][e]) for e in live}) for w in ws]
    check_ffn(x, src, cu, host, act, h, group)


def test_all_rows_on_one_expert():
    T, E, H, Hp, group = 300, 16, 256, 128, 64
    rng = np.random.default_rng(1)
    cu = np.zeros(E + 1, np.int32)
    cu[6:] = T
    ws = weights(E, H, Hp, group, rng)
    x = synth.store(rng.standard_normal((T, H)), "bf16").host.to(DEV)
    act, h = ffn(x, None, torch.from_numpy(cu).to(DEV), T, ws, E, H, Hp, group)
    check_ffn(x, None, cu, ws, act, h, group)


def test_bad_indices_are_reported_and_the_rest_holds():
    T, E, K, H, Hp, group = 12, 5, 2, 128, 64, 32
    rng = np.random.default_rng(2)
    cu, src = routed(T, E, K, rng)
    ws = weights(E, H, Hp, group, rng)
    x = synth.store(rng.standard_normal((T, H)), "bf16").host.to(DEV)
    bad = src.copy()
    bad[3], bad[7] = -1, T
    act, h = ffn(x, torch.from_numpy(bad).to(DEV), torch.from_numpy(cu).to(DEV), T * K, ws, E, H, Hp, group)
    assert L.moe_last_device_error() == L.MOE_ERR_DEVICE_BOUNDS
    assert not act[[3, 7]].any() and not h[[3, 7]].any()
    want = ffn(x, torch.from_numpy(src).to(DEV), torch.from_numpy(cu).to(DEV), T * K, ws, E, H, Hp, group)
    keep = [r for r in range(T * K) if r not in (3, 7)]
    assert torch.equal(act[keep], want[0][keep]) and torch.equal(h[keep], want[1][keep])
    # offsets past the rows, and downwards: cut off, the rows of no expert left as they were
    cut = np.array([0, 6, 4, 10, 99, 1000], np.int32)
    act, h = ffn(x, torch.from_numpy(src).to(DEV), torch.from_numpy(cut).to(DEV), 20, ws, E, H, Hp, group)
    assert L.moe_last_device_error() == L.MOE_ERR_DEVICE_BOUNDS
    short = np.array([0, 5, 9, 12, 12, 15], np.int32)
    act, h = ffn(x, torch.from_numpy(src).to(DEV), torch.from_numpy(short).to(DEV), 20, ws, E, H, Hp, group)
    assert L.moe_last_device_error() == L.MOE_ERR_DEVICE_BOUNDS
    assert (act[15:] == 55).all() and (h[15:] == 55).all()
    check_ffn(x, src, short, ws, act[:15], h[:15], group)


@pytest.mark.parametrize("T,E", [(3000, 700), (6000, 700)])
def test_offsets_that_run_up_and_down_give_nothing(T, E):
    """Every other expert would have all rows: 350 times as many as there are."""
    H, Hp, group = 64, 32, 32
    rng = np.random.default_rng(4)
    ws = weights(E, H, Hp, group, rng)
    x = synth.store(rng.standard_normal((T, H)), "bf16").host.to(DEV)
    cu = np.where(np.arange(E + 1) % 2 == 1, T, 0).astype(np.int32)
    cu[E] = T
    act, h = ffn(x, None, torch.from_numpy(cu).to(DEV), T, ws, E, H, Hp, group)
    assert L.moe_last_device_error() == L.MOE_ERR_DEVICE_BOUNDS
    assert (act == 55).all() and (h == 55).all()


@pytest.mark.parametrize("T", [3, 40, 100])
@pytest.mark.parametrize("size", ["fine", "huge", "tiny"])
def test_scales_of_any_bits(T, size):
    """Scales made elsewhere, of 8 significant bits: around 1, just below 2^125 (their 8-fold is finite, their 24-fold
    is not), and down to subnormal ones.  Rows with one entry make each sum one weight times that entry."""
    E, H, Hp, group = 1, 128, 64, 32
    rng = np.random.default_rng(T)
    ws = weights(E, H, Hp, group, rng)
    lo, hi, entry = {"fine": (0x3f00, 0x4000, 2.0 ** 6), "huge": (0x7d80, 0x7e00, 2.0 ** -94),
                     "tiny": (0x0011, 0x0180, 2.0 ** 94)}[size]
    scale = torch.from_numpy(rng.integers(lo, hi, tuple(ws[1][1].shape)).astype(np.int16)).view(torch.bfloat16)
    ws[1][1].copy_(scale)
    ws[0][0].fill_(-1)  # gate: all codes 15, that is 7, and every product 7 * 8
    ws[0][1].fill_(8 / entry)
    at = rng.integers(0, H, T)
    x = torch.zeros((T, H), dtype=torch.bfloat16)
    x[torch.arange(T), torch.from_numpy(at)] = entry
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    act, _ = ffn(x.to(DEV), None, cu, T, ws, E, H, Hp, group)
    assert L.moe_last_device_error() == L.MOE_OK
    words = ws[1][0].cpu().numpy().astype(np.int64) & 0xffffffff
    j, v, i = at // 32, at % 32 // 8, at % 8
    code = (words[0][:, 4 * v + j] >> (4 * (i // 2) + 16 * (i % 2)) & 15) - 8
    want = (56 / (1 + np.exp(-56.0)) * code * scale.double().numpy()[0][:, at // group] * entry).T
    # the weight and act are rounded to bf16 (the form for few rows rounds act alone), fp32 in between
    err = np.abs(act.double().cpu().numpy() - want)
    assert (err <= np.abs(want) * (2 * 2.0 ** -8 + 2.0 ** -15)).all()


@pytest.mark.parametrize("T,E,group", [(4096, 64, 128), (64, 64, 32)])
def test_the_same_each_time_with_many_tiles(T, E, group):
    """Codes that a warp still reads while their place is loaded again show here: wrong weights of a few outputs, in
    one call of five with 384 rows an expert when the loads were not told of the reads (a proxy fence)."""
    K, H, Hp = 6, 2048, 1408
    rng = np.random.default_rng(T)
    cu, src = routed(T, E, K, rng)
    gen = torch.Generator(device=DEV).manual_seed(T)
    ws = []
    for out, n in ((Hp, H), (Hp, H), (H, Hp)):
        blocks = -(-n // 128)
        q = torch.randint(-2 ** 31, 2 ** 31 - 1, (E, out, blocks * 16), generator=gen, device=DEV, dtype=torch.int32)
        s = torch.rand((E, out, blocks * 128 // group), generator=gen, device=DEV).mul_(0.01).bfloat16()
        ws.append((q, s))
    x = torch.randn((T, H), generator=gen, device=DEV).bfloat16()
    cu, src = torch.from_numpy(cu).to(DEV), torch.from_numpy(src).to(DEV)
    first = ffn(x, src, cu, T * K, ws, E, H, Hp, group)
    for _ in range(60):
        again = ffn(x, src, cu, T * K, ws, E, H, Hp, group)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_nan_scales_and_infinite_rows_stay_where_they_are():
    T, E, H, Hp, group = 6, 3, 128, 64, 32
    rng = np.random.default_rng(3)
    cu = np.array([0, 2, 4, 6], np.int32)
    ws = weights(E, H, Hp, group, rng)
    x = synth.store(rng.standard_normal((T, H)), "bf16").host.to(DEV)
    want = ffn(x, None, torch.from_numpy(cu).to(DEV), T, ws, E, H, Hp, group)
    ws[0][1][1, 5, 2] = float("nan")  # an output of expert 1's gate
    bad = x.clone()
    bad[4, 9] = float("inf")
    act, h = ffn(bad, None, torch.from_numpy(cu).to(DEV), T, ws, E, H, Hp, group)
    assert act[2:4, 5].isnan().all() and h[2:4].isnan().all()
    act[2:4, 5] = want[0][2:4, 5]
    assert not torch.isfinite(h[4]).any()
    keep = [0, 1, 5]
    assert torch.equal(act[:4], want[0][:4]) and torch.equal(act[5], want[0][5]) and torch.equal(h[keep], want[1][keep])
