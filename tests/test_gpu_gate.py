"""The gate with expert groups and its backward on the GPU against the oracle in
64 bits: the chosen experts bit for bit, the gates and gradients within what
fp32 arithmetic gives."""
import numpy as np
import pytest
import torch

import oracle as O
from token_dispatch_gb300 import _lib as L
from token_dispatch_gb300 import synth
from tests.gpu_util import DEV, assert_close

pytestmark = pytest.mark.gpu

# A gate is a quotient of exponentials and their sum.  With u = 2^-24: expf is
# within 2 ulp (4u), a sum of E <= 1024 positive terms taken as 32 lanes of at
# most 64 and a tree is within 70u, sums, products and quotients of the rest stay
# under 16u in all: 2^-17 = 128u covers it, relative to each gate; values below
# 2^-126 lose bits to the fp32 format itself (2^-149 each).
REL, TINY = 2.0 ** -17, 2.0 ** -140


@pytest.fixture(scope="module", autouse=True)
def built():
    from token_dispatch_gb300 import build
    build.build()


def mode_of(sigmoid, renorm, group_max=False):
    return (L.MOE_GATE_SIGMOID if sigmoid else 0) | (L.MOE_GATE_RENORM if renorm else 0) | \
        (L.MOE_GATE_GROUP_MAX if group_max else 0)


def to_dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def run_gate(logits, K, G, KG, sigmoid, bias, renorm, group_max, scale):
    T, E = logits.shape
    idx = torch.full((T, K), -7, dtype=torch.int32, device=DEV)
    gate = torch.full((T, K), -7.0, device=DEV)
    L.moe_gate(to_dev(logits), to_dev(bias), T, E, K, G, KG, mode_of(sigmoid, renorm, group_max), scale, idx, gate)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), gate.cpu().numpy()


def check(logits, K, G, KG, sigmoid, bias, renorm, group_max, scale=1.0):
    logits = np.asarray(logits, np.float32)
    bias = None if bias is None else np.asarray(bias, np.float32)
    idx, gate = run_gate(logits, K, G, KG, sigmoid, bias, renorm, group_max, scale)
    r_idx, r_gate = O.gate_group(logits, K, G, KG, sigmoid, bias, renorm, group_max, scale)
    bad = np.nonzero((idx != r_idx).any(axis=1))[0]
    assert len(bad) == 0, (len(bad), bad[:4], idx[bad[:2]], r_idx[bad[:2]])
    assert np.array_equal(np.isnan(gate), np.isnan(r_gate))
    ok = ~np.isnan(r_gate)
    assert (np.abs(gate[ok] - r_gate[ok]) <= REL * np.abs(r_gate[ok]) + TINY).all()
    return idx, gate


def draw(T, E, kind, seed):
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((T, E)) * 1.7
    if kind == "ties":  # a few values only: whole runs of equal scores
        l = np.round(l)
    elif kind == "near":  # neighbours in fp32, far inside fp32's error of a score
        l = (0.5 + 0.25 * rng.integers(0, 2, (T, E))).astype(np.float32)
        l = l + rng.integers(0, 5, (T, E)) * np.spacing(l)
    elif kind == "wide":  # scores that saturate at 1 and vanish below fp32
        l = l * 25
    elif kind == "masked":
        l[:, rng.permutation(E)[:max(1, E // 3)]] = -np.inf
        l[::5, :] = -np.inf
        l[1::5, 1:] = -np.inf
    return l.astype(np.float32)


# (T, E, K, groups, kept groups): one token; one expert; odd sizes and group
# sizes; one expert to a group; 32 groups; the most experts and choices
SIZES = [(1, 384, 8, 8, 4), (5, 1, 1, 1, 1), (300, 7, 3, 1, 1), (67, 64, 6, 8, 3), (129, 384, 8, 8, 4),
         (33, 160, 6, 8, 3), (41, 96, 5, 32, 9), (50, 24, 4, 24, 4), (19, 1024, 16, 1, 1), (21, 1020, 10, 17, 5),
         (23, 254, 8, 2, 1), (37, 1000, 16, 8, 2), (64, 256, 8, 8, 4), (40, 16, 16, 4, 4), (31, 12, 3, 3, 1)]
OPTIONS = [(False, False, False, False), (False, True, True, False), (True, True, True, False),
           (True, False, False, True), (True, True, False, True), (False, True, False, True), (True, False, True, False)]


@pytest.mark.parametrize("kind", ["plain", "ties", "near", "wide", "masked"])
@pytest.mark.parametrize("size", SIZES, ids=["T%d_E%d_K%d_G%d_%d" % s for s in SIZES])
def test_gate_matches_oracle(size, kind):
    T, E, K, G, KG = size
    for i, (sigmoid, biased, renorm, group_max) in enumerate(OPTIONS):
        l = draw(T, E, kind, 31 * i + E)
        b = np.random.default_rng(i).standard_normal(E) * 0.05 if biased else None
        if b is not None and kind == "ties":
            b = np.round(b * 20) / 16
        check(l, K, G, KG, sigmoid, b, renorm, group_max, scale=(1.0, 2.5)[i % 2])


def test_gate_of_the_wide_router_at_length():
    """Enough rows that near scores come up by themselves."""
    l = draw(20000, 384, "plain", 3)
    b = np.random.default_rng(4).standard_normal(384) * 0.05
    T, K = 20000, 8
    idx, gate = run_gate(l, K, 8, 4, True, b.astype(np.float32), True, False, 2.5)
    s = 1 / (1 + np.exp(-l.astype(np.float64)))
    c = s + b.astype(np.float32).astype(np.float64)
    top2 = np.sort(c.reshape(T, 8, 48), axis=2)[:, :, -2:].sum(axis=2)
    kept = np.argsort(-top2, axis=1, kind="stable")[:, :4]
    allowed = np.zeros((T, 8), bool)
    np.put_along_axis(allowed, kept, True, axis=1)
    ref = np.argsort(-np.where(np.repeat(allowed, 48, axis=1), c, -np.inf), axis=1, kind="stable")[:, :K]
    assert np.array_equal(idx, ref)
    q = np.take_along_axis(s, ref, axis=1)
    q = 2.5 * q / q.sum(axis=1, keepdims=True)
    assert (np.abs(gate - q) <= REL * q).all()


def test_gate_special_values():
    inf, nan = np.inf, np.nan
    l = np.array([[0.1, nan, 0.3, -inf, 2.0, 0.0, inf, 1.0],
                  [nan] * 8, [-inf] * 8, [inf] * 8,
                  [-200.0, -201.0, -inf, -202.0, -inf, -250.0, -inf, -300.0]], np.float32)
    for sigmoid in (False, True):
        for b in (None, np.linspace(0, 0.1, 8)):
            for G, KG in ((1, 1), (4, 2)):
                if not sigmoid:  # a softmax over +inf has no value; its rows choose something in range
                    idx, gate = run_gate(l, 3, G, KG, False, None if b is None else b.astype(np.float32), True, False, 1.0)
                    assert ((idx >= 0) & (idx < 8)).all() and all(len(set(r)) == 3 for r in idx.tolist())
                    assert np.isnan(gate[[0, 1, 3]]).all() and (gate[2] == 0).all()
                else:
                    check(l, 3, G, KG, True, b, False, False)
    # renormalised scores far below fp32's range keep their ratios
    idx, gate = run_gate(l[4:], 3, 1, 1, True, None, True, False, 1.0)
    r = np.exp([0.0, -1.0, -2.0])
    assert idx.tolist() == [[0, 1, 3]] and np.allclose(gate[0], r / r.sum(), rtol=REL)
    # an infinite bias takes an expert out of the choice, too
    b = np.zeros(8, np.float32)
    b[4] = -inf
    idx, _ = run_gate(np.arange(8, dtype=np.float32)[None], 4, 1, 1, True, b, False, False, 1.0)
    assert idx.tolist() == [[7, 6, 5, 3]]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=["T%d_E%d_K%d_G%d_%d" % s for s in SIZES])
def test_gate_bwd_matches_oracle(size, sigmoid, renorm):
    T, E, K, G, KG = size
    for kind in ("plain", "masked", "wide"):
        l = draw(T, E, kind, E + 5)
        idx, _ = O.gate_group(l, K, G, KG, sigmoid)
        dg = np.random.default_rng(E).standard_normal((T, K)).astype(np.float32)
        out = torch.full((T, E), 7.0, device=DEV)
        L.moe_gate_bwd(to_dev(dg), to_dev(l), to_dev(idx), T, E, K, mode_of(sigmoid, renorm), 1.7, out)
        got = out.cpu().numpy()
        ref = O.gate_group_bwd(dg.astype(np.float64), l, idx, sigmoid, renorm, 1.7)
        # each term of a difference is within REL of itself (the oracle's 1 - s is exact to 2^-53 of 1)
        s = O.gate_group(l, E, 1, 1, sigmoid)  # every score, by rank
        p = np.zeros((T, E))
        np.put_along_axis(p, s[0].astype(np.int64), s[1], axis=1)
        mag = np.abs(dg).sum(axis=1, keepdims=True) * 1.7 * (1.0 if renorm else p)
        mag = np.where(np.isnan(mag), 0, mag)
        assert (np.abs(got - ref) <= 2 * REL * mag + 1e-15 * np.abs(dg).max() + TINY).all(), kind


def test_gate_bwd_repeated_and_foreign_indices():
    l = draw(3, 16, "plain", 1)
    idx = np.array([[3, 3, 5], [0, 1, 2], [15, -1, 16]], np.int32)
    dg = np.array([[1, 2, 3], [4, 5, 6], [7, 8, 9]], np.float32)
    for sigmoid, renorm in ((True, False), (False, False)):
        out = torch.full((3, 16), 7.0, device=DEV)
        L.moe_last_device_error()
        L.moe_gate_bwd(to_dev(dg), to_dev(l), to_dev(idx), 3, 16, 3, mode_of(sigmoid, renorm), 1.0, out)
        assert L.moe_last_device_error() == L.MOE_ERR_DEVICE_BOUNDS
        assert L.moe_last_device_error() == L.MOE_OK
        ref = O.gate_group_bwd(dg[:2].astype(np.float64), l[:2], idx[:2], sigmoid, renorm)
        assert_close(out[:2].cpu().numpy(), ref, 2 * REL, "d_logits")
        last = O.gate_group_bwd(dg[2:, :1].astype(np.float64), l[2:], idx[2:, :1], sigmoid, renorm)
        assert_close(out[2:].cpu().numpy(), last, 2 * REL, "row with indices outside")


ROUTE = [("bf16", 300, 128, 384, 8, 8, 4), ("bf16", 777, 256, 64, 6, 8, 3), ("bf16", 200, 1024, 16, 4, 4, 2),
         ("bf16", 1000, 2048, 32, 4, 4, 2), ("f32", 130, 64, 12, 3, 3, 2), ("bf16", 1, 512, 8, 2, 2, 1)]


@pytest.mark.parametrize("case", ROUTE, ids=["%s_T%d_H%d_E%d_K%d_G%d_%d" % c for c in ROUTE])
def test_route_group_and_its_backward(case):
    """Every form of the router GEMM under the group gate; then the gradient
    through moe_gate_bwd and moe_route_bwd(MOE_ROUTE_LOGIT_GRAD)."""
    dtype, T, H, E, K, G, KG = case
    shape = synth.MoEShape("route", T, H, E, K, 64, dtype)
    cdt = L.MOE_BF16 if dtype == "bf16" else L.MOE_F32
    x, wr = synth.router_inputs(shape)
    xd, wd = x.host.to(DEV), wr.host.to(DEV)
    bias = (np.random.default_rng(2).standard_normal(E) * 0.05).astype(np.float32)
    logits, idx, gate = torch.empty((T, E), device=DEV), torch.empty((T, K), dtype=torch.int32, device=DEV), \
        torch.empty((T, K), device=DEV)
    n = L.moe_workspace_bytes(L.MOE_OP_ROUTE, T, H, E, K, 0)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    mode = mode_of(True, True)
    L.moe_route_group(xd, wd, to_dev(bias), T, H, E, K, cdt, G, KG, mode, 2.5, logits, idx, gate, ws, n)
    got = logits.cpu().numpy()
    ref = O.router_logits(x.ref, wr.ref)
    assert_close(got, ref, 1e-5, "logits")  # the tolerance of the router's own tests
    r_idx, r_gate = O.gate_group(got, K, G, KG, True, bias, True, False, 2.5)
    assert np.array_equal(idx.cpu().numpy(), r_idx)
    assert (np.abs(gate.cpu().numpy() - r_gate) <= REL * r_gate).all()

    dg = torch.randn((T, K), generator=torch.Generator().manual_seed(1))
    dl, dw = torch.empty((T, E), device=DEV), torch.empty((H, E), device=DEV)
    dx = torch.full((T, H), 3.0, dtype=xd.dtype, device=DEV)
    L.moe_gate_bwd(dg.to(DEV), logits, idx, T, E, K, mode, 2.5, dl)
    n = L.moe_workspace_bytes(L.MOE_OP_ROUTE_BWD, T, H, E, K, 0)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    L.moe_route_bwd(L.MOE_ROUTE_LOGIT_GRAD | L.MOE_ROUTE_DX_WRITE, dl, None, None, xd, wd, T, H, E, K, cdt, None, dw, dx,
                    ws, n)
    d = dl.cpu().numpy().astype(np.float64)
    r_dl = O.gate_group_bwd(dg.numpy().astype(np.float64), got, r_idx, True, True, 2.5)
    assert_close(d, r_dl, 4 * REL, "d_logits")
    assert_close(dw.cpu().numpy(), x.ref.T @ d, 1e-5, "dw_router")
    # dx: bf16 rounds by at most 2^-8 of the value; fp32 sums of E terms as the router's own tests
    assert_close(dx.float().cpu().numpy(), d @ wr.ref.T, 2.0 ** -8 + 1e-5 if dtype == "bf16" else 1e-5, "dx")
    L.moe_route_bwd(L.MOE_ROUTE_LOGIT_GRAD, dl, None, None, xd, wd, T, H, E, K, cdt, None, None, dx, ws, n)
    assert_close(dx.float().cpu().numpy(), 2 * (d @ wr.ref.T), 2.0 ** -7 + 1e-5 if dtype == "bf16" else 1e-5, "dx twice")
    assert L.moe_last_device_error() == L.MOE_OK


def test_gate_on_another_stream_and_in_a_graph():
    l = torch.from_numpy(draw(500, 384, "plain", 8)).to(DEV)
    b = torch.linspace(-0.05, 0.05, 384, device=DEV)
    out = [torch.empty((500, 8), dtype=torch.int32, device=DEV), torch.empty((500, 8), device=DEV)]
    dl = torch.empty((500, 384), device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        L.moe_gate(l, b, 500, 384, 8, 8, 4, mode_of(True, True), 2.5, *out, stream=s)
        L.moe_gate_bwd(out[1], l, out[0], 500, 384, 8, mode_of(True, True), 2.5, dl, stream=s)
    step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s, capture_error_mode="relaxed"):
        step()
    l.copy_(torch.from_numpy(draw(500, 384, "near", 9)))
    for t in (*out, dl):
        t.fill_(7)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (*out, dl)]
    step()
    s.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, (*out, dl)))
    r_idx, _ = O.gate_group(l.cpu().numpy(), 8, 8, 4, True, b.cpu().numpy())
    assert np.array_equal(got[0].cpu().numpy(), r_idx)


def test_gate_zeros_of_both_signs_and_the_lowest_number():
    """Equal zeros of either sign rank by index; the type's lowest number is a number."""
    low = np.finfo(np.float32).min
    l = np.zeros((6, 64), np.float32)
    l[0, 1::2] = -0.0
    l[1, ::3] = -0.0
    l[2, :] = low
    l[2, 40] = 1.0
    l[3, :60] = low
    l[4, :] = -1e-42
    l[4, 7] = 1e-44
    l[5, 5:9] = [1e-45, -1e-45, 3e-45, 0.0]
    for G, KG in ((1, 1), (8, 8), (8, 3), (1, 1)):
        for group_max in (False, True):
            check(l, 6, G, KG, False, None, True, group_max)
            check(l, 6, G, KG, True, None, False, group_max)
            check(l, 6, G, KG, True, np.zeros(64), True, group_max)


@pytest.mark.parametrize("E,K,G,KG", [(384, 8, 8, 1), (512, 16, 32, 1), (1024, 16, 2, 1), (640, 12, 16, 2)])
def test_gate_of_few_lanes(E, K, G, KG):
    """Kept groups that lie in one lane or a few: a lane gives more than it keeps at hand."""
    for sigmoid, biased in ((False, False), (True, True)):
        l = np.sort(draw(40, E, "plain", E), axis=1)
        l[::2] = l[::2, ::-1]
        b = np.random.default_rng(1).standard_normal(E) * 0.01 if biased else None
        check(l, K, G, KG, sigmoid, b, True, False)


def test_gate_offsets_past_32_bits():
    T, E, K = 2200000, 1024, 4  # 2.25e9 logits
    l = torch.empty((T, E), device=DEV)
    l[-300:].normal_(generator=torch.Generator(device=DEV).manual_seed(2))
    l[:-300] = 0
    tail = l[-300:].contiguous()

    def run(x):
        n = len(x)
        idx, gate, dl = torch.empty((n, K), dtype=torch.int32, device=DEV), torch.empty((n, K), device=DEV), torch.empty_like(x)
        L.moe_gate(x, None, n, E, K, 8, 4, mode_of(True, True), 1.0, idx, gate)
        L.moe_gate_bwd(gate, x, idx, n, E, K, mode_of(False, False), 1.0, dl)
        return idx, gate, dl
    big, small = run(l), run(tail)
    assert all(torch.equal(a[-300:], b) for a, b in zip(big, small))
    # a row of equal scores takes the first experts of the first groups, with equal gates
    assert (big[0][:-300] == torch.arange(K, device=DEV)).all() and (big[1][:-300] == 0.25).all()


def test_empty_batch():
    e = torch.empty((0, 8), device=DEV)
    i = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    L.moe_gate(e, None, 0, 8, 2, 1, 1, 0, 1.0, i, e)
    L.moe_gate_bwd(e, e, i, 0, 8, 2, 0, 1.0, e)
    assert L.moe_last_device_error() == L.MOE_OK


@pytest.mark.parametrize("E,K,G,KG", [(64, 6, 8, 3), (384, 8, 8, 4), (128, 8, 16, 5), (96, 4, 4, 2), (256, 8, 8, 2)])
def test_gate_groups_of_saturated_scores(E, K, G, KG):
    """Scores at and just below 1: many groups of equal fp32 rank, others a little below, which
    hide where the border of the kept groups is."""
    rng = np.random.default_rng(E + G)
    l = rng.uniform(4, 70, (600, E)).astype(np.float32)
    l[::3] = np.where(rng.random((200, E)) < 0.7, -5, l[::3])
    for sigmoid, b in ((True, None), (True, np.round(rng.standard_normal(E) * 2) / 64), (False, None)):
        check(l, K, G, KG, sigmoid, b, True, False)


@pytest.mark.parametrize("E,K,G,KG", [(64, 6, 8, 4), (384, 8, 8, 4), (384, 8, 8, 3), (160, 6, 8, 6), (96, 4, 6, 2)])
def test_gate_equal_groups_around_the_border(E, K, G, KG):
    """Groups come in pairs of equal rank (a group holds its neighbour's logits in another order), so that equal
    ranks lie above the border of the kept groups, on it and below it."""
    rng = np.random.default_rng(E + KG)
    l = rng.standard_normal((300, G, E // G)).astype(np.float32) * 2
    l[:, 1::2] = rng.permuted(l[:, ::2], axis=2)
    l = l.reshape(300, E)
    for sigmoid, b in ((True, None), (True, np.zeros(E)), (False, None), (False, np.zeros(E))):
        check(l, K, G, KG, sigmoid, b, True, False)


@pytest.mark.parametrize("low", [-3.4028235e38, -1e38, -3e4])
@pytest.mark.parametrize("E,K,G,KG", [(64, 6, 8, 3), (384, 8, 8, 4), (256, 8, 8, 2), (24, 3, 4, 3)])
def test_gate_groups_at_the_lowest_number(E, K, G, KG, low):
    """Masks of the type's lowest value: all but a few groups at it (fewer, as many and more than stay), half of
    a group at it, whole rows of it; and the same with numbers as large the other way."""
    rng = np.random.default_rng(E + KG)
    l = rng.standard_normal((240, G, E // G)).astype(np.float32)
    for t in range(240):
        l[t, rng.permutation(G)[:t % (G + 1)]] = low
    l[60:120, :, ::2] = low
    l[120:150] *= 1e37
    l[150:160] = -low
    l = l.reshape(240, E)
    for sigmoid in (True, False):
        for group_max in (True, False):
            for b in (None, rng.standard_normal(E) * 0.1):
                check(l, K, G, KG, sigmoid, b, not sigmoid, group_max)


@pytest.mark.parametrize("E,K,G,KG", [(64, 6, 8, 3), (384, 8, 8, 4), (96, 9, 12, 11), (24, 3, 4, 3), (256, 8, 1, 1)])
def test_gate_infinite_biases_and_groups(E, K, G, KG):
    """Biases of +inf put their experts, and so their groups, first; those of -inf and NaN take theirs out."""
    rng = np.random.default_rng(E * KG)
    l = rng.standard_normal((100, E)).astype(np.float32)
    l[::7, ::3] = -np.inf
    for values in ([np.inf, 0.1], [-np.inf, 0.1, 0.3], [np.nan, -0.1, 0.2], [np.inf, -np.inf, np.nan, 1e38, 0.5]):
        b = rng.choice(values, E, p=None if len(values) > 2 else [0.05, 0.95])
        for sigmoid in (True, False):
            for group_max in (True, False):
                check(l, K, G, KG, sigmoid, b, False, group_max)
