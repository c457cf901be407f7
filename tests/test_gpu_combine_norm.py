"""The combine fused with its norms, and its backward, on the GPU against the oracle
in 64 bits, element by element.

Tolerances.  An output of type t is rounded once: half a step, eps(t)/2 of its
value.  Before that everything is fp32 (u = 2^-24): a sum over K <= 16 rows, one
over H <= 16384 columns (at most 64 terms in a thread, then trees: under 80u
relative to the sum of magnitudes), a square root and quotient, and under ten
products.  2^-16 = 256u of the magnitudes that are added up covers a value that has
passed one such sum, 2^-15 one that has passed two."""
import numpy as np
import pytest
import torch

import oracle as O
from token_dispatch_gb300 import _lib as L
from token_dispatch_gb300 import synth
from tests.gpu_util import DEV, TDT, to64

pytestmark = pytest.mark.gpu
CDT = {"f32": L.MOE_F32, "bf16": L.MOE_BF16}
ONE, TWO = 2.0 ** -16, 2.0 ** -15


@pytest.fixture(scope="module", autouse=True)
def built():
    from token_dispatch_gb300 import build
    build.build()


class Case:
    """Inputs of a case: device tensors by name, and the same values in float64."""

    def __init__(self, dtype, T, H, K, seed=0, post=True, nxt=True, scale=True, gate=True, perm=True, residual=True,
                 gain=1.0):
        rng = np.random.default_rng(seed)
        self.dtype, self.T, self.H, self.K = dtype, T, H, K
        self.d, self.r = {}, {}

        def put(name, a, t="f32"):
            s = synth.store(a, t)
            self.d[name], self.r[name] = s.host.to(DEV), s.ref
        put("h", gain * rng.standard_normal((T * K, H)), dtype) if K else None
        put("residual", rng.standard_normal((T, H)), dtype) if residual else None
        put("dy", rng.standard_normal((T, H)), dtype)
        put("dxn", rng.standard_normal((T, H)), dtype) if nxt else None
        put("w_next", 1 + 0.3 * rng.standard_normal(H)) if nxt else None
        if K:
            put("gate", rng.random((T, K))) if gate else None
            put("row_scale", rng.standard_normal(T)) if scale else None
            put("res_scale", rng.standard_normal(H)) if scale else None
            put("w_post", 1 + 0.3 * rng.standard_normal(H)) if post else None
        self.dst = rng.permutation(T * K).astype(np.int32) if perm and K else None
        self.dst_d = torch.from_numpy(self.dst).to(DEV) if self.dst is not None else None

    def opt(self, what):
        return {n: what.get(n) for n in ("row_scale", "w_post", "res_scale", "w_next")}

    def forward(self, eps, y=None, stream=None):
        tdt, d = TDT[self.dtype], self.d
        y = torch.full((self.T, self.H), 7, dtype=tdt, device=DEV) if y is None and self.K else y
        xn = torch.full((self.T, self.H), 7, dtype=tdt, device=DEV) if "w_next" in d else None
        L.moe_combine_norm(d.get("h"), d.get("gate"), self.dst_d, d.get("row_scale"), d.get("residual"), d.get("w_post"),
                           d.get("res_scale"), d.get("w_next"), eps, self.T, self.H, self.K, CDT[self.dtype], y, xn,
                           stream=stream)
        return y, xn

    def backward(self, eps, y, skip=(), stream=None, d_res=None):
        T, H, K, d, tdt = self.T, self.H, self.K, self.d, TDT[self.dtype]

        def out(name, shape, t=torch.float32, when=True):
            return torch.full(shape, 7, dtype=t, device=DEV) if when and name not in skip else None
        o = {"d_res": d_res if d_res is not None else out("d_res", (T, H), tdt), "dh": out("dh", (T * K, H), tdt, K > 0),
             "d_gate": out("d_gate", (T, K), when=K > 0), "d_scale": out("d_scale", (T,), when=K > 0),
             "dw_post": out("dw_post", (H,), when="w_post" in d), "d_res_scale": out("d_res_scale", (H,), when="res_scale" in d),
             "dw_next": out("dw_next", (H,), when="w_next" in d)}
        sums = any(o[n] is not None for n in ("dw_post", "d_res_scale", "dw_next"))
        n = L.moe_workspace_bytes(L.MOE_OP_COMBINE_NORM_BWD, T, H, 0, K, 0) if sums else 0
        ws = torch.full((n,), 0x7f, dtype=torch.uint8, device=DEV) if sums else None
        L.moe_combine_norm_bwd(d.get("dy") if "dy" not in skip else None, d.get("dxn"), d.get("h"), d.get("gate"), self.dst_d,
                               d.get("row_scale"), y if "w_next" in d else None, d.get("w_post"), d.get("res_scale"),
                               d.get("w_next"), eps, T, H, K, CDT[self.dtype], *o.values(), ws, n, stream=stream)
        return {k: v for k, v in o.items() if v is not None}


def half(dtype):
    return torch.finfo(TDT[dtype]).eps / 2


def within(got, ref, tol, what):
    got = to64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - ref) / (tol + 1e-300)):.3g} of the bound"


def check_forward(c, eps, y=None):
    y, xn = c.forward(eps, y)
    torch.cuda.synchronize()
    r, K = c.r, c.K
    ry, rxn = O.combine_norm(r.get("h"), r.get("gate"), c.dst, K, eps, residual=r.get("residual"), **c.opt(r))
    res = np.abs(r["residual"]) if "residual" in r else 0.0
    mag = res + np.zeros_like(ry)
    if K:
        absz = O.combine_norm(np.abs(r["h"]), None if "gate" not in r else np.abs(r["gate"]), c.dst, K, eps)[0]
        z = O.combine_norm(r["h"], r.get("gate"), c.dst, K, eps)[0]
        f = O.rms(z, eps) * np.abs(r["w_post"]) if "w_post" in r else 1.0
        if "res_scale" in r:
            f = f * np.abs(r["res_scale"]) * np.abs(r["row_scale"])[:, None]
        # an error of z moves its root mean square, and so every column of the row
        spread = np.sqrt((absz ** 2).mean(axis=1, keepdims=True)) if "w_post" in r else 0.0
        mag = mag + f * (absz + spread)
        within(y, ry, half(c.dtype) * np.abs(ry) + ONE * mag, "y")
    if rxn is not None:
        f = O.rms(ry, eps) * np.abs(r["w_next"])
        spread = np.sqrt((mag ** 2).mean(axis=1, keepdims=True))
        within(xn, rxn, half(c.dtype) * np.abs(rxn) + TWO * f * (mag + spread), "xn")
    return y, xn


def check_backward(c, eps, y, **kw):
    o = c.backward(eps, y, **kw)
    torch.cuda.synchronize()
    r, K, T, H = c.r, c.K, c.T, c.H
    ry = to64(y) if "w_next" in r else None
    dy = None if "dy" in kw.get("skip", ()) else r["dy"]
    ref = O.combine_norm_bwd(dy, r.get("dxn"), r.get("h"), r.get("gate"), c.dst, K, eps, ry, **c.opt(r))
    h2 = half(c.dtype)
    Dm = np.zeros((T, H)) if dy is None else np.abs(dy)
    if "w_next" in r:
        q = O.rms(ry, eps)
        t = np.abs(r["dxn"] * r["w_next"])
        v = np.abs(ry * q)
        Dm = Dm + q * (t + v * (t * v).mean(axis=1, keepdims=True))
        within(o["dw_next"], ref["dw_next"], TWO * (np.abs(r["dxn"]) * v).sum(axis=0), "dw_next")
    if "d_res" in o:
        within(o["d_res"], ref["d_res"], h2 * np.abs(ref["d_res"]) + TWO * Dm, "d_res")
    if not K:
        return
    absz = O.combine_norm(np.abs(r["h"]), None if "gate" not in r else np.abs(r["gate"]), c.dst, K, eps)[0]
    z = O.combine_norm(r["h"], r.get("gate"), c.dst, K, eps)[0]
    rr = O.rms(z, eps) if "w_post" in r else 1.0
    um = rr * (absz + (np.sqrt((absz ** 2).mean(axis=1, keepdims=True)) if "w_post" in r else 0.0))
    one = np.ones(H)
    w, a = np.abs(r.get("w_post", one)), np.abs(r.get("res_scale", one))
    s = np.abs(r["row_scale"])[:, None] if "row_scale" in r else np.ones((T, 1))
    Pm = s * a * w * Dm
    dzm = rr * (Pm + um * (Pm * um).mean(axis=1, keepdims=True)) if "w_post" in r else Pm
    g = np.abs(r["gate"]) if "gate" in r else np.ones((T, K))
    rows = (np.arange(T * K) if c.dst is None else c.dst.astype(np.int64)).reshape(T, K)
    three = 2.0 ** -14  # D, then the row's mean, then the product below: three sums
    if "d_scale" in o:
        within(o["d_scale"], ref["d_scale"], three * (Dm * a * w * um).sum(axis=1), "d_scale")
    if "dw_post" in o:
        within(o["dw_post"], ref["dw_post"], three * (s * Dm * a * um).sum(axis=0), "dw_post")
    if "d_res_scale" in o:
        within(o["d_res_scale"], ref["d_res_scale"], three * (s * Dm * w * um).sum(axis=0), "d_res_scale")
    for k in range(K):
        if "dh" in o:
            want = ref["dh"][rows[:, k]]
            within(o["dh"][torch.from_numpy(rows[:, k]).to(DEV)], want, h2 * np.abs(want) + three * g[:, k:k + 1] * dzm, "dh")
        if "d_gate" in o:
            within(o["d_gate"][:, k], ref["d_gate"][:, k], three * (dzm * np.abs(r["h"][rows[:, k]])).sum(axis=1), "d_gate")


# (dtype, T, H, K): a vector's width to the widest row, one token upward, every
# count of rows, H that leaves the last warp ragged
SIZES = [("bf16", 1, 8, 1), ("f32", 1, 4, 2), ("bf16", 7, 72, 3), ("f32", 9, 1000, 3), ("bf16", 33, 1032, 2),
         ("bf16", 5, 2048, 6), ("f32", 3, 2052, 5), ("bf16", 3, 4096, 2), ("bf16", 7, 7168, 8), ("f32", 2, 7168, 2),
         ("bf16", 2, 8200, 4), ("bf16", 2, 16384, 16), ("f32", 2, 16384, 3), ("bf16", 400, 264, 16), ("f32", 700, 36, 1),
         ("bf16", 1300, 64, 7), ("bf16", 3, 12296, 1), ("f32", 5, 4104, 9)]
OPTIONS = {"all": {}, "prenorm": dict(post=False, scale=False), "post": dict(nxt=False), "plain": dict(post=False, nxt=False),
           "bare": dict(gate=False, perm=False, scale=False), "no_residual": dict(residual=False)}


@pytest.mark.parametrize("opt", list(OPTIONS))
@pytest.mark.parametrize("size", SIZES, ids=["%s_T%d_H%d_K%d" % s for s in SIZES])
def test_combine_norm_and_backward_match_oracle(size, opt):
    c = Case(*size, seed=size[2], **OPTIONS[opt])
    y, _ = check_forward(c, 1e-5)
    check_backward(c, 1e-5, y)


@pytest.mark.parametrize("size", [("bf16", 1, 8, 0), ("bf16", 500, 2048, 0), ("f32", 31, 7168, 0), ("bf16", 3, 16384, 0)],
                         ids=lambda s: "%s_T%d_H%d" % s[:3])
def test_norm_without_a_block(size):
    c = Case(*size)
    check_forward(c, 1e-6)
    check_backward(c, 1e-6, c.d["residual"])
    check_backward(c, 1e-6, c.d["residual"], skip=("dy",))


def test_large_and_vanishing_rows():
    """Rows of zeros have norms of zero, not NaN; eps rules rows far below it; large rows do not overflow."""
    c = Case("f32", 40, 264, 3)
    c.d["h"][:30] = 0
    c.r["h"][:30] = 0
    c.d["residual"][:20] = 0
    c.r["residual"][:20] = 0
    c.dst[:] = np.arange(120)
    c.dst_d.copy_(torch.from_numpy(c.dst))
    y, _ = check_forward(c, 1e-3)
    check_backward(c, 1e-3, y)
    for gain in (1e-12, 1e12):
        c = Case("f32", 9, 264, 3, gain=gain)
        y, _ = check_forward(c, 1e-5)
        check_backward(c, 1e-5, y)


def test_outputs_left_out_change_nothing_in_the_others():
    c = Case("bf16", 90, 520, 3)
    y, _ = c.forward(1e-5)
    whole = c.backward(1e-5, y)
    for skip in (("dw_post", "d_res_scale", "dw_next"), ("dh",), ("d_gate",), ("d_scale",), ("d_res",), ("dw_next",),
                 ("dh", "d_gate", "d_scale", "dw_post", "d_res_scale")):
        part = c.backward(1e-5, y, skip=skip)
        assert set(part) == set(whole) - set(skip)
        assert all(torch.equal(part[n], whole[n]) for n in part), skip


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(dtype):
    """y over the residual, d_res over dy or dxn."""
    c = Case(dtype, 57, 1032, 3)
    y, xn = c.forward(1e-5)
    buf = c.d["residual"].clone()
    keep, c.d["residual"] = c.d["residual"], buf
    y2, xn2 = c.forward(1e-5, y=buf)
    c.d["residual"] = keep
    assert torch.equal(y, y2) and torch.equal(xn, xn2)
    whole = c.backward(1e-5, y)
    for name in ("dy", "dxn"):
        keep = c.d[name]
        c.d[name] = keep.clone()
        got = c.backward(1e-5, y, d_res=c.d[name])
        c.d[name] = keep
        assert all(torch.equal(got[n], whole[n]) for n in whole), name


def test_rows_outside_are_reported_and_count_as_zero():
    c = Case("bf16", 20, 264, 2)
    c.dst[[3, 10]] = [-1, 40]
    c.dst_d.copy_(torch.from_numpy(c.dst))
    L.moe_last_device_error()
    y, xn = c.forward(1e-5)
    assert L.moe_last_device_error() == L.MOE_ERR_DEVICE_BOUNDS
    o = c.backward(1e-5, y)
    assert L.moe_last_device_error() == L.MOE_ERR_DEVICE_BOUNDS
    assert L.moe_last_device_error() == L.MOE_OK
    # the same with a gate of zero on any row of the right size
    lost = [r for r in range(40) if r not in c.dst]
    c.dst[[3, 10]] = lost
    c.dst_d.copy_(torch.from_numpy(c.dst))
    c.d["gate"].view(-1)[[3, 10]] = 0
    y2, xn2 = c.forward(1e-5)
    o2 = c.backward(1e-5, y)
    assert torch.equal(y, y2) and torch.equal(xn, xn2)
    assert o["d_gate"].view(-1)[[3, 10]].tolist() == [0, 0]
    for n in ("d_res", "d_scale", "dw_post", "d_res_scale", "dw_next"):
        assert torch.equal(o[n], o2[n]), n


def test_empty_batch_clears_the_column_sums():
    c = Case("bf16", 0, 264, 2)
    c.forward(1e-5)
    o = c.backward(1e-5, torch.empty((0, 264), dtype=torch.bfloat16, device=DEV))
    assert all((o[n] == 0).all() for n in ("dw_post", "d_res_scale", "dw_next"))


def test_many_rows_and_the_same_bits_every_time():
    c = Case("bf16", 3001, 1032, 3)
    y, xn = check_forward(c, 1e-5)
    check_backward(c, 1e-5, y)
    a = c.backward(1e-5, y)
    for _ in range(3):
        y2, xn2 = c.forward(1e-5)
        b = c.backward(1e-5, y)
        assert torch.equal(y, y2) and torch.equal(xn, xn2) and all(torch.equal(a[n], b[n]) for n in a)


def test_offsets_past_32_bits():
    """Rows whose element offset in h passes 2^31 (bf16: 2^32 bytes and more)."""
    T, H, K = 140000, 2048, 8
    h = torch.zeros((T * K, H), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    last = torch.randn((64 * K, H), generator=g, device=DEV).to(torch.bfloat16)
    h[-64 * K:] = last
    gate = torch.rand((T, K), generator=g, device=DEV)
    res = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.rand((H,), generator=g, device=DEV)
    y, xn = torch.empty_like(res), torch.empty_like(res)
    L.moe_combine_norm(h, gate, None, None, res, w, None, w, 1e-5, T, H, K, L.MOE_BF16, y, xn)
    ys, xs = torch.empty_like(res[:64]), torch.empty_like(res[:64])
    tail = [res[-64:].contiguous(), gate[-64:].contiguous()]
    L.moe_combine_norm(last, tail[1], None, None, tail[0], w, None, w, 1e-5, 64, H, K, L.MOE_BF16, ys, xs)
    assert torch.equal(y[-64:], ys) and torch.equal(xn[-64:], xs) and torch.equal(y[:-64], res[:-64])
    dy = res
    dh, dg = torch.empty_like(h), torch.empty_like(gate)
    L.moe_combine_norm_bwd(dy, xn, h, gate, None, None, y, w, None, w, 1e-5, T, H, K, L.MOE_BF16, None, dh, dg, None, None,
                           None, None)
    dhs, dgs = torch.empty_like(last), torch.empty_like(tail[1])
    L.moe_combine_norm_bwd(tail[0], xs, last, tail[1], None, None, ys, w, None, w, 1e-5, 64, H, K, L.MOE_BF16, None, dhs, dgs,
                           None, None, None, None)
    assert torch.equal(dh[-64 * K:], dhs) and torch.equal(dg[-64:], dgs)


# rows that pass through the ring twice, and rows of 32 values a thread, over more tokens than
# the GPU has CTAs for, so that every CTA walks several
@pytest.mark.parametrize("size", [("bf16", 700, 8200, 2), ("f32", 400, 8196, 1), ("bf16", 350, 8192, 12), ("f32", 340, 5000, 8),
                                  ("bf16", 1500, 4096, 2)], ids=lambda s: "%s_T%d_H%d_K%d" % s)
def test_many_tokens_of_wide_rows(size):
    c = Case(*size, seed=5)
    y, _ = check_forward(c, 1e-5)
    check_backward(c, 1e-5, y)


@pytest.mark.parametrize("K", [1, 4])
def test_gradient_through_the_next_norm_alone(K):
    """No dy: the next block's norm is the only reader of y."""
    c = Case("bf16", 70, 520, K)
    y, _ = c.forward(1e-5)
    check_backward(c, 1e-5, y, skip=("dy",))


def test_two_streams_at_once():
    """Two calls that run at the same time, each with its own workspace, and the default stream behind them."""
    cases = [Case("bf16", 2000, 1032, 4, seed=s) for s in (1, 2)]
    alone = []
    for c in cases:
        y, xn = c.forward(1e-5)
        alone.append((y, xn, c.backward(1e-5, y)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                y, xn = c.forward(1e-5)
                got[i] = (y, xn, c.backward(1e-5, y))
    torch.cuda.synchronize()
    for a, g in zip(alone, got):
        assert torch.equal(a[0], g[0]) and torch.equal(a[1], g[1]) and all(torch.equal(a[2][n], g[2][n]) for n in a[2])


@pytest.mark.parametrize("opt", ["all", "post"])
@pytest.mark.parametrize("size", [("bf16", 1500, 1024, 8), ("bf16", 1000, 2048, 8), ("bf16", 500, 4096, 8), ("bf16", 700, 4096, 2),
                                  ("bf16", 320, 7168, 11), ("f32", 700, 3000, 5), ("f32", 320, 4096, 6)],
                         ids=lambda s: "%s_T%d_H%d_K%d" % s if isinstance(s, tuple) else s)
def test_more_tokens_than_ctas_at_every_depth_of_the_ring(size, opt):
    """Several tokens to a CTA, with none, 2 and 4 of the next one's rows on their way, and two passes over a token."""
    c = Case(*size, seed=size[3], **OPTIONS[opt])
    y, _ = check_forward(c, 1e-5)
    check_backward(c, 1e-5, y)
