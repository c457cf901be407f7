"""The gate, the fused norms and the checkpoint together, as a training step of whole MoE
blocks, against the oracle's chain in 64 bits; and the same step captured in a graph."""
import numpy as np
import pytest
import torch

import oracle as O
from token_dispatch_gb300 import _lib as L
from token_dispatch_gb300 import layer, synth
from tests.gpu_util import DEV, TOL, assert_close, dev, host_layer_inputs, to64

pytestmark = pytest.mark.gpu

SHAPE = synth.MoEShape("block_bf16_T333_H256_E32_K4_Hp192", 333, 256, 32, 4, 192, "bf16")
GATE = layer.GroupGate(groups=8, topk_groups=4, sigmoid=True, renorm=True, scale=2.5)
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    from token_dispatch_gb300 import build
    build.build()


def inputs(seed=0):
    x, wr, wg, wu, wd = host_layer_inputs(SHAPE, seed=seed)
    rng = np.random.default_rng(seed + 50)
    f = {n: (1 + 0.2 * rng.standard_normal(SHAPE.H)).astype(np.float32) for n in ("w_pre", "w_post", "res_scale", "w_next")}
    f["sel_bias"] = (0.05 * rng.standard_normal(SHAPE.E)).astype(np.float32)
    dy = synth.upstream_grad(SHAPE, SHAPE.T, SHAPE.H, seed=seed + 1)
    dxn = synth.upstream_grad(SHAPE, SHAPE.T, SHAPE.H, seed=seed + 2)
    return (x, wr, wg, wu, wd), f, dy, dxn


def device(stored, f):
    return [dev(a) for a in stored], {n: torch.from_numpy(a).to(DEV) for n, a in f.items()}


def forward(m, d, f, **kw):
    x, wr, wg, wu, wd = d
    layer.moe_block_forward(m, x, f["w_pre"], wr, f["sel_bias"], GATE, wg, wu, wd, f["w_post"], f["res_scale"], f["w_next"],
                            EPS, **kw)


def backward(m, d, f, dy, dxn, **kw):
    x, wr, wg, wu, wd = d
    layer.moe_block_backward(m, x, f["w_pre"], wr, GATE, wg, wu, wd, dy, dxn, f["w_post"], f["res_scale"], f["w_next"], EPS,
                             **kw)


def test_block_step_matches_oracle():
    stored, f, dy, dxn = inputs()
    d, fd = device(stored, f)
    m = layer.MoEBlockBuffers(SHAPE.T, SHAPE.H, SHAPE.E, SHAPE.K, SHAPE.Hp, "bf16", DEV, train=True)
    forward(m, d, fd)
    backward(m, d, fd, dev(dy), dev(dxn))
    assert L.moe_last_device_error() == L.MOE_OK
    b, K = m.moe, SHAPE.K
    x, wr, wg, wu, wd = (a.ref for a in stored)
    w = {n: a.astype(np.float64) for n, a in f.items()}
    # forward, each step from what the GPU stored before it
    x0 = O.combine_norm(None, None, None, 0, EPS, residual=x, w_next=w["w_pre"])[1]
    assert_close(to64(m.x0), x0, TOL["bf16"], "x0")
    x0 = to64(m.x0)
    logits = to64(b.logits)
    assert_close(logits, O.router_logits(x0, wr), 1e-5, "logits")
    idx, gate = O.gate_group(logits, K, 8, 4, True, w["sel_bias"], True, False, 2.5)
    assert np.array_equal(b.idx.cpu().numpy(), idx)
    assert_close(to64(b.gate), gate, 1e-5, "gate")
    cu, dst, src, xs = O.dispatch(x0, idx, SHAPE.E)
    assert np.array_equal(b.dst_row.cpu().numpy(), dst) and np.array_equal(to64(b.xs), xs)
    h = O.expert_ffn(xs, cu, wg, wu, wd)[1]
    assert_close(to64(b.h), h, TOL["bf16"], "h")
    opt = dict(w_post=w["w_post"], res_scale=w["res_scale"], w_next=w["w_next"])
    y, xn = O.combine_norm(h, gate, dst, K, EPS, residual=x, **opt)
    assert_close(to64(m.y), y, TOL["bf16"], "y")
    assert_close(to64(m.xn), xn, TOL["bf16"], "xn")
    # backward: the whole chain in 64 bits
    g = O.combine_norm_bwd(dy.ref, dxn.ref, h, gate, dst, K, EPS, y, **opt)
    assert_close(to64(b.dh), g["dh"], TOL["bf16"], "dh")
    assert_close(to64(b.d_gate), g["d_gate"], TOL["bf16"], "d_gate")
    for n in ("dw_post", "d_res_scale", "dw_next"):
        assert_close(to64(getattr(m, n)), g[n], TOL["bf16"], n)
    dxs, dwg, dwu, dwd = O.expert_ffn_bwd(xs, cu, wg, wu, wd, g["dh"])
    dl = O.gate_group_bwd(g["d_gate"], logits, idx, True, True, 2.5)
    assert_close(to64(b.d_logits), dl, TOL["bf16"], "d_logits")
    dx0 = dxs[dst].reshape(SHAPE.T, K, SHAPE.H).sum(axis=1) + dl @ wr.T
    for n, ref in (("dw_gate", dwg), ("dw_up", dwu), ("dw_down", dwd), ("dw_router", x0.T @ dl), ("dx", dx0)):
        assert_close(to64(getattr(b, n)), ref, TOL["bf16"], n)
    pre = O.combine_norm_bwd(g["d_res"], dx0, None, None, None, 0, EPS, x, w_next=w["w_pre"])
    assert_close(to64(m.d_x), pre["d_res"], TOL["bf16"], "d_x")
    assert_close(to64(m.dw_pre), pre["dw_next"], TOL["bf16"], "dw_pre")


def expert_bwd_of(g, u, xs, cu, wg, wu, wd, dh):
    """The expert backward at given g, u and rows."""
    s = 1 / (1 + np.exp(-g))
    act, dxs = g * s * u, np.zeros_like(xs)
    dw = [np.zeros_like(wg) for _ in range(3)]
    for e in range(len(wg)):
        r = slice(int(cu[e]), int(cu[e + 1]))
        da = dh[r] @ wd[e]
        dg, du = da * u[r] * s[r] * (1 + g[r] * (1 - s[r])), da * g[r] * s[r]
        dxs[r] = dg @ wg[e].T + du @ wu[e].T
        dw[0][e], dw[1][e], dw[2][e] = xs[r].T @ dg, xs[r].T @ du, dh[r].T @ act[r]
    return [dxs] + dw


def test_two_blocks_share_buffers_through_checkpoints():
    """Two layers through one MoEBuffers: the first one's expert activations come back from its
    checkpoint; the gradients are those at the checkpointed values, and near the exact ones."""
    (stored, f, dy, dxn), (stored2, f2, _, _) = inputs(), inputs(9)
    (d, fd), (d2, fd2) = device(stored, f), device(stored2, f2)
    one = layer.MoEBlockBuffers(SHAPE.T, SHAPE.H, SHAPE.E, SHAPE.K, SHAPE.Hp, "bf16", DEV, train=True)
    two = layer.MoEBlockBuffers(SHAPE.T, SHAPE.H, SHAPE.E, SHAPE.K, SHAPE.Hp, "bf16", DEV, train=True)
    ck = layer.ExpertCheckpoint(one.moe)
    forward(one, d, fd, ckpt=ck)
    b = one.moe
    gu, xs = to64(b.gu), to64(b.xs)
    # the second layer works in the first one's expert buffers
    for n in ("gu", "act", "xs", "dxs", "dw_gate", "dw_up", "dw_down", "ws_ffn", "ws_ffn_bwd"):
        setattr(two.moe, n, getattr(b, n))
    forward(two, [one.y] + d2[1:], fd2, x0=one.xn)
    backward(two, [one.y] + d2[1:], fd2, dev(dy), dev(dxn), x0=one.xn)
    backward(one, d, fd, two.d_x, two.moe.dx, ckpt=ck)
    assert L.moe_last_device_error() == L.MOE_OK
    rgu, rxs = O.ckpt_unpack(*O.ckpt_pack(gu)), O.ckpt_unpack(*O.ckpt_pack(xs))
    assert np.array_equal(to64(b.gu), rgu) and np.array_equal(to64(b.xs), rxs)
    Hp, cu = SHAPE.Hp, b.cu.cpu().numpy()
    wg, wu, wd = (a.ref for a in stored[2:])
    got = [to64(getattr(b, n)) for n in ("dxs", "dw_gate", "dw_up", "dw_down")]
    at = expert_bwd_of(rgu[:, :Hp], rgu[:, Hp:], rxs, cu, wg, wu, wd, to64(b.dh))
    exact = expert_bwd_of(gu[:, :Hp], gu[:, Hp:], xs, cu, wg, wu, wd, to64(b.dh))
    for n, a, r, e in zip(("dxs", "dw_gate", "dw_up", "dw_down"), got, at, exact):
        assert_close(a, r, TOL["bf16"], n)
        # each stored value is off by at most 2^-7 of the largest of its 32, and the gradients are
        # at most of third degree in them: well inside 3 * 2^-7 in the 2-norm
        assert np.linalg.norm(a - e) <= (3 * 2.0 ** -7 + TOL["bf16"]) * np.linalg.norm(e), n
    with pytest.raises(ValueError):
        layer.ExpertCheckpoint(layer.MoEBuffers(8, 64, 8, 2, 64, "bf16", DEV))


def test_graph_replay_of_a_block_step_is_bit_exact():
    stored, f, dy, dxn = inputs(3)
    d, fd = device(stored, f)
    dyd, dxnd = dev(dy), dev(dxn)
    m = layer.MoEBlockBuffers(SHAPE.T, SHAPE.H, SHAPE.E, SHAPE.K, SHAPE.Hp, "bf16", DEV, train=True)
    ck = layer.ExpertCheckpoint(m.moe)
    s = torch.cuda.Stream(device=DEV)
    s.wait_stream(torch.cuda.current_stream())

    def step():
        forward(m, d, fd, ckpt=ck, stream=s)
        backward(m, d, fd, dyd, dxnd, ckpt=ck, stream=s)
    step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s, capture_error_mode="relaxed"):
        step()
    new, _, dy2, dxn2 = inputs(77)
    d[0].copy_(dev(new[0]))
    dyd.copy_(dev(dy2))
    dxnd.copy_(dev(dxn2))
    outs = {n: getattr(m, n) for n in ("x0", "y", "xn", "d_x", "dw_pre", "dw_post", "d_res_scale", "dw_next")}
    outs.update({n: getattr(m.moe, n) for n in ("idx", "gate", "d_gate", "d_logits", "dx", "dw_router", "dw_gate", "dw_down")})
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    got = {n: t.clone() for n, t in outs.items()}
    for t in outs.values():
        t.fill_(7)
    torch.cuda.synchronize()
    step()
    s.synchronize()
    assert L.moe_last_device_error() == L.MOE_OK
    for n, t in outs.items():
        assert torch.equal(got[n], t), n


def test_block_of_one_token_serves():
    """A decoding step: one token, inference buffers, in place on the residual stream's y."""
    stored, f, _, _ = inputs()
    d, fd = device(stored, f)
    m = layer.MoEBlockBuffers(1, SHAPE.H, SHAPE.E, SHAPE.K, SHAPE.Hp, "bf16", DEV)
    big = layer.MoEBlockBuffers(SHAPE.T, SHAPE.H, SHAPE.E, SHAPE.K, SHAPE.Hp, "bf16", DEV)
    forward(big, d, fd)
    for t in (0, 200):
        forward(m, [d[0][t:t + 1].contiguous()] + d[1:], fd)
        assert torch.equal(m.x0[0], big.x0[t])
        assert_close(to64(m.moe.logits), to64(big.moe.logits[t:t + 1]), 1e-5, "logits")
        assert torch.equal(m.moe.idx[0], big.moe.idx[t])
        assert_close(to64(m.y), to64(big.y[t:t + 1]), TOL["bf16"], "y")
        assert_close(to64(m.xn), to64(big.xn[t:t + 1]), TOL["bf16"], "xn")


def test_blocks_that_share_expert_buffers():
    """Two blocks on one set of expert tensors, through checkpoints: every gradient is the bits of two blocks
    with tensors of their own; a backward whose activations are gone is refused."""
    (stored, f, dy, dxn), (stored2, f2, _, _) = inputs(), inputs(9)
    (d, fd), (d2, fd2) = device(stored, f), device(stored2, f2)
    dyd, dxnd = dev(dy), dev(dxn)
    size = (SHAPE.T, SHAPE.H, SHAPE.E, SHAPE.K, SHAPE.Hp, "bf16", DEV)

    def run(share):
        one = layer.MoEBlockBuffers(*size, train=True)
        two = layer.MoEBlockBuffers(*size, train=True, experts=one.moe if share else None)
        cks = [layer.ExpertCheckpoint(one.moe), layer.ExpertCheckpoint(two.moe)]
        forward(one, d, fd, ckpt=cks[0])
        forward(two, [one.y] + d2[1:], fd2, x0=one.xn, ckpt=cks[1])
        if share:
            assert two.moe.gu is one.moe.gu and two.moe.h is not one.moe.h
            with pytest.raises(ValueError):
                layer.MoEBlockBuffers(SHAPE.T - 1, *size[1:], train=True, experts=one.moe)
            with pytest.raises(ValueError):
                backward(one, d, fd, dyd, dxnd)
        backward(two, [one.y] + d2[1:], fd2, dyd, dxnd, x0=one.xn, ckpt=cks[1])
        backward(one, d, fd, two.d_x, two.moe.dx, ckpt=cks[0])
        assert L.moe_last_device_error() == L.MOE_OK
        return [getattr(b.moe, n) for b in (one, two) for n in
                ("d_gate", "d_logits", "dx", "dw_router", "dw_gate", "dw_up", "dw_down")] + \
            [getattr(b, n) for b in (one, two) for n in ("y", "xn", "d_x", "dw_post", "d_res_scale", "dw_next")] + \
            [one.dw_pre]
    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)
