"""The expert tensors' way together: gradients of a training step, the momentum step on the three tensors, the tensors
in 4 bits, and forwards that read them; the same in captured graphs, on streams of their own and past 32-bit offsets."""
import numpy as np
import pytest
import torch

import oracle as O
from token_dispatch_gb300 import _lib as L
from token_dispatch_gb300 import layer, synth
from tests.gpu_util import DEV, TOL, assert_close, dev, host_layer_inputs, to64
from tests.test_gpu_graph import bits
from tests.test_gpu_ortho import COEF, EPS, bound, matrices

pytestmark = pytest.mark.gpu

SHAPE = synth.MoEShape("bf16_T300_H256_E8_K2_Hp192", 300, 256, 8, 2, 192, "bf16")
LR, DECAY = 0.02, 0.1


@pytest.fixture(scope="module", autouse=True)
def built():
    from token_dispatch_gb300 import build
    build.build()


def sizes(T=SHAPE.T):
    return T, SHAPE.H, SHAPE.E, SHAPE.K, SHAPE.Hp, "bf16", DEV


def f32(v):
    return float(np.float32(v))


@pytest.mark.parametrize("masters", [False, True])
def test_train_update_pack_and_serve(masters):
    """A training step, its update, the packed tensors and a prompt and a decoding step through them, each against the
    oracle from what the step before it stored."""
    x, wr, wg, wu, wd = host_layer_inputs(SHAPE)
    xd, wrd = dev(x), dev(wr)
    low = [dev(w) for w in (wg, wu, wd)]  # what the forward reads
    w = [t.float() for t in low] if masters else low
    b = layer.MoEBuffers(*sizes(), train=True)
    muon = layer.ExpertMuon(b)
    old = [to64(t) for t in w]
    m_old = [np.zeros_like(a) for a in old]
    for step in range(2):
        layer.moe_forward(b, xd, wrd, None, *low)
        layer.moe_train_backward(b, xd, wrd, *low, dev(synth.upstream_grad(SHAPE, SHAPE.T, SHAPE.H, seed=step)))
        muon.step(b, *w, LR, DECAY, low=low if masters else (None, None, None))
        assert L.moe_last_device_error() == L.MOE_OK
        for k, (t, dw, m) in enumerate(zip(w, (b.dw_gate, b.dw_up, b.dw_down), (muon.m_gate, muon.m_up, muon.m_down))):
            g = to64(dw)
            scale = f32(0.2 * np.sqrt(max(SHAPE.H, SHAPE.Hp)))
            rw, rm, _ = O.muon_step(old[k], g, m_old[k], f32(0.95), True, f32(LR), f32(DECAY), scale, 5, *COEF, EPS)
            assert (np.abs(to64(m) - rm) <= 2.0 ** -23 * (np.abs(rm) + np.abs(m_old[k])) + 1e-30).all()
            u = g + f32(0.95) * rm
            for e in range(SHAPE.E):
                off = f32(LR) * scale * bound(u[e])[1] + (2.0 ** -22 if masters else 2.0 ** -8 + 2.0 ** -22) * \
                    (np.linalg.norm(rw[e]) + np.linalg.norm(old[k][e]) * 2.0 ** -14)
                assert np.linalg.norm(to64(t)[e] - rw[e]) <= off, (step, k, e)
            if masters:
                assert torch.equal(low[k], t.bfloat16())
            old[k], m_old[k] = to64(t), to64(m)
    # 4 bits: the packed form of the new weights, and what it stands for
    w4 = layer.ExpertsW4(SHAPE.E, SHAPE.H, SHAPE.Hp, DEV, group=32).pack(*w)
    back = [torch.empty_like(t) for t in low]
    w4.unpack(*back)
    ref = []
    for k, axis in enumerate((0, 0, 1)):
        q, s = O.w4_pack(old[k], axis, 32)
        ref.append(O.w4_unpack(q, s, axis, 32, old[k].shape[1 + axis]))
        assert np.array_equal(to64(back[k]), ref[k])
    for T in (SHAPE.T, 3, 1):  # a prompt, and decoding steps
        s = layer.MoEBuffers(*sizes(T), backward=False)
        layer.moe_forward(s, xd[:T], wrd, None, w4, None, None, route_flags=L.MOE_ROUTE_RENORM)
        assert L.moe_last_device_error() == L.MOE_OK
        idx = s.idx.cpu().numpy()
        cu, dst, src, xs = O.dispatch(x.ref[:T], idx, SHAPE.E)
        assert np.array_equal(s.dst_row.cpu().numpy(), dst) and np.array_equal(s.src_tok.cpu().numpy(), src)
        act, h = O.expert_ffn(xs, cu, *ref)[:2]
        assert_close(to64(s.act), act, TOL["bf16"], "act")
        assert_close(to64(s.h), h, TOL["bf16"], "h")
        y = (to64(s.gate)[:, :, None] * h[dst].reshape(T, SHAPE.K, SHAPE.H)).sum(axis=1)
        assert_close(to64(s.y), y, TOL["bf16"], "y")


def test_block_and_mod_forwards_with_packed_experts():
    """The forwards that take tensors give with the packed form what they give with the tensors it stands for."""
    x, wr, wg, wu, wd = host_layer_inputs(SHAPE)
    w4 = layer.ExpertsW4(SHAPE.E, SHAPE.H, SHAPE.Hp, DEV).pack(dev(wg), dev(wu), dev(wd))
    back = [torch.empty_like(dev(t)) for t in (wg, wu, wd)]
    w4.unpack(*back)
    ones = torch.ones(SHAPE.H, device=DEV)
    out = []
    for w in ((w4, None, None), back):
        m = layer.MoEBlockBuffers(*sizes())
        layer.moe_block_forward(m, dev(x), ones, dev(wr), None, layer.GroupGate(), *w, w_post=ones, w_next=ones)
        d = layer.MoDBuffers(3, 100, 50, *sizes()[1:], backward=False)
        layer.mod_forward(d, dev(x), torch.full((SHAPE.H,), 0.05, device=DEV).bfloat16(), dev(wr), *w)
        out.append((m.y, m.xn, d.y))
    assert L.moe_last_device_error() == L.MOE_OK
    for a, b in zip(*out):
        assert_close(to64(a), to64(b), TOL["bf16"])


def test_graph_replays_and_shared_workspaces():
    """A decoding step, and the momentum step of two layers that share a workspace, captured and replayed on
    new inputs: bit for bit what the calls give one by one."""
    x, wr, wg, wu, wd = host_layer_inputs(SHAPE)
    w4 = layer.ExpertsW4(SHAPE.E, SHAPE.H, SHAPE.Hp, DEV).pack(dev(wg), dev(wu), dev(wd))
    s = torch.cuda.Stream(device=DEV)
    bufs = [layer.MoEBuffers(*sizes(T), backward=False) for T in (1, SHAPE.T)]
    xd, wrd = dev(x).clone(), dev(wr)
    g, m, w = (torch.from_numpy(matrices(np.random.default_rng(k), 2, 200, 300)).float().to(DEV) for k in range(3))
    small = [t[:, :60, :64].contiguous() for t in (g, m, w)]
    n = L.moe_workspace_bytes(L.MOE_OP_MUON_STEP, 0, 200, 2, 0, 300)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    outs = [(torch.empty_like(t[2]), torch.empty_like(t[1])) for t in ((g, m, w), small)]

    def step():
        for b in bufs:
            layer.moe_forward(b, xd[:b.T], wrd, None, w4, None, None, stream=s)
        for (gg, mm, ww), (w_out, m_out) in zip(((g, m, w), small), outs):
            E, M, N = gg.shape
            L.moe_muon_step(ww, gg, mm, E, M, N, L.MOE_F32, 0.9, True, 0.1, 0.0, 1.0, 5, *COEF, EPS, w_out, None, m_out, ws,
                            n, stream=s)

    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s, capture_error_mode="relaxed"):
        step()
    xd.copy_(torch.randn(xd.shape, generator=torch.Generator().manual_seed(3)).bfloat16())
    g.mul_(-0.5)
    torch.cuda.synchronize()
    for _ in range(3):  # one replay behind the other: each kernel waits for the one before it
        graph.replay()
    torch.cuda.synchronize()
    assert L.moe_last_device_error() == L.MOE_OK
    tensors = [t for b in bufs for t in (b.act, b.h, b.y)] + [t for o in outs for t in o]
    got = [t.clone() for t in tensors]
    for t in tensors:
        t.fill_(7)
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    for a, b in zip(got, tensors):
        assert torch.equal(bits(a), bits(b))


def test_two_streams_at_once():
    """Calls on two streams with buffers of their own, many times over, give what each gives alone."""
    x, wr, wg, wu, wd = host_layer_inputs(SHAPE)
    w4 = layer.ExpertsW4(SHAPE.E, SHAPE.H, SHAPE.Hp, DEV).pack(dev(wg), dev(wu), dev(wd))
    xd, wrd = dev(x), dev(wr)
    u = torch.from_numpy(matrices(np.random.default_rng(1), 3, 260, 300)).float().to(DEV)
    n = L.moe_workspace_bytes(L.MOE_OP_ORTHOGONALIZE, 0, 260, 3, 0, 300)
    streams = [torch.cuda.Stream(device=DEV) for _ in range(2)]
    sets = [(layer.MoEBuffers(*sizes(T), backward=False), torch.empty((3, 260, 300), dtype=torch.bfloat16, device=DEV),
             torch.empty(n, dtype=torch.uint8, device=DEV)) for T in (SHAPE.T, 2)]

    def work(k):
        b, o, ws = sets[k]
        layer.moe_forward(b, xd[:b.T], wrd, None, w4, None, None, stream=streams[k])
        L.moe_orthogonalize(u, 3, 260, 300, L.MOE_F32, 5, *COEF, EPS, o, ws, n, stream=streams[k])
    torch.cuda.synchronize()
    alone = []
    for k in range(2):
        work(k)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in (sets[k][0].y, sets[k][0].act, sets[k][1])])
    for _ in range(20):
        work(0)
        work(1)
    torch.cuda.synchronize()
    assert L.moe_last_device_error() == L.MOE_OK
    for k in range(2):
        for a, t in zip(alone[k], (sets[k][0].y, sets[k][0].act, sets[k][1])):
            assert torch.equal(bits(a), bits(t))


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last matrix comes out as it does alone."""
    E, M, N = 2100, 1024, 1024
    w = torch.zeros((E, M, N), dtype=torch.bfloat16, device=DEV)
    w[0].normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    w[-1] = w[0].flip(0)
    q = torch.empty((E, N, M // 8), dtype=torch.int32, device=DEV)
    s = torch.empty((E, N, M // 32), dtype=torch.bfloat16, device=DEV)
    for axis in (0, 1):
        L.moe_w4_pack(w, E, M, N, axis, 32, L.MOE_BF16, q, s)
        last = w[-1:].clone()
        q1, s1 = torch.empty_like(q[:1]), torch.empty_like(s[:1])
        L.moe_w4_pack(last, 1, M, N, axis, 32, L.MOE_BF16, q1, s1)
        assert torch.equal(q[-1], q1[0]) and torch.equal(s[-1], s1[0])
        out = torch.full_like(w, 3)
        L.moe_w4_unpack(q, s, E, M, N, axis, 32, L.MOE_BF16, out)
        one = torch.empty_like(last)
        L.moe_w4_unpack(q1, s1, 1, M, N, axis, 32, L.MOE_BF16, one)
        assert torch.equal(out[-1], one[0]) and not out[1:-1].any()
    del q, s, out
    n = L.moe_workspace_bytes(L.MOE_OP_ORTHOGONALIZE, 0, M, E, 0, N)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    o = torch.empty_like(w)
    L.moe_orthogonalize(w, E, M, N, L.MOE_BF16, 1, *COEF, EPS, o, ws, n)
    assert L.moe_last_device_error() == L.MOE_OK
    want = torch.empty_like(last)
    L.moe_orthogonalize(last, 1, M, N, L.MOE_BF16, 1, *COEF, EPS, want, ws, n)
    # alone the sum X X^T runs over the same blocks in the same order: the same bits
    assert torch.equal(o[-1], want[0]) and not o[1:-1].any()
