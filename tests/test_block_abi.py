"""Refusals of the gate, fused-norm and checkpoint calls: reported before anything
is launched, on fake addresses that nothing reads.  CPU only."""
import math

import pytest
import torch

A = 1 << 20  # a fake, 16-byte aligned address


@pytest.fixture(scope="module")
def L():
    from token_dispatch_gb300 import build
    build.build()
    from token_dispatch_gb300 import _lib
    return _lib


def test_gate_refusals(L):
    gate = L.lib().moe_gate
    ok = dict(logits=A, bias=None, T=4, E=64, K=6, G=8, KG=3, mode=0, scale=1.0, idx=A, gate=A)

    def st(**kw):
        a = dict(ok, **kw)
        return gate(a["logits"], a["bias"], a["T"], a["E"], a["K"], a["G"], a["KG"], a["mode"], a["scale"], a["idx"],
                    a["gate"], None)
    for bad in (dict(T=-1), dict(E=0), dict(E=1025, G=1, KG=1), dict(K=0), dict(K=17), dict(E=8, G=1, KG=1, K=9),
                dict(G=0), dict(G=7), dict(G=64, KG=8), dict(KG=0), dict(KG=9), dict(E=16, G=8, KG=2, K=5),
                dict(mode=2), dict(mode=0x40), dict(mode=-1), dict(scale=math.inf), dict(scale=math.nan),
                dict(logits=None), dict(idx=None), dict(gate=None)):
        assert st(**bad) == L.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(logits=A + 4), dict(bias=A + 8), dict(idx=A + 4), dict(gate=A + 4)):
        assert st(**bad) == L.MOE_ERR_MISALIGNED, bad
    assert st(T=1 << 28, K=16) == L.MOE_ERR_UNSUPPORTED
    assert st(T=0, logits=None, idx=None, gate=None) == L.MOE_OK


def test_gate_bwd_and_route_group_refusals(L):
    bwd = L.lib().moe_gate_bwd
    assert bwd(A, A, A, 0, 64, 6, 1, 1.0, A, None) == L.MOE_OK
    assert bwd(A, A, A, 4, 64, 6, 1 | L.MOE_GATE_GROUP_MAX | 4, 1.0, A, None) == L.MOE_ERR_INVALID_ARG
    assert bwd(None, A, A, 4, 64, 6, 1, 1.0, A, None) == L.MOE_ERR_INVALID_ARG
    assert bwd(A, A, A, 4, 64, 6, 1, 1.0, None, None) == L.MOE_ERR_INVALID_ARG
    assert bwd(A, A, A + 4, 4, 64, 6, 1, 1.0, A, None) == L.MOE_ERR_MISALIGNED
    rg = L.lib().moe_route_group
    f32, bf16 = L.MOE_F32, L.MOE_BF16
    assert rg(A, A, None, 4, 64, 64, 6, 7, 8, 3, 1, 1.0, A, A, A, None, 0, None) == L.MOE_ERR_INVALID_ARG
    assert rg(A, A, None, 4, 64, 64, 6, f32, 8, 3, 1, 1.0, None, A, A, None, 0, None) == L.MOE_ERR_INVALID_ARG
    assert rg(A, A, None, 4, 60, 64, 6, bf16, 8, 3, 1, 1.0, A, A, A, None, 0, None) == L.MOE_ERR_UNSUPPORTED
    assert rg(A, A, None, 4, 64, 60, 6, bf16, 1, 1, 1, 1.0, A, A, A, None, 0, None) == L.MOE_ERR_UNSUPPORTED
    assert rg(A, A, None, 1024, 2048, 32, 2, bf16, 8, 3, 1, 1.0, A, A, A, None, 0, None) == L.MOE_ERR_WORKSPACE
    rb = L.lib().moe_route_bwd
    mode = L.MOE_ROUTE_LOGIT_GRAD
    assert rb(mode, A, None, None, A, A, 4, 64, 8, 2, f32, A, A, A, A, 1 << 30, None) == L.MOE_ERR_INVALID_ARG
    assert rb(mode, A, None, None, A, A, 4, 64, 6, 2, f32, None, A, A, A, 1 << 30, None) == L.MOE_ERR_UNSUPPORTED
    assert rb(mode | L.MOE_ROUTE_GATE_RENORM, A, None, None, A, A, 4, 64, 8, 2, f32, None, A, A, A, 1 << 30,
              None) == L.MOE_ERR_INVALID_ARG


def test_combine_norm_refusals(L):
    fwd, bwd = L.lib().moe_combine_norm, L.lib().moe_combine_norm_bwd
    names = ("h", "gate", "dst_row", "row_scale", "residual", "w_post", "res_scale", "w_next", "eps", "T", "H", "K",
             "dtype", "y", "xn")
    ok = dict(zip(names, [A] * 8 + [1e-5, 4, 64, 2, L.MOE_BF16, A, A]))

    def st(**kw):
        return fwd(*[dict(ok, **kw)[n] for n in names], None)
    alone = dict(h=None, gate=None, dst_row=None, row_scale=None, w_post=None, res_scale=None, K=0, y=None)
    for bad in (dict(T=-1), dict(H=0), dict(K=17), dict(K=-1), dict(dtype=5), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=math.nan), dict(eps=math.inf), dict(h=None), dict(K=0), dict(y=None), dict(xn=None),
                dict(w_next=None), dict(alone, y=A), dict(alone, gate=A), dict(alone, residual=None),
                dict(alone, w_next=None, xn=None)):
        assert st(**bad) == L.MOE_ERR_INVALID_ARG, bad
    for n in ("h", "gate", "dst_row", "row_scale", "residual", "w_post", "res_scale", "w_next", "y", "xn"):
        assert st(**{n: A + 4}) == L.MOE_ERR_MISALIGNED, n
    for bad in (dict(H=68), dict(H=16392), dict(H=66, dtype=L.MOE_F32), dict(T=1 << 30)):
        assert st(**bad) == L.MOE_ERR_UNSUPPORTED, bad
    assert st(T=0) == L.MOE_OK

    names = ("dy", "dxn", "h", "gate", "dst_row", "row_scale", "y", "w_post", "res_scale", "w_next", "eps", "T", "H", "K",
             "dtype", "d_res", "dh", "d_gate", "d_scale", "dw_post", "d_res_scale", "dw_next", "ws", "ws_bytes")
    need = L.moe_workspace_bytes(L.MOE_OP_COMBINE_NORM_BWD, 4, 64, 0, 2, 0)
    assert need >= 2 * 64 * 4
    okb = dict(zip(names, [A] * 10 + [1e-5, 4, 64, 2, L.MOE_BF16] + [A] * 8 + [need]))

    def stb(**kw):
        return bwd(*[dict(okb, **kw)[n] for n in names], None)
    alone = dict(h=None, gate=None, dst_row=None, row_scale=None, w_post=None, res_scale=None, K=0)
    for bad in (dict(eps=0.0), dict(dxn=None), dict(w_next=None), dict(y=None), dict(h=None), dict(w_post=None),
                dict(res_scale=None), dict(dy=None, dxn=None, w_next=None, dw_next=None),
                dict(alone, dw_post=None, d_res_scale=None)):
        assert stb(**bad) == L.MOE_ERR_INVALID_ARG, bad
    for n in ("dy", "dxn", "h", "y", "d_res", "dh", "d_gate", "d_scale", "dw_post", "d_res_scale", "dw_next", "ws"):
        assert stb(**{n: A + 4}) == L.MOE_ERR_MISALIGNED, n
    assert stb(ws_bytes=need - 1) == L.MOE_ERR_WORKSPACE
    assert stb(ws=None) == L.MOE_ERR_WORKSPACE
    assert L.moe_workspace_bytes(L.MOE_OP_COMBINE_NORM_BWD, 4, 0, 0, 2, 0) == 0


def test_ckpt_refusals(L):
    pack, unpack, swiglu = L.lib().moe_ckpt_pack, L.lib().moe_ckpt_unpack, L.lib().moe_ckpt_swiglu
    f32, bf16 = L.MOE_F32, L.MOE_BF16
    for call in (lambda x, r, n, t, q, s: pack(x, r, n, t, q, s, None),
                 lambda x, r, n, t, q, s: unpack(q, s, r, n, t, x, None)):
        for bad in ((None, 4, 64, bf16, A, A), (A, -1, 64, bf16, A, A), (A, 4, 0, bf16, A, A), (A, 4, 64, 9, A, A),
                    (A, 4, 64, bf16, None, A), (A, 4, 64, bf16, A, None)):
            assert call(*bad) == L.MOE_ERR_INVALID_ARG, bad
        for bad in ((A + 4, 4, 64, bf16, A, A), (A, 4, 64, bf16, A + 8, A), (A, 4, 64, bf16, A, A + 1)):
            assert call(*bad) == L.MOE_ERR_MISALIGNED, bad
        assert call(A, 4, 60, bf16, A, A) == L.MOE_ERR_UNSUPPORTED
        assert call(A, 4, 62, f32, A, A) == L.MOE_ERR_UNSUPPORTED
        assert call(None, 0, 64, bf16, None, None) == L.MOE_OK
    assert swiglu(A, A, 4, 0, bf16, A, A, None) == L.MOE_ERR_INVALID_ARG
    assert swiglu(A, A, 4, 1 << 30, bf16, A, A, None) == L.MOE_ERR_INVALID_ARG
    assert swiglu(None, A, 4, 64, bf16, A, A, None) == L.MOE_ERR_INVALID_ARG
    assert swiglu(A, A, 4, 64, bf16, A + 4, A, None) == L.MOE_ERR_MISALIGNED
    assert swiglu(A, A, 4, 60, bf16, A, A, None) == L.MOE_ERR_UNSUPPORTED
    assert swiglu(A, A, 4, 6, f32, A, A, None) == L.MOE_ERR_UNSUPPORTED
    assert swiglu(A, A, 4, 64, bf16, None, None, None) == L.MOE_OK  # nothing asked for


def test_the_binding_refuses_tensors_it_cannot_pass_on(L):
    """Host tensors, other types, strides and short buffers never reach a kernel."""
    f32 = torch.float32
    with pytest.raises(ValueError, match="logits is not on the current CUDA device"):
        L.moe_gate(torch.zeros(4, 8), None, 4, 8, 2, 1, 1, 0, 1.0, A, A, stream=0)

    class Fake:  # a tensor's face, on "device 0"
        is_cuda = True

        def __init__(self, shape, dtype, strides=None):
            self.t = torch.empty(shape, dtype=dtype)
            if strides:
                self.t = self.t.t()
            self.dtype, self.shape = dtype, self.t.shape

        def get_device(self):
            return 0

        def __getattr__(self, name):
            return getattr(self.t, name)
    real = torch.cuda.current_device
    torch.cuda.current_device = lambda: 0
    try:
        for bad, name in ((Fake((4, 8), torch.bfloat16), "logits"), (Fake((8, 4), f32, True), "logits"),
                          (Fake((4, 7), f32), "logits")):
            with pytest.raises(ValueError, match=name):
                L.moe_gate(bad, None, 4, 8, 2, 1, 1, 0, 1.0, A, A, stream=0)
        with pytest.raises(ValueError, match="dst_row"):
            L.moe_combine_norm(A, A, Fake((8,), torch.int64), None, None, None, None, None, 1e-5, 4, 64, 2, L.MOE_BF16,
                               A, None, stream=0)
        with pytest.raises(ValueError, match="scale"):
            L.moe_ckpt_pack(A, 4, 65 * 8, L.MOE_BF16, A, Fake((4, 16), torch.uint8), stream=0)
    finally:
        torch.cuda.current_device = real
    with pytest.raises(L.MoEError):
        L.moe_ckpt_pack(A, 4, 64, 7, A, A, stream=0)
