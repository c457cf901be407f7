"""Refusals of the 4-bit weight and orthogonalised-update calls: reported before anything is
launched, on fake addresses that nothing reads.  CPU only."""
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


@pytest.mark.parametrize("call", ["moe_w4_pack", "moe_w4_unpack"])
def test_pack_refusals(L, call):
    f = getattr(L.lib(), call)
    ok = dict(w=A, E=2, rows=64, cols=72, axis=0, group=32, dtype=L.MOE_BF16, q=A, scale=A)

    def st(**kw):
        a = dict(ok, **kw)
        sizes = (a["E"], a["rows"], a["cols"], a["axis"], a["group"], a["dtype"])
        if call == "moe_w4_pack":
            return f(a["w"], *sizes, a["q"], a["scale"], None)
        return f(a["q"], a["scale"], *sizes, a["w"], None)
    for bad in (dict(E=0), dict(rows=0), dict(cols=-8), dict(axis=2), dict(axis=-1), dict(group=16), dict(group=0),
                dict(group=256), dict(dtype=2), dict(w=None), dict(q=None), dict(scale=None)):
        assert st(**bad) == L.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(w=A + 8), dict(q=A + 4), dict(scale=A + 2)):
        assert st(**bad) == L.MOE_ERR_MISALIGNED, bad
    for bad in (dict(rows=60), dict(cols=4), dict(dtype=L.MOE_F32, rows=62), dict(rows=(1 << 23) + 8), dict(E=65536)):
        assert st(**bad) == L.MOE_ERR_UNSUPPORTED, bad


def test_expert_ffn_w4_refusals(L):
    f = L.lib().moe_expert_ffn_w4
    ok = dict(x=A, src=None, T=0, cu=A, rows=4, qg=A, sg=A, qu=A, su=A, qd=A, sd=A, E=8, H=64, Hp=72, group=64,
              dtype=L.MOE_BF16, act=A, h=A, ws=None, n=0)

    def st(**kw):
        return f(*dict(ok, **kw).values(), None)
    for bad in (dict(rows=-1), dict(E=0), dict(H=0), dict(Hp=0), dict(T=-1), dict(group=48), dict(dtype=3), dict(cu=None),
                dict(qg=None), dict(sg=None), dict(qu=None), dict(su=None), dict(qd=None), dict(sd=None), dict(x=None),
                dict(act=None), dict(h=None), dict(src=A, T=0)):
        assert st(**bad) == L.MOE_ERR_INVALID_ARG, bad
    for name in ("x", "src", "cu", "qg", "sg", "qu", "su", "qd", "sd", "act", "h", "ws"):
        assert st(**{name: A + 4}, **({"T": 4} if name == "src" else {})) == L.MOE_ERR_MISALIGNED, name
    for bad in (dict(dtype=L.MOE_F32), dict(H=60), dict(Hp=68), dict(E=1025), dict(H=(1 << 20) + 8)):
        assert st(**bad) == L.MOE_ERR_UNSUPPORTED, bad
    assert st(rows=0, x=None, act=None, h=None) == L.MOE_OK


def test_orthogonalize_and_muon_refusals(L):
    o, m = L.lib().moe_orthogonalize, L.lib().moe_muon_step
    n = L.moe_workspace_bytes(L.MOE_OP_ORTHOGONALIZE, 0, 64, 2, 0, 72)
    assert n == L.moe_workspace_bytes(L.MOE_OP_MUON_STEP, 0, 64, 2, 0, 72) > 4 * 2 * 64 * 72
    assert L.moe_workspace_bytes(L.MOE_OP_ORTHOGONALIZE, 0, 0, 2, 0, 72) == 0
    base = dict(E=2, M=64, N=72, dtype=L.MOE_F32)
    newton = dict(steps=5, a=3.0, b=-4.0, c=2.0, eps=1e-7)

    def st_o(**kw):
        a = dict(dict(x=A, **base, **newton, out=A, ws=A, n=n), **kw)
        return o(*a.values(), None)

    def st_m(**kw):
        a = dict(dict(w=A, dw=A, m=A, **base, beta=0.9, nesterov=1, lr=0.1, wd=0.1, scale=1.0, **newton, w_out=A, w_low=A,
                      m_out=A, ws=A, n=n), **kw)
        return m(*a.values(), None)
    for st in (st_o, st_m):
        for bad in (dict(E=0), dict(M=0), dict(N=-1), dict(dtype=2), dict(steps=0), dict(steps=65), dict(a=math.nan),
                    dict(b=math.inf), dict(c=-math.inf), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf)):
            assert st(**bad) == L.MOE_ERR_INVALID_ARG, bad
        assert st(ws=A + 8) == L.MOE_ERR_MISALIGNED
        for bad in (dict(E=65536), dict(M=65537), dict(N=65537), dict(E=65535, M=65536, N=65536)):
            assert st(**bad) == L.MOE_ERR_UNSUPPORTED, bad
        for bad in (dict(ws=None), dict(n=n - 1), dict(n=0)):
            assert st(**bad) == L.MOE_ERR_WORKSPACE, bad
    assert st_o(x=None) == st_o(out=None) == L.MOE_ERR_INVALID_ARG
    assert st_o(x=A + 4) == st_o(out=A + 4) == L.MOE_ERR_MISALIGNED
    for bad in (dict(beta=1.0), dict(beta=-0.1), dict(beta=math.nan), dict(nesterov=2), dict(lr=math.inf),
                dict(wd=math.nan), dict(scale=math.inf), dict(w=None), dict(dw=None), dict(m=None), dict(w_out=None),
                dict(m_out=None)):
        assert st_m(**bad) == L.MOE_ERR_INVALID_ARG, bad
    for name in ("w", "dw", "m", "w_out", "w_low", "m_out"):
        assert st_m(**{name: A + 8}) == L.MOE_ERR_MISALIGNED, name


def test_bindings_check_tensors(L):
    w, q, s = torch.zeros(2, 16, 24), torch.zeros(2, 24, 16, dtype=torch.int32), torch.zeros(2, 24, 4).bfloat16()
    bf = w.bfloat16()
    for call in (lambda: L.moe_w4_pack(bf, 2, 16, 24, 0, 32, L.MOE_F32, q, s),
                 lambda: L.moe_w4_pack(w, 2, 16, 24, 0, 32, L.MOE_F32, q, s),  # not on the current CUDA device
                 lambda: L.moe_orthogonalize(w.transpose(1, 2), 2, 24, 16, L.MOE_F32, 5, 1.0, 0.0, 0.0, 0.0, bf),
                 lambda: L.moe_muon_step(w, w, w, 2, 16, 24, L.MOE_F32, 0.9, True, 0.1, 0.0, 1.0, 5, 1.0, 0.0, 0.0, 0.0, w,
                                         None, w)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(L.MoEError) as e:
        L.moe_w4_pack(A, 2, 16, 24, 0, 0, L.MOE_F32, A, A, stream=0)
    assert e.value.status == L.MOE_ERR_INVALID_ARG
