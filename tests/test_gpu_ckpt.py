"""The 8-bit activation checkpoint on the GPU: integers, powers of two and restored
values equal to the oracle's bit for bit; silu(g) u within its roundings."""
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


def pack(x, dtype):
    rows, N = x.shape
    q = torch.full((rows, N), 99, dtype=torch.int8, device=DEV)
    s = torch.full((rows, -(-N // 32)), 99, dtype=torch.uint8, device=DEV)
    L.moe_ckpt_pack(x, rows, N, CDT[dtype], q, s)
    return q, s


def check(x, dtype):
    """x: host tensor in the storage type."""
    q, s = pack(x.to(DEV), dtype)
    rq, rs = O.ckpt_pack(to64(x))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    out = torch.full(x.shape, 7, dtype=x.dtype, device=DEV)
    L.moe_ckpt_unpack(q, s, *x.shape, CDT[dtype], out)
    want = torch.from_numpy(O.ckpt_unpack(rq, rs)).to(torch.float32).to(x.dtype)
    assert np.array_equal(to64(out), to64(want), equal_nan=True)
    return q, s


SIZES = [("bf16", 1, 8), ("f32", 1, 4), ("bf16", 3, 32), ("f32", 5, 36), ("bf16", 17, 72), ("bf16", 7, 1000),
         ("f32", 9, 2808), ("bf16", 33, 2816), ("f32", 2, 64), ("bf16", 300, 24), ("bf16", 2, 16408)]


@pytest.mark.parametrize("size", SIZES, ids=["%s_R%d_N%d" % s for s in SIZES])
def test_pack_and_unpack_match_oracle(size):
    dtype, rows, N = size
    rng = np.random.default_rng(N)
    x = rng.standard_normal((rows, N)) * np.exp(2 * rng.standard_normal((rows, 1)))
    x[rng.random((rows, N)) < 0.1] = 0
    check(synth.store(x, dtype).host, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_borders_of_the_power_of_two(dtype):
    """Largest magnitudes at 127 * 2^e, one step to either side, at every exponent the
    type has; halves; zeros; the smallest and largest numbers; infinities and NaN."""
    tdt = TDT[dtype]
    step = torch.finfo(tdt).eps * 64  # of values in [64, 128)
    rows = []
    for e in list(range(-133, 122)):
        for top in (127.0, 127.0 - step, 127.0 + step, 64.0, 128.0 - step):
            rows.append([float(np.ldexp(v, e)) for v in (top, -top, 0.5, 1.5, 2.5, -0.5, -1.5, 62.5, 63.5, 0.0, 1.0, 126.5)] +
                        [0.0] * 20)
    fi = torch.finfo(tdt)
    rows += [[0.0] * 32, [-0.0] * 32, [fi.max, 1.0] + [fi.tiny] * 30, [fi.tiny] * 32, [fi.smallest_normal / 2] * 32,
             [-fi.max] * 32]
    x = torch.tensor(rows, dtype=torch.float64).to(tdt)
    check(x, dtype)
    bad = torch.ones((3, 64), dtype=tdt)
    bad[0, 3], bad[1, 40], bad[2, 63] = float("inf"), float("nan"), -float("inf")
    q, s = check(bad, dtype)
    assert s.tolist() == [[255, 121], [121, 255], [121, 255]]


@pytest.mark.parametrize("size", [("bf16", 1, 8), ("f32", 3, 4), ("bf16", 65, 40), ("f32", 31, 1404), ("bf16", 129, 1408),
                                  ("bf16", 9, 5632), ("f32", 200, 20), ("bf16", 2, 14336)], ids=lambda s: "%s_R%d_Hp%d" % s)
def test_swiglu_of_the_checkpoint(size):
    dtype, rows, Hp = size
    rng = np.random.default_rng(Hp)
    x = rng.standard_normal((rows, 2 * Hp)) * np.exp(rng.standard_normal((rows, 1)))
    x[0, :] *= 30  # silu's tails
    gu = synth.store(x, dtype).host.to(DEV)
    q, s = pack(gu, dtype)
    r = O.ckpt_unpack(q.cpu().numpy(), s.cpu().numpy())
    g, u = r[:, :Hp], r[:, Hp:]
    ref = g / (1 + np.exp(-g)) * u
    got = [torch.full((rows, 2 * Hp), 7, dtype=TDT[dtype], device=DEV), torch.full((rows, Hp), 7, dtype=TDT[dtype], device=DEV)]
    L.moe_ckpt_swiglu(q, s, rows, Hp, CDT[dtype], *got)
    assert np.array_equal(to64(got[0]), to64(torch.from_numpy(r).to(torch.float32).to(TDT[dtype])))
    # expf and the quotient are within 2 ulp each, a sum and a product round: under 8 * 2^-24 = 2^-21; below
    # 2^-126 fp32 loses bits (2^-149, times |u|), then half a step of the type
    tol = (torch.finfo(TDT[dtype]).eps / 2 + 2.0 ** -20) * np.abs(ref) + 2.0 ** -125 * (1 + np.abs(u))
    assert (np.abs(to64(got[1]) - ref) <= tol).all()
    for keep in (0, 1):  # each output alone
        part = [torch.full_like(t, 7) if i == keep else None for i, t in enumerate(got)]
        L.moe_ckpt_swiglu(q, s, rows, Hp, CDT[dtype], *part)
        assert torch.equal(part[keep], got[keep])


def test_restored_infinities_reach_the_activation():
    gu = torch.ones((2, 128), dtype=torch.bfloat16)
    gu[0, 5] = float("inf")
    gu[1, 100] = float("nan")
    q, s = pack(gu.to(DEV), "bf16")
    act = torch.empty((2, 64), dtype=torch.bfloat16, device=DEV)
    L.moe_ckpt_swiglu(q, s, 2, 64, L.MOE_BF16, None, act)
    assert act.isnan().tolist() == [[True] * 32 + [False] * 32, [False] * 32 + [True] * 32]


def test_offsets_past_32_bits():
    rows, N = 80000, 28672  # 2.3e9 values
    x = torch.empty((rows, N), dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(3))
    q, s = pack(x, "bf16")
    q2, s2 = pack(x[-100:].contiguous(), "bf16")
    assert torch.equal(q[-100:], q2) and torch.equal(s[-100:], s2)
    gu, act = torch.empty_like(x), torch.empty((rows, N // 2), dtype=torch.bfloat16, device=DEV)
    L.moe_ckpt_swiglu(q, s, rows, N // 2, L.MOE_BF16, gu, act)
    gu2, act2 = torch.empty_like(gu[:100]), torch.empty_like(act[:100])
    L.moe_ckpt_swiglu(q2, s2, 100, N // 2, L.MOE_BF16, gu2, act2)
    assert torch.equal(gu[-100:], gu2) and torch.equal(act[-100:], act2)
    L.moe_ckpt_unpack(q, s, rows, N, L.MOE_BF16, x)
    assert torch.equal(x, gu)


def test_empty_batch_and_another_stream():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    q, s = pack(e, "bf16")
    L.moe_ckpt_unpack(q, s, 0, 64, L.MOE_BF16, e)
    L.moe_ckpt_swiglu(q, s, 0, 32, L.MOE_BF16, e, e)
    x = torch.randn((500, 1408), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    ref = pack(x, "bf16")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = pack(x, "bf16")
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    assert L.moe_last_device_error() == L.MOE_OK
