"""Sizes next to the 32-bit limit are refused before anything is launched, on fake addresses that nothing reads.
CPU only."""
import pytest

A = 1 << 20  # a fake, 16-byte aligned address


@pytest.fixture(scope="module")
def L():
    from token_dispatch_gb300 import build
    build.build()
    from token_dispatch_gb300 import _lib
    return _lib


def test_ckpt_rows_whose_last_run_passes_32_bits(L):
    pack, unpack, swiglu = L.lib().moe_ckpt_pack, L.lib().moe_ckpt_unpack, L.lib().moe_ckpt_swiglu
    f32, bf16 = L.MOE_F32, L.MOE_BF16
    for N, dtype in ((0x7ffffffc, f32), (0x7fffffe4, f32), (0x7ffffff8, bf16), (0x7fffffe8, bf16)):
        for rows in (0, 1, 3):
            assert pack(A, rows, N, dtype, A, A, None) == L.MOE_ERR_UNSUPPORTED, (N, rows)
            assert unpack(A, A, rows, N, dtype, A, None) == L.MOE_ERR_UNSUPPORTED, (N, rows)
    for Hp, dtype in ((0x3ffffffc, f32), (0x3ffffff4, f32), (0x3ffffff8, bf16)):
        for rows in (0, 1, 3):
            assert swiglu(A, A, rows, Hp, dtype, A, A, None) == L.MOE_ERR_UNSUPPORTED, (Hp, rows)
    # the last width whose runs are numbers of 32 bits
    assert pack(None, 0, 0x7fffffe0, bf16, None, None, None) == L.MOE_OK
    assert unpack(None, None, 0, 0x7fffffe0, f32, None, None) == L.MOE_OK
    assert swiglu(None, None, 0, 0x3ffffff0, bf16, None, None, None) == L.MOE_OK
