"""The workspace of moe_orthogonalize and moe_muon_step is what the header states.  CPU only (152 SMs are assumed without a
GPU)."""
import pytest

PARTS = 76  # pairs of SMs


@pytest.fixture(scope="module")
def L():
    from token_dispatch_gb300 import build
    build.build()
    from token_dispatch_gb300 import _lib
    return _lib


def up(v, k):
    return -(-v // k) * k


@pytest.mark.parametrize("E,M,N", [(1, 1, 1), (64, 8, 8), (1, 64, 7168), (1, 16, 4096), (1, 1, 65536), (1, 7168, 384),
                                   (1, 300, 4800), (8, 128, 256), (3, 1001, 777), (64, 2048, 1408), (8, 4096, 14336),
                                   (25, 200, 9000), (26, 200, 9000), (2, 1024, 65536), (1, 65536, 65536)])
def test_workspace_is_what_the_header_says(L, E, M, N):
    m, n = sorted((M, N))
    got = L.moe_workspace_bytes(L.MOE_OP_ORTHOGONALIZE, 0, M, E, 0, N)
    assert got == L.moe_workspace_bytes(L.MOE_OP_MUON_STEP, 0, M, E, 0, N)
    matrices = E * (4 * m * (up(n, 64) + up(m, 64)) + 8 * up(m, 64) + 6152)
    tiles = E * (-(-m // 256)) * (-(-m // 256) + 1) // 2
    rest = got - matrices
    if tiles <= 25 and n >= 3 * 8 * 64:  # at least three parts of eight blocks of 64
        assert 0 <= rest <= PARTS * 4 * 256 * 256 + 2304
    else:
        assert 0 <= rest <= 2304  # nine parts, each on a boundary of 256 bytes
    if m >= 1024:
        assert got <= 8.3 * E * M * N + PARTS * 4 * 256 * 256
