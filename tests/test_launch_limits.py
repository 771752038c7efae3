"""Sizes whose launch would need 2^32 threads or more, on the CPU: such a launch runs what is left
modulo 2^32 without an error, so the entry points refuse them before any HIP call."""
import fp8_delayed_scaling_amd as F

A16 = 1 << 20        # a fake 16-byte aligned address: never dereferenced, validation fails first
TILES_CAST, TILES = (1 << 22) - 1, (1 << 24) - 1        # of 256 x 256, on 1024 and on 256 threads


def test_casts():
    L = F.lib()
    for rows, cols in ((TILES_CAST * 256 + 1, 16), (16, TILES_CAST * 256 + 1), (1 << 19, 1 << 19)):
        assert L.fp8_cast_transpose(A16, rows, cols, A16, 0, A16, A16, None, None, None, None) == -2
        assert L.fp8_dbias_cast_transpose(A16, rows, cols, A16, 1, A16, A16, None, None, A16, A16, 1 << 60, None) == -2
    # the largest that fit go on to the next check
    for rows, cols in ((TILES_CAST * 256, 16), (16, TILES_CAST * 256)):
        assert L.fp8_cast_transpose(None, rows, cols, A16, 0, A16, A16, None, None, None, None) == -1
        assert L.fp8_dbias_cast_transpose(A16, rows, cols, A16, 1, A16, A16, None, None, None, A16, 1 << 60, None) == -1
    # zeros for the columns of no rows take four threads each
    assert L.fp8_dbias_cast_transpose(None, 0, 1 << 30, A16, 1, None, None, None, None, A16, None, 0, None) == -2


def test_transpose():
    L = F.lib()
    assert L.fp8_transpose(A16, TILES * 256 + 1, 16, A16, None, None) == -2
    assert L.fp8_transpose(None, TILES * 256, 16, A16, None, None) == -1


def test_gemm():
    L = F.lib()

    def gemm(M, N, K, A=None):
        return L.fp8_gemm_bias(A, 0, A16, max(K, 16), A16, 0, A16, max(K, 16), None, A16, N, 0, M, N, K, None)

    assert gemm((1 << 31) - 1, 512, 16, A16) == -2
    assert gemm((1 << 31) - 1, 256, 16) == -1
    # an empty contraction writes each output by a thread of its own
    assert gemm(1 << 20, 1 << 12, 0) == -2
    assert gemm(1 << 16, 1 << 16, 0) == -2


def test_linear():
    L = F.lib()

    def fwd(M, N, K):        # two tensors' tiles in one launch
        return L.fp8_linear_fwd(A16, A16, None, M, N, K, A16, None, None, None, A16, A16, None, A16, A16, A16, None, A16, None)

    assert fwd((1 << 29), 256, 256) == -2 and fwd(256, 1 << 29, 256) == -2
    assert fwd((1 << 29) - 256, 256, 256) == -1          # x8 is missing
    bwd = L.fp8_linear_bwd(A16, 1 << 30, 256, 256, A16, None, A16, A16, A16, None, None, 0, A16, A16, A16, A16, A16, A16, 0, None)
    assert bwd == -2
