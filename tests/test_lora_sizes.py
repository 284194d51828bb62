"""The adapter calls' sizes at the ends of their types: answered or refused, not wrapped
around."""
import ctypes as ct

import pytest

P = ct.c_void_p(16)
ARG, UNSUPPORTED = 1, 3
MAX = 2 ** 63 - 1


@pytest.fixture(scope="module")
def lib():
    from w4a4_bit_gemm_hq_b200 import build_lib
    build_lib.build()
    from w4a4_bit_gemm_hq_b200 import _lib
    return _lib.lib


def test_max_tiles_of_any_number_of_adapters(lib):
    from w4a4_bit_gemm_hq_b200 import hq
    for M in (1, 5, 64, 1000, 1 << 40):
        for n in (0, 1, M - 1, M, M + 1, MAX - 1, MAX):
            want = M // 64 + min(n + 1, M)
            assert lib.hq_lora_max_tiles(M, n) == want and hq.hq_lora_max_tiles(M, n) == want
    assert lib.hq_lora_max_tiles(MAX, 1) == MAX // 64 + 2


def test_workspace_that_no_size_holds(lib):
    assert lib.hq_lora_workspace_size(1 << 40, 256) == 1 << 50
    assert lib.hq_lora_workspace_size(MAX, 256) == 2 ** 64 - 1      # more than any buffer has


@pytest.mark.parametrize("M,n", [(4, MAX), (MAX, 4), (MAX, MAX), (1 << 40, 1000)])
def test_sizes_beyond_the_limits_are_refused(lib, M, n):
    assert lib.hq_lora_plan(P, M, n, ct.c_void_p(32), ct.c_void_p(48), None) == UNSUPPORTED
    got = lib.hq_lora_apply(P, 0, M, 256, 256, P, P, 128, n, 16, None, None, P, P, None, 0, P, 0, 128, P, 1 << 62, None)
    assert got == UNSUPPORTED


def test_results_over_the_input_with_another_stride_are_refused(lib):
    """Rows of Y over other tokens' rows of X, which may still be read."""
    def call(X, Y, ld_x, ld_y, yt):
        return lib.hq_lora_apply(X, 0, 4, 256, ld_x, P, P, 128, 3, 16, None, None, P, P, None, 0, Y, yt, ld_y, P, 1 << 20, None)
    X = ct.c_void_p(4096)
    assert call(X, X, 256, 128, 0) == ARG and call(X, X, 256, 264, 0) == ARG
    assert call(X, X, 256, 256, 2) == ARG                 # fp32 rows are twice as far apart
