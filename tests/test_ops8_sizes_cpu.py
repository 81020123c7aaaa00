"""Sizes of the 8-bit entry points next to 2^31 (before any CUDA call)."""
import ctypes

import pytest

import dispatch_ffn_combine_gb300 as mk
from dispatch_ffn_combine_gb300 import build as cuda_build

A = ctypes.c_void_p(0x10000)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return mk.load_library()


@pytest.mark.parametrize("c", [(1 << 31) - 1, (1 << 31) - 64, (1 << 31) - 511, (1 << 31) - 512, 1 << 30])
def test_scale_rows_of_the_longest_rows(lib, c):
    assert lib.mk_moe_scale_pitch(c) == mk.scale_pitch(c) > 0


def _gemm8(lib, S, d, E, n, ws=None):
    return lib.mk_moe_grouped_gemm8(A, A, A, A, A, None, S, d, E, n, A, 0, ws, 0, None)


# Without a workspace an accepted size gives MK_ERR_WORKSPACE and a refused one its own status, with and without a GPU.
@pytest.mark.parametrize("S,d,E,n", [(1, 1 << 28, 1, 64), (1, (1 << 31) - 64, 1, 64), (1, 64, 1, 1 << 30),
                                     (1, 64, 1, (1 << 31) - 64), (1 << 25, 64, 1, 64), (1 << 24, 64, 1, 1 << 16)])
def test_product_refuses_what_its_counters_do_not_hold(lib, S, d, E, n):
    assert _gemm8(lib, S, d, E, n) == mk.MK_ERR_UNSUPPORTED


@pytest.mark.parametrize("S,d,E,n", [(8 * 131072, 7168, 256, 4096), (8 * 131072, 2048, 256, 7168), (320000, 7168, 256, 4096),
                                     ((1 << 25) - 1, 64, 8, 64), ((1 << 25) - 1, 16384, 8, 16384), (1, (1 << 28) - 64, 1, 64)])
def test_product_takes_the_rows_of_every_token_the_layer_takes(lib, S, d, E, n):
    """128K tokens of the large layer among them: eight rows each, more than 2^31 values."""
    assert _gemm8(lib, S, d, E, n) == mk.MK_ERR_WORKSPACE


@pytest.mark.parametrize("n,d", [(1 << 30, 64), (64, 1 << 30), (64, (1 << 31) - 64)])
def test_weights_quantiser_refuses_as_the_rows_do(lib, n, d):
    assert lib.mk_moe_quant8_weights(None, 1, n, d, A, A, None) == mk.MK_ERR_UNSUPPORTED
