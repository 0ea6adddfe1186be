"""Weights in blocks of 128 are quantized up to the size at which their values can be had back."""
import ctypes

import pytest

from moe_expert_ffn_03_gb300 import binding as B, build

A = ctypes.c_void_p(256)                     # an aligned address; none is read
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def test_rows_of_all_matrices(lib):
    def quantize(E, N, w=A):
        return lib.moe_fp8_block_quantize_weights(w, 0, E, N, 16, A, A, None)

    def back(E, N, dst=A):
        return lib.moe_fp8_block_dequantize(A, A, B.FP8_FORMATS["tiles"], E * N, N, 16, dst, 0, 16, None)

    for E, N in ((2048, 2 ** 20), (65536, 2 ** 15), (65536, 2 ** 20), (2049, 2 ** 20)):
        assert back(E, N) == INVALID and quantize(E, N) == UNSUPPORTED, (E, N)
    # the sizes before those pass this check: the next one looks at the pointers
    for E, N in ((2047, 2 ** 20), (65535, 2 ** 15)):
        assert quantize(E, N, w=None) == INVALID and back(E, N, dst=None) == INVALID, (E, N)
        assert b"dst" in lib.moe_last_error_message()
