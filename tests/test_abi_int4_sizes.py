"""Sizes of a 4-bit product whose tile and chunk counts would pass 31 bits are refused on the
host (no GPU)."""
import ctypes

from deepseek_sequential_mtp_gb300 import build, lib as binding


def test_sizes_that_pass_31_bits():
    build.build()
    lib = binding.load()
    fake = ctypes.c_void_p(1 << 20)
    m = binding.Int4Matrix(1 << 20, 1 << 20, None)
    call = lambda N, K, R=1: lib.mtp_gemm_int4w(R, N, K, 128, fake, ctypes.byref(m), fake, 0, None)  # noqa: E731
    for N, K in ((1, 0x7FFFFFE0), (0x7FFFFFFF, 32), ((1 << 30) + 1, 32), (1, (1 << 30) + 32)):
        assert call(N, K) == 7 and call(N, K, 32) == 7
