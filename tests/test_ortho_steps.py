"""lora_orthogonalize refuses steps whose c0 multiply a rounding of 64 bits to where it
shows, on the host: the calls return before anything is enqueued (the addresses are made up)."""
import ctypes

import pytest

from rank_adapter_gemm_amd import lora as L

A = [(1 << 40) + (i << 30) for i in range(3)]
STEP = (3.4445, -4.7750, 2.0315)


def call(coef, n=0, ws_bytes=0):
    flat = (ctypes.c_float * (3 * len(coef)))(*[c for step in coef for c in step])
    return L.load().lora_orthogonalize(A[0], n, 64, 16, L.LORA_F32, flat, len(coef), 1e-7, 1.0, A[1], A[2], ws_bytes, None)


@pytest.mark.parametrize("coef", [[(3.7, -4.0, 1.5)] * 16, [(-3.7, 4.0, -1.5)] * 16, [(1.1e9, 0.0, 0.0)], [(8.0, 0, 0)] * 11,
                                  [(0.01, 0, 0)] * 4 + [(8.0, 0, 0)] * 11, [(8.0, 0, 0)] * 11 + [(0.01, 0, 0)] * 5,
                                  [(3e38, 0, 0)] * 16])
def test_steps_past_64_bits_are_refused(coef):
    assert call(coef) == L.LORA_ERR_UNSUPPORTED
    assert call(coef, n=3, ws_bytes=1 << 20) == L.LORA_ERR_UNSUPPORTED


@pytest.mark.parametrize("coef", [[STEP] * 16, [(8.0, 0, 0)] * 10, [(1e9, 0, 0)], [(0.0, 1e30, 0)] * 16,
                                  [(8.0, 0, 0)] * 8 + [(0.01, 0, 0)] + [(8.0, 0, 0)] * 4, [(1e-30, 0, 0)] * 16])
def test_steps_within_64_bits_are_taken(coef):
    assert call(coef) == L.LORA_OK
