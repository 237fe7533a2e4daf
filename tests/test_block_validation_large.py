"""Backward passes whose rank octets would need a grid of 2^32 threads are
refused before anything is enqueued (made-up addresses; no GPU needed)."""
import ctypes

import pytest
import torch

from rank_adapter_gemm_amd import lora as L


def test_octets_past_2_32_threads():
    if torch.cuda.is_available():
        pytest.skip("made-up addresses stay off a GPU")
    lib = L.load()
    T, S, R, f = 16000, 16000, 8, 8
    at = lambda i: (1 << 44) + (i << 40)  # noqa: E731

    def call(d, dtype=L.LORA_BF16, dx=at(9)):
        p = (L.lora_pool_t * 2)()
        for m in range(2):
            p[m] = L.lora_pool_t(S, d, f, R, dtype, at(10 + m), at(12 + m), at(14 + m), at(16 + m))
        n = L.lora_workspace_bytes_gated_backward(T, S, R, d, f, dtype)
        assert 0 < n < 1 << 40
        return lib.lora_gated_backward(at(0), at(1), at(2), T, p, at(3), 0, at(4), at(5), at(6), dx,
                                       ctypes.POINTER(ctypes.c_void_p)(), ctypes.POINTER(ctypes.c_void_p)(), at(8), n, None)

    assert call(268800) == L.LORA_ERR_UNSUPPORTED              # 16000 x 268800 = 1.001 x 2^32
    # beside it the call gets as far as its first launch, which a host without a GPU reports
    assert call(268000) == call(268800, dx=None) == call(268800, dtype=L.LORA_F32) == L.LORA_ERR_HIP
