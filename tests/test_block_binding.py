"""Gradient lists of the binding's lora_gated_backward: two buffers each, refused
before anything else is looked at (no GPU needed)."""
import pytest

from rank_adapter_gemm_amd import lora as L

FAKE = 1 << 40


@pytest.mark.parametrize("dA,dB", [([FAKE], [FAKE, FAKE]), ([FAKE, FAKE], [FAKE]), ([FAKE] * 3, [FAKE] * 2),
                                   ([], [FAKE, FAKE]), ([FAKE, FAKE], [FAKE] * 4), ([FAKE, FAKE], None),
                                   (None, [FAKE, FAKE])])
def test_gradient_lists(dA, dB):
    p = L.lora_pool_t(4, 64, 96, 16, L.LORA_BF16, FAKE, FAKE, FAKE, FAKE)
    with pytest.raises(L.LoraError) as e:
        L.lora_gated_backward(FAKE, FAKE, FAKE, 8, [p, p], FAKE, 0, FAKE, FAKE, FAKE, FAKE, dA, dB, None)
    assert e.value.status == L.LORA_ERR_INVALID_ARGUMENT
