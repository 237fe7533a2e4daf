"""dweight and dbias of the layer norm's backward pass for rows so wide that their sums' workgroups (d = 2^29) or their
columns together (2^30) pass 32 bits.  Bounds: one row, so each sum is one value: dbias is dy itself, dweight one product
of dy and h (two roundings in fp32, steps of 2^-23), rounded once.  dx's two means add 2^20 values a thread one after
the other: at most 2^20 2^-24 of the mean of their sizes."""
import pytest
import torch

from rank_adapter_gemm_amd import lora as L

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("d", [(1 << 29) + 8, (1 << 30) + 24])
def test_rows_of_2_to_the_30_values(d):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    need = L.lora_workspace_bytes_layernorm_backward(1, d)
    if torch.cuda.mem_get_info()[0] < need + 20 * d:
        pytest.skip("not enough memory")
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    dy, z, w = (torch.randn(d, generator=g, device="cuda", dtype=BF16) for _ in range(3))
    mean, rstd = torch.full((1,), 0.25, device="cuda"), torch.full((1,), 1.5, device="cuda")
    dx, dw, db = (torch.full((d,), 77.0, device="cuda", dtype=BF16) for _ in range(3))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    L.lora_add_layernorm_backward(dy, None, z, w, mean, rstd, 1, d, L.LORA_BF16, dx, dw, db, ws)
    torch.cuda.synchronize()
    assert torch.equal(db, dy)
    parts = [slice(i, min(d, i + (1 << 26))) for i in range(0, d, 1 << 26)]
    ma = mah = size_a = size_ah = 0.0
    for p in parts:
        h, a = (z[p].float() - 0.25) * 1.5, dy[p].float() * w[p].float()
        ref = dy[p].float() * h
        assert ((dw[p].float() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -21)).all()
        ma, mah = ma + float(a.double().sum()), mah + float((a * h).double().sum())
        size_a, size_ah = size_a + float(a.abs().double().sum()), size_ah + float((a * h).abs().double().sum())
    ma, mah = ma / d, mah / d
    off = 2.0 ** -4 / d
    for p in parts:
        h, a = (z[p].float() - 0.25) * 1.5, dy[p].float() * w[p].float()
        ref = 1.5 * (a - ma - h * mah)
        tol = ref.abs() * 2.0 ** -8 + 1.6 * (off * size_a + h.abs() * off * size_ah + 2.0 ** -20 * (a.abs() + h.abs()))
        assert ((dx[p].float() - ref).abs() <= tol).all()
