"""lora_orthogonalize on bf16 matrices of any size of value: scale / (|g| + eps) need be no fp32 number, nor
g times the polynomial.  Bounds as in test_gpu_orthogonalize.py: the steps see X alone, whose size is 1."""
import pytest
import torch

from rank_adapter_gemm_amd import lora as L
from test_gpu_orthogonalize import BF16, F32, check, gradients, run

pytestmark = pytest.mark.gpu
FLT_MIN = 2.0 ** -126


def fp32(x):
    return float(torch.tensor(x, dtype=torch.float32))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("r", [8, 24, 64, 128])
@pytest.mark.parametrize("eps,scale", [(FLT_MIN, 12.8), (2.0 ** -149, 3e38), (2.0 ** -149, -1.0), (1e-7, 3e38)])
def test_zero_matrices_stay_zero_for_any_eps_and_scale(eps, scale, r, wide, dtype):
    g = gradients(3, r if wide else 136, 136 if wide else r, dtype)
    g[1].zero_()
    assert not run(g, eps=eps, scale=scale)[1].any()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("r", [16, 32, 64, 128])
def test_values_near_the_ends_of_the_type(r, wide):
    """Entries of up to 1e-38 (most of them subnormal), 1e-30, 1e30, 1e36 and 1e38, and scales as far apart."""
    g = gradients(6, r if wide else 264, 264 if wide else r, F32, seed=12)
    for i, k in enumerate((1e-38, 1e-30, 1.0, 1e30, 1e36, 1e38)):
        g[i] = g[i].double() * (k / float(g[i].abs().max()))
    g = g.to(BF16)
    assert torch.isfinite(g).all()
    eps = fp32(1e-38)
    for scale in (1.0, -12.8, 1e-30, 3e38):
        check(run(g, eps=eps, scale=scale), g, eps=eps, scale=fp32(scale))


@pytest.mark.parametrize("r", [16, 40])
def test_infinite_and_nan_matrices_beside_zero_ones(r):
    g = gradients(4, 136, r, BF16, seed=13)
    g[0, 3, 2], g[1, 4, 1] = float("inf"), float("nan")
    g[2].zero_()
    out = run(g, eps=FLT_MIN, scale=12.8)
    assert torch.isnan(out[:2]).all() and not out[2].any()
    check(out[3:], g[3:], eps=FLT_MIN, scale=fp32(12.8))
