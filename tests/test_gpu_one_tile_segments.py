"""AUTO batches of 512 to 1024 rows, whose segments one workgroup builds: the
GEMM's row order bit for bit, and the layer's result exactly (small whole
numbers), with segments on both sides of the short-segment border."""
import numpy as np
import pytest
import torch

from rank_adapter_gemm_amd import lora as L
from test_gpu_mixed import expected_gemm_order

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("T", [512, 700, 1024])
@pytest.mark.parametrize("S", [37, 1500, 16000])
@pytest.mark.parametrize("short_len", [1, 2, 16, 255])
def test_order_and_result(T, S, short_len):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rng = np.random.default_rng(T + S + short_len)
    lengths = [1] * 150 + [120, 90, 16, 15, 17] + list(rng.integers(2, 20, size=70))
    used = np.unique(np.concatenate([[0, S - 1], rng.integers(0, S, size=30)]))
    owners = rng.permutation(np.concatenate([rng.choice(used, size=len(lengths) - 30), [-1] * 30]))
    ids = np.repeat(owners, rng.permutation(lengths)).astype(np.int32)[:T]
    T = ids.size
    ids[[3, 400]] = [-7, S + 2]                        # bad ids count as -1 (base rows)
    d, f = 16, 72
    g = torch.Generator(device="cuda")
    g.manual_seed(short_len)
    whole = lambda *shape: torch.randint(-1, 2, shape, generator=g, device="cuda").to(BF16)  # noqa: E731
    x, W, A, B = whole(T, d), whole(d, f), whole(len(used), d, 8), whole(len(used), 8, f)
    pool = L.AdapterPool(S, d, f, 8, BF16)
    for i, s in enumerate(used):
        pool.upload(int(s), A[i], B[i], 8, 8.0)
    ids_dev = torch.as_tensor(ids, device="cuda")
    ws = L.Workspace(T, S, 8, f)
    y = torch.full((T, f), 7.5, dtype=BF16, device="cuda")
    L.lora_linear_forward(x, W, y, T, pool.pool, ids_dev, L.LORA_MODE_AUTO, L.LORA_FLAG_SHORT_SEGMENT(short_len),
                          ws.buf)
    seg = ws.segments(T)
    order, n_long = expected_gemm_order(ids, S, short_len)
    assert int(seg["n_fused"].cpu()[0]) == n_long
    assert np.array_equal(seg["gemm_perm"].cpu().numpy(), order)
    want = x.float() @ W.float()
    for i, s in enumerate(used):                       # sums of at most 16 + 128: exact in bf16
        t = torch.as_tensor(np.flatnonzero(ids == s), device="cuda")
        want[t] += (x[t].float() @ A[i].float()) @ B[i].float()
    assert torch.equal(y.float(), want)
    assert L.lora_get_device_error(ws.buf) == 3
