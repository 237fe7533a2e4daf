"""The fp32 pair on more workgroups than one grid dimension holds threads for:
2^24 tiles of 32 x 64 are 2^32 threads, which takes an h of 137 GB."""
import pytest
import torch

from helpers_block import Pair, within
from rank_adapter_gemm_amd import lora as L

pytestmark = pytest.mark.gpu


def test_f32_grid_past_2_32_threads():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    d, f = 8, 28672
    T = ((1 << 24) // (f // 64) + 5) * 32 + 3
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < T * f * 4 + (8 << 30):
        pytest.skip("not enough free memory")
    p = Pair(T, d, f, [8, 3], 8, torch.float32, seed=41)
    h = torch.empty(T, f, dtype=torch.float32, device="cuda")
    # rows of the first tiles, of the middle, of the last 2^24th tiles and past them
    rows = torch.tensor([0, 33, T // 2, T - 200, T - 101, T - 4, T - 1], device="cuda")
    h[rows] = 7.0
    ws = L.Workspace(T, p.S, p.R, 0, gated=True)
    L.lora_gated_forward(p.x, p.W[0], p.W[1], h, T, p.desc, p.ids_dev, 0, L.LORA_MODE_BGMV, 0, ws.buf)
    got = h[rows].clone()
    del h, ws
    torch.cuda.empty_cache()
    few = Pair(len(rows), d, f, [8, 3], 8, torch.float32, seed=41, ids=p.ids[rows.cpu().numpy()])
    few.x, few.W, few.A, few.B, few.alphas = p.x[rows], p.W, p.A, p.B, p.alphas
    ref, tol, _, _ = few.forward64("silu")
    within(got, ref, tol, "rows")
