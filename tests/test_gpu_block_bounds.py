"""The block's calls write their outputs and the bytes that the workspace
functions name, and nothing beside them: buffers of exactly those sizes between
guard bytes."""
import numpy as np
import pytest
import torch

from helpers_block import Pair
from rank_adapter_gemm_amd import lora as L
from test_gpu_gated import fp8_parts
from test_gpu_gated_backward import kept

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
GUARD = 1 << 18


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


class Guarded:
    """Buffers with GUARD bytes of 0x5a on both sides."""

    def __init__(self):
        self.raw = []

    def __call__(self, *shape, dtype=torch.uint8):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((2 * GUARD + (n + 255) // 256 * 256,), 0x5a, dtype=torch.uint8, device="cuda")
        self.raw.append((raw, n))
        return raw[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self, what):
        for i, (raw, n) in enumerate(self.raw):
            assert bool((raw[:GUARD] == 0x5a).all()) and bool((raw[GUARD + n:] == 0x5a).all()), (what, i)


SHAPES = [(1, 64, 8, 1, 8), (33, 272, 136, 3, 16), (130, 784, 520, 200, 8), (300, 144, 7304, 4, 24),
          (700, 48, 40, 37, 64), (1025, 1040, 1400, 700, 16), (2047, 1808, 264, 5, 40)]


@pytest.mark.parametrize("T,d,f,S,R", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pair_and_backward(T, d, f, S, R, dtype):
    ranks = [(7 * i) % R + 1 for i in range(S)]
    for seed, ids in enumerate((None, np.arange(T) % S, np.full(T, S - 1), np.full(T, -1))):
        p = Pair(T, d, f, ranks, R, dtype, seed=seed, ids=ids, packed=seed == 1)
        k = kept(p)
        for mode in (L.LORA_MODE_AUTO, L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
            for split in (f, 0):                          # with and without room for pieces of K
                new = Guarded()
                ws = new(L.lora_workspace_bytes_gated(T, S, R, split))
                L.lora_workspace_init(ws)
                h, g, u = (new(T, f, dtype=dtype) for _ in range(3))
                L.lora_gated_forward(p.x, p.W[0], p.W[1], h, T, p.desc, p.ids_dev, 0, mode, 0, ws, gate=g, up=u)
                new.check("forward %d %d" % (mode, split))
        new = Guarded()
        n = L.lora_workspace_bytes_gated_backward(T, S, R, d, f, L.dtype_code(dtype))
        ws = new(n)
        L.lora_workspace_init(ws)
        dx = new(T, d, dtype=dtype)
        dA, dB = [new(S, d, R, dtype=dtype) for _ in range(2)], [new(S, R, f, dtype=dtype) for _ in range(2)]
        L.lora_gated_backward(p.x, p.W[0], p.W[1], T, p.desc, p.ids_dev, 0, *k, dx, dA, dB, ws)
        new.check("backward")


@pytest.mark.parametrize("T,d,f,S,R", [s for s in SHAPES if s[1] % 16 == 0])
def test_fp8_pair_and_norm(T, d, f, S, R):
    ranks = [(7 * i) % R + 1 for i in range(S)]
    for seed, ids in enumerate((None, np.arange(T) % S, np.full(T, -1))):
        p = Pair(T, d, f, ranks, R, BF16, seed=seed, ids=ids)
        wq = fp8_parts(p)[0][2]
        for mode in (L.LORA_MODE_AUTO, L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
            new = Guarded()
            ws = new(L.lora_workspace_bytes_gated_fp8(T, S, R, d, f))
            L.lora_workspace_init(ws)
            h, g, u = (new(T, f, dtype=BF16) for _ in range(3))
            L.lora_gated_forward_fp8(p.x, None, None, wq[0].codes, wq[0].scale, wq[1].codes, wq[1].scale, h, T, p.desc,
                                     p.ids_dev, 0, mode, 0, ws, gate=g, up=u)
            new.check("fp8 %d" % mode)
        new = Guarded()
        z, y, q, s = new(T, d, dtype=BF16), new(T, d, dtype=BF16), new(T, d), new(T, dtype=F32)
        L.lora_add_rmsnorm_fp8(p.x, p.x, p.x[0].contiguous(), 1e-6, T, d, z, y, q, s)
        new.check("norm")
