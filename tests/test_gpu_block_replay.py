"""A captured call follows what its buffers hold at the replay: other rows,
other adapters of the rows (all of one, each its own, none), and a slot with
another adapter of another rank, as a server runs it; every replay is what an
eager call gives, bit for bit."""
import numpy as np
import pytest
import torch

from helpers_block import Pair, run_backward, run_forward
from rank_adapter_gemm_amd import lora as L
from test_gpu_gated import fp8_parts
from test_gpu_gated_backward import kept

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


def changes(p, seed=0):
    """Between replays: new ids, new rows and a smaller adapter in slot 0."""
    rng = np.random.default_rng(seed)
    for ids in (np.zeros(p.T), np.arange(p.T) % p.S, np.full(p.T, -1), np.sort(rng.integers(-1, p.S, size=p.T)),
                rng.integers(-2, p.S + 2, size=p.T)):
        p.ids_dev.copy_(torch.as_tensor(ids.astype(np.int32)))
        p.x.copy_(p.x.roll(1, 0).clone())
        for m in range(2):
            p.pools[m].upload(0, p.A[m][1], p.B[m][1], 1 + int(rng.integers(p.R)), 4.0, lda=p.R, ldb=p.f)
        torch.cuda.synchronize()
        yield


@pytest.mark.parametrize("T,dtype,fp8", [(5, BF16, False), (200, BF16, False), (1400, BF16, False), (40, BF16, True),
                                         (1400, BF16, True), (90, F32, False), (600, F32, False)])
def test_forward(T, dtype, fp8):
    p = Pair(T, 528, 776, [16, 16, 5, 9], 16, dtype, seed=T)
    parts = fp8_parts(p)[0] if fp8 else None
    ws, other = (L.Workspace(T, p.S, p.R, p.f, gated=True, fp8_d_in=p.d if fp8 else 0) for _ in range(2))
    h = torch.empty(T, p.f, dtype=dtype, device="cuda")

    def call():
        if fp8:                                           # the codes made within the call
            L.lora_gated_forward_fp8(p.x, None, None, parts[2][0].codes, parts[2][0].scale, parts[2][1].codes,
                                     parts[2][1].scale, h, T, p.desc, p.ids_dev, 0, 0, 0, ws.buf)
        else:
            L.lora_gated_forward(p.x, p.W[0], p.W[1], h, T, p.desc, p.ids_dev, 0, 0, 0, ws.buf)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in changes(p):
        h.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = run_forward(p, "silu", ws=other, fp8=parts, codes=False)[0]
        assert torch.equal(h, ref)
        assert L.lora_get_device_error(ws.buf) == L.lora_get_device_error(other.buf)


@pytest.mark.parametrize("T,dtype", [(5, BF16), (200, BF16), (1400, BF16), (90, F32)])
def test_backward(T, dtype):
    p = Pair(T, 528, 776, [16, 16, 5, 9], 16, dtype, seed=T)
    k = kept(p)
    ws, other = (L.Workspace(T, p.S, p.R, p.f, gated=True, backward_d_in=p.d, dtype=dtype) for _ in range(2))
    new = lambda *shape: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    dx, dA, dB = new(T, p.d), [new(p.S, p.d, p.R) for _ in range(2)], [new(p.S, p.R, p.f) for _ in range(2)]

    def call():
        L.lora_gated_backward(p.x, p.W[0], p.W[1], T, p.desc, p.ids_dev, 0, *k, dx, dA, dB, ws.buf)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in changes(p, 1):
        for t in [dx] + dA + dB:
            t.fill_(7)
        k[2].mul_(-0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = run_backward(p, "silu", *k, ws=other)
        assert torch.equal(dx, ref[0])
        for m in range(2):
            assert torch.equal(dA[m], ref[1][m]) and torch.equal(dB[m], ref[2][m])
        assert L.lora_get_device_error(ws.buf) == L.lora_get_device_error(other.buf)
