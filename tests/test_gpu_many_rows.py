"""Batches whose rows need more than 2^32 threads in one grid dimension (a
launch of that size runs a part of its workgroups without an error).  Small
whole numbers, so every sum is exact and every row is compared."""
import numpy as np
import pytest
import torch

from rank_adapter_gemm_amd import lora as L

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()
    torch.cuda.empty_cache()


def needs(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb * 1e9:
        pytest.skip("not enough free memory")


def whole(*shape, dtype=BF16, most=3, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


def two_slots(T, d, f, dtype):
    """A pool of two adapters of rank 8 (scale 1), and ids -1, 0, 1 in turn."""
    pool = L.AdapterPool(2, d, f, 8, dtype)
    A, B = whole(2, d, 8, dtype=dtype, seed=1), whole(2, 8, f, dtype=dtype, seed=2)
    for s in range(2):
        pool.upload(s, A[s], B[s], 8, 8.0)
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) % 3) - 1
    return pool, A, B, ids


def rank_vectors(x, A, ids, a=0, b=None):
    """x A of every row's own adapter, rows a to b."""
    xs, ix = x[a:b].float(), ids[a:b]
    return sum((xs @ A[s].float()) * (ix == s)[:, None] for s in range(2))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_shrink_by_rows(dtype):
    T = (1 << 23) + 700                                    # 512 threads a row
    pool, A, _, ids = two_slots(T, 8, 8, dtype)
    x = whole(T, 8, dtype=dtype)
    ws = L.Workspace(T, 2, 8)
    v = torch.full((T, 8), 7.5, device="cuda")
    L.lora_shrink(x, T, pool.pool, ids, L.LORA_MODE_BGMV, v, ws.buf)
    assert torch.equal(v, rank_vectors(x, A, ids))


def test_f32_pair_in_adapter_order():
    """AUTO on this many rows: the rank vectors by rows, through the segments' order."""
    T = (1 << 23) + 700
    pool, A, B, ids = two_slots(T, 8, 8, F32)
    x, W = whole(T, 8, dtype=F32), [whole(8, 8, dtype=F32, seed=3 + i) for i in range(2)]
    h, g, u = (torch.full((T, 8), 7.5, device="cuda") for _ in range(3))
    ws = L.Workspace(T, 2, 8, gated=True)
    L.lora_gated_forward(x, W[0], W[1], h, T, [pool.pool, pool.pool], ids, L.LORA_ACT_SILU, L.LORA_MODE_AUTO, 0, ws.buf,
                         gate=g, up=u)
    delta = sum((rank_vectors(x, A, ids) @ B[s]) * (ids == s)[:, None] for s in range(2))
    assert torch.equal(g, x @ W[0] + delta) and torch.equal(u, x @ W[1] + delta)


def test_fp8_layer_by_rows():
    """The FP8 layer's rank vectors and codes in one launch (512 threads a row)."""
    T, d = (1 << 23) + 700, 16
    pool, A, B, ids = two_slots(T, d, 8, BF16)
    x = whole(T, d, most=3)
    W = torch.zeros(d, 8, dtype=BF16, device="cuda")
    w = L.Fp8Weight(W)
    y = torch.full((T, 8), 7.5, dtype=BF16, device="cuda")
    ws = L.Workspace(T, 2, 8, 8, fp8_d_in=d)
    L.lora_linear_forward_fp8(x, w.codes, w.scale, y, T, pool.pool, ids, L.LORA_MODE_BGMV, 0, ws.buf)
    v = rank_vectors(x, A, ids)
    assert torch.equal(y, sum((v @ B[s].float()) * (ids == s)[:, None] for s in range(2)).to(BF16))


def test_fp8_rows():
    """Codes and scales of rows (256 threads each), alone and within the pair."""
    T, d = (1 << 24) + 300, 16
    x = whole(T, d, most=100)
    q, s = torch.full((T, d), 99, dtype=torch.uint8, device="cuda"), torch.full((T,), 7.5, device="cuda")
    L.lora_quantize_rows_fp8(x, T, d, q, s)
    m, e = torch.frexp(x.float().abs().amax(1))            # the smallest 2^e with amax <= 448 2^e = 0.875 2^(e + 9)
    want = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).int())
    assert torch.equal(s, torch.where(m > 0, want, s)) and float(s.max()) < 1
    assert torch.equal(q.view(torch.float8_e4m3fn).float(), (x.float() / s[:, None]).to(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_expand_by_rows(dtype):
    T = (1 << 24) + 300                                    # 256 threads a row
    pool, _, B, ids = two_slots(T, 8, 8, dtype)
    v = whole(T, 8, dtype=F32)
    y = torch.zeros(T, 8, dtype=dtype, device="cuda")
    ws = L.Workspace(T, 2, 8)
    L.lora_expand(v, T, pool.pool, ids, L.LORA_MODE_BGMV, y, ws.buf)
    assert torch.equal(y, sum((v @ B[s].float()) * (ids == s)[:, None] for s in range(2)).to(dtype))


def test_f32_gemm():
    """2^30 rows: 256 threads for every 64 rows."""
    needs(85)
    T = (1 << 30) + 192
    x, W = torch.zeros(T, 8, device="cuda"), whole(8, 8, dtype=F32, seed=3)
    near = [slice(0, 999), slice(T // 2, T // 2 + 999), slice(T - 4000, T)]
    for i, n in enumerate(near):
        x[n] = whole(x[n].shape[0], 8, dtype=F32, seed=10 + i)
    y = torch.full((T, 8), 7.5, device="cuda")
    L.lora_gemm(x, W, y, T, 8, 8, L.LORA_F32)
    for n in near:
        assert torch.equal(y[n], x[n] @ W)
    assert float(y[T // 4:T // 4 + 1000].abs().max()) == 0
    del x, y
    torch.cuda.empty_cache()


def test_grouped_shrink():
    """2^28 rows: 256 threads for every 16 rows."""
    needs(185)
    T = (1 << 28) + 64
    pool, A, _, ids = two_slots(T, 8, 8, BF16)
    x = torch.zeros(T, 8, dtype=BF16, device="cuda")
    near = [slice(0, 999), slice(T // 2, T // 2 + 999), slice(T - 4000, T)]
    for i, n in enumerate(near):
        x[n] = whole(x[n].shape[0], 8, seed=10 + i)
    ws = L.Workspace(T, 2, 8)
    L.lora_build_segments(ids, T, 2, 8, ws.buf)
    v = torch.full((T, 8), 7.5, device="cuda")
    L.lora_shrink(x, T, pool.pool, ids, L.LORA_MODE_SGMV, v, ws.buf)
    for n in near:
        assert torch.equal(v[n], rank_vectors(x, A, ids, n.start, n.stop))
    assert int((v == 7.5).sum()) == 0
    del v, ws, x
    torch.cuda.empty_cache()
