"""lora_add_rmsnorm and lora_add_rmsnorm_fp8 against the plain form in 64
bits.  Bounds: z is one fp32 sum and one rounding.  The sum of squares adds at
most 40 terms a thread (more for rows past 32768 values: d / 1024) and 10 + 16
partial sums, each off by a step; half of that enters 1 / sqrt, with six more
steps for the products, the division and the root; one rounding of y."""
import numpy as np
import pytest
import torch

from helpers_block import HALF, STEP32, within
from rank_adapter_gemm_amd import lora as L

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


def make(T, d, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 31 * T + d)
    x = torch.randn(T, d, generator=g, device="cuda").to(dtype)
    r = (3 * torch.randn(T, d, generator=g, device="cuda")).to(dtype)
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    return x, r, w


def plain(x, r, w, eps=EPS):
    z = x.double() + (r.double() if r is not None else 0)
    return z, z / torch.sqrt((z * z).mean(1, keepdim=True) + eps) * w.double()


def check(z_got, y_got, x, r, w, eps=EPS):
    z, y = plain(x, r, w, eps)
    half, d = HALF[x.dtype], x.shape[1]
    tol = (0.5 * (40 + d / 1024 + 26) + 6 + 2) * STEP32      # + 2: z's own fp32 sum
    if z_got is not None:
        within(z_got, z, (half + STEP32) * z.abs(), "z")
    within(y_got, y, (half + tol) * y.abs() + 2.0 ** -120, "y")


SIZES = [(1, 8), (1, 4096), (3, 16), (5, 504), (130, 512), (7, 1024), (64, 1032), (9, 2048), (33, 4104), (4, 8192),
         (3, 16384), (2, 16392), (2, 32768), (2, 32776), (1, 70000), (5000, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", SIZES)
def test_norm(T, d, dtype):
    x, r, w = make(T, d, dtype)
    z, y = torch.empty_like(x), torch.empty_like(x)
    L.lora_add_rmsnorm(x, r, w, EPS, T, d, L.dtype_code(dtype), z, y)
    check(z, y, x, r, w)
    y2 = torch.empty_like(x)                                 # no residual, nothing kept
    L.lora_add_rmsnorm(x, None, w, EPS, T, d, L.dtype_code(dtype), None, y2)
    check(None, y2, x, None, w)


@pytest.mark.parametrize("T,d", [(T, d) for T, d in SIZES if d % 16 == 0])
def test_codes_are_those_of_the_stored_rows(T, d):
    x, r, w = make(T, d, torch.bfloat16, seed=3)
    z, y = torch.empty_like(x), torch.empty_like(x)
    q, s = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    L.lora_add_rmsnorm_fp8(x, r, w, EPS, T, d, z, y, q, s)
    check(z, y, x, r, w)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    L.lora_quantize_rows_fp8(y, T, d, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    q3, s3 = torch.empty_like(q), torch.empty_like(s)        # codes only
    L.lora_add_rmsnorm_fp8(x, r, w, EPS, T, d, None, None, q3, s3)
    assert torch.equal(q, q3) and torch.equal(s, s3)


@pytest.mark.parametrize("d", [64, 1024, 4096, 40000])
def test_in_place(d):
    """The residual stream updated in place, y over x, and the other way round."""
    T = 37
    x, r, w = make(T, d, torch.bfloat16, seed=5)
    z, y = torch.empty_like(x), torch.empty_like(x)
    q, s = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    L.lora_add_rmsnorm_fp8(x, r, w, EPS, T, d, z, y, q, s)
    for swap in (False, True):
        xa, ra = x.clone(), r.clone()
        q2, s2 = torch.empty_like(q), torch.empty_like(s)
        zo, yo = (xa, ra) if swap else (ra, xa)
        L.lora_add_rmsnorm_fp8(xa, ra, w, EPS, T, d, zo, yo, q2, s2)
        assert torch.equal(zo, z) and torch.equal(yo, y) and torch.equal(q2, q) and torch.equal(s2, s)


def test_rows_keep_to_themselves():
    """Rows of zeros, of tiny and of huge values, and a row with NaN between them."""
    T, d = 9, 1032
    x, r, w = make(T, d, torch.bfloat16, seed=7)
    x[2] = 0
    r[2] = 0
    x[3] *= 2.0 ** -60
    r[3] *= 2.0 ** -60
    x[4] *= 2.0 ** 40
    r[4] *= 2.0 ** 40
    x[6, 17] = float("nan")
    z, y = torch.empty_like(x), torch.empty_like(x)
    L.lora_add_rmsnorm(x, r, w, EPS, T, d, L.LORA_BF16, z, y)
    assert torch.equal(y[2], torch.zeros_like(y[2])) and torch.isnan(y[6]).all()
    rest = torch.tensor([i for i in range(T) if i != 6], device="cuda")
    check(z[rest], y[rest], x[rest], r[rest], w)


def test_rows_past_the_batch_stay_and_no_rows_is_no_work():
    x, r, w = make(12, 256, torch.bfloat16, seed=9)
    z, y = torch.full_like(x, 5), torch.full_like(x, 5)
    L.lora_add_rmsnorm(x, r, w, EPS, 7, 256, L.LORA_BF16, z, y)
    assert (z[7:] == 5).all() and (y[7:] == 5).all()
    check(z[:7], y[:7], x[:7], r[:7], w)
    z.fill_(5)
    L.lora_add_rmsnorm(x, r, w, EPS, 0, 256, L.LORA_BF16, z, y)
    assert (z == 5).all()


def test_deterministic_on_another_stream_and_in_a_graph():
    T, d = 201, 4096
    x, r, w = make(T, d, torch.bfloat16, seed=11)
    q, s = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    z, y = torch.empty_like(x), torch.empty_like(x)
    L.lora_add_rmsnorm_fp8(x, r, w, EPS, T, d, z, y, q, s)
    ref = [t.clone() for t in (z, y, q, s)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for t in (z, y, q, s):
        t.zero_()
    torch.cuda.synchronize()
    L.lora_add_rmsnorm_fp8(x, r, w, EPS, T, d, z, y, q, s, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((z, y, q, s), ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lora_add_rmsnorm_fp8(x, r, w, EPS, T, d, z, y, q, s)
    for _ in range(3):
        for t in (z, y, q, s):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((z, y, q, s), ref))


def test_the_binding_refuses_tensors_the_kernels_would_misread():
    """Other types, strides, sizes and devices than the kernel reads."""
    x, r, w = make(6, 256, torch.bfloat16, seed=13)
    z, y = torch.empty_like(x), torch.empty_like(x)
    good = dict(x=x, r=r, w=w, z=z, y=y)
    wide = torch.empty(6, 512, dtype=torch.bfloat16, device="cuda")
    for name in good:
        for other in (x.float(), x.cpu(), wide[:, :256], wide[:, ::2], x[:0]):
            bad = dict(good, **{name: other})
            with pytest.raises(L.LoraError) as e:
                L.lora_add_rmsnorm(bad["x"], bad["r"], bad["w"], EPS, 6, 256, L.LORA_BF16, bad["z"], bad["y"])
            assert e.value.status == L.LORA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("d", [1792, 1800, 3584, 3592, 3600, 4088, 7168, 7184, 8176])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_widths_at_the_borders_of_the_thread_counts(d, dtype):
    """One vector a thread or two: the last widths of one count and the first of the next."""
    T = 11
    x, r, w = make(T, d, dtype, seed=d)
    z, y = torch.empty_like(x), torch.empty_like(x)
    L.lora_add_rmsnorm(x, r, w, EPS, T, d, L.dtype_code(dtype), z, y)
    check(z, y, x, r, w)
    if dtype == torch.bfloat16 and d % 16 == 0:
        z2, y2 = torch.empty_like(x), torch.empty_like(x)
        q, s = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
        q2, s2 = torch.empty_like(q), torch.empty_like(s)
        L.lora_add_rmsnorm_fp8(x, r, w, EPS, T, d, z2, y2, q, s)
        assert torch.equal(z, z2) and torch.equal(y, y2)
        L.lora_quantize_rows_fp8(y2, T, d, q2, s2)
        assert torch.equal(q, q2) and torch.equal(s, s2)
