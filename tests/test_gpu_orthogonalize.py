"""lora_orthogonalize against the steps on X itself in 64 bits.

Bounds.  The sums of G^T G add at most 2^9 terms one after the other in 64 bits:
2^-44 of the whole.  A step amplifies an error of the smallest directions by its
c0 and later ones again: at most 3e4 over 5 of the usual steps, and P is at most
485: 2^-44 * 1.5e7 < 2^-20 times the norm of a row of X.  fp32 results add one
rounding.  bf16: P enters in three parts (2^-24 with its fp32 rounding), and the
last sum adds 3 r products, a step each, of the sizes |X| |P|; one rounding."""
import pytest
import torch

from helpers_block import HALF, STEP32, within
from rank_adapter_gemm_amd import lora as L

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
USUAL = [(3.4445, -4.7750, 2.0315)] * 5
EPS = 1e-7


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


def gradients(n, rows, cols, dtype, seed=0, decades=2.0, ranks=None):
    """Matrices of singular values that fall by `decades`, ranks past a matrix's own zero."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + rows + 3 * cols)
    r, D = min(rows, cols), max(rows, cols)
    mix = torch.randn(n, r, r, generator=g, device="cuda") / r ** 0.5
    mix = mix * torch.pow(10.0, -decades * torch.arange(r, device="cuda") / r)[None, :, None]
    x = torch.matmul(torch.randn(n, D, r, generator=g, device="cuda"), mix) * 1e-3
    if ranks is not None:
        for i, k in enumerate(ranks):
            x[i, :, k:] = 0
    return (x if rows >= cols else x.transpose(1, 2)).contiguous().to(dtype)


def steps64(g, coef, eps, scale):
    """The result, and the bound's |X| |P| and row norms of X."""
    tall = g.shape[0] >= g.shape[1]
    x = g.double() / (g.double().norm() + eps)
    x0 = x if tall else x.t()
    x = x0
    m, p = x.t() @ x, None
    for a, b, c in coef:
        y = x @ (x.t() @ x)
        x = a * x + b * y + c * (y @ (x.t() @ x))
        q = a * torch.eye(m.shape[0], dtype=m.dtype, device=m.device) + b * m + c * (m @ m)
        p = q if p is None else p @ q
        m = q @ m @ q
    sizes, rows = x0.abs() @ p.abs() * abs(scale), x0.norm(dim=1, keepdim=True).expand_as(x0) * abs(scale)
    return [scale * x if tall else scale * x.t(), sizes if tall else sizes.t(), rows if tall else rows.t()]


def run(g, coef=USUAL, eps=EPS, scale=1.0, out=None, ws=None, **kw):
    n, rows, cols = g.shape
    out = torch.full_like(g, 7) if out is None else out
    if ws is None:
        ws = torch.empty(L.lora_workspace_bytes_orthogonalize(n, rows, cols), dtype=torch.uint8, device="cuda")
    L.lora_orthogonalize(g, n, rows, cols, L.dtype_code(g.dtype), coef, eps, scale, out, ws, **kw)
    return out


def check(out, g, coef=USUAL, eps=EPS, scale=1.0):
    half, r = HALF[g.dtype], min(g.shape[1:])
    for i in range(g.shape[0]):
        ref, sizes, rows = steps64(g[i], coef, eps, scale)
        tol = 2.0 ** -20 * rows + 4 * STEP32 * ref.abs()
        if g.dtype == BF16:
            tol = tol + (3 * r + 8) * STEP32 * sizes
        within(out[i], ref, tol * (1 + half) + half * ref.abs() + 2.0 ** -120, "matrix %d" % i)


SHAPES = [(1, 8, 8), (3, 16, 16), (2, 64, 8), (5, 520, 16), (2, 1032, 24), (3, 264, 32), (2, 4096, 40), (2, 2056, 64),
          (1, 776, 72), (2, 392, 96), (2, 1544, 128), (1, 128, 128), (1, 14336, 16), (70, 136, 8)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("n,D,r", SHAPES)
def test_steps(n, D, r, wide, dtype):
    g = gradients(n, r if wide else D, D if wide else r, dtype)
    check(run(g), g)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("wide", [False, True])
def test_ranks_past_a_matrix_s_own_and_zero_matrices_stay_zero(wide, dtype):
    ranks = [5, 0, 24, 1, 17]
    g = gradients(5, 24 if wide else 392, 392 if wide else 24, BF16, seed=3)
    for i, k in enumerate(ranks):
        (g[i, k:] if wide else g[i, :, k:]).zero_()
    g = g.to(dtype)
    out = run(g)
    check(out, g)
    for i, k in enumerate(ranks):
        assert not (out[i, k:] if wide else out[i, :, k:]).any()


@pytest.mark.parametrize("r", [8, 24, 64, 120])
@pytest.mark.parametrize("count", [1, 2])
def test_one_and_two_steps(r, count):
    for dtype, wide in ((BF16, False), (F32, True)):
        g = gradients(2, r if wide else 392, 392 if wide else r, dtype, seed=7)
        check(run(g, USUAL[:count]), g, USUAL[:count])


@pytest.mark.parametrize("n,D", [(300, 264), (1, 100000), (513, 24)])
def test_many_matrices_and_long_ones_of_one_tile(n, D):
    for dtype, wide in ((BF16, False), (BF16, True), (F32, True)):
        g = gradients(n, 16 if wide else D, D if wide else 16, dtype, seed=8)
        out, some = run(g), sorted({0, n // 3, n - 1})
        check(out[some], g[some])


@pytest.mark.parametrize("coef,scale", [([(1.0, 0.0, 0.0)], 1.0), ([(1.5, -0.5, 0.0)] * 9, 0.25),
                                        ([(2.0, -1.5, 0.5)] * 3, -3.0), ([(3.4445, -4.775, 2.0315), (1.5, -0.5, 0.0)], 2.0)])
def test_other_coefficients_and_counts(coef, scale):
    for dtype in (BF16, F32):
        g = gradients(3, 328, 40, dtype, seed=5, decades=1.0)
        check(run(g, coef, scale=scale), g, coef, scale=scale)


def test_singular_values_follow_the_polynomial():
    """16 cubic steps x -> 1.5 x - 0.5 x^3, each at most 1.5-fold: an error of 2^-44 of M grows to 2^-44 * 2.6e5 of P's
    directions (0.33 times the sum of 1.5^(2 k)), P is at most 657, and no singular value moves by more than the result's
    error: 1e-5, and 32 roundings of values below 1."""
    g = gradients(4, 1024, 32, F32, seed=6, decades=0.5)
    x = run(g, [(1.5, -0.5, 0.0)] * 16).double()
    want = torch.linalg.svdvals((g.double() / (g.double().norm(dim=(1, 2), keepdim=True) + EPS)).cpu())
    for _ in range(16):
        want = 1.5 * want - 0.5 * want ** 3
    got = torch.linalg.svdvals(x.cpu())
    err = float((got.sort(dim=1).values - want.sort(dim=1).values).abs().max())
    assert err < 1e-5 + 32 * 2.0 ** -24, err


def test_sizes_of_values_do_not_matter():
    """Gradients of 1e-30 and 1e30 beside ordinary ones (the squares of either are no fp32 numbers)."""
    g = gradients(3, 264, 16, F32, seed=7)
    g[1] *= 1e30
    g[2] *= 1e-30
    out = run(g, eps=1e-38)
    check(out, g, eps=float(torch.tensor(1e-38)))


def test_matrices_keep_to_themselves():
    g = gradients(4, 520, 16, BF16, seed=8)
    ref = run(g)
    g[1, 7, 3], g[2, 100, 15] = float("nan"), float("inf")
    out = run(g)
    assert torch.isnan(out[1]).all() and torch.isnan(out[2]).all()
    assert torch.equal(out[0], ref[0]) and torch.equal(out[3], ref[3])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1032, 40), (40, 1032), (16, 4104), (520, 128)])
def test_in_place_and_matrices_past_n_stay(rows, cols, dtype):
    g = gradients(3, rows, cols, dtype, seed=9)
    ref = run(g)
    h = torch.cat([g, torch.full_like(g[:1], 5)])
    ws = torch.empty(L.lora_workspace_bytes_orthogonalize(3, rows, cols), dtype=torch.uint8, device="cuda")
    L.lora_orthogonalize(h, 3, rows, cols, L.dtype_code(dtype), USUAL, EPS, 1.0, h, ws)
    assert torch.equal(h[:3], ref) and (h[3] == 5).all()
    L.lora_orthogonalize(h, 0, rows, cols, L.dtype_code(dtype), USUAL, EPS, 1.0, h, ws)
    assert torch.equal(h[:3], ref)


def test_deterministic_on_another_stream_and_in_graphs_that_share_a_workspace():
    a, b = gradients(6, 2056, 16, BF16, seed=10), gradients(3, 64, 1544, F32, seed=11)
    ra, rb = run(a), run(b)
    ws = torch.empty(max(L.lora_workspace_bytes_orthogonalize(*t.shape) for t in (a, b)), dtype=torch.uint8,
                     device="cuda")
    oa, ob = torch.empty_like(a), torch.empty_like(b)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    run(a, out=oa, ws=ws, stream=st)
    run(b, out=ob, ws=ws, stream=st)
    st.synchronize()
    assert torch.equal(oa, ra) and torch.equal(ob, rb)
    graphs = []
    for g, o in ((a, oa), (b, ob)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(g, out=o, ws=ws)
        graphs.append(graph)
    for _ in range(3):
        for t in (oa, ob):
            t.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, ra) and torch.equal(ob, rb)
    a.copy_(a.roll(1, 0).clone())                            # other gradients in the same buffer
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, ra.roll(1, 0))


def test_writes_stay_in_bounds():
    for n, rows, cols, dtype in [(1, 8, 8, BF16), (3, 72, 8, F32), (2, 24, 136, BF16), (1, 40, 1032, F32),
                                 (2, 264, 72, BF16), (1, 128, 520, BF16)]:
        g = gradients(n, rows, cols, dtype)
        raw = []

        def new(size):
            t = torch.full((size + 8192 + 256,), 0x5a, dtype=torch.uint8, device="cuda")
            raw.append((t, size))
            return t[4096:4096 + size]

        out = new(g.numel() * g.element_size()).view(dtype).view(g.shape)
        ws = new(L.lora_workspace_bytes_orthogonalize(n, rows, cols))
        check(run(g, out=out, ws=ws), g)
        assert all((t[:4096] == 0x5a).all() and (t[4096 + k:] == 0x5a).all() for t, k in raw)


def test_the_binding_refuses_tensors_the_kernels_would_misread():
    g = gradients(2, 64, 16, BF16)
    out = torch.empty_like(g)
    ws = torch.empty(L.lora_workspace_bytes_orthogonalize(2, 64, 16), dtype=torch.uint8, device="cuda")
    for other in (g.float(), g.cpu(), g.transpose(1, 2), g[:1]):
        for pair in ((other, out), (g, other)):
            with pytest.raises(L.LoraError) as e:
                L.lora_orthogonalize(pair[0], 2, 64, 16, L.LORA_BF16, USUAL, EPS, 1.0, pair[1], ws)
            assert e.value.status == L.LORA_ERR_INVALID_ARGUMENT
    with pytest.raises(L.LoraError):
        L.lora_orthogonalize(g, 2, 64, 16, L.LORA_BF16, [(1.0, 2.0)], EPS, 1.0, out, ws)
