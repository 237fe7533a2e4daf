"""lora_orthogonalize over the steps it accepts, on matrices of fewer directions than columns (the gradient of an
adapter with fewer rows in the batch than ranks): against the steps on X in extended precision, on the CPU.

Bound, relative to the norm of the row of X = g / |g| that a result's row is made of.  Directions that a matrix does not
have hold the 64-bit roundings of its sums, and every step multiplies them by its c0.  growth: the largest product of c0
over steps up to the last.  16 steps of 4 products whose sums have r <= 72 terms, root of r roundings each, are at most 2^9
roundings on the way to one value, independent too: their root, 2^4.5, and 4 deviations: 2^-53 2^6.5 growth.  Where
the steps go on from M = X^T X alone, P's products lose their symmetry by growth^2 root(r) 2^-53 in a step (P is growth
where M is nothing, and M's part there is as far off), the steps before add 0.4 of it, and a tile stands for its mirror
image: 4 deviations of 3 products, 10 root(r) 2^-53 growth^2, and M is made anew before growth^2 passes 2^22.
The result is rounded once to its type, bf16 of up to 2^11 growth also in fp32 sums of 3 r
products: 4 root(3 r) 2^-24 growth.  The reference's own roundings (2^-64) are below 2^-10 of all that."""
import numpy as np
import pytest
import torch

from helpers_block import HALF, STEP32
from rank_adapter_gemm_amd import lora as L
from test_gpu_orthogonalize import BF16, EPS, F32, run

pytestmark = pytest.mark.gpu
STEP = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


def few_directions(kind, D, r, seed):
    rng = np.random.default_rng(seed)
    if kind == "rows":                                    # exactly so: three rows of values, zeros else
        g = np.zeros((D, r), np.float32)
        g[rng.choice(D, 3, replace=False)] = rng.standard_normal((3, r))
    elif kind == "repeated":                              # exactly so: four rows, over and over
        g = rng.standard_normal((4, r)).astype(np.float32)[rng.integers(0, 4, D)]
    elif kind == "graded":                                # down to 1e-8 of the largest
        u, v = (np.linalg.qr(rng.standard_normal((k, r)))[0] for k in (D, r))
        g = (u * 10.0 ** (-8 * np.arange(r) / r)) @ v.T
    else:                                                 # up to the type's rounding
        g = rng.standard_normal((D, kind)) @ rng.standard_normal((kind, r))
    return torch.from_numpy(np.asarray(g, np.float32)) * 1e-3


def steps_extended(g, coef, eps):
    x = g.double().numpy().astype(np.longdouble)
    x = x / (np.sqrt((x * x).sum()) + np.longdouble(np.float32(eps)))
    x0 = x
    for c in coef:
        a, b, c2 = (np.longdouble(np.float32(v)) for v in c)
        m = x.T @ x
        x = a * x + x @ (b * m + c2 * (m @ m))
    return x0, x


def check_range(dtype, kinds, D, r, wide, coef):
    g = torch.stack([few_directions(k, D, r, 10 * i + r) for i, k in enumerate(kinds)]).to(dtype)
    arg = (g.transpose(1, 2) if wide else g).contiguous().cuda()
    out = run(arg, coef).cpu().double()
    out = out.transpose(1, 2) if wide else out
    growth = 1.0
    for c in coef:
        growth = max(growth, 1.0) * abs(float(np.float32(c[0])))
    growth = max(growth, 1.0)
    for i, k in enumerate(kinds):
        x0, ref = steps_extended(g[i], coef, EPS)
        ref = ref.astype(np.float64)
        rows = np.sqrt((x0 * x0).sum(1, keepdims=True)).astype(np.float64)
        tol = 2.0 ** -53 * (2.0 ** 6.5 * growth + 10 * r ** 0.5 * min(growth ** 2, 2.0 ** 22)) * rows
        tol = tol + 4 * STEP32 * np.abs(ref)
        if dtype == BF16 and growth <= 2048:              # products of P in parts, in fp32 sums
            tol = tol + 4 * (3 * r) ** 0.5 * 2.0 ** -24 * growth * rows
        tol = tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(ref) + 2.0 ** -120
        worst = float((np.abs(out[i].numpy() - ref) / tol).max())
        assert worst <= 1.0, (k, len(coef), worst, float(np.abs(out[i].numpy() - ref).max()))


@pytest.mark.parametrize("count", [5, 8, 9, 10, 12, 14, 16])
@pytest.mark.parametrize("r,wide", [(16, False), (16, True), (8, False), (32, False), (64, True), (72, False)])
def test_fp32_of_few_directions(r, wide, count):
    check_range(F32, [1, 5, "rows", "repeated", "graded"], 520, r, wide, [STEP] * count)


@pytest.mark.parametrize("count", [5, 6, 7, 8, 10, 12, 14, 16])
@pytest.mark.parametrize("r,wide", [(16, False), (16, True), (8, False), (32, False), (64, True), (72, False)])
def test_bf16_of_few_directions(r, wide, count):
    check_range(BF16, [1, 5, "rows", "repeated", "graded"], 520, r, wide, [STEP] * count)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_steps_that_grow_and_shrink(dtype):
    """Large and small c0 in turn, and steps of one kind after another."""
    for coef in ([STEP, STEP, (1.875, -1.25, 0.375)] * 4, [(1.875, -1.25, 0.375)] * 16,
                 [(0.25, 0.0, 0.0)] * 4 + [STEP] * 12, [STEP] * 11 + [(1.5, -0.5, 0.0)] * 5):
        check_range(dtype, [1, "rows", "graded"], 264, 24, False, coef)


def test_bf16_of_large_and_tiny_polynomials():
    """c1 that brings P past what its parts carry, and c0 that multiply to no fp32 number, which the scale makes up for."""
    check_range(BF16, ["rows", "graded"], 264, 24, False, [STEP] * 3 + [(0.5, 3000.0, 0.0)])
    g = few_directions("graded", 264, 24, 1).to(BF16)
    out = run(g[None].cuda(), [(2.0 ** -26, 0.0, 0.0)] * 5, scale=2.0 ** 127)[0].cpu().double()
    ref = g.double() / (g.double().norm() + float(np.float32(EPS))) * 2.0 ** -3
    assert ((out - ref).abs() <= ref.abs() * (HALF[BF16] + 2.0 ** -40) + 2.0 ** -130).all()


@pytest.mark.parametrize("count", [6, 16])
@pytest.mark.parametrize("dtype,wide", [(F32, False), (BF16, True)])
def test_the_widest(dtype, wide, count):
    check_range(dtype, [1, "repeated"], 264, 128, wide, [STEP] * count)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("r,wide", [(16, True), (24, False), (64, False), (96, True)])
def test_many_steps_in_place_in_graphs_and_in_bounds(r, wide, dtype):
    """On a workspace of exactly the named size between guard bytes, of 255s, shared by two captured calls."""
    coefs, D = ([STEP] * 12, [STEP] * 16), 520
    g = torch.stack([few_directions(k, D, r, 5) for k in (5, "rows", "graded")]).to(dtype)
    g = (g.transpose(1, 2) if wide else g).contiguous().cuda()
    ref = [run(g, c) for c in coefs]
    size = L.lora_workspace_bytes_orthogonalize(*g.shape)
    raw = torch.full((size + 8192,), 255, dtype=torch.uint8, device="cuda")
    ws, bufs, graphs = raw[4096:4096 + size], [g.clone(), g.clone()], []
    for c, b, want in zip(coefs, bufs, ref):
        run(b, c, out=b, ws=ws)
        assert torch.equal(b, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(b, c, out=b, ws=ws)
        graphs.append(graph)
    for _ in range(3):
        for b in bufs:
            b.copy_(g)
        ws.fill_(255)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[0], ref[0]) and torch.equal(bufs[1], ref[1])
    assert (raw[:4096] == 255).all() and (raw[4096 + size:] == 255).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("r,wide", [(8, False), (16, True), (40, False), (128, True)])
def test_zeros_stay_zero_and_others_nan_through_many_steps(r, wide, dtype):
    g = torch.stack([few_directions(5, 264, r, i) for i in range(4)]).to(dtype)
    g[0, :, 3:] = 0
    g[1] = 0
    g[2, 9, 1] = float("nan")
    ref = run((g[3:].transpose(1, 2) if wide else g[3:]).contiguous().cuda(), [STEP] * 16)
    out = run((g.transpose(1, 2) if wide else g).contiguous().cuda(), [STEP] * 16)
    assert torch.equal(out[3:], ref)
    out = out.transpose(1, 2) if wide else out
    assert out[0, :, :3].any() and not out[0, :, 3:].any() and not out[1].any() and torch.isnan(out[2]).all()


@pytest.mark.parametrize("count", [5, 12])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("r,wide", [(16, False), (24, True), (64, False), (72, True)])
def test_powers_of_two_change_nothing(r, wide, dtype, count):
    """eps is below every rounding of |g|; all sums scale with g to the bit, and the result does not."""
    g = torch.stack([few_directions(k, 264, r, 3) for k in (5, "rows")]).to(dtype)
    g = (g.transpose(1, 2) if wide else g).contiguous().cuda()
    ref = run(g, [STEP] * count, eps=2.0 ** -126)
    for e in (30, 70, 110, -30, -50):
        h = g.double() * 2.0 ** e
        assert torch.equal(h.to(dtype).double(), h)
        assert torch.equal(run(h.to(dtype), [STEP] * count, eps=2.0 ** -126), ref), e


@pytest.mark.parametrize("wide", [False, True])
def test_bf16_of_one_tile_by_64_bit_products(wide):
    for coef in ([STEP] * 3 + [(0.5, 3000.0, 0.0)], [(2.0 ** -21, 2.0 ** -21, 0.0)]):
        check_range(BF16, ["rows", "graded"], 264, 16, wide, coef)
