"""lora_gated_backward against the gradients' formulas in 64 bits (bounds in
helpers_block.backward64), those against differences of the forward pass, and
the whole block forward and backward as it would be trained."""
import numpy as np
import pytest
import torch

from helpers_block import ACTS, Pair, act64, backward64, run_backward, run_forward, within
from rank_adapter_gemm_amd import lora as L

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


def kept(p, seed=0):
    """gate, up and dh as a forward pass and a loss leave them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 100)
    new = lambda std: (std * torch.randn(p.T, p.f, generator=g, device="cuda")).to(p.dtype)  # noqa: E731
    return new(1.3), new(1.3), new(0.02)


def check(p, act, gate, up, dh, got, what):
    dx, tx, dA, tA, dB, tB = backward64(p, act, gate, up, dh)
    if got[0] is not None:
        within(got[0], dx, tx, what + " dx")
    if got[1] is not None:
        for m in range(2):
            within(got[1][m], dA[m], tA[m], what + " dA %d" % m)
            within(got[2][m], dB[m], tB[m], what + " dB %d" % m)


RANKS = [16, 3, 8, 0, 13, 16, 1]

SHAPES = [(1, 64, 8), (1, 1032, 712), (2, 512, 1000), (31, 264, 256), (64, 1024, 2048), (130, 520, 776),
          (300, 136, 1064), (700, 40, 8), (2048, 3336, 72), (1100, 1032, 1400), (4200, 64, 64)]


@pytest.mark.parametrize("T,d,f", SHAPES)
def test_bf16(T, d, f):
    p = Pair(T, d, f, RANKS, 16, BF16, seed=T + f)
    k = kept(p)
    got = run_backward(p, "silu", *k)
    check(p, "silu", *k, got, "bf16")
    assert L.lora_get_device_error(got[3].buf) == p.bad_row()


@pytest.mark.parametrize("T,d,f", [(1, 64, 8), (5, 136, 72), (64, 264, 256), (130, 136, 1032), (333, 520, 64)])
@pytest.mark.parametrize("act", list(ACTS))
def test_f32(T, d, f, act):
    p = Pair(T, d, f, RANKS, 16, F32, seed=T)
    k = kept(p)
    check(p, act, *k, run_backward(p, act, *k), act)


@pytest.mark.parametrize("act", list(ACTS))
def test_activations(act):
    p = Pair(150, 264, 520, RANKS, 16, BF16, seed=5)
    gate, up, dh = kept(p)
    gate[0] *= 30
    gate[1] *= 2.0 ** -30
    check(p, act, gate, up, dh, run_backward(p, act, gate, up, dh), act)


@pytest.mark.parametrize("R,ranks", [(8, [8, 1]), (24, [24, 17, 5]), (40, [33, 40, 0, 8]), (64, [64, 63, 20])])
@pytest.mark.parametrize("packed", [False, True])
def test_ranks(R, ranks, packed):
    for T, order in ((9, "random"), (520, "random"), (1500, "sorted")):
        p = Pair(T, 136, 328, ranks, R, BF16, seed=R, packed=packed, order=order)
        k = kept(p)
        check(p, "silu", *k, run_backward(p, "silu", *k), "R %d T %d" % (R, T))


def test_pools_that_differ():
    p = Pair(200, 256, 136, ([8, 0, 4], [0, 16, 3]), 16, BF16, seed=2)
    k = kept(p)
    got = run_backward(p, "silu", *k)
    check(p, "silu", *k, got, "differ")
    assert L.lora_get_device_error(got[3].buf) == p.bad_row() >= 0


def test_ids():
    """Nobody's rows, one adapter's, bad ids, long and short runs, slots without rows."""
    T, S = 530, 9
    rng = np.random.default_rng(0)
    odd = rng.integers(-1, 5, size=T).astype(np.int32)
    odd[[3, 77, 400]] = [S, -2, 10 ** 6]
    runs = np.repeat([0, -1, 2, 1, 4], [70, 33, 250, 1, T - 354]).astype(np.int32)
    for ids in (np.full(T, -1, np.int32), np.full(T, 2, np.int32), odd, runs):
        for dtype in (BF16, F32):
            p = Pair(T, 192, 264, [8, 16, 12, 16, 2, 5, 16, 0, 9], 16, dtype, seed=1, ids=ids)
            k = kept(p)
            got = run_backward(p, "silu", *k)
            check(p, "silu", *k, got, "ids")
            assert L.lora_get_device_error(got[3].buf) == p.bad_row()
            for s in range(S):
                if not (ids == s).any():
                    assert all((t[s] == 0).all() for t in got[1] + got[2])


def test_a_row_of_nan_stays_with_its_adapter():
    for dtype in (BF16, F32):
        p = Pair(300, 136, 264, [8, 16, 4], 16, dtype, seed=4, ids=np.arange(300) % 4 - 1)
        gate, up, dh = kept(p)
        dh[17] = float("nan")                              # slot 0's row
        dx, dA, dB, _ = run_backward(p, "silu", gate, up, dh)
        assert torch.isnan(dx[17]).all()
        ok = [t for t in range(300) if t != 17]
        assert torch.isfinite(dx[ok].float()).all()
        for m in range(2):
            assert torch.isnan(dA[m][0, :, :8]).all() and torch.isnan(dB[m][0, :8]).all()
            assert (dA[m][0, :, 8:] == 0).all() and (dB[m][0, 8:] == 0).all()
            assert torch.isfinite(dA[m][1:].float()).all() and torch.isfinite(dB[m][1:].float()).all()


def test_parts_and_no_rows():
    """dx alone, the adapters' alone, and a batch of no rows."""
    for dtype in (BF16, F32):
        p = Pair(90, 128, 264, [8, 8], 8, dtype, seed=6)
        k = kept(p)
        full = run_backward(p, "silu", *k)
        only = run_backward(p, "silu", *k, want_ab=False)
        assert torch.equal(only[0], full[0])
        only = run_backward(p, "silu", *k, want_dx=False)
        for m in range(2):
            assert torch.equal(only[1][m], full[1][m]) and torch.equal(only[2][m], full[2][m])
        p.T = 0
        dx, dA, dB, _ = run_backward(p, "silu", *k)
        assert all((t == 0).all() for t in dA + dB)


def test_rows_past_the_batch_stay():
    p = Pair(70, 128, 264, [8, 8], 8, BF16, seed=6)
    k = kept(p)
    ws = L.Workspace(90, 2, 8, 264, gated=True, backward_d_in=128)
    dx = torch.full((90, 128), 3.0, dtype=BF16, device="cuda")
    L.lora_gated_backward(p.x, p.W[0], p.W[1], 70, p.desc, p.ids_dev, 0, *k, dx, None, None, ws.buf)
    assert (dx[70:] == 3).all()
    check(p, "silu", *k, (dx[:70], None, None), "first rows")


@pytest.mark.parametrize("act", list(ACTS))
def test_the_formulas_against_differences(act):
    """The 64-bit gradients the kernels are held to against central differences
    of the 64-bit forward pass along random directions: the difference's own
    error is its third order, about eps^2 = 1e-8 of the sum, and 1e-16 / eps."""
    p = Pair(23, 40, 48, [8, 5, 3], 8, F32, seed=9)
    dh = kept(p)[2]
    _, _, (g, u), _ = p.forward64(act)
    dx, _, dA, _, dB, _ = backward64(p, act, g, u, dh)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    eps = 1e-4

    def loss(x, A, B):
        out = []
        for m in range(2):
            y = x @ p.W[m].double()
            for s, r in enumerate(p.ranks[m]):
                t = p.owners(s)
                sc = float(np.float32(p.alphas[s]) / np.float32(r))
                y[t] = y[t] + sc * (x[t] @ A[m][s][:, :r]) @ B[m][s][:r]
            out.append(y)
        return float((act64(act, out[0])[0] * out[1] * dh.double()).sum())

    x, A, B = p.x.double(), [a.double() for a in p.A], [b.double() for b in p.B]
    rand = lambda t: torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    D = rand(x)
    slopes = [((loss(x + eps * D, A, B) - loss(x - eps * D, A, B)) / (2 * eps), float((dx * D).sum()))]
    for m in range(2):
        D = rand(A[m])
        moved = lambda s: [A[i] + s * eps * D if i == m else A[i] for i in range(2)]  # noqa: E731, B023
        slopes.append(((loss(x, moved(1), B) - loss(x, moved(-1), B)) / (2 * eps), float((dA[m] * D).sum())))
        D = rand(B[m])
        moved = lambda s: [B[i] + s * eps * D if i == m else B[i] for i in range(2)]  # noqa: E731, B023
        slopes.append(((loss(x, A, moved(1)) - loss(x, A, moved(-1))) / (2 * eps), float((dB[m] * D).sum())))
    for diff, grad in slopes:
        assert abs(diff - grad) <= 1e-5 * (1 + abs(grad)), slopes


@pytest.mark.parametrize("T", [3, 200, 1400])
def test_repeats_other_streams_and_graphs(T):
    p = Pair(T, 520, 776, RANKS, 16, BF16, seed=T)
    k = kept(p)
    flat = lambda got: [got[0]] + got[1] + got[2]  # noqa: E731
    ref = flat(run_backward(p, "silu", *k))
    wss = [L.Workspace(T, p.S, p.R, p.f, gated=True, backward_d_in=p.d) for _ in range(2)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for st, ws in zip(streams, wss):
        with torch.cuda.stream(st):
            outs.append(flat(run_backward(p, "silu", *k, ws=ws, stream=st)))
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    bufs = [torch.empty_like(t) for t in ref]

    def call():
        L.lora_gated_backward(p.x, p.W[0], p.W[1], T, p.desc, p.ids_dev, 0, *k, bufs[0], bufs[1:3], bufs[3:], wss[0].buf)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for b in bufs:
            b.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bufs, ref))
        assert all(torch.equal(a, b) for a, b in zip(flat(run_backward(p, "silu", *k, ws=wss[1])), ref))
        torch.cuda.synchronize()


def test_a_block_forward_and_backward():
    """Norm, gated pair and down projection as a model runs them, then the
    pair's backward pass from what the forward kept."""
    T, d, f = 260, 512, 776
    p = Pair(T, d, f, [16, 8, 4], 16, BF16, seed=21)
    res = p.x.clone()
    delta = (0.5 * p.x.float().roll(1, 0)).to(BF16)
    w = torch.ones(d, dtype=BF16, device="cuda")
    y = torch.empty_like(res)
    want_z = (res.double() + delta.double())
    L.lora_add_rmsnorm(delta, res, w, 1e-6, T, d, L.LORA_BF16, res, y)
    within(res, want_z, 2.0 ** -8 * want_z.abs() + 1e-30, "residual")
    p.x = y
    h, gate, up, _ = run_forward(p, "silu", keep=True)
    ref, tol, _, _ = p.forward64("silu")
    within(h, ref, tol, "h")
    Wd = (torch.randn(f, d, device="cuda") / f ** 0.5).to(BF16)
    out = torch.empty(T, d, dtype=BF16, device="cuda")
    L.lora_gemm(h, Wd, out, T, f, d, L.LORA_BF16)
    dh = (0.01 * out.double() @ Wd.double().t()).to(BF16)      # of the loss 0.005 |out|^2
    got = run_backward(p, "silu", gate, up, dh)
    check(p, "silu", gate, up, dh, got, "block")


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_a_nan_adapter_stays_with_its_rows(what):
    """Values that are not finite in one adapter's A and B: dx of other rows, and
    other adapters' gradients, as if that adapter were sound."""
    for T, order in ((40, "random"), (700, "sorted")):
        for dtype in (BF16, F32):
            p = Pair(T, 136, 264, [16, 16, 5, 9], 16, dtype, seed=13, order=order)
            k = kept(p)
            clean = run_backward(p, "silu", *k)
            for m in range(2):
                p.A[m][1, 7, 3] = what
                p.B[m][1, 2, 100] = what
                p.pools[m].upload(1, p.A[m][1], p.B[m][1], 16, p.alphas[1], lda=16, ldb=p.f)
            got = run_backward(p, "silu", *k)
            others = torch.as_tensor(p.ids != 1, device="cuda")
            assert torch.equal(got[0][others], clean[0][others])
            assert not torch.isfinite(got[0][~others].float()).all(1).any()
            for m in range(2):
                assert torch.equal(got[1][m][[0, 2, 3]], clean[1][m][[0, 2, 3]])
                assert torch.equal(got[2][m][[0, 2, 3]], clean[2][m][[0, 2, 3]])


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gates_far_from_zero(act, dtype):
    """Where the activation is 0 or its argument, its slope is 0 or 1, also where the argument's square overflows."""
    p = Pair(6, 64, 72, [8, 3], 8, dtype, seed=3, ids=[-1] * 6)
    gate, up, dh = kept(p)
    big = [60.0, -60.0, 1e15, -1e15, 3e38, -3e38]
    for t, f in enumerate(big):
        gate[t] = f
    dh[:] = dh * 2.0 ** -40
    dx, _, _, _ = run_backward(p, act, gate, up, dh)
    for t, f in enumerate(big):
        # slope 1, act(g) = g; or both 0 (silu at -60: 60 exp(-60) < 2^-80, below every bound here)
        dg = dh[t].double() * up[t].double() * (f > 0)
        du = dh[t].double() * gate[t].double() * (f > 0)
        half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
        Wg, Wu = p.W[0].double(), p.W[1].double()
        size = dg.abs() @ Wg.t().abs() + du.abs() @ Wu.t().abs()
        ref = dg @ Wg.t() + du @ Wu.t()
        # dg and du: 4 fp32 steps and one rounding; 2 f sums of one step; dx rounded
        tol = (half + (2 * p.f + 12) * 2.0 ** -23) * size + half * ref.abs() * (1 + half) + 2.0 ** -110
        within(dx[t], ref, tol, "%s gate %g" % (act, f))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_each_part_alone_is_what_the_whole_gives(dtype):
    """dx alone and the adapters' gradients alone: bitwise those of the call for both."""
    p = Pair(150, 136, 264, RANKS, 16, dtype, seed=12)
    k = kept(p)
    dx, dA, dB, _ = run_backward(p, "silu", *k)
    only_dx, none_a, none_b, _ = run_backward(p, "silu", *k, want_ab=False)
    none_dx, only_a, only_b, _ = run_backward(p, "silu", *k, want_dx=False)
    assert none_a is None and none_b is None and none_dx is None
    assert torch.equal(dx, only_dx)
    for m in range(2):
        assert torch.equal(dA[m], only_a[m]) and torch.equal(dB[m], only_b[m])
