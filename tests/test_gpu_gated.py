"""The gated pair (lora_gated_forward, lora_gated_forward_fp8) against its
plain form in 64 bits, element by element, with bounds that count the sums
and roundings of the kernels (helpers_block.Pair.forward64)."""
import numpy as np
import pytest
import torch

from helpers_block import ACTS, Pair, run_forward, within
from rank_adapter_gemm_amd import lora as L

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


def check(p, act, got, what, bases=(None, None), extra=(0.0, 0.0)):
    h, tol_h, y, tol_y = p.forward64(act, bases, extra)
    within(got[0], h, tol_h, what + " h")
    if got[1] is not None:
        within(got[1], y[0], tol_y[0], what + " gate")
        within(got[2], y[1], tol_y[1], what + " up")


RANKS = [16, 3, 8, 0, 13, 16, 1]

# T, d, f: one token and few rows (K split), odd widths, every whole-tile plan, a tail round split over K
SHAPES = [(1, 64, 8), (1, 1032, 712), (2, 512, 1000), (31, 256, 264), (64, 1024, 2048), (130, 776, 520),
          (128, 72, 14336), (300, 136, 7304), (700, 8, 40), (2048, 64, 3456), (1100, 1032, 3400)]


@pytest.mark.parametrize("T,d,f", SHAPES)
def test_bf16(T, d, f):
    p = Pair(T, d, f, RANKS, 16, BF16, seed=T + f)
    for mode in (L.LORA_MODE_AUTO, L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
        got = run_forward(p, "silu", mode, keep=mode == L.LORA_MODE_SGMV)
        check(p, "silu", got, "mode %d" % mode)
        assert L.lora_get_device_error(got[3].buf) == p.bad_row()


@pytest.mark.parametrize("T,d,f", [(1, 64, 8), (5, 136, 72), (64, 256, 264), (130, 1032, 136), (333, 64, 520)])
@pytest.mark.parametrize("act", list(ACTS))
def test_f32(T, d, f, act):
    p = Pair(T, d, f, RANKS, 16, F32, seed=T)
    for mode in (L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
        check(p, act, run_forward(p, act, mode, keep=True), "f32")


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("T,f", [(40, 200), (600, 3400)])
def test_activations(act, T, f):
    p = Pair(T, 512, f, RANKS, 16, BF16, seed=5)
    p.x[0] *= 40                       # far into both tails of the activation
    p.x[1] *= 2.0 ** -30               # and near its zero
    check(p, act, run_forward(p, act, keep=True), act)


@pytest.mark.parametrize("R,ranks", [(8, [8, 1]), (24, [24, 17, 5]), (40, [33, 40, 0, 8]), (64, [64, 63, 20])])
@pytest.mark.parametrize("packed", [False, True])
def test_ranks(R, ranks, packed):
    for T, order in ((9, "random"), (520, "random"), (2100, "sorted")):
        p = Pair(T, 128, 1736, ranks, R, BF16, seed=R, packed=packed, order=order)
        for mode in (L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
            check(p, "silu", run_forward(p, "silu", mode), "R %d T %d" % (R, T))


def test_pools_that_differ():
    """A slot empty in one pool only: the other's term stays, the row is recorded."""
    p = Pair(200, 256, 136, ([8, 0, 4], [0, 16, 3]), 16, BF16, seed=2)
    for mode in (L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
        got = run_forward(p, "silu", mode, keep=True)
        check(p, "silu", got, "differ")
        assert L.lora_get_device_error(got[3].buf) == p.bad_row() >= 0


def test_ids():
    """No adapter at all, one adapter for all, ids out of range, runs that cross the tiles."""
    T, S = 530, 5
    rng = np.random.default_rng(0)
    odd = rng.integers(-1, S, size=T).astype(np.int32)
    odd[[3, 77, 400]] = [S, -2, 10 ** 6]
    runs = np.repeat([0, -1, 2, 1, 4], [70, 33, 250, 1, T - 354]).astype(np.int32)
    for ids in (np.full(T, -1, np.int32), np.full(T, 2, np.int32), odd, runs):
        p = Pair(T, 192, 968, [8, 16, 12, 16, 2], 16, BF16, seed=1, ids=ids)
        for mode in (L.LORA_MODE_AUTO, L.LORA_MODE_BGMV):
            got = run_forward(p, "silu", mode)
            check(p, "silu", got, "ids")
            assert L.lora_get_device_error(got[3].buf) == p.bad_row()


def test_a_row_of_nan_stays_in_its_row():
    for T in (60, 1500):
        for dtype in (BF16, F32):
            p = Pair(T, 256, 520, [8, 16, 4], 16, dtype, seed=4)
            p.x[17] = float("nan")
            p.x[18, 3] = float("inf")
            for mode in (L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
                h = run_forward(p, "silu", mode)[0]
                assert torch.isnan(h[17]).all()
                rest = torch.tensor([t for t in range(T) if t not in (17, 18)], device="cuda")
                x = p.x.clone()
                x[17:19] = 0
                p.x, kept = x, p.x
                ref, tol, _, _ = p.forward64("silu")
                p.x = kept
                within(h[rest], ref[rest], tol[rest], "rows beside")


def test_rows_past_the_batch_stay():
    p = Pair(70, 128, 264, [8, 8], 8, BF16, seed=6)
    h = torch.full((90, 264), 3.0, dtype=BF16, device="cuda")
    ws = L.Workspace(90, 2, 8, 264, gated=True)
    L.lora_gated_forward(p.x, p.W[0], p.W[1], h, 70, p.desc, p.ids_dev, 0, L.LORA_MODE_AUTO, 0, ws.buf)
    assert (h[70:] == 3).all()
    ref, tol, _, _ = p.forward64("silu")
    within(h[:70], ref, tol, "first rows")
    h.fill_(3)
    L.lora_gated_forward(p.x, p.W[0], p.W[1], h, 0, p.desc, p.ids_dev, 0, L.LORA_MODE_AUTO, 0, ws.buf)
    assert (h == 3).all()


def test_no_room_for_a_split_and_segments_ready():
    """A workspace without partials computes every tile whole; segments built
    once serve a second call."""
    p = Pair(90, 1024, 1000, [8, 16], 16, BF16, seed=8)
    ws = L.Workspace(90, 2, 16, 0, gated=True)
    got = run_forward(p, "silu", L.LORA_MODE_SGMV, ws=ws)
    check(p, "silu", got, "no partials")
    again = run_forward(p, "silu", L.LORA_MODE_SGMV, ws=ws, flags=L.LORA_FLAG_SEGMENTS_READY)
    assert torch.equal(got[0], again[0])
    L.lora_build_segments(p.ids_dev, 90, 2, 32, ws.buf)
    again = run_forward(p, "silu", L.LORA_MODE_SGMV, ws=ws, flags=L.LORA_FLAG_SEGMENTS_READY)
    assert torch.equal(got[0], again[0])


@pytest.mark.parametrize("dtype,T", [(BF16, 700), (BF16, 90), (F32, 90)])
def test_overwritten_segment_tables_stay_in_bounds(dtype, T):
    """Segments said to be ready in a workspace that holds other things: wrong
    rows, read and written in their buffers; built again, they are right."""
    p = Pair(T, 264, 520, [8, 16, 5], 16, dtype, seed=31)
    ws = L.Workspace(T, p.S, p.R, p.f, gated=True)
    words = ws.buf.numel() // 4 * 4
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    ws.buf[:words] = torch.randint(0, 256, (words,), generator=g, device="cuda").to(ws.buf.dtype)
    run_forward(p, "silu", L.LORA_MODE_SGMV, ws=ws, flags=L.LORA_FLAG_SEGMENTS_READY)
    torch.cuda.synchronize()
    L.lora_workspace_init(ws.buf)
    check(p, "silu", run_forward(p, "silu", L.LORA_MODE_SGMV, ws=ws), "built again")


@pytest.mark.parametrize("T,S", [(1, 16000), (1024, 16000), (1023, 1), (700, 64)])
def test_segments_of_one_tile(T, S):
    """Batches of up to 1024 rows, whose segments one workgroup builds: every
    row by its slot, rows of one slot in batch order, ids that are none first."""
    rng = np.random.default_rng(T + S)
    ids = rng.integers(-3, S + 3, size=T).astype(np.int32)
    ids[rng.random(T) < 0.3] = S - 1
    key = np.where((ids >= 0) & (ids < S), ids, -1)
    ws = L.Workspace(T, S, 8)
    L.lora_build_segments(torch.as_tensor(ids, device="cuda"), T, S, 8, ws.buf)
    got = ws.segments(T)
    assert np.array_equal(got["perm"].cpu().numpy(), np.argsort(key, kind="stable"))
    assert np.array_equal(np.diff(got["offsets"].cpu().numpy()), np.bincount(key + 1, minlength=S + 1))


# ---- FP8 base ----------------------------------------------------------------
def fp8_parts(p):
    from helpers_fp8 import e4m3_decode
    xq = torch.empty(p.T, p.d, dtype=torch.uint8, device="cuda")
    xs = torch.empty(p.T, dtype=torch.float32, device="cuda")
    L.lora_quantize_rows_fp8(p.x, p.T, p.d, xq, xs)
    wq = [L.Fp8Weight(w) for w in p.W]
    bases, extra = [], []
    X = torch.as_tensor(e4m3_decode(xq.cpu().numpy()), device="cuda") * xs.double()[:, None]
    for q in wq:
        W = torch.as_tensor(e4m3_decode(q.codes.cpu().numpy()), device="cuda").t() * q.scale.double()[None, :]
        size = X.abs() @ W.abs()
        bases.append((X @ W, size))
        extra.append(2.0 ** -11 * size)          # the matrix cores' sums of 64 codes' products
    return (xq, xs, wq), bases, extra


@pytest.mark.parametrize("T,d,f", [(1, 64, 8), (1, 1040, 712), (31, 256, 264), (130, 784, 520), (128, 80, 14336),
                                   (300, 144, 7304), (2048, 64, 3456), (1100, 1040, 3400)])
def test_fp8(T, d, f):
    p = Pair(T, d, f, RANKS, 16, BF16, seed=T + f)
    parts, bases, extra = fp8_parts(p)
    for mode in (L.LORA_MODE_AUTO, L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
        got = run_forward(p, "silu", mode, keep=mode == L.LORA_MODE_SGMV, fp8=parts)
        check(p, "silu", got, "fp8 mode %d" % mode, bases, extra)
        made = run_forward(p, "silu", mode, fp8=parts, codes=False)       # the codes made within the call
        assert torch.equal(made[0], got[0])


# ---- streams, graphs, repeats --------------------------------------------------
@pytest.mark.parametrize("T,fp8", [(3, False), (200, False), (1400, False), (200, True), (1400, True)])
def test_repeats_other_streams_and_graphs(T, fp8):
    p = Pair(T, 1024, 1544, RANKS, 16, BF16, seed=T)
    parts = fp8_parts(p)[0] if fp8 else None
    ref = run_forward(p, "silu", fp8=parts)[0]
    assert torch.equal(ref, run_forward(p, "silu", fp8=parts)[0])
    torch.cuda.synchronize()
    # two calls at once, each with its own workspace
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    wss = [L.Workspace(T, p.S, p.R, p.f, gated=True, fp8_d_in=p.d if fp8 else 0) for _ in streams]
    torch.cuda.synchronize()
    outs = []
    for st, ws in zip(streams, wss):
        with torch.cuda.stream(st):
            outs.append(run_forward(p, "silu", ws=ws, stream=st, fp8=parts)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    # captured and replayed, with eager work on the same inputs between
    h = torch.empty_like(ref)
    ws = wss[0]

    def call():
        if fp8:
            xq, xs, wq = parts
            L.lora_gated_forward_fp8(p.x, xq, xs, wq[0].codes, wq[0].scale, wq[1].codes, wq[1].scale, h, T, p.desc,
                                     p.ids_dev, 0, 0, 0, ws.buf)
        else:
            L.lora_gated_forward(p.x, p.W[0], p.W[1], h, T, p.desc, p.ids_dev, 0, 0, 0, ws.buf)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        h.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, ref)
        assert torch.equal(run_forward(p, "silu", ws=wss[1], fp8=parts)[0], ref)
        torch.cuda.synchronize()


def test_the_pair_is_what_the_projections_give():
    """h from the pair against act and product of lora_linear_forward's gate and
    up: those are rounded to bf16 before, so within both roundings of each."""
    p = Pair(600, 512, 1032, [16, 8, 4], 16, BF16, seed=12)
    h = run_forward(p, "silu", keep=True)
    ys = []
    for m in range(2):
        ws = L.Workspace(p.T, p.S, p.R, p.f)
        y = torch.empty(p.T, p.f, dtype=BF16, device="cuda")
        L.lora_linear_forward(p.x, p.W[m], y, p.T, p.desc[m], p.ids_dev, L.LORA_MODE_AUTO, 0, ws.buf)
        ys.append(y)
        # two roundings of nearly one value: at most one step apart, and the short segments' second rounding
        d = (y.double() - h[1 + m].double()).abs()
        assert (d <= 2.0 ** -6 * (1 + y.double().abs())).all()
    ref = torch.nn.functional.silu(ys[0].double()) * ys[1].double()
    assert ((h[0].double() - ref).abs() <= 2.0 ** -5 * (1 + ref.abs())).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,f,order", [(20, 264, "random"), (90, 264, "random"), (300, 3400, "random"), (700, 1032, "sorted"),
                                       (2100, 3400, "sorted")])
def test_a_nan_adapter_stays_with_its_rows(T, f, order, what):
    """A value that is not finite in one adapter's B (and its A): rows of other
    adapters and of none get what they get beside a sound one."""
    for fp8 in (False, True):
        p = Pair(T, 256, f, [16, 16, 5, 9], 16, BF16, seed=13, order=order)
        parts = fp8_parts(p)[0] if fp8 else None
        modes = (L.LORA_MODE_BGMV, L.LORA_MODE_SGMV)
        clean = [run_forward(p, "silu", mode, fp8=parts)[0] for mode in modes]
        for m in range(2):
            p.A[m][1, 7, 3] = what
            p.B[m][1, 2, 100] = what
            p.B[m][1, 15, 230] = -what
            p.pools[m].upload(1, p.A[m][1], p.B[m][1], 16, p.alphas[1], lda=16, ldb=p.f)
        others = torch.as_tensor(p.ids != 1, device="cuda")
        for mode, ref in zip(modes, clean):
            h = run_forward(p, "silu", mode, fp8=parts)[0]
            assert torch.equal(h[others], ref[others])
            assert not torch.isfinite(h[~others][:, [100, 230]].float()).any()


def test_the_binding_refuses_tensors_the_kernels_would_misread():
    p = Pair(6, 64, 72, [8, 8], 8, BF16, seed=3)
    ws = L.Workspace(6, 2, 8, 72, gated=True)
    h = torch.empty(6, 72, dtype=BF16, device="cuda")

    def call(x=p.x, W=p.W[0], h=h, ids=p.ids_dev, w=ws.buf, gate=None, up=None):
        L.lora_gated_forward(x, W, p.W[1], h, 6, p.desc, ids, 0, 0, 0, w, gate=gate, up=up)

    call()
    for bad in (dict(x=p.x.float()), dict(x=p.x.cpu()), dict(x=p.x[:5]), dict(W=p.W[0].t()), dict(W=p.W[0][:63]),
                dict(h=h[:5]), dict(h=h.half()), dict(ids=p.ids_dev.long()), dict(ids=p.ids_dev.cpu()),
                dict(ids=p.ids_dev[:3]), dict(w=ws.buf.cpu()), dict(w=ws.buf[:1024]), dict(gate=h[:2], up=h)):
        with pytest.raises(L.LoraError):
            call(**bad)


@pytest.mark.parametrize("T", [1, 150, 700])
def test_a_block_on_fp8_weights(T):
    """Norm with codes, gated pair on them, down projection: each step against
    the 64-bit form of what it was given, as a server runs them."""
    d, f = 512, 1040
    p = Pair(T, d, f, [16, 8, 4, 0], 16, BF16, seed=31, ids=np.arange(T) % 4 - 1)
    delta, res = (0.5 * p.x.float()).to(BF16), p.x.roll(1, 1).contiguous()
    w = (1 + 0.1 * torch.randn(d, device="cuda")).to(BF16)
    z, y = torch.empty_like(res), torch.empty_like(res)
    q, s = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    L.lora_add_rmsnorm_fp8(delta, res, w, 1e-6, T, d, z, y, q, s)
    p.x = y
    parts, bases, extra = fp8_parts(p)
    assert torch.equal(parts[0], q) and torch.equal(parts[1], s)
    got = run_forward(p, "silu", fp8=(q, s, parts[2]))
    check(p, "silu", got, "h", bases, extra)
    Wd = (torch.randn(f, d, device="cuda") / f ** 0.5).to(BF16)
    down = Pair(1, f, d, [16, 8, 4], 16, BF16, seed=32).pools[0]
    wd, out = L.Fp8Weight(Wd), torch.empty(T, d, dtype=BF16, device="cuda")
    ids = torch.where(p.ids_dev < 3, p.ids_dev, -1)
    ws = L.Workspace(T, 3, 16, d, fp8_d_in=f)
    L.lora_linear_forward_fp8(got[0], wd.codes, wd.scale, out, T, down.pool, ids, L.LORA_MODE_AUTO, 0, ws.buf)
    nxt, codes, scales = torch.empty_like(y), torch.empty_like(q), torch.empty_like(s)
    L.lora_add_rmsnorm_fp8(out, z, w, 1e-6, T, d, z, nxt, codes, scales)
    assert torch.isfinite(nxt.float()).all()
    want = out.double() + (delta.double() + res.double()).to(BF16).double()
    assert ((z.double() - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -7 * (delta.double() + res.double()).abs()).all()
