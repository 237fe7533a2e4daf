"""lora_linear_act_forward and its FP8 form against the plain form in 64 bits,
element by element, with bounds that count the sums and roundings of the kernels
(helpers_act.Layer.forward64)."""
import numpy as np
import pytest
import torch

from helpers_act import ACTS, Layer, run_forward
from helpers_block import within
from rank_adapter_gemm_amd import lora as L

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
MODES = (L.LORA_MODE_AUTO, L.LORA_MODE_BGMV, L.LORA_MODE_SGMV)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


def check(p, act, got, what, bias=True, residual=True, base=None, extra=0.0):
    y, tol_y, pre, tol_p = p.forward64(act, bias, residual, base, extra)
    within(got[0], y, tol_y, what + " y")
    if got[1] is not None:
        within(got[1], pre, tol_p, what + " pre")


RANKS = [16, 3, 8, 0, 13, 16, 1]

# T, d, f: one token and few rows (K split), odd widths, every whole-tile plan (256 x 256, 256 x 128, 128 x 128,
# 128 x 64), a tail round split over K
SHAPES = [(1, 64, 8), (1, 4096, 4096), (1, 1032, 712), (2, 512, 1000), (31, 256, 264), (64, 1024, 2048),
          (130, 776, 520), (128, 72, 14336), (300, 136, 7304), (700, 8, 40), (3580, 64, 4090 // 8 * 8), (1790, 72, 4096),
          (890, 136, 4096), (890, 136, 2048), (1100, 1032, 3400), (2048, 1032, 8712)]


@pytest.mark.parametrize("T,d,f", SHAPES)
def test_bf16(T, d, f):
    p = Layer(T, d, f, RANKS, 16, BF16, seed=T + f)
    for mode in MODES:
        got = run_forward(p, "gelu", mode, keep=mode == L.LORA_MODE_SGMV)
        check(p, "gelu", got, "mode %d" % mode)
        assert L.lora_get_device_error(got[2].buf) == p.bad_row()


# grids of few tiles: K ranges in whole rounds of workgroups (two of 112 tiles, three of 80, one of 224), and tiles of
# 64 columns where K is too short for ranges
@pytest.mark.parametrize("T,d,f", [(100, 1040, 14336), (65, 1288, 10240), (192, 520, 14336), (127, 264, 14328)])
@pytest.mark.parametrize("fp8", [False, True])
def test_grids_of_few_tiles(T, d, f, fp8):
    d = d // 16 * 16 if fp8 else d
    p = Layer(T, d, f, RANKS, 16, BF16, seed=T + d)
    parts, base, extra = p.fp8() if fp8 else (None, None, 0.0)
    for mode in MODES[1:]:
        got = run_forward(p, "gelu_tanh", mode, keep=True, fp8=parts)
        check(p, "gelu_tanh", got, "mode %d" % mode, base=base, extra=extra)
        assert L.lora_get_device_error(got[2].buf) == p.bad_row()


@pytest.mark.parametrize("T,d,f", [(1, 64, 8), (5, 136, 72), (64, 256, 264), (130, 1032, 136), (333, 64, 520),
                                   (900, 264, 2056)])
@pytest.mark.parametrize("act", list(ACTS))
def test_f32(T, d, f, act):
    p = Layer(T, d, f, RANKS, 16, F32, seed=T)
    for mode in MODES[1:]:
        got = run_forward(p, act, mode, keep=True)
        check(p, act, got, "f32")
        assert L.lora_get_device_error(got[2].buf) == p.bad_row()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("T,f", [(40, 200), (600, 3400)])
def test_activations(act, T, f):
    p = Layer(T, 512, f, RANKS, 16, BF16, seed=5)
    p.x[0] *= 40                       # far into both tails of the activation
    p.x[1] *= 2.0 ** -30               # and near its zero
    check(p, act, run_forward(p, act, keep=True), act)


@pytest.mark.parametrize("dtype,T,f", [(BF16, 3, 264), (BF16, 200, 264), (BF16, 900, 4096), (F32, 90, 264),
                                       (F32, 2100, 264)])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
def test_parts_left_out(dtype, T, f, bias, residual):
    p = Layer(T, 264, f, RANKS, 16, dtype, seed=6)
    for act in ("none", "silu"):
        got = run_forward(p, act, bias=bias, residual=residual, keep=bias)
        check(p, act, got, act, bias, residual)


@pytest.mark.parametrize("R,ranks", [(8, [8, 1]), (24, [24, 17, 5]), (40, [33, 40, 0, 8]), (128, [128, 65, 20])])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ranks(R, ranks, packed, dtype):
    for T, order in ((9, "random"), (520, "random"), (2100, "sorted")):
        p = Layer(T, 128, 3464, ranks, R, dtype, seed=R, packed=packed, order=order)
        for mode in MODES[1:]:
            check(p, "silu", run_forward(p, "silu", mode), "R %d T %d" % (R, T))


@pytest.mark.parametrize("T,f", [(250, 4096), (1020, 4104), (3600, 4096)])
@pytest.mark.parametrize("S", [40, 300])
def test_blocks_of_many_adapters(T, f, S):
    """Every row its own adapter, or short runs: the terms of such blocks are added row by row."""
    ranks = [(5 * i) % 16 + 1 for i in range(S)]
    for ids in (np.arange(T) % S, np.repeat(np.arange(T // 7 + 1), 7)[:T] % S):
        p = Layer(T, 136, f, ranks, 16, BF16, seed=S, ids=ids)
        for mode in MODES:
            check(p, "gelu_tanh", run_forward(p, "gelu_tanh", mode), "mode %d" % mode)


def test_ids():
    """No adapter at all, one adapter for all, ids out of range, runs that cross the tiles."""
    T, S = 530, 5
    rng = np.random.default_rng(0)
    odd = rng.integers(-1, S, size=T).astype(np.int32)
    odd[[3, 77, 400]] = [S, -2, 10 ** 6]
    runs = np.repeat([0, -1, 2, 1, 4], [70, 33, 250, 1, T - 354]).astype(np.int32)
    for ids in (np.full(T, -1, np.int32), np.full(T, 2, np.int32), odd, runs):
        for dtype in (BF16, F32):
            p = Layer(T, 192, 968, [8, 16, 12, 16, 2], 16, dtype, seed=1, ids=ids)
            for mode in MODES[:2]:
                got = run_forward(p, "silu", mode)
                check(p, "silu", got, "ids")
                assert L.lora_get_device_error(got[2].buf) == p.bad_row()


def test_rows_of_nan_and_an_adapter_of_infinities_keep_to_themselves():
    for T, dtype in ((60, BF16), (1500, BF16), (60, F32), (600, F32)):
        ids = np.arange(T, dtype=np.int32) % 3
        p = Layer(T, 256, 4096, [8, 16, 4], 16, dtype, seed=4, ids=ids)
        p.x[17] = float("nan")
        p.B[1, 2, 5] = float("inf")
        p.pool.upload(1, p.A[1], p.B[1], 16, p.alphas[1], lda=p.R, ldb=p.f)
        for mode in MODES:
            y = run_forward(p, "silu", mode)[0]
            assert torch.isnan(y[17]).all()
            hit = torch.as_tensor(ids == 1, device="cuda")
            rest = torch.as_tensor(np.flatnonzero((ids != 1) & (np.arange(T) != 17)), device="cuda")
            assert not torch.isfinite(y[hit, 5]).any()
            x, B = p.x.clone(), p.B.clone()
            p.x[17], p.B[1, 2, 5] = 0, 0
            ref, tol, _, _ = p.forward64("silu")
            p.x, p.B = x, B
            within(y[rest], ref[rest], tol[rest], "rows beside")


def test_rows_past_the_batch_stay():
    for dtype in (BF16, F32):
        p = Layer(70, 128, 264, [8, 8], 8, dtype, seed=6)
        y, pre = (torch.full((90, 264), 3.0, dtype=dtype, device="cuda") for _ in range(2))
        ws = L.Workspace(90, 2, 8, 264)
        L.lora_linear_act_forward(p.x, p.W, p.bias, None, y, 70, p.desc, p.ids_dev, 0, L.LORA_MODE_AUTO, 0, ws.buf,
                                  pre=pre)
        assert (y[70:] == 3).all() and (pre[70:] == 3).all()
        check(p, "silu", (y[:70], pre[:70]), "first rows", residual=False)
        y.fill_(3)
        L.lora_linear_act_forward(p.x, p.W, p.bias, None, y, 0, p.desc, p.ids_dev, 0, L.LORA_MODE_AUTO, 0, ws.buf)
        assert (y == 3).all()


@pytest.mark.parametrize("dtype,T,f", [(BF16, 1, 4096), (BF16, 150, 1000), (BF16, 900, 4096), (F32, 40, 520)])
def test_residual_stream_in_place(dtype, T, f):
    p = Layer(T, 520, f, RANKS, 16, dtype, seed=7)
    ref = run_forward(p, "none")[0]
    stream = p.residual
    L.lora_linear_act_forward(p.x, p.W, p.bias, stream, stream, T, p.desc, p.ids_dev, ACTS["none"], 0, 0,
                              L.Workspace(T, p.S, p.R, f).buf)
    assert torch.equal(stream, ref)


def test_no_room_for_a_split_and_segments_ready():
    """A workspace without partials computes every tile whole; segments built once serve later calls."""
    for T in (90, 1):
        p = Layer(T, 1024, 1000, [8, 16], 16, BF16, seed=8)
        ws = L.Workspace(T, 2, 16, 0)
        got = run_forward(p, "silu", L.LORA_MODE_SGMV, ws=ws)
        check(p, "silu", got, "no partials")
        check(p, "silu", run_forward(p, "silu", L.LORA_MODE_BGMV, ws=ws), "no partials, rows in their order")
        L.lora_build_segments(p.ids_dev, T, 2, 16, ws.buf)
        again = run_forward(p, "silu", L.LORA_MODE_SGMV, ws=ws, flags=L.LORA_FLAG_SEGMENTS_READY)
        assert torch.equal(got[0], again[0])
    # segments that a mixed batch's forward built (its own row order beside them)
    p = Layer(700, 264, 4096, [(3 * i) % 16 + 1 for i in range(60)], 16, BF16, seed=9)
    ws = L.Workspace(700, 60, 16, 4096)
    ref = run_forward(p, "silu", ws=ws)[0]
    y = torch.empty_like(ref)
    L.lora_linear_forward(p.x, p.W, y, 700, p.desc, p.ids_dev, L.LORA_MODE_AUTO, 0, ws.buf)
    assert torch.equal(run_forward(p, "silu", ws=ws, flags=L.LORA_FLAG_SEGMENTS_READY)[0], ref)


@pytest.mark.parametrize("dtype,T", [(BF16, 700), (BF16, 90), (F32, 90)])
def test_overwritten_segment_tables_stay_in_bounds(dtype, T):
    p = Layer(T, 264, 520, [8, 16, 5], 16, dtype, seed=31)
    ws = L.Workspace(T, p.S, p.R, p.f)
    words = ws.buf.numel() // 4 * 4
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    ws.buf[:words] = torch.randint(0, 256, (words,), generator=g, device="cuda").to(ws.buf.dtype)
    run_forward(p, "silu", L.LORA_MODE_SGMV, ws=ws, flags=L.LORA_FLAG_SEGMENTS_READY)
    torch.cuda.synchronize()
    L.lora_workspace_init(ws.buf)
    check(p, "silu", run_forward(p, "silu", L.LORA_MODE_SGMV, ws=ws), "built again")


@pytest.mark.parametrize("T,d,f", [(1, 64, 8), (1, 4096, 4096), (1, 1040, 712), (31, 256, 264), (130, 784, 520),
                                   (128, 80, 14336), (300, 144, 7304), (3580, 64, 4088), (1790, 80, 4096),
                                   (1100, 1040, 3400)])
def test_fp8(T, d, f):
    p = Layer(T, d, f, RANKS, 16, BF16, seed=T + f)
    parts, base, extra = p.fp8()
    for mode in MODES:
        got = run_forward(p, "gelu", mode, keep=mode == L.LORA_MODE_SGMV, fp8=parts)
        check(p, "gelu", got, "fp8 mode %d" % mode, base=base, extra=extra)
        assert L.lora_get_device_error(got[2].buf) == p.bad_row()
        made = run_forward(p, "gelu", mode, fp8=parts, codes=False)       # the codes made within the call
        assert torch.equal(made[0], got[0])
        assert L.lora_get_device_error(made[2].buf) == p.bad_row()


@pytest.mark.parametrize("T", [250, 3600])
def test_fp8_blocks_of_many_adapters_and_a_wide_rank(T):
    for S, R in ((60, 16), (3, 64), (2, 128)):
        ranks = [(7 * i) % R + 1 for i in range(S)]
        p = Layer(T, 144, 4096, ranks, R, BF16, seed=S, ids=np.arange(T) % S)
        parts, base, extra = p.fp8()
        for mode in MODES[1:]:
            got = run_forward(p, "none", mode, fp8=parts, keep=True)
            check(p, "none", got, "S %d mode %d" % (S, mode), base=base, extra=extra)


# ---- streams, graphs, repeats --------------------------------------------------
@pytest.mark.parametrize("T,fp8,dtype", [(1, False, BF16), (200, False, BF16), (1400, False, BF16), (200, True, BF16),
                                         (1400, True, BF16), (90, False, F32)])
def test_repeats_other_streams_and_graphs(T, fp8, dtype):
    p = Layer(T, 1024, 3400, RANKS, 16, dtype, seed=T)
    parts = p.fp8()[0] if fp8 else None
    ref = run_forward(p, "silu", fp8=parts)[0]
    assert torch.equal(ref, run_forward(p, "silu", fp8=parts)[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]     # two calls at once, each with its own workspace
    wss = [L.Workspace(T, p.S, p.R, p.f, fp8_d_in=p.d if fp8 else 0) for _ in streams]
    torch.cuda.synchronize()
    outs = []
    for st, ws in zip(streams, wss):
        with torch.cuda.stream(st):
            outs.append(run_forward(p, "silu", ws=ws, stream=st, fp8=parts)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    # captured, and replayed on what the buffers then hold: other rows, ids and adapters
    y = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_forward(p, "silu", ws=wss[0], fp8=parts, codes=False, y=y)
    rng = np.random.default_rng(0)
    for ids in (p.ids, np.zeros(T), np.arange(T) % p.S, np.full(T, -1), rng.integers(-2, p.S + 2, size=T)):
        p.ids_dev.copy_(torch.as_tensor(np.asarray(ids).astype(np.int32)))
        p.x.copy_(p.x.roll(1, 1).clone())
        p.residual.copy_(p.residual.roll(1, 1).clone())
        p.pool.upload(0, p.A[1], p.B[1], 1 + int(rng.integers(p.R)), 4.0, lda=p.R, ldb=p.f)
        y.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = run_forward(p, "silu", ws=wss[1], fp8=parts, codes=False)[0]
        assert torch.equal(y, eager)


class Guarded:
    """Buffers with 256 KiB of 0x5a on both sides."""

    def __init__(self):
        self.raw = []

    def __call__(self, *shape, dtype=torch.uint8):
        n, guard = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size(), 1 << 18
        raw = torch.full((2 * guard + (n + 255) // 256 * 256,), 0x5a, dtype=torch.uint8, device="cuda")
        self.raw.append((raw, n))
        return raw[guard:guard + n].view(dtype).view(shape)

    def check(self):
        guard = 1 << 18
        for raw, n in self.raw:
            assert bool((raw[:guard] == 0x5a).all()) and bool((raw[guard + n:] == 0x5a).all())


@pytest.mark.parametrize("T,d,f,S,R", [(1, 64, 8, 1, 8), (33, 272, 136, 3, 16), (130, 784, 520, 200, 8),
                                       (300, 144, 7304, 4, 24), (700, 48, 40, 37, 64), (2047, 1808, 264, 5, 40)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_writes_stay_in_bounds(T, d, f, S, R, dtype):
    ranks = [(7 * i) % R + 1 for i in range(S)]
    p = Layer(T, d, f, ranks, R, dtype, seed=1)
    for mode in MODES:
        for split in (f, 0):                              # with and without room for pieces of K
            for fp8 in (False, True)[:1 + (dtype == BF16)]:
                new = Guarded()
                n = L.lora_workspace_bytes_fp8(T, S, R, d, split) if fp8 else L.lora_workspace_bytes(T, S, R, split)
                ws, y, pre = new(n), new(T, f, dtype=dtype), new(T, f, dtype=dtype)
                L.lora_workspace_init(ws)
                if fp8:
                    w = L.Fp8Weight(p.W)
                    L.lora_linear_act_forward_fp8(p.x, None, None, w.codes, w.scale, p.bias, p.residual, y, T, p.desc,
                                                  p.ids_dev, 0, mode, 0, ws, pre=pre)
                else:
                    L.lora_linear_act_forward(p.x, p.W, p.bias, p.residual, y, T, p.desc, p.ids_dev, 0, mode, 0, ws,
                                              pre=pre)
                new.check()


def test_the_binding_refuses_tensors_the_kernels_would_misread():
    p = Layer(6, 64, 128, [8, 8], 8, BF16, seed=13)
    ws = L.Workspace(6, 2, 8, 128)
    good = dict(x=p.x, W=p.W, bias=p.bias, residual=p.residual, y=torch.empty_like(p.residual),
                pre=torch.empty_like(p.residual), ids=p.ids_dev)
    for name, t in good.items():
        for other in (t.double(), t.cpu(), torch.stack([t, t], -1)[..., 0], t[:0]):
            v = dict(good, **{name: other})
            with pytest.raises(L.LoraError) as e:
                L.lora_linear_act_forward(v["x"], v["W"], v["bias"], v["residual"], v["y"], 6, p.desc, v["ids"], 0, 0, 0,
                                          ws.buf, pre=v["pre"])
            assert e.value.status == L.LORA_ERR_INVALID_ARGUMENT
