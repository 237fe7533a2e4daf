"""lora_linear_act_backward against the gradients' formulas in 64 bits (bounds in
helpers_act.backward64), those against differences of the forward pass, and a
biased block forward, backward and updated as it would be trained."""
import numpy as np
import pytest
import torch

from helpers_act import ACTS, Layer, act64, backward64, run_backward, run_forward
from helpers_block import STEP32, within
from rank_adapter_gemm_amd import lora as L
from test_gpu_linear_act import Guarded

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


def kept(p, seed=0):
    """The activation's argument and dy as a forward pass and a loss leave them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 100)
    new = lambda std: (std * torch.randn(p.T, p.f, generator=g, device="cuda")).to(p.dtype)  # noqa: E731
    return new(1.3), new(0.02)


def check(p, act, pre, dy, got, what):
    for name, (ref, tol), out in zip(("dx", "dA", "dB", "dbias"), backward64(p, act, pre, dy), got):
        if out is not None:
            within(out, ref, tol, what + " " + name)


RANKS = [16, 3, 8, 0, 13, 16, 1]

SHAPES = [(1, 64, 8), (1, 1032, 712), (2, 512, 1000), (31, 264, 256), (64, 1024, 2048), (130, 520, 776),
          (300, 136, 1064), (700, 40, 8), (2048, 3336, 72), (1100, 1032, 1400), (4200, 64, 64), (1797, 1800, 8208),
          (3500, 3800, 72), (2000, 3496, 136), (2000, 1080, 520)]


@pytest.mark.parametrize("T,d,f", SHAPES)
@pytest.mark.parametrize("act", ["none", "silu"])
def test_bf16(T, d, f, act):
    p = Layer(T, d, f, RANKS, 16, BF16, seed=T + f)
    k = kept(p)
    got = run_backward(p, act, *k)
    check(p, act, *k, got, "bf16")
    assert L.lora_get_device_error(got[4].buf) == p.bad_row()


@pytest.mark.parametrize("T,d,f", [(777, 1048, 1032), (129, 2056, 1288), (500, 4096, 520)])
def test_ranges_of_the_sum_in_whole_rounds(T, d, f):
    for act in ("none", "gelu"):
        p = Layer(T, d, f, RANKS, 16, BF16, seed=T + d)
        k = kept(p)
        check(p, act, *k, run_backward(p, act, *k), "bf16")


# 306 whole tiles of 256 x 256: the adapters' gradients run beside the last round, two column tiles a workgroup (35 and
# 7 of them here); one adapter of over 1024 rows, and none with rows
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("ids", ["random", "one", "none"])
@pytest.mark.parametrize("R", [16, 32])
def test_gradients_beside_dx(act, ids, R):
    T, d, f = 4100, 4360, 888
    ranks = [min(R, r) for r in (32, 3, 8, 0, 13, 30, 1)]
    p = Layer(T, d, f, ranks, R, BF16, seed=R,
              ids=None if ids == "random" else np.full(T, 0 if ids == "one" else -1, np.int32))
    k = kept(p)
    got = run_backward(p, act, *k)
    check(p, act, *k, got, ids)
    assert L.lora_get_device_error(got[4].buf) == p.bad_row()
    again = run_backward(p, act, *k)
    assert all(torch.equal(a, b) for a, b in zip(got[:4], again[:4]))


@pytest.mark.parametrize("T,d,f", [(1, 64, 8), (5, 136, 72), (64, 264, 256), (130, 136, 1032), (333, 520, 64),
                                   (700, 264, 520)])
@pytest.mark.parametrize("act", list(ACTS))
def test_f32(T, d, f, act):
    p = Layer(T, d, f, RANKS, 16, F32, seed=T)
    k = kept(p)
    got = run_backward(p, act, *k)
    check(p, act, *k, got, act)
    assert L.lora_get_device_error(got[4].buf) == p.bad_row()


@pytest.mark.parametrize("act", list(ACTS))
def test_activations(act):
    p = Layer(260, 136, 520, RANKS, 16, BF16, seed=3)
    pre, dy = kept(p)
    pre[0], pre[1], pre[2] = pre[0] * 60, pre[1] * 2.0 ** -30, 0
    check(p, act, pre, dy, run_backward(p, act, pre, dy), act)


@pytest.mark.parametrize("R,ranks", [(8, [8, 1]), (24, [24, 17, 5]), (40, [33, 40, 0, 8]), (64, [64, 63]),
                                     (72, [72, 9]), (96, [96, 80, 1]), (128, [128, 65, 20])])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ranks(R, ranks, packed, dtype):
    for T in (9, 300, 1500 if dtype == BF16 else 150):
        p = Layer(T, 136, 264, ranks, R, dtype, seed=R + T, packed=packed)
        for act in ("none", "gelu"):
            k = kept(p)
            check(p, act, *k, run_backward(p, act, *k), "R %d T %d" % (R, T))


@pytest.mark.parametrize("T,S", [(777, 24), (1500, 300), (1100, 2)])
def test_many_adapters_and_long_segments(T, S):
    ranks = [(5 * i) % 24 + 1 for i in range(S)]
    for ids in (None, np.arange(T) % S, np.sort(np.arange(T) % S), np.full(T, S - 1), np.full(T, -1)):
        p = Layer(T, 520, 1032, ranks, 24, BF16, seed=S, ids=ids)
        k = kept(p)
        check(p, "gelu_tanh", *k, run_backward(p, "gelu_tanh", *k), "S %d" % S)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_what_is_asked_for(dtype, act):
    p = Layer(200, 264, 520, RANKS, 16, dtype, seed=6)
    k = kept(p)
    full = run_backward(p, act, *k)
    check(p, act, *k, full, "all")
    for want in (("dx",), ("ab",), ("bias",), ("dx", "ab"), ("ab", "bias"), ()):
        got = run_backward(p, act, *k, want=want)
        for a, b in zip(got[:4], full):
            assert a is None or torch.equal(a, b)


def test_no_rows_give_zeros():
    for dtype in (BF16, F32):
        p = Layer(4, 64, 72, [8, 3], 8, dtype, seed=7)
        p.T = 0
        _, dA, dB, db, _ = run_backward(p, "silu", *[t[:0] for t in (p.residual, p.residual)], want=("ab", "bias"))
        assert not dA.any() and not dB.any() and not db.any()


def test_rows_of_nan_keep_to_themselves():
    """A row's NaN reaches its dx, its adapter's gradients and dbias, nothing of another row or adapter."""
    for T, dtype in ((300, BF16), (90, F32)):
        p = Layer(T, 136, 264, [8, 16, 4], 16, dtype, seed=8, ids=np.arange(T) % 3)
        pre, dy = kept(p)
        ref = run_backward(p, "silu", pre, dy)
        dy[17] = float("nan")                                # a row of slot 2
        dx, dA, dB, db, _ = run_backward(p, "silu", pre, dy)
        rest = torch.tensor([t for t in range(T) if t != 17], device="cuda")
        assert torch.isnan(dx[17]).all() and torch.equal(dx[rest], ref[0][rest]) and torch.isnan(db).all()
        assert torch.equal(dA[:2], ref[1][:2]) and torch.equal(dB[:2], ref[2][:2])


def test_gradients_are_those_of_differences():
    """Central differences of the forward formula in 64 bits, along x, A, B and the bias; and of the residual dy itself."""
    for act in ACTS:
        p = Layer(9, 40, 24, [8, 5], 8, F32, seed=11)
        y, pre, _ = run_forward(p, act, keep=True)
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        dy = torch.randn(p.T, p.f, generator=g, device="cuda")
        dx, dA, dB, db, _ = run_backward(p, act, pre, dy)

        def loss(x, A, B, bias):
            q = x @ p.W.double() + bias
            for s, r in enumerate(p.ranks):
                t = torch.as_tensor(np.flatnonzero(p.ids == s), device="cuda")
                q = q.index_add(0, t, p.scale(s) * ((x[t] @ A[s, :, :r]) @ B[s, :r]))
            return (act64(act, q)[0] * dy.double()).sum()

        at = [t.double() for t in (p.x, p.A, p.B, p.bias)]
        for i, grad in enumerate((dx, dA, dB, db)):
            step = torch.randn(grad.shape, generator=g, device="cuda").double()
            lo, hi = list(at), list(at)
            lo[i], hi[i] = at[i] - 1e-5 * step, at[i] + 1e-5 * step
            diff = float(loss(*hi) - loss(*lo)) / 2e-5
            # sums of 40 to 400 fp32 products of order 1, and the difference's own 1e-10 / 1e-5
            assert abs(diff - float((grad.double() * step).sum())) < 1e-3 * (1 + float(grad.double().norm() * step.norm()))


@pytest.mark.parametrize("T,d,f,S,R", [(1, 64, 8, 1, 8), (33, 272, 136, 3, 16), (130, 784, 520, 200, 8),
                                       (300, 144, 2304, 4, 24), (700, 48, 40, 37, 64), (1025, 1040, 1400, 700, 72)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_writes_stay_in_bounds(T, d, f, S, R, dtype):
    ranks = [(7 * i) % R + 1 for i in range(S)]
    for ids in (None, np.arange(T) % S, np.full(T, S - 1), np.full(T, -1)):
        p = Layer(T, d, f, ranks, R, dtype, seed=1, ids=ids)
        pre, dy = kept(p)
        for act in ("none", "silu"):
            new = Guarded()
            ws = new(L.lora_workspace_bytes_linear_act_backward(T, S, R, d, f, L.dtype_code(dtype)))
            L.lora_workspace_init(ws)
            dx, dA, dB, db = (new(*s, dtype=dtype) for s in ((T, d), (S, d, R), (S, R, f), (f,)))
            L.lora_linear_act_backward(p.x, p.W, T, p.desc, p.ids_dev, ACTS[act], pre, dy, dx, dA, dB, db, ws)
            new.check()


@pytest.mark.parametrize("T,dtype,act", [(3, BF16, "none"), (700, BF16, "none"), (700, BF16, "silu"), (90, F32, "gelu")])
def test_repeats_other_streams_and_graphs(T, dtype, act):
    p = Layer(T, 528, 776, [16, 16, 5, 9], 16, dtype, seed=T)
    pre, dy = kept(p)
    ref = run_backward(p, act, pre, dy)[:4]
    wss = [L.Workspace(T, p.S, p.R, p.f, linear_backward_d_in=p.d, dtype=dtype) for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for ws in wss:                                           # two calls at once
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            outs.append(run_backward(p, act, pre, dy, ws=ws, stream=st)[:4])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, ref))
    graph = torch.cuda.CUDAGraph()
    out = [torch.empty_like(t) for t in ref]
    with torch.cuda.graph(graph):
        L.lora_linear_act_backward(p.x, p.W, T, p.desc, p.ids_dev, ACTS[act], pre, dy, *out, wss[0].buf)
    rng = np.random.default_rng(0)
    for ids in (p.ids, np.zeros(T), np.arange(T) % p.S, np.full(T, -1), rng.integers(-2, p.S + 2, size=T)):
        p.ids_dev.copy_(torch.as_tensor(np.asarray(ids).astype(np.int32)))
        p.x.copy_(p.x.roll(1, 1).clone())
        dy.copy_(dy.roll(1, 1).clone())
        p.pool.upload(0, p.A[1], p.B[1], 1 + int(rng.integers(p.R)), 4.0, lda=p.R, ldb=p.f)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = run_backward(p, act, pre, dy, ws=wss[1])
        assert all(torch.equal(a, b) for a, b in zip(out, eager))


def test_the_binding_refuses_tensors_the_kernels_would_misread():
    p = Layer(6, 64, 128, [8, 8], 8, BF16, seed=13)
    pre, dy = kept(p)
    ws = L.Workspace(6, 2, 8, 128, linear_backward_d_in=64)
    good = dict(x=p.x, W=p.W, ids=p.ids_dev, pre=pre, dy=dy, dx=torch.empty_like(p.x), dA=torch.empty_like(p.A),
                dB=torch.empty_like(p.B), db=torch.empty_like(p.bias))
    for name, t in good.items():
        for other in (t.double(), t.cpu(), torch.stack([t, t], -1)[..., 0], t[:0]):
            v = dict(good, **{name: other})
            with pytest.raises(L.LoraError) as e:
                L.lora_linear_act_backward(v["x"], v["W"], 6, p.desc, v["ids"], 0, v["pre"], v["dy"], v["dx"], v["dA"],
                                           v["dB"], v["db"], ws.buf)
            assert e.value.status == L.LORA_ERR_INVALID_ARGUMENT
    with pytest.raises(L.LoraError):
        L.Workspace(6, 2, 8, 128, linear_backward_d_in=64, gated=True)


# ---- the block as it is trained ----------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_training_step_of_the_biased_block(dtype):
    """Norm, first layer with GELU, second layer onto the residual stream; backward through all three; orthogonalised
    updates of the adapters, uploaded.  Every stage against its 64-bit formula on the values the stage before left."""
    T, d, f, R, S, eps = 300, 136, 264, 16, 3, 1e-5
    rng = np.random.default_rng(0)
    ids = rng.integers(-1, S, size=T).astype(np.int32)
    one = Layer(T, d, f, [16, 9, 4], R, dtype, seed=1, ids=ids)
    two = Layer(T, f, d, [16, 9, 4], R, dtype, seed=2, ids=ids)
    new = lambda *shape: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    x, stream, weight, bias = one.x, two.residual, 1 + 0.1 * one.bias[:1].expand(d), 0.1 * one.bias[:d]
    weight, bias = weight.contiguous(), bias.contiguous()
    z, y, mean, rstd = new(T, d), new(T, d), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    code = L.dtype_code(dtype)
    L.lora_add_layernorm(x, stream, weight, bias, eps, T, d, code, z, y, mean, rstd)
    one.x, two.residual = y, z
    h, pre, _ = run_forward(one, "gelu", residual=False, keep=True)
    two.x = h
    out = run_forward(two, "none")[0]
    for p, got, act, res in ((one, h, "gelu", False), (two, out, "none", True)):
        ref, tol, _, _ = p.forward64(act, residual=res)
        within(got, ref, tol, "forward")
    # backward: the loss's gradient reaches the second layer and, past it, the stream
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    dout = (0.02 * torch.randn(T, d, generator=g, device="cuda")).to(dtype)
    back2 = run_backward(two, "none", None, dout)
    check(two, "none", None, dout, back2, "second layer")
    back1 = run_backward(one, "gelu", pre, back2[0])
    check(one, "gelu", pre, back2[0], back1, "first layer")
    dz, dw, db = new(T, d), new(d), new(d)
    ws = torch.empty(L.lora_workspace_bytes_layernorm_backward(T, d), dtype=torch.uint8, device="cuda")
    L.lora_add_layernorm_backward(back1[0], dout, z, weight, mean, rstd, T, d, code, dz, dw, db, ws)
    from test_gpu_layernorm import check_backward
    check_backward((dz, dw, db), back1[0], dout, z, weight, mean, rstd)
    # updates of both layers' adapters, and a forward pass with them
    from test_gpu_orthogonalize import USUAL, check as check_update, run as update
    for p, back in ((one, back1), (two, back2)):
        for grad, par in ((back[1], p.A), (back[2], p.B)):
            step = update(grad, scale=0.2)
            check_update(step, grad, scale=0.2)
            par -= (0.05 * step.float()).to(dtype)
        for s, r in enumerate(p.ranks):
            assert not (p.A[s, :, r:] != 0).logical_and(back[1][s, :, r:] != 0).any()
            p.pool.upload(s, p.A[s], p.B[s], r, p.alphas[s], lda=R, ldb=p.f)
    again = run_forward(one, "gelu", residual=False)[0]
    ref, tol, _, _ = one.forward64("gelu", residual=False)
    within(again, ref, tol, "with updated adapters")
    assert not torch.equal(again, h)
