"""lora_add_layernorm, its FP8 form and its backward pass against the plain
form in 64 bits.

Forward bounds: a sum over a row adds at most N = 66 + d / 1024 terms one after
the other (40 a thread, or d / 1024; 26 in the reduction), each off by a step.
So the mean is off by dm = N steps of mean|z|; z - mean by dm, z's own sum and
the difference; the variance by what the row's rms of that does to the squares
and N steps; half of it enters 1 / sqrt with 6 steps; then two products, a sum
with the bias and one rounding.

Backward bounds: the same counts on a = dy w and a h; h is off by three steps of
its two factors.  dweight and dbias add at most T / 256 + 64 + 24 terms one after
the other."""
import pytest
import torch

from helpers_block import HALF, STEP32, within
from rank_adapter_gemm_amd import lora as L

pytestmark = pytest.mark.gpu
EPS = 1e-5
BF16, F32 = torch.bfloat16, torch.float32
TINY = 2.0 ** -120


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


def make(T, d, dtype, seed=0, shift=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 31 * T + d)
    x = (torch.randn(T, d, generator=g, device="cuda") + shift).to(dtype)
    r = (3 * torch.randn(T, d, generator=g, device="cuda")).to(dtype)
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    b = (0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    return x, r, w, b


def check(got, x, r, w, b, eps=EPS):
    """z, y, mean, rstd as the kernel gave them (None: not looked at)."""
    z_got, y_got, mean_got, rstd_got = got
    half, d = HALF[x.dtype], x.shape[1]
    z = x.double() + (r.double() if r is not None else 0)
    mean = z.mean(1, keepdim=True)
    c = z - mean
    var = c.square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    n = (66 + d / 1024) * STEP32
    dm = (n + STEP32) * z.abs().mean(1, keepdim=True)
    dc = dm + 2 * STEP32 * (z.abs() + c.abs())
    rms = dc.square().mean(1, keepdim=True).sqrt()
    dvar = 2 * var.sqrt() * rms + rms * rms + (n + 2 * STEP32) * var
    rel = 0.5 * dvar / (var + eps) * 1.01 + 6 * STEP32
    if z_got is not None:
        within(z_got, z, (half + STEP32) * z.abs(), "z")
    if mean_got is not None:
        within(mean_got[:, None], mean, dm + TINY, "mean")
        within(rstd_got[:, None], rstd, rel * rstd, "rstd")
    bias = b.double() if b is not None else torch.zeros_like(w).double()
    h = c * rstd * w.double()
    y = h + bias
    tol = w.double().abs() * (dc * rstd * (1 + rel)) + h.abs() * (rel + 3 * STEP32) + STEP32 * y.abs()
    if y_got is not None:
        within(y_got, y, tol * (1 + half) + half * y.abs() + TINY, "y")


def forward(x, r, w, b, keep=True, **kw):
    T, d = x.shape
    z, y = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty(T, device="cuda") for _ in range(2)) if keep else (None, None)
    L.lora_add_layernorm(x, r, w, b, EPS, T, d, L.dtype_code(x.dtype), z, y, mean, rstd, **kw)
    return z, y, mean, rstd


SIZES = [(1, 8), (1, 4096), (3, 16), (5, 504), (130, 512), (7, 1024), (64, 1032), (9, 2048), (33, 4104), (4, 8192),
         (3, 16384), (2, 16392), (2, 32768), (2, 32776), (1, 70000), (5000, 64), (11, 1800), (11, 3592), (11, 7184)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d", SIZES)
def test_forward(T, d, dtype):
    x, r, w, b = make(T, d, dtype)
    check(forward(x, r, w, b), x, r, w, b)
    y = torch.empty_like(x)                                  # no residual, no bias, nothing kept
    L.lora_add_layernorm(x, None, w, None, EPS, T, d, L.dtype_code(dtype), None, y)
    check((None, y, None, None), x, None, w, None)


@pytest.mark.parametrize("T,d", [(T, d) for T, d in SIZES if d % 16 == 0])
def test_codes_are_those_of_the_stored_rows(T, d):
    x, r, w, b = make(T, d, BF16, seed=3)
    z, y, mean, rstd = forward(x, r, w, b)
    z2, y2, mean2, rstd2 = (torch.empty_like(t) for t in (z, y, mean, rstd))
    q, s = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    L.lora_add_layernorm_fp8(x, r, w, b, EPS, T, d, z2, y2, q, s, mean2, rstd2)
    assert torch.equal(z, z2) and torch.equal(y, y2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    L.lora_quantize_rows_fp8(y, T, d, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    q3, s3 = torch.empty_like(q), torch.empty_like(s)        # codes only
    L.lora_add_layernorm_fp8(x, r, w, b, EPS, T, d, None, None, q3, s3)
    assert torch.equal(q, q3) and torch.equal(s, s3)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_far_from_zero(dtype):
    """A mean 30 times the spread: a variance from the squares' mean would be lost in it."""
    x, _, w, b = make(33, 1032, dtype, shift=30.0)
    check(forward(x, None, w, b), x, None, w, b)


@pytest.mark.parametrize("d", [64, 1024, 4096, 40000])
def test_in_place(d):
    T = 37
    x, r, w, b = make(T, d, BF16, seed=5)
    z, y, _, _ = forward(x, r, w, b)
    for swap in (False, True):
        xa, ra = x.clone(), r.clone()
        zo, yo = (xa, ra) if swap else (ra, xa)
        L.lora_add_layernorm(xa, ra, w, b, EPS, T, d, L.LORA_BF16, zo, yo)
        assert torch.equal(zo, z) and torch.equal(yo, y)


def test_rows_keep_to_themselves():
    """Rows of one value, of tiny values, and a row with NaN and one with an infinity between them."""
    T, d = 9, 1032
    x, r, w, b = make(T, d, BF16, seed=7)
    x[2], r[2] = 1.5, 0
    x[3] *= 2.0 ** -60
    r[3] *= 2.0 ** -60
    x[6, 17] = float("nan")
    x[7, 3] = float("inf")
    z, y, mean, rstd = forward(x, r, w, b)
    assert torch.isnan(y[6]).all() and torch.isnan(y[7]).all()
    assert torch.equal(y[2], b)
    rest = torch.tensor([0, 1, 2, 3, 4, 5, 8], device="cuda")
    check((z[rest], y[rest], mean[rest], rstd[rest]), x[rest], r[rest], w, b)


def test_rows_past_the_batch_stay_and_no_rows_is_no_work():
    x, r, w, b = make(12, 256, BF16, seed=9)
    z, y = torch.full_like(x, 5), torch.full_like(x, 5)
    mean, rstd = (torch.full((12,), 5.0, device="cuda") for _ in range(2))
    L.lora_add_layernorm(x, r, w, b, EPS, 7, 256, L.LORA_BF16, z, y, mean, rstd)
    assert all((t[7:] == 5).all() for t in (z, y, mean, rstd))
    check((z[:7], y[:7], mean[:7], rstd[:7]), x[:7], r[:7], w, b)
    z.fill_(5)
    L.lora_add_layernorm(x, r, w, b, EPS, 0, 256, L.LORA_BF16, z, y, mean, rstd)
    assert (z == 5).all()


# ---- the backward pass ------------------------------------------------------


def make_backward(T, d, dtype, seed=0):
    x, r, w, b = make(T, d, dtype, seed)
    z, _, mean, rstd = forward(x, r, w, b)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 7)
    dy = torch.randn(T, d, generator=g, device="cuda").to(dtype)
    dres = torch.randn(T, d, generator=g, device="cuda").to(dtype)
    return dy, dres, z, w, mean, rstd


def backward(dy, dres, z, w, mean, rstd, sums=True, ws=None, dx=None, **kw):
    T, d = z.shape
    dx = torch.full_like(z, 7) if dx is None else dx
    dw, db = (torch.full_like(w, 7) for _ in range(2)) if sums else (None, None)
    if ws is None and sums:
        ws = torch.empty(L.lora_workspace_bytes_layernorm_backward(T, d), dtype=torch.uint8, device="cuda")
    L.lora_add_layernorm_backward(dy, dres, z, w, mean, rstd, T, d, L.dtype_code(z.dtype), dx, dw, db, ws, **kw)
    return dx, dw, db


def check_backward(got, dy, dres, z, w, mean, rstd):
    dx_got, dw_got, db_got = got
    T, d = z.shape
    half, n = HALF[z.dtype], (66 + d / 1024) * STEP32
    dy, w, rs = dy.double(), w.double(), rstd.double()[:, None]
    c = z.double() - mean.double()[:, None]
    h, dh = c * rs, 2 * STEP32 * (c.abs() * rs) + STEP32 * z.double().abs() * rs
    a = dy * w
    ma, mah = a.mean(1, keepdim=True), (a * h).mean(1, keepdim=True)
    dma = (n + 2 * STEP32) * a.abs().mean(1, keepdim=True)
    dmah = (n + 3 * STEP32) * (a * h).abs().mean(1, keepdim=True) + (a.abs() * dh).mean(1, keepdim=True)
    dx = rs * (a - ma - h * mah)
    tol = rs * (2 * STEP32 * (a.abs() + ma.abs() + (h * mah).abs()) + dma + h.abs() * dmah + dh * mah.abs()) + \
        2 * STEP32 * dx.abs()
    if dres is not None:
        dx = dx + dres.double()
        tol = tol + STEP32 * dx.abs()
    within(dx_got, dx, tol * (1 + half) + half * dx.abs() + TINY, "dx")
    if dw_got is None:
        return
    m = (T / 256 + 88) * STEP32
    dw, db = (dy * h).sum(0), dy.sum(0)
    within(dw_got, dw, (m * (dy * h).abs().sum(0) + (dy.abs() * dh).sum(0)) * (1 + half) + half * dw.abs() + TINY,
           "dweight")
    within(db_got, db, m * dy.abs().sum(0) * (1 + half) + half * db.abs() + TINY, "dbias")


BACK_SIZES = SIZES + [(1023, 264), (1030, 520), (2500, 1032), (1027, 16400), (4500, 24)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d", BACK_SIZES)
def test_backward(T, d, dtype):
    p = make_backward(T, d, dtype)
    check_backward(backward(*p), *p)
    bare = (p[0], None) + p[2:]
    full = backward(*bare)
    check_backward(full, *bare)
    assert torch.equal(backward(*bare, sums=False)[0], full[0])


def test_backward_is_the_formula_s_gradient_and_that_of_differences():
    """Against 64-bit differentiation of the forward formula, and central differences of it."""
    T, d = 6, 72
    x, r, w, b = make(T, d, F32, seed=21)
    z, _, mean, rstd = forward(x, r, w, b)
    dy, dres = (torch.randn(T, d, device="cuda") for _ in range(2))
    dx, dw, db = backward(dy, dres, z, w, mean, rstd)

    def loss(x, w, b):
        z = x + r.double()
        c = z - z.mean(1, keepdim=True)
        y = c / torch.sqrt(c.square().mean(1, keepdim=True) + EPS) * w + b
        return (y * dy.double()).sum() + (z * dres.double()).sum()

    v = [t.double().requires_grad_() for t in (x, w, b)]
    loss(*v).backward()
    # 72-term sums of fp32: a few hundred steps of values of order 1 to 10
    for got, leaf in zip((dx, dw, db), v):
        assert (got.double() - leaf.grad).abs().max() < 2e-4
    with torch.no_grad():
        for i, got in enumerate((dx, dw, db)):
            step = torch.randn_like(got).double()
            lo, hi = [t.detach() for t in v], [t.detach() for t in v]
            lo[i], hi[i] = lo[i] - 1e-5 * step, hi[i] + 1e-5 * step
            diff = (loss(*hi) - loss(*lo)) / 2e-5
            assert abs(diff - (got.double() * step).sum()) < 2e-3 * (1 + got.double().norm() * step.norm())


@pytest.mark.parametrize("d", [64, 1024, 4096, 40000])
def test_backward_in_place(d):
    p = make_backward(41, d, BF16, seed=5)
    ref = backward(*p)
    for i in range(3):                                       # over dy, dresidual and z
        q = [t.clone() for t in p]
        got = backward(*q, dx=q[i])
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_backward_of_no_rows_and_rows_past_the_batch():
    p = make_backward(12, 256, BF16, seed=9)
    dx, dw, db = torch.full_like(p[2], 5), torch.full_like(p[3], 5), torch.full_like(p[3], 5)
    ws = torch.empty(L.lora_workspace_bytes_layernorm_backward(12, 256), dtype=torch.uint8, device="cuda")
    L.lora_add_layernorm_backward(*p, 7, 256, L.LORA_BF16, dx, dw, db, ws)
    assert (dx[7:] == 5).all()
    check_backward((dx[:7], dw, db), *[t[:7] if t.shape[0] == 12 else t for t in p])
    dx.fill_(5)
    L.lora_add_layernorm_backward(*p, 0, 256, L.LORA_BF16, dx, dw, db, ws)
    assert (dx == 5).all() and (dw == 0).all() and (db == 0).all()


def test_backward_rows_keep_to_themselves():
    """A row's NaN reaches its own dx and the sums over rows, no other row's dx."""
    p = make_backward(9, 520, BF16, seed=13)
    p[0][4, 11] = float("nan")
    dx, dw, db = backward(*p)
    rest = torch.tensor([0, 1, 2, 3, 5, 6, 7, 8], device="cuda")
    assert torch.isnan(dx[4]).all() and torch.isnan(dw[11]) and torch.isnan(db[11])
    assert torch.isfinite(dx[rest].float()).all() and torch.isfinite(db[:11].float()).all()


def test_deterministic_on_another_stream_and_in_a_graph():
    T, d = 2201, 4096
    p = make_backward(T, d, BF16, seed=11)
    x, r, w, b = make(T, d, BF16, seed=11)
    z, y, mean, rstd = forward(x, r, w, b)
    dx, dw, db = backward(*p)
    ws = torch.empty(L.lora_workspace_bytes_layernorm_backward(T, d), dtype=torch.uint8, device="cuda")
    outs = (z, y, mean, rstd, dx, dw, db)
    ref = [t.clone() for t in outs]

    def call(**kw):
        L.lora_add_layernorm(x, r, w, b, EPS, T, d, L.LORA_BF16, z, y, mean, rstd, **kw)
        L.lora_add_layernorm_backward(p[0], p[1], z, w, mean, rstd, T, d, L.LORA_BF16, dx, dw, db, ws, **kw)

    def same():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
        for t in outs:
            t.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()

    same()
    call(stream=torch.cuda.Stream())
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        graph.replay()
        same()


def test_writes_stay_in_bounds():
    """Outputs and a workspace of exactly the named size between guard bytes."""
    for T, d, dtype in [(1, 8, BF16), (3, 520, F32), (1030, 136, BF16), (2, 33000, F32)]:
        p = make_backward(T, d, dtype, seed=2)
        raw = []

        def new(n, dt):
            size = n * torch.empty((), dtype=dt).element_size()
            t = torch.full((size + 8192 + 256,), 0x5a, dtype=torch.uint8, device="cuda")
            raw.append((t, size))
            return t[4096:4096 + size].view(dt)

        dx, dw, db = new(T * d, dtype), new(d, dtype), new(d, dtype)
        ws = new(L.lora_workspace_bytes_layernorm_backward(T, d), torch.uint8)
        L.lora_add_layernorm_backward(*p, T, d, L.dtype_code(dtype), dx, dw, db, ws)
        assert all((t[:4096] == 0x5a).all() and (t[4096 + n:] == 0x5a).all() for t, n in raw)


def test_the_binding_refuses_tensors_the_kernels_would_misread():
    x, r, w, b = make(6, 256, BF16, seed=13)
    p = make_backward(6, 256, BF16)
    ws = torch.empty(L.lora_workspace_bytes_layernorm_backward(6, 256), dtype=torch.uint8, device="cuda")
    wide = torch.empty(6, 512, dtype=BF16, device="cuda")
    names = ["x", "r", "w", "b", "z", "y", "mean", "rstd"]
    good = dict(zip(names, (x, r, w, b, torch.empty_like(x), torch.empty_like(x), p[4], p[5])))
    back = dict(zip(["dy", "dres", "z", "w", "mean", "rstd", "dx", "dw", "db"],
                    p + (torch.empty_like(x), torch.empty_like(w), torch.empty_like(w))))
    for other in (x.double(), x.cpu(), wide[:, :256], wide[:, ::2], x[:0]):
        for name in good:
            v = dict(good, **{name: other})
            with pytest.raises(L.LoraError) as e:
                L.lora_add_layernorm(v["x"], v["r"], v["w"], v["b"], EPS, 6, 256, L.LORA_BF16, v["z"], v["y"],
                                     v["mean"], v["rstd"])
            assert e.value.status == L.LORA_ERR_INVALID_ARGUMENT
        for name in back:
            v = dict(back, **{name: other})
            with pytest.raises(L.LoraError) as e:
                L.lora_add_layernorm_backward(v["dy"], v["dres"], v["z"], v["w"], v["mean"], v["rstd"], 6, 256,
                                              L.LORA_BF16, v["dx"], v["dw"], v["db"], ws)
            assert e.value.status == L.LORA_ERR_INVALID_ARGUMENT
