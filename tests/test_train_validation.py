"""Refusals of the layer norm's, its backward pass's and the orthogonalised
update's entry points, on the host: every call below returns before anything is
enqueued (the addresses are made up)."""
import ctypes

import pytest

from rank_adapter_gemm_amd import lora as L

FAKE = 1 << 40
INVALID, UNSUPPORTED, SMALL, OK = (L.LORA_ERR_INVALID_ARGUMENT, L.LORA_ERR_UNSUPPORTED,
                                   L.LORA_ERR_WORKSPACE_TOO_SMALL, L.LORA_OK)
A = [FAKE + (i << 30) for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    return L.load()


def test_layernorm(lib):
    def call(x=A[0], r=A[1], w=A[2], b=A[3], eps=1e-6, T=4, d=64, dt=L.LORA_BF16, z=A[4], y=A[5], m=A[6], s=A[7]):
        return lib.lora_add_layernorm(x, r, w, b, eps, T, d, dt, z, y, m, s, None)

    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(T=-1), dict(d=0), dict(d=-8), dict(d=60), dict(dt=2),
                dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=A[0] + 2),
                dict(r=A[1] + 8), dict(w=A[2] + 4), dict(b=A[3] + 8), dict(z=A[4] + 8), dict(y=A[5] + 2),
                dict(m=None), dict(s=None), dict(m=A[6] + 4), dict(s=A[7] + 8),
                # outputs that meet another buffer
                dict(z=A[5]), dict(y=A[2]), dict(y=A[3]), dict(z=A[3]), dict(z=A[0] + 16), dict(y=A[1] + 16),
                dict(m=A[7]), dict(m=A[0]), dict(s=A[4]), dict(s=A[5] + 16), dict(m=A[3])):
        assert call(**bad) == INVALID, bad
    assert call(T=0, x=None, r=None, w=None, b=None, z=None, y=None, m=None, s=None) == OK


def test_layernorm_fp8(lib):
    def call(x=A[0], r=A[1], w=A[2], b=A[3], eps=1e-6, T=4, d=64, z=A[4], y=A[5], q=A[6], qs=A[7], m=A[8], s=A[9]):
        return lib.lora_add_layernorm_fp8(x, r, w, b, eps, T, d, z, y, q, qs, m, s, None)

    for bad in (dict(q=None), dict(qs=None), dict(d=72), dict(q=A[6] + 8), dict(qs=A[7] + 4), dict(x=None),
                dict(eps=0.0), dict(z=A[5]), dict(q=A[5]), dict(q=A[3]), dict(qs=A[3]), dict(m=A[7]), dict(s=A[6] + 16),
                dict(m=None)):
        assert call(**bad) == INVALID, bad
    assert call(T=0, x=None, w=None, q=None, qs=None, m=None, s=None) == OK


def test_layernorm_backward(lib):
    need = L.lora_workspace_bytes_layernorm_backward(4, 64)
    assert need >= 4 * 2 * 64 * 4 and need % 256 == 0
    for bad in ((-1, 64), (4, 0), (4, 60), (4, -8)):
        assert L.lora_workspace_bytes_layernorm_backward(*bad) == 0

    def call(dy=A[0], dr=A[1], z=A[2], w=A[3], m=A[4], s=A[5], T=4, d=64, dt=L.LORA_BF16, dx=A[6], dw=A[7], db=A[8],
             ws=A[9], n=need):
        return lib.lora_add_layernorm_backward(dy, dr, z, w, m, s, T, d, dt, dx, dw, db, ws, n, None)

    for bad in (dict(dy=None), dict(z=None), dict(w=None), dict(m=None), dict(s=None), dict(dx=None), dict(T=-1),
                dict(d=0), dict(d=60), dict(dt=2), dict(dy=A[0] + 2), dict(dr=A[1] + 8), dict(z=A[2] + 4),
                dict(w=A[3] + 8), dict(m=A[4] + 4), dict(s=A[5] + 4), dict(dx=A[6] + 8), dict(dw=A[7] + 8),
                dict(db=A[8] + 2), dict(ws=None), dict(ws=A[9] + 8),
                # outputs that meet another buffer
                dict(dx=A[7]), dict(dw=A[8]), dict(dx=A[3]), dict(dx=A[4]), dict(dx=A[0] + 16), dict(dx=A[2] + 32),
                dict(dw=A[0]), dict(db=A[3]), dict(ws=A[2]), dict(ws=A[6]), dict(ws=A[7]), dict(dw=A[1] + 16)):
        assert call(**bad) == INVALID, bad
    assert call(n=need - 1) == SMALL
    assert call(T=0, dw=None, db=None, dy=None, z=None, w=None, m=None, s=None, dx=None, ws=None, n=0) == OK
    assert call(T=0, dw=A[7], db=A[7]) == INVALID


def test_orthogonalize(lib):
    need = L.lora_workspace_bytes_orthogonalize(3, 64, 16)
    assert need >= 3 * 16 * 16 * 8 and need % 256 == 0
    for bad in ((-1, 64, 16), (3, 0, 16), (3, 64, 0), (3, 60, 16), (3, 64, 12), (3, 136, 136), (3, 1 << 28, 16)):
        assert L.lora_workspace_bytes_orthogonalize(*bad) == 0, bad
    assert L.lora_workspace_bytes_orthogonalize(0, 64, 16) > 0
    good = (ctypes.c_float * 48)(*[1.0] * 48)

    def call(g=A[0], n=3, rows=64, cols=16, dt=L.LORA_BF16, coef=good, steps=5, eps=1e-7, scale=1.0, out=A[1], ws=A[2],
             nb=need):
        return lib.lora_orthogonalize(g, n, rows, cols, dt, coef, steps, eps, scale, out, ws, nb, None)

    inf, nan = float("inf"), float("nan")
    odd = (ctypes.c_float * 48)(*([1.0] * 14 + [nan] + [1.0] * 33))
    for bad in (dict(g=None), dict(out=None), dict(ws=None), dict(coef=None), dict(n=-1), dict(rows=0), dict(rows=60),
                dict(cols=12), dict(dt=2), dict(steps=0), dict(steps=17), dict(eps=0.0), dict(eps=inf), dict(eps=nan),
                dict(scale=nan), dict(scale=-inf), dict(coef=odd), dict(g=A[0] + 8), dict(out=A[1] + 8),
                dict(ws=A[2] + 8), dict(out=A[0] + 16), dict(ws=A[0]), dict(ws=A[1])):
        assert call(**bad) == INVALID, bad
    for bad in (dict(rows=136, cols=136), dict(rows=1 << 28)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(nb=need - 1) == SMALL
    assert call(n=0, g=None, out=None, ws=None, nb=0) == OK


def test_the_binding_refuses_tensors_the_kernels_would_misread():
    """On a host without a GPU no tensor is on the current device."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("covered on the GPU")
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    w, f = torch.ones(64, dtype=torch.bfloat16), torch.zeros(4)
    for call in (lambda: L.lora_add_layernorm(t, t, w, w, 1e-6, 4, 64, L.LORA_BF16, t, t, f, f),
                 lambda: L.lora_add_layernorm_fp8(t, t, w, w, 1e-6, 4, 64, t, t, t, f),
                 lambda: L.lora_add_layernorm_backward(t, t, t, w, f, f, 4, 64, L.LORA_BF16, t, w, w, t),
                 lambda: L.lora_orthogonalize(t, 1, 64, 8, L.LORA_BF16, [(1, 1, 1)], 1e-7, 1.0, t, t)):
        with pytest.raises(L.LoraError) as e:
            call()
        assert e.value.status == INVALID


def pool(**change):
    f = dict(n_slots=4, d_in=64, d_out=96, max_rank=16, dtype=L.LORA_BF16)
    f.update(change)
    P = [FAKE + (i << 32) for i in range(8, 12)]
    return L.lora_pool_t(f["n_slots"], f["d_in"], f["d_out"], f["max_rank"], f["dtype"], *P)


def test_linear_act_forward(lib):
    need = L.lora_workspace_bytes(8, 4, 16, 0)
    p0 = pool()

    def call(x=A[0], w=A[1], b=A[2], r=A[3], y=A[4], pre=A[5], T=8, p=p0, ids=A[6], act=3, mode=0, flags=0, ws=A[7],
             n=need):
        return lib.lora_linear_act_forward(x, w, b, r, y, pre, T, p, ids, act, mode, flags, ws, n, None)

    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(ids=None), dict(T=-1), dict(act=4), dict(act=-1),
                dict(mode=3), dict(flags=2), dict(flags=0x1000), dict(ws=None), dict(ws=A[7] + 8), dict(x=A[0] + 2),
                dict(w=A[1] + 8), dict(b=A[2] + 4), dict(r=A[3] + 8), dict(y=A[4] + 8), dict(pre=A[5] + 8), dict(p=None),
                dict(p=pool(d_in=60)), dict(p=pool(dtype=2)), dict(p=pool(max_rank=12)),
                # outputs that meet another buffer (a residual that only partly is y's)
                dict(y=A[0]), dict(y=A[1]), dict(y=A[2]), dict(y=A[5]), dict(y=A[7]), dict(pre=A[3]), dict(pre=A[0]),
                dict(y=A[6]), dict(r=A[4] + 16), dict(ws=A[3]), dict(ws=A[2]), dict(y=p0.b), dict(pre=p0.scale)):
        assert call(**bad) == INVALID, bad
    assert call(n=need - 1) == SMALL
    assert call(T=0, x=None, w=None, b=None, r=None, y=None, pre=None, ids=None) == OK


def test_linear_act_forward_fp8(lib):
    need, lean = L.lora_workspace_bytes_fp8(8, 4, 16, 64, 0), L.lora_workspace_bytes(8, 4, 16, 0)
    p0 = pool()

    def call(x=A[0], xq=None, xs=None, w=A[1], wsc=A[8], b=A[2], r=A[3], y=A[4], pre=A[5], T=8, p=p0, ids=A[6], act=3,
             mode=0, flags=0, ws=A[7], n=need):
        return lib.lora_linear_act_forward_fp8(x, xq, xs, w, wsc, b, r, y, pre, T, p, ids, act, mode, flags, ws, n, None)

    for bad in (dict(x=None), dict(w=None), dict(wsc=None), dict(y=None), dict(ids=None), dict(xq=A[9]), dict(xs=A[9]),
                dict(act=4), dict(mode=3), dict(flags=2), dict(ws=None), dict(x=A[0] + 2), dict(xq=A[9] + 1, xs=A[10]),
                dict(xq=A[9], xs=A[10] + 4), dict(w=A[1] + 8), dict(wsc=A[8] + 4), dict(b=A[2] + 4), dict(r=A[3] + 8),
                dict(y=A[4] + 8), dict(pre=A[5] + 8), dict(p=pool(d_in=72)), dict(p=pool(dtype=0)),
                dict(y=A[0]), dict(y=A[1]), dict(y=A[8]), dict(y=A[9], xq=A[9], xs=A[10]),
                dict(pre=A[10], xq=A[9], xs=A[10]), dict(r=A[4] + 16), dict(ws=A[3])):
        assert call(**bad) == INVALID, bad
    assert call(n=need - 1) == SMALL
    assert call(n=lean - 1, xq=A[9], xs=A[10]) == SMALL
    assert call(T=0, x=None) == OK


def test_linear_act_refuses_rows_of_more_tiles_than_a_grid_holds(lib):
    T, far = (1 << 31) - 1, [(1 << 40) + (i << 44) for i in range(8)]
    p = pool(d_in=8, d_out=264, n_slots=1)
    assert lib.lora_linear_act_forward(far[0], far[1], None, None, far[2], None, T, p, far[3], 3, 0, 0, far[4], 1 << 42,
                                       None) == UNSUPPORTED


def test_linear_act_backward(lib):
    need = L.lora_workspace_bytes_linear_act_backward(8, 4, 16, 64, 96, L.LORA_BF16)
    assert need >= 2 * 8 * 96 * 2 + 8 * 16 * 4
    for bad in ((-1, 4, 16, 64, 96, 1), (8, 0, 16, 64, 96, 1), (8, 4, 12, 64, 96, 1), (8, 4, 136, 64, 96, 1),
                (8, 4, 16, 60, 96, 1), (8, 4, 16, 64, 0, 1), (8, 4, 16, 64, 96, 2)):
        assert L.lora_workspace_bytes_linear_act_backward(*bad) == 0, bad
    p0 = pool()

    def call(x=A[0], w=A[1], T=8, p=p0, ids=A[2], act=0, pre=A[3], dy=A[4], dx=A[5], dA=A[6], dB=A[7], db=A[8], ws=A[9],
             n=need):
        return lib.lora_linear_act_backward(x, w, T, p, ids, act, pre, dy, dx, dA, dB, db, ws, n, None)

    for bad in (dict(x=None), dict(w=None), dict(T=-1), dict(ids=None), dict(act=4), dict(act=-1), dict(pre=None),
                dict(dy=None), dict(dA=None), dict(dB=None), dict(dx=A[5] + 8), dict(dy=A[4] + 2), dict(pre=A[3] + 8),
                dict(dA=A[6] + 8), dict(dB=A[7] + 8), dict(db=A[8] + 8), dict(ws=None), dict(ws=A[9] + 4), dict(p=None),
                dict(p=pool(d_in=60)), dict(p=pool(dtype=2)),
                # outputs that meet another buffer
                dict(dx=A[0]), dict(dx=A[4]), dict(dx=A[6]), dict(dA=A[7]), dict(db=A[6]), dict(db=A[3]), dict(dB=A[1]),
                dict(ws=A[4]), dict(ws=A[8]), dict(dA=p0.a), dict(db=p0.scale), dict(dx=A[4] + 16)):
        assert call(**bad) == INVALID, bad
    assert call(n=1024) == SMALL
    assert call(T=0, x=None, w=None, ids=None, pre=None, dy=None, dx=None, dA=None, dB=None, db=None) == OK
    assert call(T=0, dA=A[6], dB=A[6], db=None) == INVALID
