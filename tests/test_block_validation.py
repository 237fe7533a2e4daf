"""Refusals of the feed-forward block's entry points, on the host: every call
below returns before anything is enqueued (the addresses are made up)."""
import ctypes

import pytest

from rank_adapter_gemm_amd import lora as L

FAKE = 1 << 40
INVALID, UNSUPPORTED, SMALL, OK = (L.LORA_ERR_INVALID_ARGUMENT, L.LORA_ERR_UNSUPPORTED,
                                   L.LORA_ERR_WORKSPACE_TOO_SMALL, L.LORA_OK)


@pytest.fixture(scope="module")
def lib():
    return L.load()


def pools(**change):
    """Gate's and up's descriptors; change: field -> (gate's, up's)."""
    arr = (L.lora_pool_t * 2)()
    for m in range(2):
        f = dict(n_slots=4, d_in=64, d_out=96, max_rank=16, dtype=L.LORA_BF16)
        f.update({k: v[m] for k, v in change.items()})
        arr[m] = L.lora_pool_t(f["n_slots"], f["d_in"], f["d_out"], f["max_rank"], f["dtype"], FAKE, FAKE, FAKE, FAKE)
    return arr


def test_norm(lib):
    def call(x=FAKE, r=FAKE, w=FAKE, eps=1e-6, T=4, d=64, dt=L.LORA_BF16, z=FAKE, y=FAKE + 4096):
        return lib.lora_add_rmsnorm(x, r, w, eps, T, d, dt, z, y, None)

    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(T=-1), dict(d=0), dict(d=-8), dict(d=60), dict(dt=2),
                dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=FAKE + 2),
                dict(r=FAKE + 8), dict(w=FAKE + 4), dict(z=FAKE + 8), dict(y=FAKE + 2), dict(z=FAKE, y=FAKE)):
        assert call(**bad) == INVALID, bad
    assert call(T=0, x=None, r=None, w=None, z=None, y=None) == OK


def test_norm_fp8(lib):
    def call(x=FAKE, r=FAKE, w=FAKE, eps=1e-6, T=4, d=64, z=FAKE, y=FAKE + 4096, q=FAKE, s=FAKE):
        return lib.lora_add_rmsnorm_fp8(x, r, w, eps, T, d, z, y, q, s, None)

    for bad in (dict(q=None), dict(s=None), dict(d=72), dict(q=FAKE + 8), dict(s=FAKE + 4), dict(x=None),
                dict(eps=0.0), dict(z=FAKE, y=FAKE)):
        assert call(**bad) == INVALID, bad
    assert call(T=0, x=None, w=None, q=None, s=None) == OK


def test_gated_workspace_bytes():
    assert L.lora_workspace_bytes_gated(-1, 4, 16, 64) == 0
    assert L.lora_workspace_bytes_gated(8, 0, 16, 64) == 0
    assert L.lora_workspace_bytes_gated(8, 4, 72, 64) == 0          # two slices of 72 ranks exceed 128
    assert L.lora_workspace_bytes_gated(8, 4, 12, 64) == 0
    assert L.lora_workspace_bytes_gated(8, 4, 16, -8) == 0
    assert L.lora_workspace_bytes_gated(8, 4, 16, 1 << 30) == 0
    assert L.lora_workspace_bytes_gated_fp8(8, 4, 16, 72, 64) == 0
    n = L.lora_workspace_bytes_gated(100, 4, 16, 64)
    assert n >= 100 * 2 * 16 * 4 and n % 256 == 0
    assert L.lora_workspace_bytes_gated_fp8(100, 4, 16, 64, 64) >= n + 100 * 64


def test_gated_forward(lib):
    need = L.lora_workspace_bytes_gated(8, 4, 16, 0)

    def call(x=FAKE, wg=FAKE, wu=FAKE, h=FAKE, g=None, u=None, T=8, p=pools(), ids=FAKE, act=0, mode=0, flags=0,
             ws=FAKE, n=need):
        return lib.lora_gated_forward(x, wg, wu, h, g, u, T, p, ids, act, mode, flags, ws, n, None)

    for bad in (dict(x=None), dict(wg=None), dict(wu=None), dict(h=None), dict(ids=None), dict(g=FAKE), dict(u=FAKE),
                dict(T=-1), dict(act=3), dict(act=-1), dict(mode=3), dict(flags=2), dict(flags=0x1000), dict(ws=None),
                dict(ws=FAKE + 8), dict(x=FAKE + 2), dict(wg=FAKE + 8), dict(wu=FAKE + 8), dict(h=FAKE + 8),
                dict(g=FAKE + 8, u=FAKE), dict(g=FAKE, u=FAKE + 8), dict(p=None),
                dict(p=pools(d_out=(96, 104))), dict(p=pools(d_in=(64, 72))), dict(p=pools(n_slots=(4, 5))),
                dict(p=pools(max_rank=(16, 8))), dict(p=pools(dtype=(1, 0))), dict(p=pools(d_in=(60, 60)))):
        assert call(**bad) == INVALID, bad
    assert call(p=pools(max_rank=(72, 72))) == UNSUPPORTED
    assert call(n=need - 1) == SMALL
    assert call(T=0, x=None, wg=None, wu=None, h=None, ids=None) == OK


def test_gated_forward_fp8(lib):
    need = L.lora_workspace_bytes_gated_fp8(8, 4, 16, 64, 0)
    lean = L.lora_workspace_bytes_gated(8, 4, 16, 0)

    def call(x=FAKE, xq=None, xs=None, qg=FAKE, sg=FAKE, qu=FAKE, su=FAKE, h=FAKE, g=None, u=None, T=8, p=pools(),
             ids=FAKE, act=0, mode=0, flags=0, ws=FAKE, n=need):
        return lib.lora_gated_forward_fp8(x, xq, xs, qg, sg, qu, su, h, g, u, T, p, ids, act, mode, flags, ws, n,
                                          None)

    for bad in (dict(x=None), dict(xq=FAKE), dict(xs=FAKE), dict(qg=None), dict(sg=None), dict(qu=None),
                dict(su=None), dict(h=None), dict(ids=None), dict(g=FAKE), dict(act=5), dict(flags=4),
                dict(qg=FAKE + 8), dict(su=FAKE + 4), dict(xq=FAKE + 1, xs=FAKE), dict(p=pools(d_in=(72, 72))),
                dict(p=pools(dtype=(0, 0)))):
        assert call(**bad) == INVALID, bad
    assert call(n=need - 1) == SMALL
    assert call(n=lean - 1, xq=FAKE, xs=FAKE) == SMALL              # no room for codes is asked where they are given
    assert call(T=0, x=None) == OK


def test_the_binding_takes_two_pools():
    p = pools()
    with pytest.raises(L.LoraError):
        L.lora_gated_forward(FAKE, FAKE, FAKE, FAKE, 1, [p[0]], FAKE, 0, 0, 0, None)


def test_gated_backward(lib):
    need = L.lora_workspace_bytes_gated_backward(8, 4, 16, 64, 96, L.LORA_BF16)
    assert need >= 2 * 8 * 96 * 2 + 8 * 32 * 4
    for bad in ((-1, 4, 16, 64, 96, 1), (8, 0, 16, 64, 96, 1), (8, 4, 72, 64, 96, 1), (8, 4, 16, 60, 96, 1),
                (8, 4, 16, 64, 0, 1), (8, 4, 16, 64, 96, 2)):
        assert L.lora_workspace_bytes_gated_backward(*bad) == 0, bad
    two = (ctypes.c_void_p * 2)(FAKE, FAKE)
    one = (ctypes.c_void_p * 2)(FAKE, None)
    odd = (ctypes.c_void_p * 2)(FAKE, FAKE + 8)

    def call(x=FAKE, wg=FAKE, wu=FAKE, T=8, p=pools(), ids=FAKE, act=0, g=FAKE, u=FAKE, dh=FAKE, dx=FAKE, dA=two,
             dB=two, ws=FAKE, n=need):
        return lib.lora_gated_backward(x, wg, wu, T, p, ids, act, g, u, dh, dx, dA, dB, ws, n, None)

    for bad in (dict(x=None), dict(wg=None), dict(wu=None), dict(T=-1), dict(ids=None), dict(act=3), dict(g=None),
                dict(u=None), dict(dh=None), dict(dA=None), dict(dB=None), dict(dA=one), dict(dB=one), dict(dA=odd),
                dict(dB=odd), dict(dx=FAKE + 8), dict(dh=FAKE + 2), dict(g=FAKE + 8), dict(ws=None), dict(ws=FAKE + 4),
                dict(p=None), dict(p=pools(d_out=(96, 104))), dict(p=pools(dtype=(1, 0)))):
        assert call(**bad) == INVALID, bad
    assert call(p=pools(max_rank=(72, 72))) == UNSUPPORTED
    assert call(n=1024) == SMALL
    assert call(T=0, x=None, dA=None, dB=None) == OK


def test_the_binding_refuses_tensors_the_kernels_would_misread():
    """On a host without a GPU no tensor is on the current device; addresses pass."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("covered on the GPU")
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    for call in (lambda: L.lora_add_rmsnorm(t, t, w, 1e-6, 4, 64, L.LORA_BF16, t, t),
                 lambda: L.lora_add_rmsnorm_fp8(t, t, w, 1e-6, 4, 64, t, t, t, t),
                 lambda: L.lora_gated_forward(t, t, t, t, 4, list(pools()), t, 0, 0, 0, t),
                 lambda: L.lora_gated_backward(t, t, t, 4, list(pools()), t, 0, t, t, t, t, [t, t], [t, t], t)):
        with pytest.raises(L.LoraError) as e:
            call()
        assert e.value.status == INVALID


def test_outputs_are_buffers_of_their_own(lib):
    """An output that is another's buffer, or an input's that is still read."""
    a = [FAKE + (i << 20) for i in range(12)]
    x, wg, wu, h, g, u, ids, ws = a[:8]
    n = L.lora_workspace_bytes_gated_fp8(8, 4, 16, 64, 0)
    for bx, bh, bg, bu in ((h, h, None, None), (x, h, g, g), (x, h, x, u), (x, h, g, x), (x, h, h, u), (x, h, g, h)):
        assert lib.lora_gated_forward(bx, wg, wu, bh, bg, bu, 8, pools(), ids, 0, 0, 0, ws, n, None) == INVALID
        assert lib.lora_gated_forward_fp8(bx, None, None, wg, wg, wu, wu, bh, bg, bu, 8, pools(), ids, 0, 0, 0, ws, n,
                                          None) == INVALID
    n = L.lora_workspace_bytes_gated_backward(8, 4, 16, 64, 96, L.LORA_BF16)
    dx, d0, d1, d2 = a[8:]
    d3 = FAKE + (12 << 20)

    def back(dx, dA, dB):
        return lib.lora_gated_backward(x, wg, wu, 8, pools(), ids, 0, g, u, h, dx, (ctypes.c_void_p * 2)(*dA),
                                       (ctypes.c_void_p * 2)(*dB), ws, n, None)

    for bad in (x, g, u, h, d0, d1, d2, d3):
        assert back(bad, (d0, d1), (d2, d3)) == INVALID
    for dA, dB in (((d0, d0), (d2, d3)), ((d0, d1), (d2, d2)), ((d0, d1), (d0, d3)), ((d0, d1), (d2, d1))):
        assert back(dx, dA, dB) == INVALID
