"""Outputs of the feed-forward block's entry points that share bytes with
another buffer of the same call are refused on the host (the addresses are made
up; nothing is enqueued).  A kernel reads such a buffer in some workgroups
while others write it, so the result would go by their order."""
import ctypes

import pytest
import torch

from rank_adapter_gemm_amd import lora as L

INVALID = L.LORA_ERR_INVALID_ARGUMENT
T, K, N, R, S = 8, 64, 96, 16, 4
STEP = 1 << 28


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("made-up addresses stay off a GPU")
    return L.load()


def places(names, size):
    """Names -> addresses far apart."""
    assert max(size.values(), default=0) < STEP
    return {n: (1 << 40) + i * STEP for i, n in enumerate(names)}


def pools(at):
    arr = (L.lora_pool_t * 2)()
    for m in range(2):
        arr[m] = L.lora_pool_t(S, K, N, R, L.LORA_BF16, at["a%d" % m], at["b%d" % m], at["scale%d" % m],
                               at["rank%d" % m])
    return arr


POOLS = ["a0", "a1", "b0", "b1", "scale0", "scale1", "rank0", "rank1"]
POOL_BYTES = dict(a0=S * R * K * 2, a1=S * R * K * 2, b0=S * R * N * 2, b1=S * R * N * 2, scale0=4 * S, scale1=4 * S,
                  rank0=4 * S, rank1=4 * S)


def meetings(size, outs, ins):
    """Every output over every other buffer: at its start, one 16-byte chunk
    before its end, and ending one chunk into it."""
    for i, o in enumerate(outs):
        for other in ins + outs[:i]:
            yield o, other, 0
            if size[other] > 16:
                yield o, other, (size[other] - 1) // 16 * 16
            yield o, other, -((size[o] - 1) // 16 * 16)


def test_backward(lib):
    names = ["x", "wg", "wu", "ids", "gate", "up", "dh"] + POOLS + ["dx", "dA0", "dA1", "dB0", "dB1", "ws"]
    n = L.lora_workspace_bytes_gated_backward(T, S, R, K, N, L.LORA_BF16)
    size = dict(x=T * K * 2, wg=K * N * 2, wu=K * N * 2, ids=4 * T, gate=T * N * 2, up=T * N * 2, dh=T * N * 2,
                dx=T * K * 2, dA0=S * K * R * 2, dA1=S * K * R * 2, dB0=S * R * N * 2, dB1=S * R * N * 2, ws=n,
                **POOL_BYTES)
    base = places(names, size)

    def call(at):
        two = lambda p: (ctypes.c_void_p * 2)(at[p + "0"], at[p + "1"])  # noqa: E731
        return lib.lora_gated_backward(at["x"], at["wg"], at["wu"], T, pools(at), at["ids"], 0, at["gate"], at["up"],
                                       at["dh"], at["dx"], two("dA"), two("dB"), at["ws"], n, None)

    for o, other, by in meetings(size, ["dx", "dA0", "dA1", "dB0", "dB1", "ws"], ["x", "wg", "wu", "ids", "gate", "up", "dh"] + POOLS):
        assert call(dict(base, **{o: base[other] + by})) == INVALID, (o, other, by)


def pair_buffers(n):
    names = ["x", "xq", "xs", "wg", "sg", "wu", "su", "ids"] + POOLS + ["h", "gate", "up", "ws"]
    size = dict(x=T * K * 2, xq=T * K, xs=4 * T, wg=K * N * 2, sg=4 * N, wu=K * N * 2, su=4 * N, ids=4 * T,
                h=T * N * 2, gate=T * N * 2, up=T * N * 2, ws=n, **POOL_BYTES)
    return places(names, size), size


def test_gated_forward(lib):
    n = L.lora_workspace_bytes_gated(T, S, R, N)
    base, size = pair_buffers(n)

    def call(at):
        return lib.lora_gated_forward(at["x"], at["wg"], at["wu"], at["h"], at["gate"], at["up"], T, pools(at),
                                      at["ids"], 0, 0, 0, at["ws"], n, None)

    for o, other, by in meetings(size, ["h", "gate", "up", "ws"], ["x", "wg", "wu", "ids"] + POOLS):
        assert call(dict(base, **{o: base[other] + by})) == INVALID, (o, other, by)


def test_gated_forward_fp8(lib):
    n = L.lora_workspace_bytes_gated_fp8(T, S, R, K, N)
    base, size = pair_buffers(n)
    size.update(wg=K * N, wu=K * N)

    def call(at):
        return lib.lora_gated_forward_fp8(at["x"], at["xq"], at["xs"], at["wg"], at["sg"], at["wu"], at["su"], at["h"],
                                          at["gate"], at["up"], T, pools(at), at["ids"], 0, 0, 0, at["ws"], n, None)

    ins = ["x", "xq", "xs", "wg", "sg", "wu", "su", "ids"] + POOLS
    for o, other, by in meetings(size, ["h", "gate", "up", "ws"], ins):
        assert call(dict(base, **{o: base[other] + by})) == INVALID, (o, other, by)
    no_codes = dict(base, xq=None, xs=None)
    assert call(dict(no_codes, h=base["x"])) == INVALID


def norm_buffers(d, T=T):
    names = ["x", "r", "w", "z", "y", "q", "s"]
    return places(names, {}), dict(x=T * d * 2, r=T * d * 2, w=d * 2, z=T * d * 2, y=T * d * 2, q=T * d, s=4 * T)


def test_norm(lib):
    """z and y may be x's or the residual's own buffers, row for row, and nothing else."""
    base, size = norm_buffers(K)
    size.pop("q"), size.pop("s")

    def call(at):
        return lib.lora_add_rmsnorm(at["x"], at["r"], at["w"], 1e-6, T, K, L.LORA_BF16, at["z"], at["y"], None)

    for o, other, by in meetings(size, ["z", "y"], ["x", "r", "w"]):
        if by == 0 and other in ("x", "r"):
            continue
        assert call(dict(base, **{o: base[other] + by})) == INVALID, (o, other, by)
    # in place on rows that the other input is half a buffer into
    assert call(dict(base, z=base["x"], r=base["x"] + size["x"] // 2)) == INVALID


def test_norm_fp8(lib):
    base, size = norm_buffers(K)

    def call(at):
        return lib.lora_add_rmsnorm_fp8(at["x"], at["r"], at["w"], 1e-6, T, K, at["z"], at["y"], at["q"], at["s"], None)

    for o, other, by in meetings(size, ["z", "y", "q", "s"], ["x", "r", "w"]):
        if by == 0 and o in ("z", "y") and other in ("x", "r"):
            continue
        assert call(dict(base, **{o: base[other] + by})) == INVALID, (o, other, by)
    assert call(dict(base, y=None, q=base["x"])) == INVALID
    assert call(dict(base, r=None, z=None, s=base["w"])) == INVALID
