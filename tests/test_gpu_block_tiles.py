"""The gated pair and its backward pass on every tile plan: the sizes below are
those at which the planner takes the large tiles (whole, and in pieces of K),
the 33 to 64-row tiles, several stretches of one adapter's rows and more than
one step of ranks.  Bounds as in helpers_block."""
import numpy as np
import pytest
import torch

from helpers_block import ACTS, Pair, run_backward, run_forward
from rank_adapter_gemm_amd import lora as L
from test_gpu_gated import check as check_forward
from test_gpu_gated import fp8_parts
from test_gpu_gated_backward import check as check_backward
from test_gpu_gated_backward import kept

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


def sorted_ids(T, lengths):
    """Slot i's lengths[i] rows one after the other, shuffled over the batch; the rest have no adapter."""
    ids = np.full(T, -1, np.int32)
    ids[:sum(lengths)] = np.repeat(np.arange(len(lengths), dtype=np.int32), lengths)
    return ids


# ---- backward: dx's plans ----------------------------------------------------
# T, d, f: 256 x 256 tiles in pieces of K (f past 4096, its own odd end), whole 256 x 256 tiles, these with a
# last round in pieces, 256 x 128 tiles whole, and with a last round in pieces, 128 x 64 tiles with one
DX = [(1797, 1800, 4104), (3500, 3800, 72), (4000, 4296, 520), (2000, 3496, 136), (1990, 4104, 520), (2000, 1080, 520)]


@pytest.mark.parametrize("T,d,f", DX)
@pytest.mark.parametrize("slots", [3, 40])
def test_dx_on_large_tiles(T, d, f, slots):
    """3 slots: the low-rank term of a split tile in its first piece; 40: in the reduction (under 64 rows a slot)
    where T allows, both on the matrix cores in whole tiles."""
    ranks = [16, 5, 11] if slots == 3 else [(3 * i) % 16 + 1 for i in range(slots)]
    p = Pair(T, d, f, ranks, 16, BF16, seed=T + slots)
    k = kept(p)
    check_backward(p, "silu", *k, run_backward(p, "silu", *k), "dx")


@pytest.mark.parametrize("T,d,f", [(1797, 1800, 4104)])
def test_many_short_segments_in_pieces(T, d, f):
    """Fewer than 64 rows an adapter on average, sorted and shuffled."""
    for order in ("sorted", "random"):
        p = Pair(T, d, f, [(5 * i) % 24 + 1 for i in range(31)], 24, BF16, seed=8, order=order)
        k = kept(p)
        check_backward(p, "gelu", *k, run_backward(p, "gelu", *k), order)


@pytest.mark.parametrize("R", [16, 64])
@pytest.mark.parametrize("lengths", [(1025, 1), (1024, 1024, 2100), (4097,)])
def test_an_adapter_of_many_rows(R, lengths):
    T = sum(lengths) + 45
    rng = np.random.default_rng(R)
    for ids in (sorted_ids(T, lengths), rng.permutation(sorted_ids(T, lengths))):
        p = Pair(T, 136, 264, [R - 3 * i for i in range(len(lengths))], R, BF16, seed=R, ids=ids)
        k = kept(p)
        check_backward(p, "silu", *k, run_backward(p, "silu", *k), "long")


@pytest.mark.parametrize("R,ranks", [(24, [24, 17, 5, 8]), (64, [64, 63, 20, 1])])
@pytest.mark.parametrize("packed", [False, True])
def test_f32_ranks(R, ranks, packed):
    """More than one block of 16 ranks in 32 bits, both ways."""
    for T in (37, 150):
        p = Pair(T, 136, 328, ranks, R, F32, seed=R, packed=packed)
        for mode in (L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
            check_forward(p, "gelu", run_forward(p, "gelu", mode, keep=True), "R %d T %d" % (R, T))
        k = kept(p)
        check_backward(p, "gelu", *k, run_backward(p, "gelu", *k), "R %d T %d" % (R, T))


# ---- the pair on FP8 weights ---------------------------------------------------
@pytest.mark.parametrize("R,ranks", [(24, [24, 17, 5]), (40, [33, 40, 0, 8]), (64, [64, 63, 20])])
@pytest.mark.parametrize("packed", [False, True])
def test_fp8_ranks(R, ranks, packed):
    """Adapters of more than one step of 16 ranks; 3580 rows are on whole 256 x 256 tiles, 2100 on 256 x 128."""
    for T, f, order in ((9, 1736, "random"), (60, 712, "random"), (520, 1736, "random"), (2100, 1736, "sorted"),
                        (3580, 1920, "sorted")):
        p = Pair(T, 144, f, ranks, R, BF16, seed=R, packed=packed, order=order)
        parts, bases, extra = fp8_parts(p)
        for mode in (L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
            check_forward(p, "silu", run_forward(p, "silu", mode, fp8=parts), "R %d T %d" % (R, T), bases, extra)


# T, d, f: 33 and 64 rows, whole and in pieces, many tiles
@pytest.mark.parametrize("T,d,f", [(33, 144, 712), (64, 1040, 712), (33, 1040, 1000), (64, 272, 10312)])
@pytest.mark.parametrize("act", list(ACTS))
def test_fp8_64_rows(T, d, f, act):
    p = Pair(T, d, f, [16, 3, 8, 0, 13], 16, BF16, seed=T + f)
    parts, bases, extra = fp8_parts(p)
    for mode in (L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
        check_forward(p, act, run_forward(p, act, mode, keep=True, fp8=parts), act, bases, extra)


@pytest.mark.parametrize("T", [50, 200, 2100])
def test_fp8_pools_that_differ(T):
    """A slot empty in one pool only: the other's term stays, the row is recorded."""
    p = Pair(T, 256, 1736, ([8, 0, 4], [0, 16, 3]), 16, BF16, seed=2)
    parts, bases, extra = fp8_parts(p)
    for act in ACTS:
        for mode in (L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
            got = run_forward(p, act, mode, keep=True, fp8=parts)
            check_forward(p, act, got, "differ", bases, extra)
            assert L.lora_get_device_error(got[3].buf) == p.bad_row() >= 0


# ---- 256 x 256 tiles with a last round in pieces of K ---------------------------
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("order", ["random", "sorted"])
def test_a_last_round_of_large_tiles_in_pieces(fp8, order):
    p = Pair(4090, 1040, 2168, [16, 9, 4, 13], 16, BF16, seed=17, order=order)
    parts, bases, extra = fp8_parts(p) if fp8 else (None, (None, None), (0.0, 0.0))
    for mode in (L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
        check_forward(p, "silu", run_forward(p, "silu", mode, keep=True, fp8=parts), "pieces", bases, extra)


@pytest.mark.parametrize("T", [33, 64])
def test_64_rows(T):
    """The bf16 pair's 64-row tiles, whole and in pieces."""
    for d, f in ((136, 712), (1032, 712), (264, 10312)):
        p = Pair(T, d, f, [16, 3, 8, 0, 13], 16, BF16, seed=T)
        for mode in (L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
            check_forward(p, "gelu_tanh", run_forward(p, "gelu_tanh", mode, keep=True), "64 rows")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_than_2_20_workgroups_of_rows(dtype):
    """Rows past one grid dimension of the row kernels, and adapters of 200000 rows."""
    p = Pair(600011, 16, 24, [8, 3, 5], 8, dtype, seed=51)
    for mode in (L.LORA_MODE_BGMV, L.LORA_MODE_SGMV):
        check_forward(p, "silu", run_forward(p, "silu", mode, keep=True), "forward")
    k = kept(p)
    check_backward(p, "silu", *k, run_backward(p, "silu", *k), "backward")
