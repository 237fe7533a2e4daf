"""The adapters' gradients keep dg and du to 2^-17 (two bf16 parts): against 64
bits with bounds that leave no room for a rounding of dg or du to bf16, so the
only full rounding is the output's."""
import numpy as np
import pytest
import torch

from helpers_block import HALF, STEP32, Pair, act64, run_backward, within
from rank_adapter_gemm_amd import lora as L
from test_gpu_gated_backward import kept

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
TWO = 2.0 ** -17      # left of a value by two bf16 parts: half a step of a remainder under 2^-8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load()


def check(p, act, gate, up, dh, dA, dB):
    half, step = HALF[BF16], STEP32
    x, dh, g, u = p.x.double(), dh.double(), gate.double(), up.double()
    a, slope = act64(act, g)
    act_dev = 32 * step * (1 + g.abs())                # as helpers_block.backward64
    dy = [dh * u * slope, dh * a]
    ddy = [TWO * dy[0].abs() + act_dev * (dh * u).abs(),
           TWO * dy[1].abs() + act_dev * (dh * a).abs() + dh.abs() * g.abs() * 2.0 ** -46]
    for m in range(2):
        for s, r in enumerate(p.ranks[m]):
            t = p.owners(s)
            if not r or not len(t):
                continue
            A, B, xt, yt = p.A[m][s, :, :r].double(), p.B[m][s, :r].double(), x[t], dy[m][t]
            sc = float(np.float32(p.alphas[s]) / np.float32(r))
            n = len(t) + 8
            dv = sc * (yt @ B.t())
            tv = sc * (ddy[m][t] @ B.t().abs() + (2 * p.f + 8) * step * (yt.abs() @ B.t().abs())) + TWO * dv.abs()
            da = xt.t() @ dv
            ta = xt.t().abs() @ tv + 2 * n * step * (xt.t().abs() @ dv.abs())
            within(dA[m][s, :, :r], da, ta * (1 + half) + half * da.abs() + 2.0 ** -120, "dA %d %d" % (m, s))
            v = xt @ A
            tv = (p.d + 8) * step * (xt.abs() @ A.abs()) + TWO * v.abs()
            db = sc * (v.t() @ yt)
            # the second parts' product, 2^-8 of v by 2^-8 of dy, is not summed
            tb = sc * (tv.t() @ yt.abs() + v.t().abs() @ ddy[m][t]
                       + (3 * n * step + 2.0 ** -16) * (v.t().abs() @ yt.abs()))
            within(dB[m][s, :r], db, tb * (1 + half) + half * db.abs() + 2.0 ** -120, "dB %d %d" % (m, s))


@pytest.mark.parametrize("T,d,f,R", [(1, 312, 136, 56), (1, 2552, 1144, 16), (3, 800, 344, 40), (23, 2168, 344, 64),
                                     (62, 952, 1528, 8), (300, 136, 1064, 24), (2100, 72, 264, 32)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_adapter_gradients(T, d, f, R, act):
    p = Pair(T, d, f, [R, max(1, R - 5), 1], R, BF16, seed=T + R, ids=np.arange(T) % 3)
    gate, up, dh = kept(p)
    _, dA, dB, _ = run_backward(p, act, gate, up, dh)
    check(p, act, gate, up, dh, dA, dB)


def test_values_past_the_types_largest():
    """dg past bf16's largest finite value rounds to infinity, with nothing beside it: its row's gradients are
    infinite or NaN, others' as they were."""
    p = Pair(6, 64, 72, [8, 8], 8, BF16, seed=3, ids=[0, 0, 0, 1, 1, 1])
    gate, up, dh = kept(p)
    clean = run_backward(p, "silu", gate, up, dh)
    # dg = 1.9995 2^127: in fp32's range, nearer to 2^128 than to the largest bf16, 1.9922 2^127
    gate[1, 5], up[1, 5], dh[1, 5] = 30.0, 1.40625 * 2.0 ** 64, 1.421875 * 2.0 ** 63
    dx, dA, dB, _ = run_backward(p, "silu", gate, up, dh)
    assert not torch.isfinite(dx[1].float()).any()
    assert not torch.isfinite(dB[0][0, :, 5].float()).any()
    ok = torch.tensor([0, 2, 3, 4, 5], device="cuda")
    assert torch.equal(dx[ok], clean[0][ok])
    for m in range(2):
        assert torch.equal(dA[m][1], clean[1][m][1]) and torch.equal(dB[m][1], clean[2][m][1])
        cols = [n for n in range(72) if n != 5]
        assert torch.equal(dB[m][0][:, cols], clean[2][m][0][:, cols])
