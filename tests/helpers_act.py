"""Test plumbing of the linear layer with bias, activation and residual: seeded
batches of one projection with its pool, the plain 64-bit forms and the error
bounds of the kernels' arithmetic (steps of the type, counted)."""
import math

import numpy as np
import torch

from helpers_block import HALF, STEP32
from helpers_block import act64 as act64_of
from rank_adapter_gemm_amd import lora as L

ACTS = {"none": L.LORA_ACT_NONE, "silu": L.LORA_ACT_SILU, "gelu": L.LORA_ACT_GELU, "gelu_tanh": L.LORA_ACT_GELU_TANH}
TINY = 2.0 ** -120


def act64(name, p):
    """The activation and its derivative, in 64 bits."""
    return (p, torch.ones_like(p)) if name == "none" else act64_of(name, p)


class Layer:
    """x, W, bias, residual and adapters.  ranks: per slot, 0 leaves it empty.  ids: None = random with base rows."""

    def __init__(self, T, d, f, ranks, R, dtype=torch.bfloat16, seed=0, ids=None, packed=False, order="random"):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.T, self.d, self.f, self.R, self.dtype, self.ranks = T, d, f, R, dtype, list(ranks)
        self.S = len(self.ranks)

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

        self.x = normal(T, d)
        self.W = normal(d, f, std=1.3 / math.sqrt(d))
        self.A = normal(self.S, d, R, std=1.3 / math.sqrt(d))
        self.B = normal(self.S, R, f, std=0.5 / math.sqrt(R))
        self.bias, self.residual = normal(f, std=0.5), normal(T, f, std=3.0)
        if ids is None:
            ids = rng.integers(0, self.S, size=T).astype(np.int32)
            ids[rng.random(T) < 0.15] = -1
            if order == "sorted":
                ids = np.sort(ids)
        self.ids = np.asarray(ids, np.int32)
        self.ids_dev = torch.as_tensor(self.ids, device="cuda")
        self.alphas = [1.5 * (i % 3 + 1) for i in range(self.S)]
        cap = [max(8, (r + 7) // 8 * 8) for r in self.ranks] if packed else None
        self.pool = L.AdapterPool(self.S, d, f, R, dtype, capacity=cap)
        for s, r in enumerate(self.ranks):
            if r:
                self.pool.upload(s, self.A[s], self.B[s], r, self.alphas[s], lda=R, ldb=f)
        self.desc = self.pool.pool

    def scale(self, s):
        return float(np.float32(self.alphas[s]) / np.float32(self.ranks[s]))

    def adapters(self):
        """Each usable slot with rows: its number, rank, rows, A, B and scale."""
        for s, r in enumerate(self.ranks):
            t = torch.as_tensor(np.flatnonzero(self.ids == s), device="cuda")
            if r and len(t):
                yield s, r, t, self.A[s, :, :r].double(), self.B[s, :r].double(), self.scale(s)

    def bad_row(self):
        """The smallest row naming no usable slot, or -1."""
        bad = [t for t, i in enumerate(self.ids) if i < -1 or i >= self.S or (i >= 0 and self.ranks[i] == 0)]
        return bad[0] if bad else -1

    def forward64(self, act, bias=True, residual=True, base=None, extra=0.0):
        """y, act's argument and their bounds: K + R + 9 sums of one fp32 step each of the products' sizes, the
        activation's few steps, one sum with the residual, one rounding.  base: the base product and its products'
        sizes (FP8), extra: its error beside that."""
        half, x = HALF[self.dtype], self.x.double()
        if base is None:
            W = self.W.double()
            p, size = x @ W, x.abs() @ W.abs()
        else:
            p, size = (t.clone() for t in base)
        for _, _, t, A, B, sc in self.adapters():
            p[t] += sc * ((x[t] @ A) @ B)
            size[t] += abs(sc) * ((x[t].abs() @ A.abs()) @ B.abs())
        if bias:
            p, size = p + self.bias.double(), size + self.bias.double().abs()
        dev = (self.d + self.R + 9) * STEP32 * size + extra
        a, _ = act64(act, p)
        a_dev = dev
        if act != "none":
            # v_exp / v_rcp or expf: |x| 2^-23 for the exponent's argument and 8 steps beside it
            a_dev = dev * 1.2 + (8 + p.abs()) * STEP32 * (a.abs() + p.abs() * 2.0 ** -23)
        y = a
        if residual:
            y = a + self.residual.double()
            a_dev = a_dev + STEP32 * (y.abs() + a_dev)
        return y, a_dev * (1 + half) + half * y.abs() + TINY, p, dev * (1 + half) + half * p.abs() + TINY

    def fp8(self):
        """The codes and scales of x and W, their product in 64 bits, and the matrix cores' error of it."""
        from helpers_fp8 import e4m3_decode
        xq = torch.empty(self.T, self.d, dtype=torch.uint8, device="cuda")
        xs = torch.empty(self.T, dtype=torch.float32, device="cuda")
        L.lora_quantize_rows_fp8(self.x, self.T, self.d, xq, xs)
        wq = L.Fp8Weight(self.W)
        X = torch.as_tensor(e4m3_decode(xq.cpu().numpy()), device="cuda") * xs.double()[:, None]
        W = torch.as_tensor(e4m3_decode(wq.codes.cpu().numpy()), device="cuda").t() * wq.scale.double()[None, :]
        size = X.abs() @ W.abs()
        return (xq, xs, wq), (X @ W, size), 2.0 ** -11 * size


def run_forward(p, act, mode=L.LORA_MODE_AUTO, keep=False, bias=True, residual=True, ws=None, flags=0, stream=None,
                fp8=None, codes=True, fill=7.0, y=None):
    """lora_linear_act_forward (fp8: (codes, scales, weight)): y, the kept argument and the workspace."""
    new = lambda: torch.full((p.T, p.f), fill, dtype=p.dtype, device="cuda")  # noqa: E731
    y, pre = new() if y is None else y, new() if keep else None
    if ws is None:
        ws = L.Workspace(p.T, p.S, p.R, p.f, fp8_d_in=p.d if fp8 else 0, stream=stream)
    b, r = p.bias if bias else None, p.residual if residual else None
    if fp8:
        xq, xs, wq = fp8
        L.lora_linear_act_forward_fp8(p.x, xq if codes else None, xs if codes else None, wq.codes, wq.scale, b, r, y,
                                      p.T, p.desc, p.ids_dev, ACTS[act], mode, flags, ws.buf, pre=pre, stream=stream)
    else:
        L.lora_linear_act_forward(p.x, p.W, b, r, y, p.T, p.desc, p.ids_dev, ACTS[act], mode, flags, ws.buf, pre=pre,
                                  stream=stream)
    return y, pre, ws


def backward64(p, act, pre, dy):
    """The gradients in 64 bits for pre as given, and their bounds (as helpers_block.backward64): dp is a few fp32
    steps and, in bf16, one rounding off in dx, 2^-17 elsewhere (none without an activation); every sum adds one
    step per term; vectors of rank width reach the matrix cores as two bf16 parts (2^-17 left out)."""
    half, step, bf16 = HALF[p.dtype], STEP32, p.dtype == torch.bfloat16
    split = 2.0 ** -17 if bf16 else 0.0
    x, dp = p.x.double(), dy.double()
    ddp = rounded = torch.zeros_like(dp)
    if act != "none":
        g = pre.double()
        _, slope = act64(act, g)
        size = dp.abs()
        dp = dp * slope
        ddp = 32 * step * (1 + g.abs()) * size + split * dp.abs()
        rounded = ddp + half * dp.abs()
    W = p.W.double()
    dx = dp @ W.t()
    tx = rounded @ W.t().abs() + (p.f + p.R + 8) * step * (dp.abs() @ W.t().abs())
    dA = torch.zeros(p.S, p.d, p.R, dtype=torch.float64, device="cuda")
    dB = torch.zeros(p.S, p.R, p.f, dtype=torch.float64, device="cuda")
    tA, tB = torch.zeros_like(dA), torch.zeros_like(dB)
    for s, r, t, A, B, sc in p.adapters():
        dv = sc * (dp[t] @ B.t())
        tv = sc * (ddp[t] @ B.t().abs() + (p.f + 8) * step * (dp[t].abs() @ B.t().abs())) + split * dv.abs()
        dx[t] += dv @ A.t()
        tx[t] += tv @ A.t().abs() + (p.R + 8) * step * (dv.abs() @ A.t().abs())
        n = len(t) + 8
        dA[s, :, :r] = x[t].t() @ dv
        tA[s, :, :r] = x[t].t().abs() @ tv + n * step * (x[t].t().abs() @ dv.abs())
        v = x[t] @ A
        dev_v = (p.d + 8) * step * (x[t].abs() @ A.abs()) + split * v.abs()
        dB[s, :r] = sc * (v.t() @ dp[t])
        tB[s, :r] = sc * (dev_v.t() @ dp[t].abs() + v.t().abs() @ ddp[t] + n * step * (v.t().abs() @ dp[t].abs()))
    db, n = dp.sum(0), p.T / 256 + 256
    tb = (ddp if bf16 else rounded).sum(0) + n * step * dp.abs().sum(0)
    end = lambda v, t: (v, t * (1 + half) + half * v.abs() + TINY)  # noqa: E731
    return end(dx, tx), end(dA, tA), end(dB, tB), end(db, tb)


def run_backward(p, act, pre, dy, ws=None, stream=None, want=("dx", "ab", "bias"), fill=7.0):
    """lora_linear_act_backward: dx, dA, dB, dbias and the workspace."""
    new = lambda *shape: torch.full(shape, fill, dtype=p.dtype, device="cuda")  # noqa: E731
    dx = new(p.T, p.d) if "dx" in want else None
    dA, dB = (new(p.S, p.d, p.R), new(p.S, p.R, p.f)) if "ab" in want else (None, None)
    db = new(p.f) if "bias" in want else None
    if ws is None:
        ws = L.Workspace(p.T, p.S, p.R, p.f, linear_backward_d_in=p.d, dtype=p.dtype, stream=stream)
    L.lora_linear_act_backward(p.x, p.W, p.T, p.desc, p.ids_dev, ACTS[act], pre if act != "none" else None, dy, dx, dA,
                               dB, db, ws.buf, stream=stream)
    return dx, dA, dB, db, ws
