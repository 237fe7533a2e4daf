"""Feed-forward block test plumbing: seeded batches of a gate and an up
projection with their pools, the plain 64-bit forms and the error bounds of
the kernels' arithmetic (steps of the type, counted)."""
import math

import numpy as np
import torch

from rank_adapter_gemm_amd import lora as L

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}     # one rounding, relative
STEP32 = 2.0 ** -23                                               # one fp32 sum or product, any rounding
ACTS = {"silu": L.LORA_ACT_SILU, "gelu": L.LORA_ACT_GELU, "gelu_tanh": L.LORA_ACT_GELU_TANH}


def act64(name, g):
    """The activation and its derivative, in 64 bits."""
    if name == "silu":
        q = torch.sigmoid(g)
        return g * q, q * (1 + g * (1 - q))
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def within(got, ref, tol, what):
    """|got - ref| <= tol elementwise (finite everywhere)."""
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), what + ": not finite"
    bad = err > tol
    if bad.any():
        i = int(torch.argmax(err / tol.clamp_min(1e-300)))
        raise AssertionError("%s: %d of %d off; worst at %d: |err| %.3e > tol %.3e (ref %.4e)" % (
            what, int(bad.sum()), err.numel(), i, err.flatten()[i], tol.flatten()[i], ref.flatten()[i]))


class Pair:
    """x, gate and up with their adapters.  ranks: per slot, or (gate's, up's)
    lists; 0 leaves the slot empty.  ids: None = random with base rows."""

    def __init__(self, T, d, f, ranks, R, dtype=torch.bfloat16, seed=0, ids=None, packed=False, order="random"):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.T, self.d, self.f, self.R, self.dtype = T, d, f, R, dtype
        self.ranks = ranks if isinstance(ranks, tuple) else (list(ranks), list(ranks))
        self.S = len(self.ranks[0])

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

        self.x = normal(T, d)
        self.W = [normal(d, f, std=1.3 / math.sqrt(d)) for _ in range(2)]
        self.A = [normal(self.S, d, R, std=1.3 / math.sqrt(d)) for _ in range(2)]
        self.B = [normal(self.S, R, f, std=0.5 / math.sqrt(R)) for _ in range(2)]
        if ids is None:
            ids = rng.integers(0, self.S, size=T).astype(np.int32)
            ids[rng.random(T) < 0.15] = -1
            if order == "sorted":
                ids = np.sort(ids)
        self.ids = np.asarray(ids, np.int32)
        self.ids_dev = torch.as_tensor(self.ids, device="cuda")
        self.alphas = [1.5 * (i % 3 + 1) for i in range(self.S)]
        self.pools = []
        for m in range(2):
            cap = [max(8, (r + 7) // 8 * 8) for r in self.ranks[m]] if packed else None
            pool = L.AdapterPool(self.S, d, f, R, dtype, capacity=cap)
            for s, r in enumerate(self.ranks[m]):
                if r:
                    pool.upload(s, self.A[m][s], self.B[m][s], r, self.alphas[s], lda=R, ldb=f)
            self.pools.append(pool)
        self.desc = [p.pool for p in self.pools]

    def owners(self, slot):
        return torch.as_tensor(np.flatnonzero(self.ids == slot), device="cuda")

    def bad_row(self):
        """The smallest row naming no usable slot of both pools, or -1."""
        bad = [t for t, i in enumerate(self.ids) if i < -1 or i >= self.S or
               (i >= 0 and min(self.ranks[0][i], self.ranks[1][i]) == 0)]
        return bad[0] if bad else -1

    def project64(self, m, base=None):
        """One projection in 64 bits and the sum of its products' sizes."""
        x = self.x.double()
        if base is None:
            W = self.W[m].double()
            y, size = x @ W, x.abs() @ W.abs()
        else:
            y, size = base
            y, size = y.clone(), size.clone()
        for s, r in enumerate(self.ranks[m]):
            t = self.owners(s)
            if r and len(t):
                A, B = self.A[m][s, :, :r].double(), self.B[m][s, :r].double()
                sc = float(np.float32(self.alphas[s]) / np.float32(r))
                y[t] += sc * ((x[t] @ A) @ B)
                size[t] += abs(sc) * ((x[t].abs() @ A.abs()) @ B.abs())
        return y, size

    def forward64(self, act, bases=(None, None), extra=(0.0, 0.0)):
        """h, g, u and their bounds: K + R + 8 sums of one fp32 step each of
        the products' sizes, the activation's few steps, one rounding."""
        half = HALF[self.dtype]
        y, dev = [], []
        for m in range(2):
            v, size = self.project64(m, bases[m])
            y.append(v)
            dev.append((self.d + self.R + 8) * STEP32 * size + extra[m])
        a, slope = act64(act, y[0])
        h = a * y[1]
        # v_exp / v_rcp or expf: |x| 2^-23 for the exponent's argument and 8 steps beside it
        a_dev = dev[0] * 1.2 + (8 + y[0].abs()) * STEP32 * (a.abs() + y[0].abs() * 2.0 ** -23)
        h_dev = a_dev * (y[1].abs() + dev[1]) + a.abs() * dev[1]
        tiny = 2.0 ** -120
        tol_h = h_dev * (1 + half) + half * h.abs() + tiny
        return h, tol_h, y, [dev[m] * (1 + half) + half * y[m].abs() + tiny for m in range(2)]


def run_forward(p, act, mode=L.LORA_MODE_AUTO, keep=False, ws=None, flags=0, stream=None, fp8=None, codes=True,
                fill=7.0):
    """lora_gated_forward (fp8: the pair's (codes, scales) of W and x)."""
    new = lambda: torch.full((p.T, p.f), fill, dtype=p.dtype, device="cuda")  # noqa: E731
    h, gate, up = new(), new() if keep else None, new() if keep else None
    if ws is None:
        ws = L.Workspace(p.T, p.S, p.R, p.f, gated=True, fp8_d_in=p.d if fp8 else 0, stream=stream)
    if fp8:
        xq, xs, wq = fp8
        L.lora_gated_forward_fp8(p.x, xq if codes else None, xs if codes else None, wq[0].codes, wq[0].scale,
                                 wq[1].codes, wq[1].scale, h, p.T, p.desc, p.ids_dev, ACTS[act], mode, flags, ws.buf,
                                 gate=gate, up=up, stream=stream)
    else:
        L.lora_gated_forward(p.x, p.W[0], p.W[1], h, p.T, p.desc, p.ids_dev, ACTS[act], mode, flags, ws.buf,
                             gate=gate, up=up, stream=stream)
    return h, gate, up, ws


def backward64(p, act, gate, up, dh):
    """The gradients in 64 bits for gate and up as given, and their bounds:
    dg and du are a few fp32 steps and one rounding off; every sum adds one
    step per term; vectors of rank width reach the matrix cores as two bf16
    parts at least (2^-17 of the value left out)."""
    half, step, split = HALF[p.dtype], STEP32, 2.0 ** -17
    x, dh = p.x.double(), dh.double()
    g, u = gate.double(), up.double()
    a, slope = act64(act, g)
    dy = [dh * u * slope, dh * a]
    act_dev = 32 * step * (1 + g.abs())
    ddy = [half * dy[0].abs() + act_dev * (dh * u).abs(), half * dy[1].abs() + act_dev * (dh * a).abs()
           + dh.abs() * g.abs() * 2.0 ** -46]
    if p.dtype == torch.float32:
        split = 0.0
    dx, tx = torch.zeros_like(x), torch.zeros_like(x)
    dA, tA, dB, tB = [], [], [], []
    for m in range(2):
        W = p.W[m].double()
        size = dy[m].abs() @ W.t().abs()
        dx += dy[m] @ W.t()
        tx += ddy[m] @ W.t().abs() + (2 * p.f + 2 * p.R + 8) * step * size
        da = torch.zeros(p.S, p.d, p.R, dtype=torch.float64, device="cuda")
        db = torch.zeros(p.S, p.R, p.f, dtype=torch.float64, device="cuda")
        ta, tb = torch.zeros_like(da), torch.zeros_like(db)
        for s, r in enumerate(p.ranks[m]):
            t = p.owners(s)
            if not r or not len(t):
                continue
            A, B = p.A[m][s, :, :r].double(), p.B[m][s, :r].double()
            sc = float(np.float32(p.alphas[s]) / np.float32(r))
            dv = sc * (dy[m][t] @ B.t())
            tv = sc * (ddy[m][t] @ B.t().abs() + (p.f + 8) * step * (dy[m][t].abs() @ B.t().abs())) + split * dv.abs()
            dx[t] += dv @ A.t()
            tx[t] += tv @ A.t().abs() + (2 * p.R + 8) * step * (dv.abs() @ A.t().abs())
            n = len(t) + 8
            da[s, :, :r] = x[t].t() @ dv
            ta[s, :, :r] = x[t].t().abs() @ tv + n * step * (x[t].t().abs() @ dv.abs())
            v = x[t] @ A
            dev_v = (p.d + 8) * step * (x[t].abs() @ A.abs()) + split * v.abs()
            db[s, :r] = sc * (v.t() @ dy[m][t])
            tb[s, :r] = sc * (dev_v.t() @ dy[m][t].abs() + v.t().abs() @ ddy[m][t] +
                              n * step * (v.t().abs() @ dy[m][t].abs()))
        dA.append(da)
        dB.append(db)
        tA.append(ta * (1 + half) + half * da.abs() + 2.0 ** -120)
        tB.append(tb * (1 + half) + half * db.abs() + 2.0 ** -120)
    return dx, tx * (1 + half) + half * dx.abs() + 2.0 ** -120, dA, tA, dB, tB


def run_backward(p, act, gate, up, dh, ws=None, stream=None, want_dx=True, want_ab=True, fill=7.0):
    new = lambda *shape: torch.full(shape, fill, dtype=p.dtype, device="cuda")  # noqa: E731
    dx = new(p.T, p.d) if want_dx else None
    dA = [new(p.S, p.d, p.R) for _ in range(2)] if want_ab else None
    dB = [new(p.S, p.R, p.f) for _ in range(2)] if want_ab else None
    if ws is None:
        ws = L.Workspace(p.T, p.S, p.R, p.f, gated=True, backward_d_in=p.d, dtype=p.dtype, stream=stream)
    L.lora_gated_backward(p.x, p.W[0], p.W[1], p.T, p.desc, p.ids_dev, ACTS[act], gate, up, dh, dx, dA, dB, ws.buf,
                          stream=stream)
    return dx, dA, dB, ws
