"""The operators of an adapter-serving feed-forward block, as they are measured.

Three operators of one path: the residual addition with its root-mean-square
norm (with E4M3 codes of the result where the base weights are FP8), the gated
feed-forward pair of projections with every row's own low-rank adapter, and
that pair's backward pass.  `run` computes them in their plain form, or, where
`own` is true, by the calls a user makes of rank_adapter_gemm_amd.

    z = x + residual;  y = z / sqrt(mean(z^2) + eps) * weight
    g = x Wg + s_a (x Ag_a) Bg_a;  u = x Wu + s_a (x Au_a) Bu_a;  h = act(g) * u
    dg = dh * u * act'(g);  du = dh * act(g)
    dv = s_a dg B_a^T;  dx = dg Wg^T + dv A_a^T (+ the same of up)
    dA_a = x_a^T dv_a;  dB_a = s_a (x_a A_a)^T dg_a
"""
import math
import random

import torch

own = False
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp8": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of an 8B-sized model between two blocks: latency alone
        dict(name="norm_token", op="norm", dtype="bf16", T=1, d=4096),
        # an odd number of rows, a width that is no power of two, 32 bits
        dict(name="norm_f32_odd", op="norm", dtype="f32", T=1111, d=1544),
        # the decode rows of an 8B-sized layer whose weights are FP8
        dict(name="norm_fp8_decode", op="norm", dtype="fp8", T=192, d=4096),
        # the rows of 64 prompts at once, FP8 weights: bandwidth alone
        dict(name="norm_fp8_prefill", op="norm", dtype="fp8", T=34811, d=4096),
        # one token through gate and up of an 8B-sized layer
        dict(name="gated_token", op="gated", dtype="bf16", T=1, d=4096, f=14336, slots=32, rank=16, ranks="full",
             rows="tokens", act="silu", save=False),
        # 512 decode rows and prompts of a 70B-sized layer, ranks 8 to 64
        dict(name="gated_mixed_70b", op="gated", dtype="bf16", T=4608, d=8192, f=28672, slots=32, rank=64,
             ranks="ragged", rows="mixed", act="silu", save=False),
        # odd sizes in 32 bits, with gate and up kept for a backward pass
        dict(name="gated_f32_odd", op="gated", dtype="f32", T=333, d=1032, f=2744, slots=5, rank=24, ranks="ragged",
             rows="mixed", act="gelu", save=True),
        # the decode rows of an 8B-sized layer, FP8 weights
        dict(name="gated_fp8_decode", op="gated", dtype="fp8", T=192, d=4096, f=14336, slots=64, rank=16,
             ranks="full", rows="tokens", act="silu", save=False),
        # decode rows and prompts of an 8B-sized layer together, FP8 weights
        dict(name="gated_fp8_mixed", op="gated", dtype="fp8", T=2240, d=4096, f=14336, slots=64, rank=16,
             ranks="full", rows="mixed", act="silu", save=False),
        # a training step of four adapters on an 8B-sized layer
        dict(name="backward_8b", op="backward", dtype="bf16", T=2048, d=4096, f=14336, slots=4, rank=16,
             ranks="full", rows="prompts", act="silu"),
        # many adapters of odd ranks and few rows each
        dict(name="backward_ragged", op="backward", dtype="bf16", T=777, d=1048, f=2744, slots=24, rank=40,
             ranks="ragged", rows="mixed", act="gelu_tanh"),
        # the same in 32 bits
        dict(name="backward_f32", op="backward", dtype="f32", T=190, d=520, f=1384, slots=6, rank=16, ranks="ragged",
             rows="tokens", act="gelu"),
    ]


def _spread(rng, low, high, step):
    """A multiple of `step` in [low, high], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return min(high, max(low, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "gated", "gated", "gated", "backward", "backward"])
    if op == "norm":
        dtype = rng.choice(["bf16", "f32", "fp8"])
        d = _spread(rng, 64, 28672, 16 if dtype == "fp8" else 8)
        most = min(34811, 34811 * 4096 // d // (2 if dtype == "f32" else 1))
        return dict(op=op, dtype=dtype, T=_spread(rng, 1, most, 1), d=d)
    dtype = rng.choice(["bf16", "f32", "bf16", "fp8"] if op == "gated" else ["bf16", "bf16", "f32"])
    # 32 bits stand for checks and small models
    wide = 1024 if dtype == "f32" else 8192
    while True:
        d = _spread(rng, 128, wide, 16 if dtype == "fp8" else 8)
        f = _spread(rng, 128, wide * 7 // 2, 8)
        T = _spread(rng, 1, 400 if dtype == "f32" else 6000, 1)
        if T * d * f <= 4608 * 8192 * 28672 // (8 if op == "backward" else 2):
            break
    case = dict(op=op, dtype=dtype, T=T, d=d, f=f, slots=_spread(rng, 1, 32, 1), rank=_spread(rng, 8, 64, 8),
                ranks=rng.choice(["full", "ragged"]), rows=rng.choice(["tokens", "prompts", "mixed"]),
                act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]))
    if op == "gated":
        case["save"] = rng.random() < 0.25
    return case


def _lengths(case, rng):
    """Rows of each request: single tokens, prompts, or a ninth of single tokens and prompts."""
    T, kind = case["T"], case["rows"]
    lengths = [1] * (T if kind == "tokens" else T // 9 if kind == "mixed" else 0)
    left = T - len(lengths)
    while left > 0:
        n = min(left, rng.randint(64, 1024))
        lengths.append(n)
        left -= n
    rng.shuffle(lengths)
    return lengths


def _normal(gen, shape, std, dtype):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def _e4m3(x):
    """E4M3 codes and the power-of-two scale of each row of x: the smallest 2^e with amax <= 448 * 2^e."""
    m, e = torch.frexp(x.float().abs().amax(1))
    e = torch.where(m > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -127))
    scale = torch.ldexp(torch.ones_like(m), e)
    return (x.float() / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, T, d = TYPES[case["dtype"]], case["T"], case["d"]
    s = dict(case)
    if case["op"] == "norm":
        # a block's output beside the wider residual stream it is added to
        s["x"] = _normal(gen, (T, d), 1.0, dtype)
        s["residual"] = _normal(gen, (T, d), 3.0, dtype)
        s["weight"] = (1.0 + _normal(gen, (d,), 0.2, torch.float32)).to(dtype)
        s["handle"] = _norm_handle(s) if own else None
        return s
    rng = random.Random(seed)
    f, S, R = case["f"], case["slots"], case["rank"]
    ranks = [R if case["ranks"] == "full" else rng.randint(1, R) for _ in range(S)]
    lengths = _lengths(case, rng)
    owners = [rng.randrange(S) if rng.random() < 0.9 else -1 for _ in lengths]
    s["ids"] = torch.repeat_interleave(torch.tensor(owners, dtype=torch.int32), torch.tensor(lengths)).cuda()
    s["rank_list"], s["alpha_list"] = ranks, [2.0 * r for r in ranks]
    s["scale"] = torch.full((S,), 2.0, device="cuda")
    kept = (torch.arange(R)[None, :] < torch.tensor(ranks)[:, None]).cuda()
    s["x"] = _normal(gen, (T, d), 1.0, dtype)
    for p in ("gate", "up"):
        s["W_" + p] = _normal(gen, (d, f), 1.3 / math.sqrt(d), dtype)
        s["A_" + p] = _normal(gen, (S, d, R), 1.3 / math.sqrt(d), dtype) * kept[:, None, :]
        s["B_" + p] = _normal(gen, (S, R, f), 0.3 / math.sqrt(R), dtype) * kept[:, :, None]
    if case["dtype"] == "fp8":
        s["xq"], s["x_scale"] = _e4m3(s["x"])  # as the norm leaves them
        for p in ("gate", "up"):
            s["Wq_" + p], s["W_scale_" + p] = _e4m3(s.pop("W_" + p).t().contiguous())
    if case["op"] == "backward":
        s["gate"] = _normal(gen, (T, f), 1.3, dtype)  # as the forward pass kept them
        s["up"] = _normal(gen, (T, f), 1.3, dtype)
        s["dh"] = _normal(gen, (T, f), 0.01, dtype)
    s["handle"] = _gated_handle(s) if own else None
    return s


# ---- the plain forms ------------------------------------------------------


def _norm_plain(s):
    z = s["x"].float() + s["residual"].float()
    y = (z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * s["weight"].float()).to(s["x"].dtype)
    out = {"residual": z.to(s["x"].dtype), "y": y}
    if s["dtype"] == "fp8":
        out["codes"], out["scale"] = _e4m3(y)  # the codes are those of the rounded y
    return out


def _act(name, g):
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_slope(name, g):
    if name == "silu":
        q = torch.sigmoid(g)
        return q * (1.0 + g * (1.0 - q))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _owned(s):
    """[T, slots * rank]: a row's scale at its own adapter's ranks, zero at the others'."""
    S, R = s["slots"], s["rank"]
    slot = torch.arange(S * R, device="cuda") // R
    return (s["ids"][:, None] == slot[None, :]) * s["scale"].repeat_interleave(R)[None, :]


def _wide(s, p):
    """All slots' A as one [d, slots * rank] and all slots' B as one [slots * rank, f], in 32 bits."""
    A, B = s["A_" + p].float(), s["B_" + p].float()
    return A.permute(1, 0, 2).reshape(A.shape[1], -1), B.reshape(-1, B.shape[2])


def _project(s, p, owned):
    if s["dtype"] == "fp8":
        base = (s["xq"].float() * s["x_scale"][:, None]) @ (s["Wq_" + p].float() * s["W_scale_" + p][:, None]).t()
    else:
        base = s["x"].float() @ s["W_" + p].float()
    A, B = _wide(s, p)
    return base + ((s["x"].float() @ A) * owned) @ B


def _gated_plain(s):
    owned, dtype = _owned(s), s["x"].dtype
    g, u = _project(s, "gate", owned), _project(s, "up", owned)
    out = {"h": (_act(s["act"], g) * u).to(dtype)}
    if s["save"]:
        out["gate"], out["up"] = g.to(dtype), u.to(dtype)
    return out


def _backward_plain(s):
    owned, dtype, S, R = _owned(s), s["x"].dtype, s["slots"], s["rank"]
    x, g, u, dh = (s[k].float() for k in ("x", "gate", "up", "dh"))
    grads = {"gate": dh * u * _act_slope(s["act"], g), "up": dh * _act(s["act"], g)}
    dx, out = 0.0, {}
    kept = (torch.arange(S * R, device="cuda") % R) < torch.tensor(s["rank_list"], device="cuda").repeat_interleave(R)
    for p in ("gate", "up"):
        A, B = _wide(s, p)
        dv = (grads[p] @ B.t()) * owned
        dx = dx + grads[p] @ s["W_" + p].float().t() + dv @ A.t()
        dA = (x.t() @ dv) * kept[None, :]
        dB = (((x @ A) * owned).t() @ grads[p]) * kept[:, None]
        out["dA_" + p] = dA.reshape(-1, S, R).permute(1, 0, 2).contiguous().to(dtype)
        out["dB_" + p] = dB.reshape(S, R, -1).to(dtype)
    out["dx"] = dx.to(dtype)
    return out


# ---- the framework's calls ------------------------------------------------


def _norm_handle(s):
    from rank_adapter_gemm_amd import lora as L
    x, fp8 = s["x"], s["dtype"] == "fp8"
    return dict(L=L, residual=torch.empty_like(x), y=torch.empty_like(x),
                codes=torch.empty(x.shape, dtype=torch.uint8, device="cuda") if fp8 else None,
                scale=torch.empty(x.shape[0], dtype=torch.float32, device="cuda") if fp8 else None)


def _norm_own(s):
    h, T, d = s["handle"], s["T"], s["d"]
    L = h["L"]
    if s["dtype"] == "fp8":
        L.lora_add_rmsnorm_fp8(s["x"], s["residual"], s["weight"], EPS, T, d, h["residual"], h["y"], h["codes"],
                               h["scale"])
        return {"residual": h["residual"], "y": h["y"], "codes": h["codes"].view(torch.float8_e4m3fn),
                "scale": h["scale"]}
    L.lora_add_rmsnorm(s["x"], s["residual"], s["weight"], EPS, T, d, L.dtype_code(s["x"].dtype), h["residual"],
                       h["y"])
    return {"residual": h["residual"], "y": h["y"]}


def _gated_handle(s):
    from rank_adapter_gemm_amd import lora as L
    T, d, f, S, R, dtype = s["T"], s["d"], s["f"], s["slots"], s["rank"], s["x"].dtype
    new = lambda *shape: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    pools = []
    for p in ("gate", "up"):
        pool = L.AdapterPool(S, d, f, R, dtype)
        for i in range(S):
            pool.upload(i, s["A_" + p][i], s["B_" + p][i], s["rank_list"][i], s["alpha_list"][i], lda=R, ldb=f)
        pools.append(pool)
    h = dict(L=L, pools=pools, descriptors=[p.pool for p in pools],
             act={"silu": L.LORA_ACT_SILU, "gelu": L.LORA_ACT_GELU, "gelu_tanh": L.LORA_ACT_GELU_TANH}[s["act"]])
    if s["op"] == "backward":
        h["ws"] = L.Workspace(T, S, R, f, gated=True, backward_d_in=d, dtype=dtype)
        h["dx"] = new(T, d)
        h["dA"], h["dB"] = [new(S, d, R), new(S, d, R)], [new(S, R, f), new(S, R, f)]
        return h
    h["ws"] = L.Workspace(T, S, R, f, gated=True, fp8_d_in=d if s["dtype"] == "fp8" else 0)
    h["h"] = new(T, f)
    h["gate"], h["up"] = (new(T, f), new(T, f)) if s["save"] else (None, None)
    if s["dtype"] == "fp8":
        for k in ("xq", "Wq_gate", "Wq_up"):
            h[k] = s[k].view(torch.uint8)
    return h


def _gated_own(s):
    h = s["handle"]
    L = h["L"]
    if s["dtype"] == "fp8":
        L.lora_gated_forward_fp8(s["x"], h["xq"], s["x_scale"], h["Wq_gate"], s["W_scale_gate"], h["Wq_up"],
                                 s["W_scale_up"], h["h"], s["T"], h["descriptors"], s["ids"], h["act"],
                                 L.LORA_MODE_AUTO, 0, h["ws"].buf, gate=h["gate"], up=h["up"])
    else:
        L.lora_gated_forward(s["x"], s["W_gate"], s["W_up"], h["h"], s["T"], h["descriptors"], s["ids"], h["act"],
                             L.LORA_MODE_AUTO, 0, h["ws"].buf, gate=h["gate"], up=h["up"])
    out = {"h": h["h"]}
    if s["save"]:
        out["gate"], out["up"] = h["gate"], h["up"]
    return out


def _backward_own(s):
    h = s["handle"]
    h["L"].lora_gated_backward(s["x"], s["W_gate"], s["W_up"], s["T"], h["descriptors"], s["ids"], h["act"],
                               s["gate"], s["up"], s["dh"], h["dx"], h["dA"], h["dB"], h["ws"].buf)
    return {"dx": h["dx"], "dA_gate": h["dA"][0], "dA_up": h["dA"][1], "dB_gate": h["dB"][0], "dB_up": h["dB"][1]}


def run(state):
    if own:
        return {"norm": _norm_own, "gated": _gated_own, "backward": _backward_own}[state["op"]](state)
    return {"norm": _norm_plain, "gated": _gated_plain, "backward": _backward_plain}[state["op"]](state)


def work(case):
    T, d = case["T"], case["d"]
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        # x, residual, weight in; the new residual and y (and codes with a scale a row) out
        more = T * (d + 4) if case["dtype"] == "fp8" else 0
        return {"bytes": e * (4 * T * d + d) + more, "flops": 5 * T * d}
    f, S, R = case["f"], case["slots"], case["rank"]
    used = min(S, T if case["rows"] == "tokens" else max(1, T // 544) + (T // 9 if case["rows"] == "mixed" else 0))
    r = R if case["ranks"] == "full" else (R + 1) // 2
    adapters = 2 * used * r * (d + f) * e
    if case["op"] == "gated":
        we = 1 if case["dtype"] == "fp8" else e
        out = T * f * e * (3 if case["save"] else 1)
        codes = T * (d + 4) + 8 * f if case["dtype"] == "fp8" else 0
        return {"bytes": T * d * e + codes + 2 * d * f * we + adapters + out + 4 * T,
                "flops": 4 * T * d * f + 4 * T * r * (d + f)}
    # x, gate, up, dh and the weights in; dx and every slot's gradients out
    out = T * d * e + 2 * S * R * (d + f) * e
    return {"bytes": T * d * e + 3 * T * f * e + 2 * d * f * e + adapters + out + 4 * T,
            "flops": 4 * T * d * f + 4 * T * r * (3 * d + 2 * f)}


# ---- the definitions in 64 bits, one adapter at a time ---------------------


def _rows_of(s, slot):
    return torch.nonzero(s["ids"] == slot).flatten()


def _exact_project(s, p):
    x = s["x"].double()
    if s["dtype"] == "fp8":
        codes, weights = s["xq"].double(), s["Wq_" + p].double()
        y = torch.matmul(codes, weights.transpose(0, 1))
        y *= s["x_scale"].double().unsqueeze(1)
        y *= s["W_scale_" + p].double()
    else:
        y = torch.matmul(x, s["W_" + p].double())
    for slot, r in enumerate(s["rank_list"]):
        t = _rows_of(s, slot)
        if len(t):
            v = torch.matmul(x[t], s["A_" + p][slot, :, :r].double())
            y[t] += s["alpha_list"][slot] / r * torch.matmul(v, s["B_" + p][slot, :r].double())
    return y


def _exact_act(name, g):
    """The activation and its derivative."""
    if name == "silu":
        q = 1.0 / (1.0 + torch.exp(-g))
        return g * q, q + g * q * (1.0 - q)
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * torch.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    q = 1.0 / (1.0 + torch.exp(-2.0 * k * (g + 0.044715 * g ** 3)))  # (1 + tanh) / 2
    return g * q, q + g * 2.0 * q * (1.0 - q) * k * (1.0 + 0.134145 * g ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        z = s["x"].double() + s["residual"].double()
        y = z / torch.sqrt((z * z).sum(1, keepdim=True) / case["d"] + EPS) * s["weight"].double()
        out = {"residual": z, "y": y}
        if case["dtype"] == "fp8":
            amax = y.to(torch.bfloat16).double().abs().max(1).values  # of y as it is stored
            scale = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
            out["codes"], out["scale"] = y / scale.unsqueeze(1), scale
        return out
    if case["op"] == "gated":
        g, u = _exact_project(s, "gate"), _exact_project(s, "up")
        out = {"h": _exact_act(case["act"], g)[0] * u}
        if case["save"]:
            out["gate"], out["up"] = g, u
        return out
    x, dh = s["x"].double(), s["dh"].double()
    act, slope = _exact_act(case["act"], s["gate"].double())
    grads = {"gate": dh * s["up"].double() * slope, "up": dh * act}
    out = {}
    dx = torch.zeros_like(x)
    for p, dy in grads.items():
        dx += torch.matmul(dy, s["W_" + p].double().transpose(0, 1))
        dA, dB = torch.zeros_like(s["A_" + p]).double(), torch.zeros_like(s["B_" + p]).double()
        for slot, r in enumerate(s["rank_list"]):
            t = _rows_of(s, slot)
            if not len(t):
                continue
            A, B = s["A_" + p][slot, :, :r].double(), s["B_" + p][slot, :r].double()
            scale = s["alpha_list"][slot] / r
            dv = scale * torch.matmul(dy[t], B.transpose(0, 1))
            dx[t] += torch.matmul(dv, A.transpose(0, 1))
            dA[slot, :, :r] = torch.matmul(x[t].transpose(0, 1), dv)
            dB[slot, :r] = scale * torch.matmul(torch.matmul(x[t], A).transpose(0, 1), dy[t])
        out["dA_" + p], out["dB_" + p] = dA, dB
    out["dx"] = dx
    return out
