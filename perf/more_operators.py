"""The operators of a biased feed-forward block with adapters, served and trained, as they are measured.

Five operators of one path: the residual addition with its layer norm (with
E4M3 codes of the result where the base weights are FP8) and its backward
pass, the linear layer with bias, activation and residual beside every row's
own low-rank adapter, that layer's backward pass, and the orthogonalised
update made of the adapters' gradients.  `run` computes them in their plain
form, or, where `own` is true, by the calls a user makes of
rank_adapter_gemm_amd.

    z = x + residual;  y = (z - mean(z)) / sqrt(var(z) + eps) * weight + bias
    h = (z - mean) * rstd;  a = dy * weight
    dx = rstd * (a - mean(a) - h * mean(a * h)) + dresidual;  dweight = sum dy * h;  dbias = sum dy
    p = x W + bias + s_a (x A_a) B_a;  y = act(p) + residual
    dp = dy * act'(p);  dv = s_a dp B_a^T;  dx = dp W^T + dv A_a^T
    dA_a = x_a^T dv_a;  dB_a = s_a (x_a A_a)^T dp_a;  dbias = sum dp
    X = G / (|G| + eps), then, step by step, X = c0 X + c1 (X X^T) X + c2 (X X^T)^2 X
"""
import math
import random

import torch

own = False
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp8": torch.bfloat16, "f32": torch.float32}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
ORTHO_EPS = 1e-7


def listed():
    return [
        # one token of an 8B-sized model between two blocks: latency alone
        dict(name="norm_token", op="norm", dtype="bf16", T=1, d=4096),
        # the rows of many prompts at once, FP8 weights after them: bandwidth alone
        dict(name="norm_fp8_prefill", op="norm", dtype="fp8", T=12345, d=8192),
        # a training batch of an 8B-sized model
        dict(name="norm_backward", op="norm_backward", dtype="bf16", T=34811, d=4096, residual=True),
        # an odd number of rows, a width that is no power of two, 32 bits
        dict(name="norm_backward_odd", op="norm_backward", dtype="f32", T=1111, d=1544, residual=False),
        # one token through the second layer of an 8B-sized block, onto the residual stream
        dict(name="linear_token", op="linear", dtype="bf16", T=1, d=14336, f=4096, slots=32, rank=16, ranks="full",
             rows="tokens", act="none", residual=True, save=False),
        # 512 decode rows and prompts through the first layer of a 70B-sized block
        dict(name="linear_mixed_70b", op="linear", dtype="bf16", T=4608, d=8192, f=28672, slots=32, rank=64,
             ranks="ragged", rows="mixed", act="gelu", residual=False, save=False),
        # the decode rows of an 8B-sized layer, FP8 weights
        dict(name="linear_fp8_decode", op="linear", dtype="fp8", T=192, d=4096, f=14336, slots=64, rank=16,
             ranks="full", rows="tokens", act="gelu_tanh", residual=False, save=False),
        # odd sizes in 32 bits, with the activation's argument kept for a backward pass
        dict(name="linear_f32_odd", op="linear", dtype="f32", T=333, d=1032, f=2744, slots=5, rank=24, ranks="ragged",
             rows="mixed", act="gelu", residual=True, save=True),
        # a training step of four adapters on the second layer of an 8B-sized block
        dict(name="linear_backward_8b", op="linear_backward", dtype="bf16", T=2048, d=14336, f=4096, slots=4, rank=16,
             ranks="full", rows="prompts", act="none"),
        # many adapters of odd ranks and few rows each, through an activation
        dict(name="linear_backward_ragged", op="linear_backward", dtype="bf16", T=777, d=1048, f=2744, slots=24,
             rank=40, ranks="ragged", rows="mixed", act="gelu_tanh"),
        # the gradients of A of 32 adapters of an 8B-sized layer
        dict(name="ortho_a", op="ortho", dtype="bf16", n=32, d=4096, r=16, ranks="full", wide=False),
        # the gradients of B of a few adapters of large and odd ranks, in 32 bits
        dict(name="ortho_b_f32", op="ortho", dtype="f32", n=8, d=14336, r=64, ranks="ragged", wide=True),
    ]


def _spread(rng, low, high, step):
    """A multiple of `step` in [low, high], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return min(high, max(low, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "linear", "linear", "linear_backward", "ortho", "ortho"])
    if op in ("norm", "norm_backward"):
        dtype = rng.choice(["bf16", "f32", "fp8"] if op == "norm" else ["bf16", "f32"])
        d = _spread(rng, 64, 28672, 16 if dtype == "fp8" else 8)
        most = min(34811, 34811 * 4096 // d // (2 if dtype == "f32" else 1))
        case = dict(op=op, dtype=dtype, T=_spread(rng, 1, most, 1), d=d)
        if op == "norm_backward":
            case["residual"] = rng.random() < 0.5
        return case
    if op == "ortho":
        dtype = rng.choice(["bf16", "f32"])
        r = _spread(rng, 8, 128 if dtype == "bf16" else 64, 8)
        d = _spread(rng, 128, 28672, 8)
        most = max(1, min(64, 8 * 14336 * 64 * 64 // (d * r * r)))
        return dict(op=op, dtype=dtype, n=_spread(rng, 1, most, 1), d=d, r=r, ranks=rng.choice(["full", "ragged"]),
                    wide=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "f32", "bf16", "fp8"] if op == "linear" else ["bf16", "bf16", "f32"])
    # 32 bits stand for checks and small models
    wide = 1024 if dtype == "f32" else 8192
    while True:
        d = _spread(rng, 128, 2 * wide, 16 if dtype == "fp8" else 8)
        f = _spread(rng, 128, wide * 7 // 2, 8)
        T = _spread(rng, 1, 400 if dtype == "f32" else 6000, 1)
        if T * d * f <= 4608 * 8192 * 28672 // (4 if op == "linear_backward" else 1):
            break
    case = dict(op=op, dtype=dtype, T=T, d=d, f=f, slots=_spread(rng, 1, 32, 1), rank=_spread(rng, 8, 64, 8),
                ranks=rng.choice(["full", "ragged"]), rows=rng.choice(["tokens", "prompts", "mixed"]),
                act=rng.choice(["none", "silu", "gelu", "gelu_tanh"]))
    if op == "linear":
        case["residual"] = rng.random() < 0.5
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
    dtype, d = TYPES[case["dtype"]], case["d"]
    s = dict(case)
    if case["op"] in ("norm", "norm_backward"):
        T = case["T"]
        s["weight"] = (1.0 + _normal(gen, (d,), 0.2, torch.float32)).to(dtype)
        if case["op"] == "norm":
            # a block's output beside the wider residual stream it is added to
            s["x"] = _normal(gen, (T, d), 1.0, dtype)
            s["residual"] = _normal(gen, (T, d), 3.0, dtype)
            s["bias"] = _normal(gen, (d,), 0.2, dtype)
        else:
            # the residual stream as the forward pass left it, a row's mean included
            z = _normal(gen, (T, d), 3.0, torch.float32).add_(_normal(gen, (T, 1), 0.5, torch.float32))
            s["z"] = z.to(dtype)
            var, s["mean"] = torch.var_mean(z, 1, correction=0)
            s["rstd"] = torch.rsqrt(var + EPS)
            s["dy"] = _normal(gen, (T, d), 0.01, dtype)
            s["dresidual"] = _normal(gen, (T, d), 0.01, dtype) if case["residual"] else None
        s["handle"] = _HANDLES[case["op"]](s) if own else None
        return s
    rng = random.Random(seed)
    if case["op"] == "ortho":
        # gradients of falling singular values, as an adapter's are; ranks past an adapter's are zero
        n, r = case["n"], case["r"]
        kept = [r if case["ranks"] == "full" else rng.randint(1, r) for _ in range(n)]
        kept = (torch.arange(r)[None, :] < torch.tensor(kept)[:, None]).cuda()
        fall = torch.pow(10.0, -2.0 * torch.arange(r, device="cuda") / r)
        mix = _normal(gen, (n, r, r), 1e-3 / math.sqrt(r), torch.float32) * fall[None, :, None]
        g = torch.matmul(_normal(gen, (n, d, r), 1.0, torch.float32), mix) * kept[:, None, :]
        s["g"] = (g.transpose(1, 2) if case["wide"] else g).contiguous().to(dtype)
        s["handle"] = _HANDLES["ortho"](s) if own else None
        return s
    T, f, S, R = case["T"], case["f"], case["slots"], case["rank"]
    ranks = [R if case["ranks"] == "full" else rng.randint(1, R) for _ in range(S)]
    lengths = _lengths(case, rng)
    owners = [rng.randrange(S) if rng.random() < 0.9 else -1 for _ in lengths]
    s["ids"] = torch.repeat_interleave(torch.tensor(owners, dtype=torch.int32), torch.tensor(lengths)).cuda()
    s["rank_list"], s["alpha_list"] = ranks, [2.0 * r for r in ranks]
    s["scale"] = torch.full((S,), 2.0, device="cuda")
    kept = (torch.arange(R)[None, :] < torch.tensor(ranks)[:, None]).cuda()
    s["x"] = _normal(gen, (T, d), 1.0, dtype)
    s["W"] = _normal(gen, (d, f), 1.3 / math.sqrt(d), dtype)
    s["A"] = _normal(gen, (S, d, R), 1.3 / math.sqrt(d), dtype) * kept[:, None, :]
    s["B"] = _normal(gen, (S, R, f), 0.3 / math.sqrt(R), dtype) * kept[:, :, None]
    if case["op"] == "linear":
        s["bias"] = _normal(gen, (f,), 0.5, dtype)
        s["residual"] = _normal(gen, (T, f), 3.0, dtype) if case["residual"] else None
        if case["dtype"] == "fp8":
            s["xq"], s["x_scale"] = _e4m3(s["x"])  # as the norm leaves them
            s["Wq"], s["W_scale"] = _e4m3(s.pop("W").t().contiguous())
    else:
        # as the forward pass kept it; a layer without activation keeps nothing
        s["pre"] = _normal(gen, (T, f), 1.3, dtype) if case["act"] != "none" else None
        s["dy"] = _normal(gen, (T, f), 0.01, dtype)
    s["handle"] = _HANDLES[case["op"]](s) if own else None
    return s


# ---- the plain forms ------------------------------------------------------


def _norm_plain(s):
    z = s["x"].float() + s["residual"].float()
    c = z - z.mean(1, keepdim=True)
    y = c * torch.rsqrt(c.square().mean(1, keepdim=True) + EPS) * s["weight"].float() + s["bias"].float()
    y = y.to(s["x"].dtype)
    out = {"residual": z.to(s["x"].dtype), "y": y}
    if s["dtype"] == "fp8":
        codes, out["scale"] = _e4m3(y)  # the codes are those of the rounded y
        out["codes"] = codes
    return out


def _norm_backward_plain(s):
    dtype = s["z"].dtype
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    h = (s["z"].float() - s["mean"][:, None]) * rstd
    a = dy * s["weight"].float()
    dx = rstd * (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return {"dx": dx.to(dtype), "dweight": (dy * h).sum(0).to(dtype), "dbias": dy.sum(0).to(dtype)}


def _act(name, p):
    if name == "none":
        return p
    if name == "silu":
        return p * torch.sigmoid(p)
    if name == "gelu":
        return 0.5 * p * (1.0 + torch.erf(p * math.sqrt(0.5)))
    return 0.5 * p * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (p + 0.044715 * p * p * p)))


def _act_slope(name, p):
    if name == "silu":
        q = torch.sigmoid(p)
        return q * (1.0 + p * (1.0 - q))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(p * math.sqrt(0.5))) + p * torch.exp(-0.5 * p * p) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (p + 0.044715 * p * p * p))
    return 0.5 * (1.0 + t) + 0.5 * p * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * p * p)


def _owned(s):
    """[T, slots * rank]: a row's scale at its own adapter's ranks, zero at the others'."""
    S, R = s["slots"], s["rank"]
    slot = torch.arange(S * R, device="cuda") // R
    return (s["ids"][:, None] == slot[None, :]) * s["scale"].repeat_interleave(R)[None, :]


def _wide(s):
    """All slots' A as one [d, slots * rank] and all slots' B as one [slots * rank, f], in 32 bits."""
    A, B = s["A"].float(), s["B"].float()
    return A.permute(1, 0, 2).reshape(A.shape[1], -1), B.reshape(-1, B.shape[2])


def _linear_plain(s):
    dtype = s["x"].dtype
    if s["dtype"] == "fp8":
        p = (s["xq"].float() * s["x_scale"][:, None]) @ (s["Wq"].float() * s["W_scale"][:, None]).t()
    else:
        p = s["x"].float() @ s["W"].float()
    A, B = _wide(s)
    p = p + s["bias"].float() + ((s["x"].float() @ A) * _owned(s)) @ B
    y = _act(s["act"], p)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(dtype)}
    if s["save"]:
        out["pre"] = p.to(dtype)
    return out


def _linear_backward_plain(s):
    dtype, S, R = s["x"].dtype, s["slots"], s["rank"]
    owned = _owned(s)
    x, dp = s["x"].float(), s["dy"].float()
    if s["act"] != "none":
        dp = dp * _act_slope(s["act"], s["pre"].float())
    kept = (torch.arange(S * R, device="cuda") % R) < torch.tensor(s["rank_list"], device="cuda").repeat_interleave(R)
    A, B = _wide(s)
    dv = (dp @ B.t()) * owned
    dx = dp @ s["W"].float().t() + dv @ A.t()
    dA = (x.t() @ dv) * kept[None, :]
    dB = (((x @ A) * owned).t() @ dp) * kept[:, None]
    return {"dx": dx.to(dtype), "dA": dA.reshape(-1, S, R).permute(1, 0, 2).contiguous().to(dtype),
            "dB": dB.reshape(S, R, -1).to(dtype), "dbias": dp.sum(0).to(dtype)}


def _ortho_plain(s):
    x = s["g"].float()
    if not s["wide"]:
        x = x.transpose(1, 2)
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + ORTHO_EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        m = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * m + c * torch.matmul(m, m), x)
    if not s["wide"]:
        x = x.transpose(1, 2)
    return {"update": x.contiguous().to(s["g"].dtype)}


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
        L.lora_add_layernorm_fp8(s["x"], s["residual"], s["weight"], s["bias"], EPS, T, d, h["residual"], h["y"],
                                 h["codes"], h["scale"])
        return {"residual": h["residual"], "y": h["y"], "scale": h["scale"],
                "codes": h["codes"].view(torch.float8_e4m3fn)}
    L.lora_add_layernorm(s["x"], s["residual"], s["weight"], s["bias"], EPS, T, d, L.dtype_code(s["x"].dtype),
                         h["residual"], h["y"])
    return {"residual": h["residual"], "y": h["y"]}


def _norm_backward_handle(s):
    from rank_adapter_gemm_amd import lora as L
    T, d = s["T"], s["d"]
    ws = torch.empty(L.lora_workspace_bytes_layernorm_backward(T, d), dtype=torch.uint8, device="cuda")
    return dict(L=L, ws=ws, dx=torch.empty_like(s["z"]), dweight=torch.empty_like(s["weight"]),
                dbias=torch.empty_like(s["weight"]))


def _norm_backward_own(s):
    h = s["handle"]
    L = h["L"]
    L.lora_add_layernorm_backward(s["dy"], s["dresidual"], s["z"], s["weight"], s["mean"], s["rstd"], s["T"], s["d"],
                                  L.dtype_code(s["z"].dtype), h["dx"], h["dweight"], h["dbias"], h["ws"])
    return {"dx": h["dx"], "dweight": h["dweight"], "dbias": h["dbias"]}


def _linear_handle(s):
    from rank_adapter_gemm_amd import lora as L
    T, d, f, S, R, dtype = s["T"], s["d"], s["f"], s["slots"], s["rank"], s["x"].dtype
    new = lambda *shape: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    pool = L.AdapterPool(S, d, f, R, dtype)
    for i in range(S):
        pool.upload(i, s["A"][i], s["B"][i], s["rank_list"][i], s["alpha_list"][i], lda=R, ldb=f)
    h = dict(L=L, pool=pool, act={"none": L.LORA_ACT_NONE, "silu": L.LORA_ACT_SILU, "gelu": L.LORA_ACT_GELU,
                                  "gelu_tanh": L.LORA_ACT_GELU_TANH}[s["act"]])
    if s["op"] == "linear_backward":
        h["ws"] = L.Workspace(T, S, R, f, linear_backward_d_in=d, dtype=dtype)
        h["dx"], h["dA"], h["dB"], h["dbias"] = new(T, d), new(S, d, R), new(S, R, f), new(f)
        return h
    h["ws"] = L.Workspace(T, S, R, f, fp8_d_in=d if s["dtype"] == "fp8" else 0)
    h["y"], h["pre"] = new(T, f), new(T, f) if s["save"] else None
    if s["dtype"] == "fp8":
        h["xq"], h["Wq"] = s["xq"].view(torch.uint8), s["Wq"].view(torch.uint8)
    return h


def _linear_own(s):
    h = s["handle"]
    L = h["L"]
    if s["dtype"] == "fp8":
        L.lora_linear_act_forward_fp8(s["x"], h["xq"], s["x_scale"], h["Wq"], s["W_scale"], s["bias"], s["residual"],
                                      h["y"], s["T"], h["pool"].pool, s["ids"], h["act"], L.LORA_MODE_AUTO, 0,
                                      h["ws"].buf, pre=h["pre"])
    else:
        L.lora_linear_act_forward(s["x"], s["W"], s["bias"], s["residual"], h["y"], s["T"], h["pool"].pool, s["ids"],
                                  h["act"], L.LORA_MODE_AUTO, 0, h["ws"].buf, pre=h["pre"])
    out = {"y": h["y"]}
    if s["save"]:
        out["pre"] = h["pre"]
    return out


def _linear_backward_own(s):
    h = s["handle"]
    h["L"].lora_linear_act_backward(s["x"], s["W"], s["T"], h["pool"].pool, s["ids"], h["act"], s["pre"], s["dy"],
                                    h["dx"], h["dA"], h["dB"], h["dbias"], h["ws"].buf)
    return {"dx": h["dx"], "dA": h["dA"], "dB": h["dB"], "dbias": h["dbias"]}


def _ortho_handle(s):
    from rank_adapter_gemm_amd import lora as L
    n, rows, cols = s["g"].shape
    ws = torch.empty(L.lora_workspace_bytes_orthogonalize(n, rows, cols), dtype=torch.uint8, device="cuda")
    return dict(L=L, ws=ws, update=torch.empty_like(s["g"]))


def _ortho_own(s):
    h = s["handle"]
    L = h["L"]
    n, rows, cols = s["g"].shape
    L.lora_orthogonalize(s["g"], n, rows, cols, L.dtype_code(s["g"].dtype), [COEFFICIENTS] * STEPS, ORTHO_EPS, 1.0,
                         h["update"], h["ws"])
    return {"update": h["update"]}


_HANDLES = {"norm": _norm_handle, "norm_backward": _norm_backward_handle, "linear": _linear_handle,
            "linear_backward": _linear_handle, "ortho": _ortho_handle}
_PLAIN = {"norm": _norm_plain, "norm_backward": _norm_backward_plain, "linear": _linear_plain,
          "linear_backward": _linear_backward_plain, "ortho": _ortho_plain}
_OWN = {"norm": _norm_own, "norm_backward": _norm_backward_own, "linear": _linear_own,
        "linear_backward": _linear_backward_own, "ortho": _ortho_own}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def work(case):
    d = case["d"]
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        # x, residual, weight and bias in; the new residual and y (and codes with a scale a row) out
        T = case["T"]
        more = T * (d + 4) if case["dtype"] == "fp8" else 0
        return {"bytes": e * (4 * T * d + 2 * d) + more, "flops": 8 * T * d}
    if case["op"] == "norm_backward":
        # dy, z (and the residual's gradient) in, dx and the weights' gradients out
        T = case["T"]
        return {"bytes": e * ((4 if case["residual"] else 3) * T * d + 3 * d) + 8 * T, "flops": 14 * T * d}
    if case["op"] == "ortho":
        # the gradients in, the update out; the Gram matrix and one product with its polynomial
        n, r = case["n"], case["r"]
        return {"bytes": 2 * n * d * r * e, "flops": 3 * n * d * r * r + 17 * n * r ** 3}
    T, f, S, R = case["T"], case["f"], case["slots"], case["rank"]
    used = min(S, T if case["rows"] == "tokens" else max(1, T // 544) + (T // 9 if case["rows"] == "mixed" else 0))
    r = R if case["ranks"] == "full" else (R + 1) // 2
    adapters = used * r * (d + f) * e
    if case["op"] == "linear":
        we = 1 if case["dtype"] == "fp8" else e
        out = T * f * e * (1 + case["save"] + case["residual"])
        codes = T * (d + 4) + 4 * f if case["dtype"] == "fp8" else 0
        return {"bytes": T * d * e + codes + d * f * we + f * e + adapters + out + 4 * T,
                "flops": 2 * T * d * f + 2 * T * r * (d + f)}
    # x, dy (and the activation's argument) and the weight in; dx and every slot's gradients out
    rows = T * f * e * (1 if case["act"] == "none" else 2)
    out = T * d * e + S * R * (d + f) * e + f * e
    return {"bytes": T * d * e + rows + d * f * e + adapters + out + 4 * T,
            "flops": 2 * T * d * f + 2 * T * r * (3 * d + 2 * f)}


# ---- the definitions in 64 bits, one adapter or matrix at a time ------------


def _exact_act(name, p):
    """The activation and its derivative."""
    if name == "none":
        return p, torch.ones_like(p)
    if name == "silu":
        q = 1.0 / (1.0 + torch.exp(-p))
        return p * q, q + p * q * (1.0 - q)
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-p / math.sqrt(2.0))
        return p * cdf, cdf + p * torch.exp(-p * p / 2.0) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    q = 1.0 / (1.0 + torch.exp(-2.0 * k * (p + 0.044715 * p ** 3)))  # (1 + tanh) / 2
    return p * q, q + p * 2.0 * q * (1.0 - q) * k * (1.0 + 0.134145 * p ** 2)


def _exact_norm(s):
    z = s["x"].double() + s["residual"].double()
    var, mean = torch.var_mean(z, 1, correction=0, keepdim=True)
    y = (z - mean) / torch.sqrt(var + EPS) * s["weight"].double() + s["bias"].double()
    out = {"residual": z, "y": y}
    if s["dtype"] == "fp8":
        amax = y.to(torch.bfloat16).double().abs().max(1).values  # of y as it is stored
        scale = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
        out["scale"], out["codes"] = scale, y / scale.unsqueeze(1)
    return out


def _exact_norm_backward(s):
    d = s["d"]
    dy, rstd = s["dy"].double(), s["rstd"].double().unsqueeze(1)
    h = (s["z"].double() - s["mean"].double().unsqueeze(1)) * rstd
    dh = dy * s["weight"].double()
    dx = (dh - (dh.sum(1, keepdim=True) + h * (dh * h).sum(1, keepdim=True)) / d) * rstd
    if s["dresidual"] is not None:
        dx += s["dresidual"].double()
    return {"dx": dx, "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}


def _adapters(s):
    """Each slot's rows, A, B and scale."""
    for slot, r in enumerate(s["rank_list"]):
        t = torch.nonzero(s["ids"] == slot).flatten()
        if len(t):
            yield slot, r, t, s["A"][slot, :, :r].double(), s["B"][slot, :r].double(), s["alpha_list"][slot] / r


def _exact_linear(s):
    x = s["x"].double()
    if s["dtype"] == "fp8":
        p = torch.matmul(s["xq"].double(), s["Wq"].double().transpose(0, 1))
        p *= s["x_scale"].double().unsqueeze(1)
        p *= s["W_scale"].double()
    else:
        p = torch.matmul(x, s["W"].double())
    p += s["bias"].double()
    for _, _, t, A, B, scale in _adapters(s):
        p[t] += scale * torch.matmul(torch.matmul(x[t], A), B)
    y = _exact_act(s["act"], p)[0]
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return {"y": y, "pre": p} if s["save"] else {"y": y}


def _exact_linear_backward(s):
    x, dp = s["x"].double(), s["dy"].double()
    if s["act"] != "none":
        dp = dp * _exact_act(s["act"], s["pre"].double())[1]
    dx = torch.matmul(dp, s["W"].double().transpose(0, 1))
    dA, dB = torch.zeros_like(s["A"]).double(), torch.zeros_like(s["B"]).double()
    for slot, r, t, A, B, scale in _adapters(s):
        dv = scale * torch.matmul(dp[t], B.transpose(0, 1))
        dx[t] += torch.matmul(dv, A.transpose(0, 1))
        dA[slot, :, :r] = torch.matmul(x[t].transpose(0, 1), dv)
        dB[slot, :r] = scale * torch.matmul(torch.matmul(x[t], A).transpose(0, 1), dp[t])
    return {"dx": dx, "dA": dA, "dB": dB, "dbias": dp.sum(0)}


def _exact_ortho(s):
    a, b, c = COEFFICIENTS
    out = []
    for g in s["g"].double():
        x = g / (torch.linalg.vector_norm(g) + ORTHO_EPS)
        for _ in range(STEPS):
            # from the side that is shorter
            if x.shape[0] <= x.shape[1]:
                y = torch.matmul(torch.matmul(x, x.transpose(0, 1)), x)
                z = torch.matmul(torch.matmul(x, x.transpose(0, 1)), y)
            else:
                y = torch.matmul(x, torch.matmul(x.transpose(0, 1), x))
                z = torch.matmul(y, torch.matmul(x.transpose(0, 1), x))
            x = a * x + b * y + c * z
        out.append(x)
    return {"update": torch.stack(out)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "linear": _exact_linear,
            "linear_backward": _exact_linear_backward, "ortho": _exact_ortho}[case["op"]](s)
