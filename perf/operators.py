"""Cases, plain forms and exact values of the training operators of a gated
feed-forward sub-layer: the SwiGLU block's backward pass, the layer norm in
front of it (forward and backward) and the orthogonalised update of its weight
matrices.

``run`` makes the calls of ``transformer_ffn_fusion_amd`` when ``own`` is true
and computes the same operators from elementary torch operations in 32 bits
otherwise.
"""
import math

import torch

own = False

# Coefficients of one Newton-Schulz step, X <- a X + b (X X^T) X + c (X X^T)^2 X.
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315
NS_EPS = 1e-7
LN_EPS = 1e-5

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a few tokens through a toy-sized block: nothing but launches and latency
        {"name": "swiglu_bwd_tiny", "op": "swiglu_backward", "M": 8, "N": 128, "O": 512, "P": 128},
        # a padded-out micro-batch on a mid-sized block: no dimension fills whole tiles
        {"name": "swiglu_bwd_ragged", "op": "swiglu_backward", "M": 1013, "N": 2056, "O": 1400, "P": 1992},
        # one tensor-parallel shard of a 4096-wide block, 4096 tokens: a training step's ordinary call
        {"name": "swiglu_bwd_shard", "op": "swiglu_backward", "M": 4096, "N": 4096, "O": 1792, "P": 4096},
        # the shard of an 8192-wide block, 8192 tokens: the largest call
        {"name": "swiglu_bwd_large", "op": "swiglu_backward", "M": 8192, "N": 8192, "O": 3584, "P": 8192},
        # the norm in front of the block while decoding 16 sequences
        {"name": "ln_fwd_decode", "op": "layernorm_forward", "M": 16, "N": 4096, "dtype": "bf16"},
        # the norm of a training step of the large block
        {"name": "ln_fwd_large", "op": "layernorm_forward", "M": 8192, "N": 8192, "dtype": "bf16"},
        # its gradient in 32 bits, an odd number of tokens
        {"name": "ln_bwd_f32_ragged", "op": "layernorm_backward", "M": 1013, "N": 2056, "dtype": "f32"},
        # its gradient in the large block's training step
        {"name": "ln_bwd_large", "op": "layernorm_backward", "M": 8192, "N": 8192, "dtype": "bf16"},
        # the update of a toy-sized weight (wide), gradients kept in 32 bits
        {"name": "ortho_tiny_f32", "op": "orthogonalize", "B": 1, "R": 128, "C": 512, "dtype": "f32"},
        # the stacked updates of eight experts' sharded first matrices (tall)
        {"name": "ortho_experts", "op": "orthogonalize", "B": 8, "R": 4096, "C": 256, "dtype": "bf16"},
        # the update of the 4096-wide shard's gate matrix (tall)
        {"name": "ortho_shard", "op": "orthogonalize", "B": 1, "R": 4096, "C": 1792, "dtype": "bf16"},
        # the update of the 8192-wide shard's last matrix (wide), gradients kept in 32 bits
        {"name": "ortho_large_f32", "op": "orthogonalize", "B": 1, "R": 3584, "C": 8192, "dtype": "f32"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _of_eight(rng, lo, hi):
    return max(8, 8 * (_log_uniform(rng, lo, hi) // 8))


def draw(rng):
    op = rng.choice(["swiglu_backward", "layernorm_forward", "layernorm_backward", "orthogonalize"])
    most = {"swiglu_backward": listed()[3], "layernorm_forward": listed()[5],
            "layernorm_backward": listed()[7], "orthogonalize": listed()[11]}[op]
    while True:
        if op == "swiglu_backward":
            case = {"op": op, "M": _log_uniform(rng, 1, 8192), "N": _of_eight(rng, 64, 8192),
                    "O": _of_eight(rng, 64, 4096), "P": _of_eight(rng, 64, 8192)}
        elif op == "orthogonalize":
            case = {"op": op, "B": _log_uniform(rng, 1, 8), "R": _of_eight(rng, 64, 8192),
                    "C": _of_eight(rng, 64, 8192), "dtype": rng.choice(["bf16", "f32"])}
        else:
            case = {"op": op, "M": _log_uniform(rng, 1, 16384), "N": _of_eight(rng, 64, 16384),
                    "dtype": rng.choice(["bf16", "f32"])}
        w, top = work(case), work(most)
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"]:
            return case


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _inputs(case, seed):
    """The operator's inputs alone, from the seed."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op == "swiglu_backward":
        M, N, O, P = case["M"], case["N"], case["O"], case["P"]
        bf = torch.bfloat16
        return {
            "X": _normal(gen, M, N).to(bf),                       # normalised activations
            "Wg": (_normal(gen, N, O) / math.sqrt(N)).to(bf),
            "Wu": (_normal(gen, N, O) / math.sqrt(N)).to(bf),
            "Wd": (_normal(gen, O, P) / math.sqrt(O)).to(bf),
            "dY": (_normal(gen, M, P) * 2.0 ** -10).to(bf),       # the gradient of a mean over many tokens
        }
    dt = DTYPES[case["dtype"]]
    if op in ("layernorm_forward", "layernorm_backward"):
        M, N = case["M"], case["N"]
        # a residual stream: an offset and a few channels that are much larger than the rest
        channel = 1.0 + 20.0 * (torch.rand(N, generator=gen, device="cuda") < 0.005).float()
        x = ((_normal(gen, M, N) + 0.3) * channel).to(dt)
        gamma = (1.0 + 0.1 * _normal(gen, N)).to(dt)
        if op == "layernorm_forward":
            return {"X": x, "gamma": gamma, "beta": (0.1 * _normal(gen, N)).to(dt)}
        wide = x.double()                                        # what the forward pass kept
        mean = wide.mean(1)
        rstd = 1.0 / torch.sqrt((wide - mean[:, None]).square().mean(1) + LN_EPS)
        return {"X": x, "dY": (_normal(gen, M, N) * 2.0 ** -10).to(dt), "gamma": gamma,
                "mean": mean.float(), "rstd": rstd.float()}
    # a weight's gradient: activations times output gradients over some tokens, with channels
    # of unequal size, so that its singular values spread over orders of magnitude
    B, R, C = case["B"], case["R"], case["C"]
    tokens = max(R, C)
    g = torch.empty(B, R, C, device="cuda", dtype=dt)
    for e in range(B):
        x = _normal(gen, R, tokens) * torch.exp(0.5 * _normal(gen, R, 1))
        d = _normal(gen, tokens, C) * torch.exp(0.5 * _normal(gen, 1, C))
        g[e] = ((x @ d) * (2.0 ** -10 / tokens)).to(dt)
    return {"G": g}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"] = case["op"]
    # buffers that a training loop keeps from step to step
    like = torch.empty_like
    if case["op"] == "swiglu_backward":
        s["out"] = {"dX": like(s["X"]), "dWg": like(s["Wg"]), "dWu": like(s["Wu"]), "dWd": like(s["Wd"])}
    elif case["op"] == "layernorm_forward":
        row = torch.empty(case["M"], device="cuda", dtype=torch.float32)
        s["out"] = {"Y": like(s["X"]), "mean": row, "rstd": like(row)}
    elif case["op"] == "layernorm_backward":
        col = torch.empty(case["N"], device="cuda", dtype=torch.float32)
        s["out"] = {"dX": like(s["X"]), "dgamma": col, "dbeta": like(col)}
    else:
        s["out"] = {"U": torch.empty(case["B"], case["R"], case["C"], device="cuda", dtype=torch.bfloat16)}
    return s


def _run_own(s):
    import transformer_ffn_fusion_amd as ffn
    o = s["out"]
    if s["op"] == "swiglu_backward":
        if "ws" not in s:   # the workspace that a program keeps
            (M, N), (O, P) = s["X"].shape, s["Wd"].shape
            s["ws"] = ffn.workspace(ffn.ffn_swiglu_backward_workspace_size(M, N, O, P))
        ffn.ffn_swiglu_backward(s["X"], s["Wg"], s["Wu"], s["Wd"], s["dY"], o["dX"], o["dWg"], o["dWu"],
                                o["dWd"], ws=s["ws"])
    elif s["op"] == "layernorm_forward":
        ffn.ffn_layernorm_forward(s["X"], s["gamma"], s["beta"], o["Y"], o["mean"], o["rstd"], eps=LN_EPS)
    elif s["op"] == "layernorm_backward":
        if "ws" not in s:
            s["ws"] = ffn.workspace(ffn.ffn_layernorm_backward_workspace_size(*s["X"].shape))
        ffn.ffn_layernorm_backward(s["X"], s["dY"], s["gamma"], s["mean"], s["rstd"], o["dX"], o["dgamma"],
                                   o["dbeta"], ws=s["ws"])
    else:
        if "ws" not in s:
            s["ws"] = ffn.workspace(ffn.ffn_orthogonalize_workspace_size(*s["G"].shape))
        ffn.ffn_orthogonalize(s["G"], o["U"], ws=s["ws"])
    return o


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "swiglu_backward":
        x, dy = s["X"].float(), s["dY"].float()
        wg, wu, wd = s["Wg"].float(), s["Wu"].float(), s["Wd"].float()
        gate, up = x @ wg, x @ wu
        sig = 1.0 / (1.0 + torch.exp(-gate))
        silu = gate * sig
        dh = dy @ wd.t()
        da = dh * up * (sig + silu * (1.0 - sig))
        db = dh * silu
        xt = x.t()
        out = {"dX": da @ wg.t() + db @ wu.t(), "dWg": xt @ da, "dWu": xt @ db, "dWd": (silu * up).t() @ dy}
        return {k: v.to(s["X"].dtype) for k, v in out.items()}
    if op == "layernorm_forward":
        x = s["X"].float()
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((c * c).mean(1) + LN_EPS)
        y = c * rstd[:, None] * s["gamma"].float() + s["beta"].float()
        return {"Y": y.to(s["X"].dtype), "mean": mean, "rstd": rstd}
    if op == "layernorm_backward":
        dy = s["dY"].float()
        xhat = (s["X"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        t = dy * s["gamma"].float()
        dx = s["rstd"][:, None] * (t - t.mean(1, keepdim=True) - xhat * (t * xhat).mean(1, keepdim=True))
        return {"dX": dx.to(s["X"].dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}
    g = s["G"]
    x = g.float()
    tall = g.shape[1] > g.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    norm = torch.sqrt(x.double().square().sum((1, 2), keepdim=True)) + NS_EPS
    x = x / norm.float()
    for _ in range(5):
        sym = torch.bmm(x, x.transpose(1, 2).contiguous())
        poly = NS_B * sym + NS_C * torch.bmm(sym, sym)
        x = NS_A * x + torch.bmm(poly, x)
    if tall:
        x = x.transpose(1, 2).contiguous()
    return {"U": x.to(torch.bfloat16)}


def work(case):
    op = case["op"]
    if op == "swiglu_backward":
        M, N, O, P = case["M"], case["N"], case["O"], case["P"]
        # read X, dY and the weights, write a gradient for all but dY; eight products
        return {"bytes": 2 * (2 * M * N + M * P + 4 * N * O + 2 * O * P), "flops": 12 * M * N * O + 4 * M * O * P}
    size = 4 if case["dtype"] == "f32" else 2
    if op == "layernorm_forward":
        M, N = case["M"], case["N"]
        return {"bytes": 2 * M * N * size + 2 * N * size + 8 * M, "flops": 8 * M * N}
    if op == "layernorm_backward":
        M, N = case["M"], case["N"]
        return {"bytes": 3 * M * N * size + N * size + 8 * M + 8 * N, "flops": 14 * M * N}
    B, R, C = case["B"], case["R"], case["C"]
    m, n = min(R, C), max(R, C)
    # five steps; the two symmetric products need one triangle each
    return {"bytes": B * R * C * (size + 2), "flops": 5 * B * (3 * m * m * n + m * m * m)}


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    w = {k: v.double() for k, v in s.items()}
    if op == "swiglu_backward":
        a = torch.mm(w["X"], w["Wg"])
        b = torch.mm(w["X"], w["Wu"])
        p = torch.sigmoid(a)
        dh = torch.mm(w["dY"], w["Wd"].t())
        h = a * p * b
        db = dh * a * p
        # d/da of a p(a) is p (1 + a (1 - p))
        da = dh * b * p * (1 + a * (1 - p))
        del a, b, p, dh
        return {"dX": torch.mm(da, w["Wg"].t()).addmm_(db, w["Wu"].t()), "dWg": torch.mm(w["X"].t(), da),
                "dWu": torch.mm(w["X"].t(), db), "dWd": torch.mm(h.t(), w["dY"])}
    if op == "layernorm_forward":
        var, mean = torch.var_mean(w["X"], dim=1, unbiased=False)
        rstd = (var + LN_EPS).pow(-0.5)
        y = (w["X"] - mean.unsqueeze(1)) * rstd.unsqueeze(1)
        return {"Y": torch.addcmul(w["beta"], y, w["gamma"]), "mean": mean, "rstd": rstd}
    if op == "layernorm_backward":
        n = case["N"]
        z = (w["X"] - w["mean"].unsqueeze(1)).mul_(w["rstd"].unsqueeze(1))
        g = w["dY"] * w["gamma"]
        s1, s2 = g.sum(1) / n, (g * z).sum(1) / n
        dx = (g - s1.unsqueeze(1) - z * s2.unsqueeze(1)) * w["rstd"].unsqueeze(1)
        return {"dX": dx, "dgamma": (w["dY"] * z).sum(0), "dbeta": w["dY"].sum(0)}
    out = []
    for g in w["G"]:
        x = g / (torch.linalg.vector_norm(g) + NS_EPS)
        wide = x.shape[0] <= x.shape[1]
        eye = torch.eye(min(x.shape), dtype=torch.float64, device=x.device)
        for _ in range(5):
            k = torch.mm(x, x.t()) if wide else torch.mm(x.t(), x)
            q = NS_A * eye + NS_B * k + NS_C * torch.mm(k, k)
            x = torch.mm(q, x) if wide else torch.mm(x, q)
        out.append(x)
    return {"U": torch.stack(out)}
