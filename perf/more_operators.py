"""Cases, plain forms and exact values of the operators around an expert sub-layer: the RMS norm with
the residual's addition (forward, 8-bit output, backward), tokens sorted by expert and back (dispatch,
combine and their gradients), and products of few rows with 4-bit weights.

``run`` makes the calls of ``transformer_ffn_fusion_amd`` when ``own`` is true and computes the same
operators from elementary torch operations in 32 bits otherwise.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100      # of a group's largest magnitude
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def listed():
    return [
        # the norm in front of the block while decoding 16 sequences: launch and latency alone
        {"name": "rms_fwd_decode", "op": "rmsnorm_forward", "M": 16, "N": 4096, "dtype": "bf16", "residual": True},
        # a 4096-token prompt, normed straight into 8-bit rows with a scale per 128 columns
        {"name": "rms_q8_prompt", "op": "rmsnorm_q8_forward", "M": 4096, "N": 4096, "dtype": "bf16",
         "residual": True, "group": 128},
        # its gradient in 32 bits, an odd number of tokens
        {"name": "rms_bwd_f32_ragged", "op": "rmsnorm_backward", "M": 1013, "N": 2056, "dtype": "f32",
         "residual": True},
        # its gradient in the 8192-wide block's training step
        {"name": "rms_bwd_large", "op": "rmsnorm_backward", "M": 8192, "N": 8192, "dtype": "bf16", "residual": True},
        # 16 decoded tokens to the top 2 of 8 experts
        {"name": "dispatch_decode", "op": "moe_dispatch", "M": 16, "N": 4096, "E": 8, "k": 2, "dtype": "bf16",
         "group": 0, "drop": 0.0},
        # 16384 tokens as 8-bit rows with scales, top 6 of 64 experts, an eighth of which are elsewhere
        {"name": "dispatch_q8_many", "op": "moe_dispatch", "M": 16384, "N": 2048, "E": 64, "k": 6, "dtype": "e4m3",
         "group": 128, "drop": 0.125},
        # back to token order in 32 bits: odd sizes, dropped entries
        {"name": "combine_f32_ragged", "op": "moe_combine", "M": 1013, "N": 2056, "E": 24, "k": 3, "dtype": "f32",
         "drop": 0.1, "residual": True},
        # the gradient of the weighted sum over 16384 tokens, top 2 of 8
        {"name": "combine_bwd_large", "op": "moe_combine_backward", "M": 16384, "N": 4096, "E": 8, "k": 2,
         "dtype": "bf16", "drop": 0.0},
        # one token through a 4096 x 4096 matrix of 4-bit integers with zero points
        {"name": "q4_single", "op": "q4_matvec", "M": 1, "K": 4096, "C": 4096, "code": "int4", "group": 128,
         "zero": True, "act": "none"},
        # five tokens, 4-bit floats in groups of 32, no dimension fills whole tiles
        {"name": "q4_e2m1_ragged", "op": "q4_matvec", "M": 5, "K": 1992, "C": 1400, "code": "e2m1", "group": 32,
         "zero": False, "act": "gelu_tanh"},
        # 16 tokens through the gated pair of the 8192-wide block's shard
        {"name": "q4_swiglu_large", "op": "q4_swiglu", "M": 16, "K": 8192, "C": 3584, "code": "int4", "group": 128,
         "zero": False},
        # 16 tokens' top 2 of 8 experts through the experts' gated pairs
        {"name": "q4_swiglu_experts", "op": "moe_q4_swiglu", "M": 16, "k": 2, "E": 8, "K": 4096, "C": 2048,
         "code": "int4", "group": 128, "zero": False},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _of(rng, step, lo, hi):
    return max(step, step * (_log_uniform(rng, lo, hi) // step))


def draw(rng):
    """The largest listed case of each family bounds the drawn ones."""
    op = rng.choice(["rmsnorm_forward", "rmsnorm_q8_forward", "rmsnorm_backward", "moe_dispatch",
                     "moe_dispatch_backward", "moe_combine", "moe_combine_backward", "moe_route_backward",
                     "q4_matvec", "q4_swiglu", "moe_q4_matvec", "moe_q4_swiglu"])
    tops = {c["name"]: c for c in listed()}
    while True:
        if op.startswith("rmsnorm"):
            top = tops["rms_bwd_large"]
            case = {"op": op, "M": _log_uniform(rng, 1, 16384), "N": _of(rng, 8, 64, 16384),
                    "dtype": rng.choice(["bf16", "f32"]), "residual": rng.random() < 0.75}
            if op == "rmsnorm_q8_forward":
                case["group"] = rng.choice([0, 128])
        elif op.startswith("moe") and "q4" not in op:
            top = tops["combine_bwd_large"]
            E = _log_uniform(rng, 2, 256)
            case = {"op": op, "M": _log_uniform(rng, 1, 32768), "E": E, "k": rng.randint(1, min(8, E)),
                    "drop": rng.choice([0.0, 0.1, 0.75])}
            if op != "moe_route_backward":
                case["N"] = _of(rng, 8, 64, 8192)
                case["dtype"] = rng.choice(["bf16", "f32"])
            if op == "moe_dispatch":
                case["dtype"] = rng.choice(["bf16", "f32", "e4m3"])
                case["group"] = 128 if case["dtype"] == "e4m3" else 0
            if op == "moe_combine":
                case["residual"] = rng.random() < 0.5
        else:
            top = tops["q4_swiglu_experts"]
            code = rng.choice(["int4", "e2m1"])
            case = {"op": op, "M": rng.randint(1, 16), "K": _of(rng, 8, 64, 8192), "C": _of(rng, 8, 64, 8192),
                    "code": code, "group": rng.choice([32, 64, 128]),
                    "zero": code == "int4" and rng.random() < 0.5}
            if op.startswith("moe"):
                case["E"] = _log_uniform(rng, 2, 64)
                case["k"] = rng.randint(1, min(4, case["E"]))
            if op == "q4_matvec":
                case["act"] = rng.choice(["none", "relu", "gelu_tanh"])
        w, most = work(case), work(top)
        if w["bytes"] <= most["bytes"] and w["flops"] <= max(most["flops"], w["bytes"]):
            return case


# ---------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _route(gen, M, E, k, drop):
    """Expert ids (M x k int32, -1 where the entry is dropped) and gate weights, of a gate that prefers
    some experts."""
    logits = _normal(gen, M, E) + _normal(gen, E)
    top, ids = logits.topk(k, dim=1)
    gone = torch.rand(M, k, generator=gen, device="cuda") < drop
    return torch.where(gone, -1, ids).to(torch.int32), torch.softmax(top, dim=1)


def _sort(ids, E):
    """(positions, offsets, sorted entries) of expert ids: by expert, then by entry; dropped ones at -1."""
    n = ids.numel()
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(n, device=ids.device)
    pos = torch.where(key < E, place, -1).to(torch.int32).reshape(ids.shape)
    experts = torch.arange(E + 1, device=ids.device)
    off = (key[:, None] < experts[None, :]).sum(0) if n * (E + 1) <= 1 << 22 else torch.searchsorted(key[order], experts)
    return pos, off.to(torch.int32), order.to(torch.int32)


def _q4_weight(gen, lead, K, C, case):
    """Codes in the packed layout, scales and zero points: tiles of 16 columns x 128 k, a tile's codes
    as 64 lanes of four 32-bit words (one word: 8 codes of one column)."""
    ct, kt, per = -(-C // 16), -(-K // 128), 128 // case["group"]
    codes = torch.randint(0, 256, (*lead, ct, kt, 1024), generator=gen, device="cuda", dtype=torch.uint8)
    spread = 4.6 if case["code"] == "int4" else 3.0           # the codes' own spread
    scale = torch.exp(0.3 * _normal(gen, *lead, ct, kt, 16, per)) / (spread * math.sqrt(K))
    zero = None
    if case["zero"]:
        zero = torch.randint(4, 12, (*lead, ct, kt, 16, per), generator=gen, device="cuda").to(torch.bfloat16)
    return codes, scale.to(torch.bfloat16), zero


def _inputs(case, seed):
    """The operator's inputs alone, from the seed."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M = case["op"], case["M"]
    bf = torch.bfloat16
    if op.startswith("rmsnorm"):
        N, dt = case["N"], DTYPES[case["dtype"]]
        # a residual stream: a few channels that are much larger than the rest
        channel = 1.0 + 20.0 * (torch.rand(N, generator=gen, device="cuda") < 0.005).float()
        x = (_normal(gen, M, N) * channel).to(dt)
        s = {"X": x, "gamma": (1.0 + 0.1 * _normal(gen, N)).to(dt)}
        if op == "rmsnorm_backward":
            s["S"] = s.pop("X")
            s["rstd"] = torch.rsqrt(s["S"].double().square().mean(1) + EPS).float()    # what the forward kept
            s["dY"] = (_normal(gen, M, N) * 2.0 ** -10).to(dt)
            s["dS"] = (_normal(gen, M, N) * 2.0 ** -10).to(dt) if case["residual"] else None
        else:
            s["R"] = (0.5 * _normal(gen, M, N)).to(dt) if case["residual"] else None   # the sub-layer's output
        return s
    if "q4" in op:
        K, C = case["K"], case["C"]
        lead = (case["E"],) if "E" in case else ()
        s = {}
        rows = M
        if lead:      # the rows that the dispatch of M tokens gives, by expert
            ids, _ = _route(gen, M, case["E"], case["k"], 0.0)
            s["offsets"] = _sort(ids, case["E"])[1]
            rows = M * case["k"]
        s["X"] = _normal(gen, rows, K).to(bf)
        if op.endswith("matvec"):
            s["W"], s["s"], s["z"] = _q4_weight(gen, lead, K, C, case)
            s["bias"] = (0.1 * _normal(gen, C)).to(bf) if not lead else None
        else:
            s["Wg"], s["sg"], s["zg"] = _q4_weight(gen, lead, K, C, case)
            s["Wu"], s["su"], s["zu"] = _q4_weight(gen, lead, K, C, case)
        return s
    E, k = case["E"], case["k"]
    ids, w = _route(gen, M, E, k, case["drop"])
    if op == "moe_route_backward":
        return {"ids": ids, "w": w, "dw": _normal(gen, M, k)}
    N, dt = case["N"], DTYPES[case["dtype"]]
    if op == "moe_dispatch":
        s = {"ids": ids, "scale": None}
        x = _normal(gen, M, N)
        if case["group"]:
            s["scale"] = torch.exp(_normal(gen, M, -(-N // case["group"]))) / E4M3_MAX
            x = (x * 100.0).clamp(-E4M3_MAX, E4M3_MAX)
        s["X"] = x.to(dt)
        return s
    s = {"pos": _sort(ids, E)[0]}
    if op == "moe_dispatch_backward":
        s["rows"] = (_normal(gen, M * k, N) * 2.0 ** -10).to(dt)
    else:
        s["w"] = w
        s["rows"] = _normal(gen, M * k, N).to(dt)
        if op == "moe_combine":
            s["R"] = _normal(gen, M, N).to(dt) if case["residual"] else None
        else:
            s["dY"] = (_normal(gen, M, N) * 2.0 ** -10).to(dt)
    return s


def _outputs(case, s):
    """Buffers that a program keeps from call to call; rows that a call leaves alone hold zeros."""
    op, M, f32, i32 = case["op"], case["M"], torch.float32, torch.int32

    def new(*shape, dtype):
        return torch.zeros(*shape, device="cuda", dtype=f32).to(dtype)
    if op.startswith("rmsnorm"):
        N, dt = case["N"], DTYPES[case["dtype"]]
        if op == "rmsnorm_backward":
            return {"dX": new(M, N, dtype=dt), "dgamma": new(N, dtype=f32)}
        o = {"rstd": new(M, dtype=f32)}
        if case["residual"]:
            o["S"] = new(M, N, dtype=dt)
        if op == "rmsnorm_forward":
            o["Y"] = new(M, N, dtype=dt)
        else:
            o["Q"] = new(M, N, dtype=torch.float8_e4m3fn)
            o["scale"] = new(M, -(-N // case["group"]) if case["group"] else 1, dtype=f32)
        return o
    if "q4" in op:
        return {"Y": new(s["X"].shape[0], case["C"], dtype=torch.bfloat16)}
    E, k = case["E"], case["k"]
    if op == "moe_route_backward":
        return {"dlogits": new(M, E, dtype=f32)}
    N, dt = case["N"], DTYPES[case["dtype"]]
    if op == "moe_dispatch":
        o = {"Xs": new(M * k, N, dtype=dt), "offsets": new(E + 1, dtype=i32), "positions": new(M, k, dtype=i32),
             "entries": new(M * k, dtype=i32)}
        if case["group"]:
            o["scale"] = new(M * k, s["scale"].shape[1], dtype=f32)
        return o
    if op == "moe_combine_backward":
        return {"dYs": new(M * k, N, dtype=dt), "dw": new(M, k, dtype=f32)}
    return {"Y": new(M, N, dtype=dt)}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["out"] = _outputs(case, s)
    s["case"] = dict(case)
    return s


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    import transformer_ffn_fusion_amd as ffn
    o, c = s["out"], s["case"]
    op = c["op"]
    if op == "rmsnorm_forward":
        ffn.ffn_rmsnorm_forward(s["X"], s["gamma"], o["Y"], R=s["R"], S=o.get("S"), rstd=o["rstd"], eps=EPS)
    elif op == "rmsnorm_q8_forward":
        ffn.ffn_rmsnorm_q8_forward(s["X"], s["gamma"], o["Q"], o["scale"], R=s["R"], S=o.get("S"), rstd=o["rstd"],
                                   group=c["group"], eps=EPS)
    elif op == "rmsnorm_backward":
        if "ws" not in s:   # the workspace that a program keeps
            s["ws"] = ffn.workspace(ffn.ffn_rmsnorm_backward_workspace_size(*s["S"].shape))
        ffn.ffn_rmsnorm_backward(s["S"], s["dY"], s["gamma"], s["rstd"], o["dX"], o["dgamma"], dS=s["dS"], ws=s["ws"])
    elif op == "moe_dispatch":
        if "ws" not in s:
            s["ws"] = ffn.workspace(ffn.moe_dispatch_workspace_size(c["M"], c["E"], c["k"]))
        ffn.moe_dispatch(s["X"], s["ids"], o["Xs"], o["offsets"], o["entries"], o["positions"], scale=s["scale"],
                         scale_sorted=o.get("scale"), ws=s["ws"])
    elif op == "moe_dispatch_backward":
        ffn.moe_dispatch_backward(s["rows"], s["pos"], o["Y"])
    elif op == "moe_combine":
        ffn.moe_combine(s["rows"], s["pos"], o["Y"], topk_w=s["w"], R=s["R"])
    elif op == "moe_combine_backward":
        ffn.moe_combine_backward(s["dY"], s["rows"], s["pos"], s["w"], o["dYs"], o["dw"])
    elif op == "moe_route_backward":
        ffn.moe_route_backward(s["ids"], s["w"], s["dw"], o["dlogits"])
    elif op == "q4_matvec":
        ffn.ffn_q4_matvec(s["X"], s["W"], s["s"], o["Y"], zero=s["z"], bias=s["bias"], act=c["act"], code=c["code"])
    elif op == "q4_swiglu":
        ffn.ffn_q4_swiglu(s["X"], s["Wg"], s["sg"], s["Wu"], s["su"], o["Y"], zero_g=s["zg"], zero_u=s["zu"],
                          code=c["code"])
    elif op == "moe_q4_matvec":
        ffn.moe_q4_matvec(s["X"], s["offsets"], s["W"], s["s"], o["Y"], zero=s["z"], code=c["code"])
    else:
        ffn.moe_q4_swiglu(s["X"], s["offsets"], s["Wg"], s["sg"], s["Wu"], s["su"], o["Y"], zero_g=s["zg"],
                          zero_u=s["zu"], code=c["code"])
    return o


# ---------------------------------------------------------------- plain forms

def _q4_plain(codes, scale, zero, K, C, code):
    """The weights (... x K x C, fp32) of the packed layout."""
    lead = codes.shape[:-3]
    ct, kt, per = codes.shape[-3], codes.shape[-2], scale.shape[-1]
    word = codes.view(torch.int32).reshape(*lead, ct, kt, 4, 16, 4, 1)   # tile, tile, lane / 16, lane % 16, step
    # the place of each of a word's eight codes: floats in order, integers even ones first
    place = [0, 1, 2, 3, 4, 5, 6, 7] if code == "e2m1" else [0, 4, 1, 5, 2, 6, 3, 7]
    q = (word >> (4 * torch.tensor(place, device=codes.device, dtype=torch.int32))) & 15
    n = len(lead)
    # k = 128 tile + 32 step + 8 (lane / 16) + e, column = 16 tile + lane % 16
    q = q.permute(*range(n), n + 1, n + 4, n + 2, n + 5, n, n + 3).reshape(*lead, kt * 128, ct * 16)

    def wide(a):    # one value per group to one per k
        a = a.float().permute(*range(n), n + 1, n + 3, n, n + 2).reshape(*lead, kt * per, 1, ct * 16)
        return a.expand(*lead, kt * per, 128 // per, ct * 16).reshape(*lead, kt * 128, ct * 16)
    if code == "e2m1":
        w = torch.tensor(E2M1, device=codes.device)[q.long()]
    else:
        w = q.float() - (8.0 if zero is None else wide(zero))
    return (w * wide(scale))[..., :K, :C]


def _of_experts(X, W, offsets):
    """X's rows times the matrix of the expert that each belongs to, and which belong to one."""
    row = torch.arange(X.shape[0], device=X.device)
    expert = (row[:, None] >= offsets[None, 1:]).sum(1)
    all_of_them = torch.matmul(X.float(), W.contiguous())      # E x rows x C
    return all_of_them[expert.clamp(max=W.shape[0] - 1), row]


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _rows_of(rows, pos):
    """rows[pos] in fp32, zeros where the entry is dropped: M x k x N."""
    kept = (pos >= 0).unsqueeze(-1)
    return torch.where(kept, rows[pos.clamp(min=0).long()].float(), 0.0)


def run(s):
    if own:
        return _run_own(s)
    o, c = s["out"], s["case"]
    op = c["op"]
    if op.startswith("rmsnorm"):
        dt = s["gamma"].dtype
        gamma = s["gamma"].float()
        if op == "rmsnorm_backward":
            z = s["S"].float() * s["rstd"][:, None]
            dy = s["dY"].float()
            t = dy * gamma
            dx = s["rstd"][:, None] * (t - z * (t * z).mean(1, keepdim=True))
            if s["dS"] is not None:
                dx = dx + s["dS"].float()
            return {"dX": dx.to(dt), "dgamma": (dy * z).sum(0)}
        out = {}
        x = s["X"].float()
        if s["R"] is not None:
            out["S"] = (x + s["R"].float()).to(dt)
            x = out["S"].float()
        rstd = 1.0 / torch.sqrt((x * x).mean(1) + EPS)
        out["rstd"] = rstd
        y = x * rstd[:, None] * gamma
        if op == "rmsnorm_forward":
            out["Y"] = y.to(dt)
            return out
        M, N = y.shape
        g = c["group"] or N
        pad = torch.nn.functional.pad(y, (0, -N % g)).reshape(M, -1, g)
        scale = pad.abs().amax(2).clamp(min=SCALE_FLOOR) / E4M3_MAX
        q = (pad / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).reshape(M, -1)[:, :N]
        out["Q"], out["scale"] = q.contiguous().to(torch.float8_e4m3fn), scale
        return out
    if op == "moe_dispatch":
        pos, off, order = _sort(s["ids"], c["E"])
        k = c["k"]
        live = torch.arange(order.numel(), device=order.device) < off[-1]     # the kept entries come first
        token = torch.div(order, k, rounding_mode="floor").long()
        bytes_ = s["X"].view(torch.uint8)
        out = {"Xs": torch.where(live[:, None], bytes_[token], o["Xs"].view(torch.uint8)).view(s["X"].dtype),
               "offsets": off, "positions": pos, "entries": torch.where(live, order, o["entries"])}
        if s["scale"] is not None:
            out["scale"] = torch.where(live[:, None], s["scale"][token], o["scale"])
        return out
    if op == "moe_dispatch_backward":
        return {"Y": _rows_of(s["rows"], s["pos"]).sum(1).to(s["rows"].dtype)}
    if op == "moe_combine":
        y = (_rows_of(s["rows"], s["pos"]) * s["w"][:, :, None]).sum(1)
        if s["R"] is not None:
            y = y + s["R"].float()
        return {"Y": y.to(s["rows"].dtype)}
    if op == "moe_combine_backward":
        dy = s["dY"].float()[:, None, :]
        n = s["rows"].shape[0]
        at = torch.where(s["pos"] >= 0, s["pos"], n).reshape(-1).long()       # dropped entries: a row past the end
        rows = torch.zeros(n + 1, dy.shape[2], device=dy.device, dtype=s["rows"].dtype)
        rows[at] = (dy * s["w"][:, :, None]).to(rows.dtype).reshape(-1, dy.shape[2])
        return {"dYs": rows[:n], "dw": (_rows_of(s["rows"], s["pos"]) * dy).sum(2)}
    if op == "moe_route_backward":
        d = s["w"] * (s["dw"] - (s["w"] * s["dw"]).sum(1, keepdim=True))
        at = torch.where(s["ids"] >= 0, s["ids"], c["E"]).long()              # dropped entries: a column past the end
        return {"dlogits": torch.zeros(c["M"], c["E"] + 1, device=d.device).scatter_add(1, at, d)[:, :c["E"]].contiguous()}
    K, C, code = c["K"], c["C"], c["code"]
    if op == "q4_matvec":
        y = s["X"].float() @ _q4_plain(s["W"], s["s"], s["z"], K, C, code) + s["bias"].float()
        return {"Y": _act(y, c["act"]).to(torch.bfloat16)}
    if op == "q4_swiglu":
        x = s["X"].float()
        a, b = (x @ _q4_plain(s["W" + n], s["s" + n], s["z" + n], K, C, code) for n in "gu")
        return {"Y": (_silu(a) * b).to(torch.bfloat16)}
    if op == "moe_q4_matvec":
        return {"Y": _of_experts(s["X"], _q4_plain(s["W"], s["s"], s["z"], K, C, code), s["offsets"]).to(torch.bfloat16)}
    a, b = (_of_experts(s["X"], _q4_plain(s["W" + n], s["s" + n], s["z" + n], K, C, code), s["offsets"]) for n in "gu")
    return {"Y": (_silu(a) * b).to(torch.bfloat16)}


# ---------------------------------------------------------------- what a call cannot do without

def work(case):
    op, M = case["op"], case["M"]
    if op.startswith("rmsnorm"):
        N = case["N"]
        size = 4 if case["dtype"] == "f32" else 2
        r = 1 if case["residual"] else 0
        if op == "rmsnorm_forward":     # x and r in, y and s out
            return {"bytes": (2 + 2 * r) * M * N * size + N * size + 4 * M, "flops": (4 + r) * M * N}
        if op == "rmsnorm_q8_forward":
            g = -(-N // case["group"]) if case["group"] else 1
            return {"bytes": (1 + 2 * r) * M * N * size + M * N + 4 * M * g + N * size + 4 * M, "flops": (6 + r) * M * N}
        return {"bytes": (3 + r) * M * N * size + N * size + 4 * M + 4 * N, "flops": (9 + r) * M * N}
    if "q4" in op:
        K, C = case["K"], case["C"]
        rows, pair = M, 2 if op.endswith("swiglu") else 1
        weights = pair * K * C
        if "E" in case:    # each expert's matrices once, of those that have rows
            rows = M * case["k"]
            weights *= min(case["E"], rows)
        per_group = 4 if case["zero"] else 2
        return {"bytes": weights // 2 + per_group * weights // case["group"] + 2 * rows * (K + C),
                "flops": 2 * rows * K * C * pair}
    E, k = case["E"], case["k"]
    kept = M * k * (1.0 - case["drop"])
    if op == "moe_route_backward":
        return {"bytes": 12 * M * k + 4 * M * E, "flops": 4 * M * k}
    N = case["N"]
    size = {"f32": 4, "bf16": 2, "e4m3": 1}[case["dtype"]]
    if op == "moe_dispatch":
        g = 4 * -(-N // case["group"]) if case["group"] else 0
        return {"bytes": (M + kept) * (N * size + g) + 12 * M * k, "flops": 0}
    if op == "moe_combine_backward":
        return {"bytes": (M + 2 * kept) * N * size + 12 * M * k, "flops": 3 * kept * N}
    r = 1 if case.get("residual") else 0
    return {"bytes": ((1 + r) * M + kept) * N * size + 8 * M * k, "flops": 2 * kept * N}


# ---------------------------------------------------------------- exact values

def _to_e4m3(v):
    """The nearest number of four exponent and three mantissa bits, ties to the even one, in fp64."""
    _, e = torch.frexp(v)                         # |v| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _q4_exact(codes, scale, zero, K, C, code):
    """One matrix of the packed layout in fp64, from each k's and column's own place in it."""
    k = torch.arange(K, device=codes.device)[:, None]
    col = torch.arange(C, device=codes.device)[None, :]
    lane = 16 * ((k % 32) // 8) + col % 16
    e = k % 8
    nibble = e if code == "e2m1" else e // 2 + 4 * (e % 2)
    byte = codes[col // 16, k // 128, 16 * lane + 4 * ((k % 128) // 32) + nibble // 2].long()
    q = torch.where(nibble % 2 == 1, byte // 16, byte % 16)
    at = (col // 16, k // 128, col % 16, (k % 128) // (128 // scale.shape[-1]))
    if code == "e2m1":
        m, ex = (q % 2).double(), (q % 8) // 2
        v = torch.where(ex == 0, 0.5 * m, torch.ldexp(1.0 + 0.5 * m, ex - 1))
        v = torch.where(q >= 8, -v, v)
    else:
        v = q.double() - (8.0 if zero is None else zero.double()[at])
    return v * scale.double()[at]


def exact(case, seed):
    s = _inputs(case, seed)
    o = _outputs(case, s)
    op = case["op"]
    if op.startswith("rmsnorm"):
        gamma = s["gamma"].double()
        if op == "rmsnorm_backward":
            r = s["rstd"].double().unsqueeze(1)
            dy, x = s["dY"].double(), s["S"].double()
            g = dy * gamma
            dx = r * g - x * r.pow(3) * (torch.linalg.vecdot(g, x) / case["N"]).unsqueeze(1)
            if s["dS"] is not None:
                dx += s["dS"].double()
            return {"dX": dx, "dgamma": torch.linalg.vecdot(dy, x * r, dim=0)}
        out = {}
        x = s["X"]
        if s["R"] is not None:       # the sum as it is kept is what is normed
            out["S"] = x.double() + s["R"].double()
            x = out["S"].to(x.dtype)
        x = x.double()
        out["rstd"] = (torch.linalg.vecdot(x, x) / case["N"] + EPS).pow(-0.5)
        y = x * out["rstd"].unsqueeze(1) * gamma
        if op == "rmsnorm_forward":
            out["Y"] = y
            return out
        g = case["group"] or case["N"]
        parts = y.split(g, dim=1)
        out["scale"] = torch.stack([p.abs().amax(1) for p in parts], 1).clamp(min=SCALE_FLOOR) / E4M3_MAX
        out["Q"] = torch.cat([_to_e4m3(p / out["scale"][:, i:i + 1]) for i, p in enumerate(parts)], 1)
        return out
    if op == "moe_dispatch":
        E, k = case["E"], case["k"]
        flat = s["ids"].reshape(-1)
        hit = [torch.nonzero(flat == e).reshape(-1) for e in range(E)]
        n = torch.tensor([0] + [h.numel() for h in hit], device=flat.device).cumsum(0)
        order = torch.cat(hit)
        pos = torch.full_like(flat, -1)
        pos[order] = torch.arange(order.numel(), device=flat.device, dtype=pos.dtype)
        xs, entries = o["Xs"].double(), o["entries"]
        xs[:order.numel()] = s["X"].double()[order // k]
        entries[:order.numel()] = order.to(entries.dtype)
        out = {"Xs": xs, "offsets": n.to(torch.int32), "positions": pos.reshape(s["ids"].shape), "entries": entries}
        if s["scale"] is not None:
            sc = o["scale"].double()
            sc[:order.numel()] = s["scale"].double()[order // k]
            out["scale"] = sc
        return out
    if op == "moe_route_backward":
        w, dw, E = s["w"].double(), s["dw"].double(), case["E"]
        slope = torch.diag_embed(w) - w.unsqueeze(2) * w.unsqueeze(1)          # the softmax's own derivative
        d = torch.matmul(slope, dw.unsqueeze(2)).squeeze(2)
        place = s["ids"].unsqueeze(2) == torch.arange(E, device=w.device)      # M x k x E
        return {"dlogits": (place * d.unsqueeze(2)).sum(1)}
    if "q4" not in op:
        k, N = case["k"], case["N"]
        wide = torch.cat([s["rows"].double(), torch.zeros(1, N, device="cuda", dtype=torch.float64)])  # -1: zeros
        if op == "moe_combine_backward":
            dy = s["dY"].double()
            rows = torch.zeros_like(wide)
            dw = []
            for j in range(k):
                p = s["pos"][:, j].long()
                rows[p] = dy * s["w"][:, j:j + 1].double()
                dw.append(torch.linalg.vecdot(wide[p], dy))
            return {"dYs": rows[:-1], "dw": torch.stack(dw, 1)}
        y = torch.zeros(case["M"], N, device="cuda", dtype=torch.float64)
        if s.get("R") is not None:
            y += s["R"].double()
        for j in range(k):
            part = wide[s["pos"][:, j].long()]
            y += part if op == "moe_dispatch_backward" else part * s["w"][:, j:j + 1].double()
        return {"Y": y}
    K, C, code = case["K"], case["C"], case["code"]
    x = s["X"].double()
    names = ("g", "u") if op.endswith("swiglu") else ("",)
    lists = [(0, x.shape[0], None)]
    if "E" in case:
        off = s["offsets"].tolist()
        lists = [(off[e], off[e + 1], e) for e in range(case["E"])]
    y = o["Y"].double()
    for lo, hi, e in lists:
        if lo == hi:
            continue
        p = []
        for n in names:
            W, sc, z = (s[v + n] for v in ("W", "s", "z"))
            if e is not None:
                W, sc, z = W[e], sc[e], None if z is None else z[e]
            p.append(torch.mm(x[lo:hi], _q4_exact(W, sc, z, K, C, code)))
        if len(p) == 2:
            v = p[0] * torch.sigmoid(p[0]) * p[1]
        else:
            v = p[0] if s["bias"] is None else p[0] + s["bias"].double()
            act = case.get("act", "none")
            if act == "relu":
                v = v.clamp(min=0)
            elif act == "gelu_tanh":
                v = v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v.pow(3)))
        y[lo:hi] = v
    return {"Y": y}
