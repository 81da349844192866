"""GPU parity of the RMS norm with the residual's addition, of its 8-bit output and of its gradients
against their fp64 forms, within the bounds of sublayer_ref."""
from __future__ import annotations

import pytest

import transformer_ffn_fusion_amd as ffn

import sublayer_ref as ref

pytestmark = pytest.mark.gpu
SHAPES = [(1, 8), (1, 4096), (3, 72), (5, 512), (7, 520), (13, 1032), (33, 2056), (6, 4104), (5, 8192), (3, 8200),
          (2, 16384), (3, 12296), (700, 9000), (1030, 136), (1100, 8192), (1025, 4104), (1030, 12296), (2053, 24),
          (4100, 264), (300, 16376), (1040, 8200), (1030, 16384), (1100, 2056), (1030, 6008)]


def make(M, N, dtype, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N, generator=g) * (1 + 30 * (torch.rand(N, generator=g) < 0.05))     # a few large channels
    return {k: v.to(dtype).cuda() for k, v in dict(
        X=x, R=0.5 * torch.randn(M, N, generator=g), dY=torch.randn(M, N, generator=g),
        dS=torch.randn(M, N, generator=g), gamma=1 + 0.3 * torch.randn(N, generator=g)).items()}


def nan(*shape, like=None, dtype=None):
    import torch
    return torch.full(shape, float("nan"), device="cuda", dtype=dtype or torch.float32) if like is None \
        else torch.full_like(like, float("nan"))


def forward(x, residual=True, eps=1e-5, **over):
    import torch
    out = {"Y": nan(like=x["X"]), "rstd": nan(x["X"].shape[0])}
    if residual:
        out["S"] = nan(like=x["X"])
    out.update(over)
    ffn.ffn_rmsnorm_forward(x["X"], x["gamma"], out["Y"], R=x["R"] if residual else None, S=out.get("S"),
                            rstd=out["rstd"], eps=eps)
    torch.cuda.synchronize()
    return out


def forward_q8(x, group, residual=True, eps=1e-5):
    import torch
    M, N = x["X"].shape
    out = {"Q": nan(M, N).to(torch.float8_e4m3fn), "scale": nan(M, -(-N // 128) if group else 1), "rstd": nan(M)}
    if residual:
        out["S"] = nan(like=x["X"])
    ffn.ffn_rmsnorm_q8_forward(x["X"], x["gamma"], out["Q"], out["scale"], R=x["R"] if residual else None,
                               S=out.get("S"), rstd=out["rstd"], group=group, eps=eps)
    torch.cuda.synchronize()
    return out


def backward(S, x, rstd, dS=None, ws=None, dX=None):
    import torch
    out = {"dX": nan(like=S) if dX is None else dX, "dgamma": nan(S.shape[1])}
    ffn.ffn_rmsnorm_backward(S, x["dY"], x["gamma"], rstd, out["dX"], out["dgamma"], dS=dS, ws=ws)
    torch.cuda.synchronize()
    return out


def summed(x):
    return (x["X"].cpu().float() + x["R"].cpu().float()).to(x["X"].dtype)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, dtype):
    import torch
    print(f"case RMS norm {shape} {dtype}", flush=True)
    x = make(*shape, getattr(torch, dtype), seed=shape[0] + shape[1])
    f = forward(x)
    assert torch.equal(f["S"].cpu(), summed(x))
    ref.check(f, ref.rmsnorm_forward(f["S"], x["gamma"], 1e-5), f"{shape} forward")
    b = backward(f["S"], x, f["rstd"], x["dS"])
    ref.check(b, ref.rmsnorm_backward(f["S"], x["dY"], x["gamma"], f["rstd"], x["dS"]), f"{shape} backward")
    f = forward(x, residual=False)
    ref.check(f, ref.rmsnorm_forward(x["X"], x["gamma"], 1e-5), f"{shape} forward, no residual")
    b = backward(x["X"], x, f["rstd"])
    ref.check(b, ref.rmsnorm_backward(x["X"], x["dY"], x["gamma"], f["rstd"]), f"{shape} backward, no residual")


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("shape", SHAPES)
def test_8_bit_output(shape, group, dtype):
    import torch
    print(f"case RMS norm, 8 bits {shape} group {group} {dtype}", flush=True)
    x = make(*shape, getattr(torch, dtype), seed=3 * shape[0] + shape[1])
    x["X"][0] = 0      # a row without values, and one with a group without values
    x["R"][0] = 0
    x["X"][-1, :min(128, shape[1])] = 0
    x["R"][-1, :min(128, shape[1])] = 0
    for residual in (True, False):
        f = forward_q8(x, group, residual)
        S = f["S"] if residual else x["X"]
        if residual:
            assert torch.equal(S.cpu(), summed(x))
        ref.check_q8(f["Q"], f["scale"], S, x["gamma"], 1e-5, group, f"{shape} group {group}")
        ref.check(f, {"rstd": ref.rmsnorm_forward(S, x["gamma"], 1e-5)["rstd"]}, f"{shape}")
        assert not bool(f["Q"][0].float().any())


@pytest.mark.parametrize("M,N", [(255, 16384), (256, 16384), (257, 16384), (511, 8200), (513, 8192)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_backward_around_whole_turns(M, N, dtype):
    import torch
    print(f"case RMS norm backward {M} x {N} {dtype}", flush=True)
    x = make(M, N, getattr(torch, dtype), seed=M)
    f = forward(x)
    b = backward(f["S"], x, f["rstd"], x["dS"])
    ref.check(b, ref.rmsnorm_backward(f["S"], x["dY"], x["gamma"], f["rstd"], x["dS"]), f"{M} x {N}")


def test_rstd_is_optional_and_calls_repeat_bitwise():
    import torch
    x = make(301, 1288, torch.bfloat16, seed=2)
    f = forward(x)
    Y, S = torch.empty_like(x["X"]), torch.empty_like(x["X"])
    ffn.ffn_rmsnorm_forward(x["X"], x["gamma"], Y, R=x["R"], S=S)
    ws = ffn.workspace(ffn.ffn_rmsnorm_backward_workspace_size(301, 1288))
    first = backward(f["S"], x, f["rstd"], x["dS"], ws)
    ws.fill_(0xFF)
    again = backward(f["S"], x, f["rstd"], x["dS"], ws)
    assert torch.equal(Y, f["Y"]) and torch.equal(S, f["S"])
    assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("M,N,dtype", [(37, 1544, "bfloat16"), (37, 1544, "float32"), (1100, 4104, "bfloat16"),
                                       (1030, 12296, "float32"), (300, 16384, "float32"), (2053, 520, "bfloat16")])
def test_in_place(M, N, dtype):
    import torch
    print(f"case RMS norm in place {M} x {N} {dtype}", flush=True)
    x = make(M, N, getattr(torch, dtype), seed=M + N)
    f = forward(x)
    for name in ("X", "R"):                       # S over either summand
        y = x[name].clone()
        again = forward({**x, name: y}, S=y)
        assert all(torch.equal(again[k], f[k]) for k in f), name
    plain = forward(x, residual=False)
    y = x["X"].clone()
    assert torch.equal(forward({**x, "X": y}, residual=False, Y=y)["Y"], plain["Y"])
    b = backward(f["S"], x, f["rstd"], x["dS"])
    for name in ("S", "dY", "dS"):
        z = {"S": f["S"], "dY": x["dY"], "dS": x["dS"]}
        z[name] = z[name].clone()
        again = backward(z["S"], {**x, "dY": z["dY"]}, f["rstd"], z["dS"], dX=z[name])
        assert all(torch.equal(again[k], b[k]) for k in b), name


@pytest.mark.parametrize("N", [72, 520, 4104, 12296])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_rows_of_zeros_tiny_and_large_rows(N, dtype):
    """Padded rows give zeros, and a finite gradient; rows far below eps and at 2^55 keep their digits."""
    import torch
    print(f"case RMS norm, unusual rows, N = {N} {dtype}", flush=True)
    x = make(21, N, getattr(torch, dtype), seed=N)
    x["X"][4] = 0
    x["X"][5] *= 2.0 ** -60
    x["X"][6] *= 2.0 ** 50
    f = forward(x, residual=False, eps=1e-6)
    ref.check(f, ref.rmsnorm_forward(x["X"], x["gamma"], 1e-6), f"N = {N}")
    assert not bool(f["Y"][4].any())
    b = backward(x["X"], x, f["rstd"])
    ref.check(b, ref.rmsnorm_backward(x["X"], x["dY"], x["gamma"], f["rstd"]), f"N = {N}")
    q = forward_q8(x, 128, residual=False, eps=1e-6)
    ref.check_q8(q["Q"], q["scale"], x["X"], x["gamma"], 1e-6, 128, f"N = {N}")


def test_nan_rows_stay_alone():
    import torch
    x = make(40, 520, torch.bfloat16, seed=8)
    clean, clean8 = forward(x), forward_q8(x, 128)
    x["X"][11, 3] = float("nan")
    f, f8 = forward(x), forward_q8(x, 128)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[11] = False
    assert torch.equal(f["Y"][keep], clean["Y"][keep]) and torch.equal(f8["scale"][keep], clean8["scale"][keep])
    assert torch.equal(f8["Q"].view(torch.uint8)[keep], clean8["Q"].view(torch.uint8)[keep])
    assert bool(torch.isnan(f["Y"][11].float()).all()) and bool(torch.isnan(f8["Q"][11].float()).all())


def test_no_rows():
    import torch
    x = make(0, 64, torch.bfloat16)
    f = forward(x)
    forward_q8(x, 128)
    b = backward(f["S"], x, f["rstd"], x["dS"])
    assert not bool(b["dgamma"].any())


def test_differences():
    """Directional differences of the fp64 forward against the gradients."""
    import torch
    x = make(11, 72, torch.float32, seed=10)
    f = forward(x)
    b = backward(f["S"], x, f["rstd"], x["dS"])
    w = {"S": ref.d(f["S"]), "gamma": ref.d(x["gamma"])}
    dy, ds = ref.d(x["dY"]), ref.d(x["dS"])

    def loss(v):
        y = v["S"] * (v["S"].square().mean(1, keepdim=True) + 1e-5).pow(-0.5) * v["gamma"]
        return float((y * dy).sum() + (v["S"] * ds).sum())
    g = torch.Generator().manual_seed(3)
    for src, grad in (("S", "dX"), ("gamma", "dgamma")):
        v = torch.randn(w[src].shape, generator=g).double()
        num = (loss({**w, src: w[src] + 1e-5 * v}) - loss({**w, src: w[src] - 1e-5 * v})) / 2e-5
        got = float((ref.d(b[grad]) * v).sum())
        # fp32 statistics and sums: a few hundred roundings of the magnitudes; the third derivative's
        # share of the differences is below 1e-5
        slack = 300 * ref.U_F32 * float((ref.d(b[grad]).abs() * v.abs()).sum() + 30)
        print(f"  {grad}: {got:.7f}, by differences {num:.7f}", flush=True)
        assert abs(got - num) <= slack + 1e-5


@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("M,N", [(40, 520), (1, 8), (130, 8192), (1100, 264), (300, 4104), (260, 8200), (260, 12296),
                                 (260, 16384)])
def test_codes_of_bf16_rows_are_exact(M, N, group):
    """Halfway points between two codes are hit exactly by products of few bits: they go to the even code."""
    import torch
    print(f"case RMS norm, exact codes {M} x {N} group {group}", flush=True)
    x = make(M, N, torch.bfloat16, seed=M + N)
    x["X"][0] = 0
    x["R"][0] = 0
    x["X"][M // 2, :8] *= 2.0 ** 20
    for residual in (True, False):
        f = forward_q8(x, group, residual)
        want = ref.q8_codes(f["S"] if residual else x["X"], x["gamma"], group)
        off = int((ref.d(f["Q"].cpu().float()) != want).sum())
        assert off == 0, f"{off} codes differ"


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("M,N", [(4100, 2056), (6200, 4104), (4100, 8200), (4100, 12296), (16500, 264), (8300, 520),
                                 (12400, 1032)])
def test_workgroups_that_walk_several_rows(M, N, dtype):
    """More rows than the grid takes at once (2048 workgroups), three turns and more: the next row's loads in
    flight, the sums' slots in turn, outputs over inputs.  Every row is bitwise that of a call whose workgroups
    take one turn; some rows of each turn are checked in fp64."""
    import torch
    dt = getattr(torch, dtype)
    print(f"case RMS norm, several turns {M} x {N} {dtype}", flush=True)
    x = make(M, N, dt, seed=M + N)
    x["X"][M - 3] = 0
    x["R"][M - 3] = 0
    rows = torch.cat([torch.arange(0, M, 211), torch.arange(2040, M, 2048), torch.arange(M - 4, M)]).cuda()

    def of(out, i):
        return {k: v[i] for k, v in out.items()}

    for residual in (True, False):
        S = None
        for call in (forward, lambda y, r: forward_q8(y, 128, r), lambda y, r: forward_q8(y, 0, r)):
            f = call(x, residual)
            for lo in range(0, M, 1024):
                lo = min(lo, M - 1024)
                part = slice(lo, lo + 1024)
                one = call({**{k: x[k][part] for k in ("X", "R")}, "gamma": x["gamma"]}, residual)
                for k in f:
                    a, b = (v if v.element_size() > 1 else v.view(torch.uint8) for v in (f[k][part], one[k]))
                    assert torch.equal(a, b), (k, lo)
            S = f["S"] if residual else x["X"]
            if residual:
                assert torch.equal(S, (x["X"].float() + x["R"].float()).to(dt))
            want = ref.rmsnorm_forward(S[rows], x["gamma"], 1e-5)
            if "Y" in f:
                ref.check(of({k: f[k] for k in want}, rows), want, f"{M} x {N}")
                plain = f
            else:
                group = 0 if f["scale"].shape[1] == 1 and N > 128 else 128
                ref.check_q8(f["Q"][rows], f["scale"][rows], S[rows], x["gamma"], 1e-5, group, f"{M} x {N} {group}")
                if dt == torch.bfloat16:
                    assert torch.equal(ref.d(f["Q"][rows].cpu().float()), ref.q8_codes(S[rows], x["gamma"], group))
        if residual:
            for name in ("X", "R"):
                y = x[name].clone()
                again = forward({**x, name: y}, S=y)
                assert all(torch.equal(again[k], plain[k]) for k in plain), name
        else:
            y = x["X"].clone()
            assert torch.equal(forward({**x, "X": y}, residual=False, Y=y)["Y"], plain["Y"])


def test_rows_past_32_bit_offsets():
    """4.3 x 10^9 values: rows at both ends and where 2^31 and 2^32 values or bytes end."""
    import torch
    M, N = (1 << 18) + 77, 16384
    print(f"case RMS norm {M} x {N}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, M, 1 << 16):
        part = X[lo:lo + (1 << 16)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda", dtype=torch.bfloat16))
    gamma = (1 + 0.3 * torch.randn(N, generator=g, device="cuda")).to(torch.bfloat16)
    at = torch.cat([torch.arange(max(0, b - 3), b + 3) for b in (0, 1 << 16, 1 << 17, 1 << 18)] + [torch.arange(M - 4, M)]).unique().cuda()
    S, rstd = torch.zeros_like(X), torch.zeros(M, device="cuda")
    Q, scale = torch.zeros(M, N, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(M, 128, device="cuda")
    ffn.ffn_rmsnorm_q8_forward(X, gamma, Q, scale, R=X, S=S, rstd=rstd)
    assert torch.equal(S[at], X[at] + X[at])
    ref.check_q8(Q[at], scale[at], S[at], gamma, 1e-5, 128, "8 bits")
    assert torch.equal(ref.d(Q[at].cpu().float()), ref.q8_codes(S[at], gamma, 128))
    del Q
    Y = torch.zeros_like(X)
    ffn.ffn_rmsnorm_forward(S, gamma, Y)
    ref.check({"Y": Y[at]}, {"Y": ref.rmsnorm_forward(S[at], gamma, 1e-5)["Y"]}, "forward")
    dX, dgamma = torch.zeros_like(X), torch.empty(N, device="cuda")
    ffn.ffn_rmsnorm_backward(S, Y, gamma, rstd, dX, dgamma, dS=X)
    ref.check({"dX": dX[at]}, {"dX": ref.rmsnorm_backward(S[at], Y[at], gamma, rstd[at], X[at])["dX"]}, "backward")
    total = sum((Y[lo:lo + 4096].double() * S[lo:lo + 4096].double() * rstd[lo:lo + 4096, None].double()).sum(0) for lo in range(0, M, 4096))
    mags = sum((Y[lo:lo + 4096].double() * S[lo:lo + 4096].double()).abs().mul_(rstd[lo:lo + 4096, None].double()).sum(0) for lo in range(0, M, 4096))
    # a workgroup's 1025 rows one after the other, then 256 partial sums; a product's two roundings
    ref.check({"dgamma": dgamma}, {"dgamma": (total.cpu(), (1025 + 256 + 4) * ref.SUM * mags.cpu())}, "dgamma")
