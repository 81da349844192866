"""GPU parity of the layer norm and its gradients against their fp64 forms, within the bounds of
training_ref."""
from __future__ import annotations

import pytest

import transformer_ffn_fusion_amd as ffn

import training_ref as ref

pytestmark = pytest.mark.gpu
SHAPES = [(1, 8), (1, 4096), (3, 72), (5, 512), (7, 520), (13, 1032), (2, 2048), (33, 2056), (6, 4104),
          (5, 8192), (3, 8200), (2, 16384), (3, 12296), (700, 9000), (1030, 136), (1100, 8192), (1025, 4104), (1030, 12296), (2053, 24), (700, 1024)]


def make(M, N, dtype, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N, generator=g) + 0.5
    x = x * (1 + 30 * (torch.rand(N, generator=g) < 0.05))     # a few large channels
    return {k: v.to(dtype).cuda() for k, v in dict(
        X=x, dY=torch.randn(M, N, generator=g), gamma=1 + 0.3 * torch.randn(N, generator=g),
        beta=0.3 * torch.randn(N, generator=g)).items()}


def forward(x, eps=1e-5, Y=None):
    import torch
    M = x["X"].shape[0]
    nan = torch.full((M,), float("nan"), device="cuda")
    out = dict(Y=torch.full_like(x["X"], float("nan")) if Y is None else Y, mean=nan, rstd=nan.clone())
    ffn.ffn_layernorm_forward(x["X"], x["gamma"], x["beta"], out["Y"], out["mean"], out["rstd"], eps=eps)
    torch.cuda.synchronize()
    return out


def backward(x, mean, rstd, ws=None, dX=None):
    import torch
    nan = torch.full((x["X"].shape[1],), float("nan"), device="cuda")
    out = dict(dX=torch.full_like(x["X"], float("nan")) if dX is None else dX, dgamma=nan, dbeta=nan.clone())
    ffn.ffn_layernorm_backward(x["X"], x["dY"], x["gamma"], mean, rstd, out["dX"], out["dgamma"],
                               out["dbeta"], ws=ws)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, dtype):
    import torch
    print(f"case layer norm {shape} {dtype}", flush=True)
    x = make(*shape, getattr(torch, dtype), seed=shape[0] + shape[1])
    f = forward(x)
    ref.check(f, ref.layernorm_forward(x["X"], x["gamma"], x["beta"], 1e-5), f"{shape} forward")
    b = backward(x, f["mean"], f["rstd"])
    ref.check(b, ref.layernorm_backward(x["X"], x["dY"], x["gamma"], f["mean"], f["rstd"]),
              f"{shape} backward")


@pytest.mark.parametrize("M,N", [(256, 16384), (257, 16384), (300, 16376), (511, 8200), (512, 8192), (513, 8192)])
def test_backward_one_two_and_three_turns(M, N):
    """Around one, two and three rows a workgroup, where the number of workgroups changes."""
    import torch
    x = make(M, N, torch.float32, seed=M)
    f = forward(x)
    b = backward(x, f["mean"], f["rstd"])
    ref.check(b, ref.layernorm_backward(x["X"], x["dY"], x["gamma"], f["mean"], f["rstd"]), f"{M} x {N}")


def test_statistics_are_optional_and_calls_repeat_bitwise():
    import torch
    x = make(301, 1288, torch.bfloat16, seed=2)
    f = forward(x)
    Y = torch.empty_like(x["X"])
    ffn.ffn_layernorm_forward(x["X"], x["gamma"], x["beta"], Y)
    ws = ffn.workspace(ffn.ffn_layernorm_backward_workspace_size(301, 1288))
    first = backward(x, f["mean"], f["rstd"], ws)
    ws.fill_(0xFF)
    again = backward(x, f["mean"], f["rstd"], ws)
    assert torch.equal(Y, f["Y"])
    assert all(torch.equal(first[k], again[k]) for k in first)


def test_in_place():
    import torch
    for dtype in (torch.bfloat16, torch.float32):
        x = make(37, 1544, dtype, seed=4)
        f = forward(x)
        y = x["X"].clone()
        ffn.ffn_layernorm_forward(y, x["gamma"], x["beta"], y)
        assert torch.equal(y, f["Y"])
        b = backward(x, f["mean"], f["rstd"])
        for name in ("X", "dY"):
            z = {**x, name: x[name].clone()}
            assert torch.equal(backward(z, f["mean"], f["rstd"], dX=z[name])["dX"], b["dX"])


def test_constant_rows_and_large_offsets():
    """Rows without spread: y = beta, and a finite gradient; an offset of 1000 costs no digits
    beyond fp32's of the inputs."""
    import torch
    x = make(9, 264, torch.float32, seed=6)
    x["X"][4] = 3.0
    x["X"][5] = 0.0
    x["X"][6] += 1000.0
    f = forward(x)
    ref.check(f, ref.layernorm_forward(x["X"], x["gamma"], x["beta"], 1e-5), "offsets")
    assert torch.equal(f["Y"][4], x["beta"]) and torch.equal(f["Y"][5], x["beta"])
    b = backward(x, f["mean"], f["rstd"])
    ref.check(b, ref.layernorm_backward(x["X"], x["dY"], x["gamma"], f["mean"], f["rstd"]), "offsets")


def test_nan_rows_stay_alone():
    import torch
    x = make(40, 520, torch.bfloat16, seed=8)
    clean = forward(x)
    x["X"][11, 3] = float("nan")
    x["X"][12, 5] = float("inf")
    f = forward(x)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[11:13] = False
    assert torch.equal(f["Y"][keep], clean["Y"][keep])
    assert bool(torch.isnan(f["Y"][11:13].float()).all())


def test_no_rows():
    import torch
    x = make(0, 64, torch.bfloat16)
    f = forward(x)
    b = backward(x, f["mean"], f["rstd"])
    assert not bool(b["dgamma"].any()) and not bool(b["dbeta"].any())


def test_differences():
    """Directional differences of the fp64 forward against the gradients."""
    import torch
    x = make(11, 72, torch.float32, seed=10)
    f = forward(x)
    b = backward(x, f["mean"], f["rstd"])
    w = {k: ref.d(v) for k, v in x.items()}

    def loss(v):
        c = v["X"] - v["X"].mean(1, keepdim=True)
        y = c * (c.square().mean(1, keepdim=True) + 1e-5).pow(-0.5) * v["gamma"] + v["beta"]
        return float((y * w["dY"]).sum())
    g = torch.Generator().manual_seed(3)
    for src, grad in (("X", "dX"), ("gamma", "dgamma"), ("beta", "dbeta")):
        v = torch.randn(w[src].shape, generator=g).double()
        num = (loss({**w, src: w[src] + 1e-5 * v}) - loss({**w, src: w[src] - 1e-5 * v})) / 2e-5
        got = float((ref.d(b[grad]) * v).sum())
        # fp32 statistics and sums: a few hundred roundings of the magnitudes
        slack = 300 * ref.U_F32 * float((ref.d(b[grad]).abs() * v.abs()).sum() + 30)
        print(f"  {grad}: {got:.7f}, by differences {num:.7f}", flush=True)
        assert abs(got - num) <= slack + 1e-5


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("N", [72, 520, 1544, 8200, 12296])
def test_backward_where_mean_times_rstd_leaves_fp32(N, dtype):
    """Constant rows far from 0: z is 0 and dX finite, although mean * rstd is past fp32's largest
    value (2^112 * 1e6); N that does not fill the waves' columns.  (The sum of N times 2^112 is a
    whole multiple of it and within fp32: the mean is exact.)"""
    import torch
    print(f"case layer norm backward, constant rows, N = {N} {dtype}", flush=True)
    x = make(21, N, getattr(torch, dtype), seed=N)
    x["X"][4] = 2.0 ** 112
    x["X"][17] = -2.0 ** 112
    f = forward(x, eps=1e-12)
    assert float(f["mean"][4]) == 2.0 ** 112 and float(f["mean"][17]) == -2.0 ** 112
    assert torch.equal(f["Y"][4], x["beta"]) and torch.equal(f["Y"][17], x["beta"])
    b = backward(x, f["mean"], f["rstd"])
    ref.check(b, ref.layernorm_backward(x["X"], x["dY"], x["gamma"], f["mean"], f["rstd"]), f"N = {N}")


@pytest.mark.parametrize("M,N,dtype", [
    (1100, 4104, "bfloat16"), (2053, 520, "float32"), (5000, 24, "bfloat16"),   # many rows, the next rows in flight
    (1030, 12296, "bfloat16"), (1030, 12296, "float32"),                        # ... of eight waves
    (5, 12296, "float32"), (300, 16384, "float32"), (520, 8200, "float32"),     # x and dy read again for dx
])
def test_in_place_many_and_wide_rows(M, N, dtype):
    import torch
    print(f"case layer norm in place {M} x {N} {dtype}", flush=True)
    x = make(M, N, getattr(torch, dtype), seed=M + N)
    f = forward(x)
    y = x["X"].clone()
    again = forward({**x, "X": y}, Y=y)
    assert all(torch.equal(again[k], f[k]) for k in f)
    b = backward(x, f["mean"], f["rstd"])
    for name in ("X", "dY"):
        z = {**x, name: x[name].clone()}
        again = backward(z, f["mean"], f["rstd"], dX=z[name])
        assert all(torch.equal(again[k], b[k]) for k in b), name
