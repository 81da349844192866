"""Refusals of the training operators, on the CPU: the binding's checks of tensors, the C ABI's
checks of pointers, sizes and workspaces (no call reaches a launch)."""
from __future__ import annotations

import pytest
import torch

import transformer_ffn_fusion_amd as ffn

BF, F32 = torch.bfloat16, torch.float32
E_INVAL, E_WS, E_UNSUP, E_ALIGN = -1, -2, -3, -4
FAKE, FAKE2 = 0x10000, 0x20000
M, N, O, P = 32, 64, 128, 72


def meta(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


def swiglu_args():
    return dict(X=meta(M, N), Wg=meta(N, O), Wu=meta(N, O), Wd=meta(O, P), dY=meta(M, P), dX=meta(M, N),
                dWg=meta(N, O), dWu=meta(N, O), dWd=meta(O, P))


@pytest.mark.parametrize("name,bad,msg", [
    ("X", meta(M, N, 1), "dimensions"),
    ("X", meta(M, N, dtype=F32), "dtype"),
    ("Wg", None, "None"),
    ("Wu", meta(N, O + 8), "shape"),
    ("Wd", meta(P, O).t(), "contiguous"),
    ("dY", meta(M + 1, P), "shape"),
    ("dX", meta(M, N, dtype=F32), "dtype"),
    ("dWg", meta(N, O, dtype=torch.float16), "dtype"),
    ("dWu", meta(N, O, dtype=F32), "dtype"),        # the weight gradients share one type
    ("dWd", meta(O, P, dtype=F32), "dtype"),
    ("dWg", meta(N, 2 * O)[:, ::2], "contiguous"),
])
def test_swiglu_backward_binding_refuses(name, bad, msg):
    a = swiglu_args()
    a[name] = bad
    with pytest.raises((ValueError, TypeError), match=msg):
        ffn.ffn_swiglu_backward(**a)


def ln_args(dt=BF):
    return dict(X=meta(M, N, dtype=dt), gamma=meta(N, dtype=dt), beta=meta(N, dtype=dt), Y=meta(M, N, dtype=dt),
                mean=meta(M, dtype=F32), rstd=meta(M, dtype=F32))


@pytest.mark.parametrize("name,bad,msg", [
    ("X", meta(M), "dimensions"),
    ("X", meta(M, N, dtype=torch.float16), "dtype"),
    ("gamma", meta(N, dtype=F32), "dtype"),
    ("beta", meta(N + 8), "shape"),
    ("Y", meta(N, M).t(), "contiguous"),
    ("mean", meta(M), "dtype"),
    ("rstd", meta(M + 1, dtype=F32), "shape"),
    ("gamma", None, "None"),
])
def test_layernorm_forward_binding_refuses(name, bad, msg):
    a = ln_args()
    a[name] = bad
    with pytest.raises((ValueError, TypeError), match=msg):
        ffn.ffn_layernorm_forward(**a)


@pytest.mark.parametrize("name,bad,msg", [
    ("dY", meta(M, N, dtype=F32), "dtype"),
    ("mean", None, "None"),
    ("rstd", meta(M, dtype=BF), "dtype"),
    ("dX", meta(M, N + 8), "shape"),
    ("dgamma", meta(N), "dtype"),
    ("dbeta", meta(1, N, dtype=F32), "shape"),
    ("ws", meta(64, dtype=F32), "uint8"),
])
def test_layernorm_backward_binding_refuses(name, bad, msg):
    a = dict(X=meta(M, N), dY=meta(M, N), gamma=meta(N), mean=meta(M, dtype=F32), rstd=meta(M, dtype=F32),
             dX=meta(M, N), dgamma=meta(N, dtype=F32), dbeta=meta(N, dtype=F32))
    a[name] = bad
    with pytest.raises((ValueError, TypeError), match=msg):
        ffn.ffn_layernorm_backward(**a)


@pytest.mark.parametrize("G,U,msg", [
    (None, meta(N, O), "None"),
    (meta(N), meta(N), "dimensions"),
    (meta(2, 2, N, O), meta(2, 2, N, O), "dimensions"),
    (meta(N, O, dtype=torch.float16), meta(N, O), "dtype"),
    (meta(N, O), meta(N, O, dtype=F32), "dtype"),
    (meta(N, O), meta(O, N), "shape"),
    (meta(O, N).t(), meta(N, O), "contiguous"),
])
def test_orthogonalize_binding_refuses(G, U, msg):
    with pytest.raises((ValueError, TypeError), match=msg):
        ffn.ffn_orthogonalize(G, U)


def test_binding_needs_gpu_tensors():
    with pytest.raises(ValueError, match="on the GPU"):
        ffn.ffn_swiglu_backward(**swiglu_args())
    with pytest.raises(ValueError, match="on the GPU"):
        ffn.ffn_layernorm_forward(**ln_args())
    with pytest.raises(ValueError, match="on the GPU"):
        ffn.ffn_orthogonalize(torch.zeros(8, 8), torch.zeros(8, 8, dtype=BF))


def _swiglu(M=64, N=64, O=64, P=64, dtype=ffn.BF16, gd=ffn.BF16, ws=FAKE, wsb=1 << 30, **ps):
    p = dict(X=FAKE, Wg=FAKE, Wu=FAKE, Wd=FAKE, dY=FAKE, dX=FAKE2, dWg=FAKE2, dWu=FAKE2, dWd=FAKE2)
    p.update(ps)
    return ffn.lib().ffn_swiglu_backward(*p.values(), M, N, O, P, dtype, gd, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), E_INVAL), (dict(Wu=None), E_INVAL), (dict(dWd=None), E_INVAL), (dict(dX=None), E_INVAL),
    (dict(ws=None), E_INVAL), (dict(M=-1), E_INVAL), (dict(O=0), E_INVAL), (dict(dtype=9), E_INVAL),
    (dict(gd=9), E_INVAL), (dict(dtype=ffn.F32), E_UNSUP), (dict(N=12), E_UNSUP), (dict(P=4), E_UNSUP),
    (dict(N=1 << 23, O=8), E_UNSUP), (dict(N=8, O=1 << 22, P=8), E_UNSUP),
    (dict(dY=FAKE + 8), E_ALIGN), (dict(dWg=FAKE2 + 4), E_ALIGN), (dict(ws=FAKE + 16), E_ALIGN),
    (dict(wsb=ffn.ffn_swiglu_backward_workspace_size(64, 64, 64, 64) - 1), E_WS),
])
def test_swiglu_backward_abi_refuses(kw, code):
    assert _swiglu(**kw) == code and ffn.ffn_last_error() != ""


def _ln_fwd(M=64, N=64, dtype=ffn.BF16, eps=1e-5, X=FAKE, gamma=FAKE, beta=FAKE, Y=FAKE2, mean=FAKE2, rstd=FAKE2):
    return ffn.lib().ffn_layernorm_forward(X, gamma, beta, Y, mean, rstd, M, N, dtype, eps, None)


def _ln_bwd(M=64, N=64, dtype=ffn.BF16, ws=FAKE, wsb=1 << 30, **ps):
    p = dict(X=FAKE, dY=FAKE, gamma=FAKE, mean=FAKE, rstd=FAKE, dX=FAKE2, dgamma=FAKE2, dbeta=FAKE2)
    p.update(ps)
    return ffn.lib().ffn_layernorm_backward(*p.values(), M, N, dtype, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), E_INVAL), (dict(beta=None), E_INVAL), (dict(M=-1), E_INVAL), (dict(N=0), E_INVAL),
    (dict(N=20), E_UNSUP), (dict(N=16392), E_UNSUP), (dict(M=1 << 31), E_UNSUP), (dict(dtype=3), E_INVAL),
    (dict(eps=-1.0), E_INVAL), (dict(eps=float("nan")), E_INVAL), (dict(Y=FAKE2 + 8), E_ALIGN),
    (dict(mean=FAKE2 + 4), E_ALIGN),
])
def test_layernorm_forward_abi_refuses(kw, code):
    assert _ln_fwd(**kw) == code and ffn.ffn_last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(dY=None), E_INVAL), (dict(mean=None), E_INVAL), (dict(dgamma=None), E_INVAL), (dict(ws=None), E_INVAL),
    (dict(N=20), E_UNSUP), (dict(N=16392), E_UNSUP), (dict(dtype=3), E_INVAL), (dict(gamma=FAKE + 8), E_ALIGN),
    (dict(ws=FAKE + 16), E_ALIGN),
    (dict(wsb=ffn.ffn_layernorm_backward_workspace_size(64, 64) - 1), E_WS),
])
def test_layernorm_backward_abi_refuses(kw, code):
    assert _ln_bwd(**kw) == code and ffn.ffn_last_error() != ""


def _ortho(B=1, R=64, C=128, dtype=ffn.BF16, steps=5, G=FAKE, U=FAKE2, ws=FAKE, wsb=1 << 40):
    return ffn.lib().ffn_orthogonalize(G, U, B, R, C, dtype, steps, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(G=None), E_INVAL), (dict(U=None), E_INVAL), (dict(ws=None), E_INVAL), (dict(B=-1), E_INVAL),
    (dict(R=0), E_INVAL), (dict(R=12), E_UNSUP), (dict(C=1 << 22), E_UNSUP), (dict(B=65536), E_UNSUP),
    (dict(R=1 << 16, C=1 << 16), E_UNSUP), (dict(steps=0), E_INVAL), (dict(steps=33), E_INVAL),
    (dict(dtype=5), E_INVAL), (dict(G=FAKE + 8), E_ALIGN), (dict(U=FAKE2 + 2), E_ALIGN), (dict(ws=FAKE + 64), E_ALIGN),
    (dict(wsb=ffn.ffn_orthogonalize_workspace_size(1, 64, 128) - 1), E_WS),
])
def test_orthogonalize_abi_refuses(kw, code):
    assert _ortho(**kw) == code and ffn.ffn_last_error() != ""


def test_workspace_sizes_of_invalid_shapes_are_zero():
    assert ffn.ffn_swiglu_backward_workspace_size(4, 4, 64, 64) == 0
    assert ffn.ffn_swiglu_backward_workspace_size(4, 64, 64, 64, ffn.F32) == 0
    assert ffn.ffn_layernorm_backward_workspace_size(4, 12) == 0
    assert ffn.ffn_orthogonalize_workspace_size(1, 64, 12) == 0
    # sizes grow with the shape and cover what the calls keep there
    assert ffn.ffn_swiglu_backward_workspace_size(64, 64, 128, 64) >= 64 * 128 * (4 + 2 + 4)
    assert ffn.ffn_orthogonalize_workspace_size(3, 136, 264) >= 3 * (3 * 136 * 264 * 2 + 2 * 136 * 136 * 2)
    # up to 128 x 512 a matrix stays in one workgroup
    for R, C in ((128, 512), (512, 128), (8, 8)):
        assert ffn.ffn_orthogonalize_workspace_size(3, R, C) == 256
    assert ffn.ffn_orthogonalize_workspace_size(3, 136, 512) > 256 < ffn.ffn_orthogonalize_workspace_size(3, 128, 520)
    assert ffn.ffn_orthogonalize_workspace_size(0, 1024, 1024) >= 256


# 1 MiB apart, as far as every array below reaches
def _at(i):
    return (i + 1) << 20


@pytest.mark.parametrize("over,by", [
    ("dX", "X"), ("dWg", "Wg"), ("dWu", "dWg"), ("dWd", "dY"), ("dX", "dWd"), ("ws", "X"), ("dWu", "ws"),
])
@pytest.mark.parametrize("shift", [0, 4096, -4096])
def test_swiglu_backward_refuses_overlaps(over, by, shift):
    names = ["X", "Wg", "Wu", "Wd", "dY", "dX", "dWg", "dWu", "dWd", "ws"]
    at = {n: _at(4 * i) for i, n in enumerate(names)}
    at[over] = at[by] + shift
    assert _swiglu(wsb=1 << 20, **at) == E_INVAL and "overlap" in ffn.ffn_last_error()


@pytest.mark.parametrize("over,by,shift", [
    ("Y", "X", 16), ("Y", "X", -16), ("Y", "gamma", 0), ("mean", "X", 0), ("rstd", "mean", 0), ("mean", "beta", 0),
    ("rstd", "Y", 0),
])
def test_layernorm_forward_refuses_overlaps(over, by, shift):
    at = {n: _at(i) for i, n in enumerate(["X", "gamma", "beta", "Y", "mean", "rstd"])}
    at[over] = at[by] + shift
    assert _ln_fwd(**at) == E_INVAL and "overlap" in ffn.ffn_last_error()


@pytest.mark.parametrize("over,by,shift", [
    ("dX", "X", 128), ("dX", "dY", -128), ("dX", "gamma", 0), ("dgamma", "gamma", 0), ("dbeta", "dgamma", 0),
    ("dbeta", "X", 0), ("dgamma", "mean", 0), ("ws", "dX", 0), ("ws", "rstd", 0),
])
def test_layernorm_backward_refuses_overlaps(over, by, shift):
    names = ["X", "dY", "gamma", "mean", "rstd", "dX", "dgamma", "dbeta", "ws"]
    at = {n: _at(i) for i, n in enumerate(names)}
    at[over] = at[by] + shift
    assert _ln_bwd(wsb=1 << 20, **at) == E_INVAL and "overlap" in ffn.ffn_last_error()


@pytest.mark.parametrize("R,C", [(64, 128), (136, 264)])
def test_orthogonalize_refuses_overlaps(R, C):
    size = 2 * R * C
    for kw in (dict(U=_at(0)), dict(U=_at(0) + size - 16), dict(U=_at(0) - size + 16), dict(ws=_at(0)),
               dict(ws=_at(1)), dict(U=_at(0) + size, dtype=ffn.F32)):
        args = dict(G=_at(0), U=_at(1), ws=_at(2), wsb=1 << 20, R=R, C=C)
        assert _ortho(**{**args, **kw}) == E_INVAL and "overlap" in ffn.ffn_last_error()


@pytest.mark.parametrize("R,C", [(64, 128), (136, 264)])
@pytest.mark.parametrize("steps", [9, 12, 16, 32])
def test_orthogonalize_refuses_steps_that_grow_noise_past_the_answer(R, C, steps):
    """A gradient of low rank: what is rounded in directions that it does not have grows by 3.4445 a step."""
    assert _ortho(R=R, C=C, steps=steps) == E_UNSUP and "steps" in ffn.ffn_last_error()
    # the most steps that are taken reach the next check
    assert _ortho(R=R, C=C, steps=8, wsb=0) == E_WS
