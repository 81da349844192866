"""GPU parity of the SwiGLU backward against its fp64 form, element by element, within the bounds
of training_ref (one bf16 rounding of h, da or db, one of the output, fp32 sums)."""
from __future__ import annotations

import pytest

import transformer_ffn_fusion_amd as ffn

import training_ref as ref

pytestmark = pytest.mark.gpu
NAMES = ("dX", "dWg", "dWu", "dWd")


def make(M, N, O, P, seed=0, grad_f32=False, spread=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g)
    x = dict(X=r(M, N), Wg=spread * r(N, O) / N ** 0.5, Wu=r(N, O) / N ** 0.5, Wd=r(O, P) / O ** 0.5,
             dY=r(M, P))
    x = {k: v.bfloat16().cuda() for k, v in x.items()}
    gd = torch.float32 if grad_f32 else torch.bfloat16
    # outputs start as NaN: every element has to be written
    out = dict(dX=torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda"),
               dWg=torch.full((N, O), float("nan"), dtype=gd, device="cuda"),
               dWu=torch.full((N, O), float("nan"), dtype=gd, device="cuda"),
               dWd=torch.full((O, P), float("nan"), dtype=gd, device="cuda"))
    return x, out


def run(x, out, ws=None):
    import torch
    ffn.ffn_swiglu_backward(*x.values(), *out.values(), ws=ws)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("grad_f32", [False, True])
@pytest.mark.parametrize("shape", [
    (1, 8, 8, 8),              # the least of everything
    (1, 64, 128, 64),          # one token
    (17, 72, 40, 88),          # inside one tile, every k-tile short
    (64, 64, 448, 64),
    (63, 128, 64, 192),        # M one below a k-tile
    (65, 200, 136, 72),        # M one above
    (130, 264, 456, 136),      # tiles that end inside every dimension
    (257, 136, 264, 520),
    (300, 520, 1032, 264),     # more hidden columns than a large tile
])
def test_shapes(shape, grad_f32):
    print(f"case swiglu backward {shape} fp32 gradients {grad_f32}", flush=True)
    x, out = make(*shape, seed=sum(shape), grad_f32=grad_f32)
    ref.check(run(x, out), ref.swiglu_backward(*x.values(), grad_f32=grad_f32), str(shape))


@pytest.mark.parametrize("shape", [
    (2056, 2072, 1048, 2056),    # tiles of 256 x 128 with ragged edges
    (3000, 1000, 2800, 1000),    # of 256 x 256; two whole rounds of small ones and a split rest; joins
    (1013, 2056, 1400, 1992),    # joins
    (8, 128, 512, 128),          # joins of few rows
    (20, 2048, 1024, 1536),
    (70, 2056, 264, 2000),       # few tiles, deep: dh and the gated step apart, split
    (2100, 72, 4104, 88),        # many tiles, shallow: dh and the gated step together, in rounds
    (2100, 1032, 4104, 1000),    # ... and a shape where they are apart
    (1030, 264, 1096, 200),
])
def test_large_shapes(shape):
    print(f"case swiglu backward {shape}", flush=True)
    x, out = make(*shape, seed=3)
    ref.check(run(x, out), ref.swiglu_backward(*x.values()), str(shape))


def test_saturated_gates():
    # gates from far below to far above 0: sigmoid at 0 and 1, exp out of fp32's range
    x, out = make(96, 64, 256, 64, seed=5, spread=60.0)
    ref.check(run(x, out), ref.swiglu_backward(*x.values()), "saturated")


def test_repeat_bitwise_and_dirty_workspace():
    import torch
    shape = (200, 264, 392, 136)
    x, out = make(*shape, seed=7)
    ws = ffn.workspace(ffn.ffn_swiglu_backward_workspace_size(*shape))
    first = {k: v.clone() for k, v in run(x, out, ws).items()}
    ws.fill_(0xFF)   # NaN patterns: nothing may be read before it is written
    for v in out.values():
        v.fill_(float("nan"))
    run(x, out, ws)
    assert all(torch.equal(first[k], out[k]) for k in NAMES)


def test_no_rows_zero_fills():
    import torch
    for grad_f32 in (False, True):
        x, out = make(0, 64, 136, 72, grad_f32=grad_f32)
        run(x, out)
        assert all(not bool(out[k].any()) for k in NAMES[1:]) and not bool(torch.isnan(out["dWd"]).any())


def test_workspace_and_outputs_end_where_they_end():
    import torch
    shape = (70, 72, 136, 200)
    x, out = make(*shape, seed=9)
    need = ffn.ffn_swiglu_backward_workspace_size(*shape)
    raw = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    big = {k: torch.full((v.numel() + 512,), 7.0, dtype=v.dtype, device="cuda") for k, v in out.items()}
    for k, v in out.items():
        out[k] = big[k][:v.numel()].view(v.shape)
    ref.check(run(x, out, raw[:need]), ref.swiglu_backward(*x.values()), "guarded")
    assert bool((raw[need:] == 0xA5).all())
    assert all(bool((big[k][out[k].numel():] == 7.0).all()) for k in NAMES)


def test_differences():
    """Directional differences of the forward against the gradients, fp64 on the inputs' values."""
    import torch
    shape = (24, 40, 56, 32)
    x, out = make(*shape, seed=11, grad_f32=True)
    run(x, out)
    w = {k: ref.d(v) for k, v in x.items()}

    def loss(v):
        a = v["X"] @ v["Wg"]
        return float(((a * torch.sigmoid(a) * (v["X"] @ v["Wu"])) @ v["Wd"] * w["dY"]).sum())
    bounds = ref.swiglu_backward(*x.values(), grad_f32=True)
    g = torch.Generator().manual_seed(1)
    for src, grad in (("X", "dX"), ("Wg", "dWg"), ("Wu", "dWu"), ("Wd", "dWd")):
        v = torch.randn(w[src].shape, generator=g).double()
        step = 1e-5
        num = (loss({**w, src: w[src] + step * v}) - loss({**w, src: w[src] - step * v})) / (2 * step)
        got = float((ref.d(out[grad]) * v).sum())
        slack = float((bounds[grad][1] * v.abs()).sum())
        print(f"  {grad}: {got:.6f}, by differences {num:.6f}, bound {slack:.2e}", flush=True)
        assert abs(got - num) <= slack + 1e-6 * abs(num)


def test_infinite_and_nan_inputs_stay_in_their_rows():
    """A NaN token reaches its own row of dX and the weight gradients, no other row of dX."""
    import torch
    shape = (70, 72, 136, 200)
    x, out = make(*shape, seed=13)
    clean = {k: v.clone() for k, v in run(x, out).items()}
    x["X"][33] = float("nan")
    run(x, out)
    keep = torch.arange(70, device="cuda") != 33
    assert torch.equal(out["dX"][keep], clean["dX"][keep]) and bool(torch.isnan(out["dX"][33]).all())
    assert bool(torch.isnan(out["dWg"]).all())


@pytest.mark.parametrize("shape", [
    (9, 4296, 3776, 3896),       # dWg | dWu and dWd in tiles of 256 x 256
    (898, 4296, 3936, 4072),     # ... dWg | dWu with a split rest
    (5393, 144, 3192, 4792),     # dWg | dWu in tiles of 256 x 128, in five joined splits
    (3163, 8, 3464, 4504),       # ... of 128 x 128, in nine
    (1697, 4528, 1488, 208),     # dWd of 128 x 128, in three
    (542, 4264, 3728, 4552),     # ... with a split rest
    (1013, 2056, 1400, 1992),    # the three output products in one launch
])
def test_fp32_gradients_of_every_tile(shape):
    print(f"case swiglu backward {shape} fp32 gradients", flush=True)
    x, out = make(*shape, seed=4, grad_f32=True)
    ref.check(run(x, out), ref.swiglu_backward(*x.values(), grad_f32=True), str(shape))
