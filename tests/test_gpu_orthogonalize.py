"""GPU parity of the orthogonalised update against the fp64 iteration (bounds: training_ref)."""
from __future__ import annotations

import pytest

import transformer_ffn_fusion_amd as ffn

import training_ref as ref

pytestmark = pytest.mark.gpu


def gradient(R, C, seed=0, rank=None, spread=0.5):
    """X^T dA over `rank` tokens, channels of unequal size."""
    import torch
    g = torch.Generator().manual_seed(seed)
    T = rank or 2 * max(R, C)
    x = torch.randn(R, T, generator=g) * torch.exp(spread * torch.randn(R, 1, generator=g))
    y = torch.randn(T, C, generator=g) * torch.exp(spread * torch.randn(1, C, generator=g))
    return x @ y / T


def run(G, steps=5, ws=None):
    import torch
    U = torch.full(G.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    ffn.ffn_orthogonalize(G, U, steps=steps, ws=ws)
    torch.cuda.synchronize()
    return U


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("shape", [
    (8, 8), (8, 264), (264, 8), (64, 64), (72, 200), (200, 72), (128, 512), (136, 136), (264, 520),
    (520, 264), (392, 400), (1032, 256),
])
def test_shapes(shape, dtype):
    import torch
    print(f"case orthogonalize {shape} {dtype}", flush=True)
    G = gradient(*shape, seed=sum(shape)).to(getattr(torch, dtype)).cuda()
    ref.check_orthogonalize(run(G), G, 5, str(shape))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("shape", [
    (8, 512), (512, 8), (16, 32), (40, 96), (96, 40), (104, 456), (456, 104), (128, 128), (512, 128),
    (128, 504), (504, 120), (128, 520), (520, 128), (136, 512), (512, 136),
])
def test_one_workgroup_shapes_and_just_beyond(shape, dtype):
    import torch
    print(f"case orthogonalize {shape} {dtype}", flush=True)
    G = gradient(*shape, seed=sum(shape) + 1).to(getattr(torch, dtype)).cuda()
    ref.check_orthogonalize(run(G), G, 5, str(shape))


@pytest.mark.parametrize("steps", [1, 2, 6])
@pytest.mark.parametrize("shape", [(72, 200), (200, 72)])
def test_one_workgroup_steps(shape, steps):
    G = gradient(*shape, seed=steps).cuda()
    ref.check_orthogonalize(run(G, steps), G, steps, f"{shape} {steps} steps")


@pytest.mark.parametrize("kind", ["rank 1", "rank 16", "orthogonal", "one large direction", "huge"])
def test_one_workgroup_spectra(kind):
    import torch
    R, C = 120, 328
    if kind == "rank 1":
        G = gradient(R, C, 13, rank=1)
    elif kind == "rank 16":
        G = gradient(R, C, 14, rank=16)
    elif kind == "orthogonal":
        G = torch.linalg.qr(torch.randn(C, R, generator=torch.Generator().manual_seed(15)))[0].t().contiguous()
    elif kind == "one large direction":
        G = gradient(R, C, 16) + 100 * gradient(R, C, 17, rank=1)
    else:
        G = gradient(R, C, 18) * 1e30   # squares leave fp32's range
    G = G.cuda()
    ref.check_orthogonalize(run(G), G, 5, kind)


def test_one_workgroup_large_stack():
    import torch
    G = torch.stack([gradient(72, 40, s) * 10.0 ** (s % 7 - 3) for s in range(20)]).cuda()
    G = G.repeat(40, 1, 1)   # 800 matrices, more than the CUs
    U = run(G)
    assert torch.equal(U, U[:20].repeat(40, 1, 1))
    for e in range(20):
        ref.check_orthogonalize(U[e], G[e], 5, f"matrix {e}")


@pytest.mark.parametrize("steps", [1, 2, 3, 6])
def test_steps(steps):
    G = gradient(136, 264, seed=steps).cuda()
    ref.check_orthogonalize(run(G, steps), G, steps, f"{steps} steps")


def test_large_tiles():
    # tiles of 256 x 256 for the outer product, joined splits of small ones for the symmetric one
    G = gradient(2056, 4136, seed=1).bfloat16().cuda()
    ref.check_orthogonalize(run(G), G, 5, "2056 x 4136")
    Gt = G.t().contiguous()
    ref.check_orthogonalize(run(Gt), Gt, 5, "4136 x 2056")


def test_joined_large_tiles():
    # 3584 rows: the symmetric product takes tiles of 256 x 256 in two joined splits
    G = gradient(3400, 8200, seed=2, rank=4096).bfloat16().cuda()
    U = run(G)
    assert bool(torch_isfinite(U).all())
    # the fp64 iteration on the GPU: 3400 x 8200 is too long for the host
    import torch
    X = G.double() / (torch.linalg.vector_norm(G.double()) + ref.NS_EPS)
    for _ in range(5):
        A = X @ X.t().contiguous()
        X = ref.NS[0] * X + (ref.NS[1] * A + ref.NS[2] * (A @ A)) @ X
    rel = float(torch.linalg.vector_norm(U.double() - X) / torch.linalg.vector_norm(X))
    print(f"  3400 x 8200: relative error {rel:.2e}", flush=True)
    assert rel <= ref.NS_REL


def torch_isfinite(t):
    import torch
    return torch.isfinite(t.float())


@pytest.mark.parametrize("kind", ["rank 1", "rank 16", "orthogonal", "one large direction", "tiny", "huge"])
def test_spectra(kind):
    import torch
    R, C = 200, 328
    if kind == "rank 1":
        G = gradient(R, C, 3, rank=1)
    elif kind == "rank 16":
        G = gradient(R, C, 4, rank=16)
    elif kind == "orthogonal":
        G = torch.linalg.qr(torch.randn(C, R, generator=torch.Generator().manual_seed(5)))[0].t().contiguous()
    elif kind == "one large direction":
        G = gradient(R, C, 6) + 100 * gradient(R, C, 7, rank=1)
    else:
        G = gradient(R, C, 8) * (1e-25 if kind == "tiny" else 1e30)   # squares leave fp32's range
    G = G.cuda()
    if kind == "tiny":   # far below the norm's epsilon: X = G / 1e-7, grown by 3.4445 each step
        got, want = ref.d(run(G)), ref.orthogonalize(G)
        assert float((got - want).abs().max()) <= 1e-9 and float(want.abs().max()) < 1e-10
        return
    ref.check_orthogonalize(run(G), G, 5, kind)


def test_stack_is_each_alone_bitwise():
    import torch
    G = torch.stack([gradient(136, 72, s) * 10.0 ** s for s in range(5)]).cuda()
    U = run(G)
    for e in range(5):
        ref.check_orthogonalize(U[e], G[e], 5, f"matrix {e}")
        assert torch.equal(run(G[e].contiguous()), U[e])


def test_repeat_bitwise_dirty_workspace_and_guard():
    import torch
    G = gradient(200, 136, 9).cuda()
    need = ffn.ffn_orthogonalize_workspace_size(1, 200, 136)
    raw = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    raw[need:] = 0xA5
    first = run(G, ws=raw[:need])
    raw[:need] = 0xFF
    assert torch.equal(run(G, ws=raw[:need]), first)
    assert bool((raw[need:] == 0xA5).all())


def test_zeros_nan_and_infinity():
    import torch
    G = torch.stack([gradient(72, 136, s) for s in range(4)]).cuda()
    G[0] = 0.0
    G[1, 3, 5] = float("nan")
    G[2, 70, 2] = float("inf")
    U = run(G)
    assert not bool(U[0].any())
    assert bool(torch.isnan(U[1].float()).all()) and bool(torch.isnan(U[2].float()).all())
    ref.check_orthogonalize(U[3], G[3], 5, "beside them")


def test_empty_stack():
    import torch
    ffn.ffn_orthogonalize(torch.empty(0, 8, 8, device="cuda"), torch.empty(0, 8, 8, dtype=torch.bfloat16, device="cuda"))


SMALL_NORMS = [1e-7, 1e-10, 1e-12, 1e-16, 1e-25, 1e-36]


@pytest.mark.parametrize("norm", SMALL_NORMS)
@pytest.mark.parametrize("shape", [(120, 328), (512, 128), (200, 328), (1032, 264)])
def test_small_norms(shape, norm):
    """||G|| around the norm's epsilon and far below it: X = G / (||G|| + 1e-7) is small then, and as
    accurate as any other, in one workgroup and in tiles."""
    import torch
    print(f"case orthogonalize {shape} of norm {norm}", flush=True)
    G = gradient(*shape, seed=21).double()
    G = (G * (norm / torch.linalg.vector_norm(G))).float().cuda()
    for steps in (1, 5, 8):
        ref.check_orthogonalize(run(G, steps), G, steps, f"{shape} norm {norm} {steps} steps")


@pytest.mark.parametrize("shape", [(72, 136), (136, 264)])
def test_stack_of_unlike_norms_is_each_alone_bitwise(shape):
    import torch
    G = torch.stack([gradient(*shape, seed=30 + s) * 10.0 ** p for s, p in enumerate((0, -12, -30, 20, -9))])
    G = torch.cat([G, torch.zeros_like(G[:1]), G[:1]]).cuda()
    G[2, 3, 5] = float("nan")
    U = run(G)
    assert bool(torch.isnan(U[2].float()).all()) and not bool(U[5].any())
    for e in (0, 1, 3, 4, 6):
        ref.check_orthogonalize(U[e], G[e], 5, f"matrix {e}")
        assert torch.equal(run(G[e].contiguous()), U[e])


# Directions that G does not have: what a step rounds there is multiplied by a = 3.4445 in each
# later one.  A rounding of X's pair is 2^-24 of an element at most; one of the product's fp32 sum
# over m terms (m / 32 additions of the matrix instruction, 2^-23 each, truncated; taken as
# independent, 1 / sqrt 3 in the mean, of partial sums that grow to |b + c| = 2.74 times an
# element): 2^-23 * 2.74 / 3 * sqrt(m / 32), 2.3 * 2^-23 at m = 200.  After the first step's rounding
# `steps` - 1 more multiply it, and the later ones' add 1 / sqrt(1 - 1 / 3.4445^2) = 1.05 and the
# pair's own: below 2.5 * 1.41 * 2^-23 * sqrt(m / 200) * 3.4445^(steps - 1) of a U of rank 1.
def low_rank_bound(m, steps):
    noise = 2.5 * 1.41 * 2.0 ** -23 * max(1.0, (m / 200) ** 0.5) * ref.NS[0] ** (steps - 1)
    return (ref.NS_REL ** 2 + noise ** 2) ** 0.5


@pytest.mark.parametrize("steps", [5, 8])
@pytest.mark.parametrize("rank", [1, 4, 16])
@pytest.mark.parametrize("shape", [(120, 328), (512, 128), (200, 328), (1032, 264), (1024, 1536), (2056, 4136)])
def test_low_rank_up_to_the_most_steps(shape, rank, steps):
    import torch
    print(f"case orthogonalize {shape} rank {rank} {steps} steps", flush=True)
    G = gradient(*shape, seed=40 + rank, rank=rank).cuda()
    want, got = ref.orthogonalize(G, steps), ref.d(run(G, steps))
    rel = float(torch.linalg.vector_norm(got - want) / torch.linalg.vector_norm(want))
    bound = low_rank_bound(min(shape), steps)
    print(f"  relative error {rel:.2e} (bound {bound:.1e})", flush=True)
    assert rel <= bound
