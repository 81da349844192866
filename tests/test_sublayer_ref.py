"""The plain fp64 forms of the operators around an expert sub-layer against automatic differentiation
and against the definitions, on the CPU."""
from __future__ import annotations

import pytest
import torch

import sublayer_ref as ref

F64 = torch.float64


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def close(a, b):
    assert a.shape == b.shape and float((a - b).abs().max()) <= 1e-12 * max(1.0, float(b.abs().max()))


def test_rmsnorm_gradients_are_those_of_the_forward():
    S, dY, dS, gamma = rand(7, 24), rand(7, 24, seed=1), rand(7, 24, seed=2), 1 + 0.1 * rand(24, seed=3)
    s, g = S.clone().requires_grad_(), gamma.clone().requires_grad_()
    y = s * (s.square().mean(1, keepdim=True) + 1e-3).pow(-0.5) * g
    ((y * dY).sum() + (s * dS).sum()).backward()
    close(ref.rmsnorm_forward(S, gamma, 1e-3)["Y"][0], y.detach())
    rstd = (S.square().mean(1) + 1e-3).pow(-0.5)
    got = ref.rmsnorm_backward(S, dY, gamma, rstd, dS)
    close(got["dX"][0], s.grad)
    close(got["dgamma"][0], g.grad)


def test_dispatch_and_combine_gradients_are_those_of_the_forward():
    M, N, E, k = 9, 8, 5, 3
    ids = torch.randint(-1, E + 1, (M, k), generator=torch.Generator().manual_seed(1))
    pos, off, entries = ref.sort(ids, E)
    assert int(off[-1]) == entries.numel() == int((pos >= 0).sum())
    X = rand(M, N).requires_grad_()
    Xs = X[(entries // k).long()]
    dXs = rand(*Xs.shape, seed=1)
    (Xs * dXs).sum().backward()
    close(ref.combine(dXs, pos)["Y"][0], X.grad)
    Ys, w, R, dY = rand(*Xs.shape, seed=2).requires_grad_(), rand(M, k, seed=3).requires_grad_(), rand(M, N, seed=4), rand(M, N, seed=5)
    kept = pos >= 0
    rows = torch.where(kept[:, :, None], Ys[pos.clamp(min=0).long()], 0.0)
    Y = R + (rows * torch.where(kept, w, 0.0)[:, :, None]).sum(1)
    close(ref.combine(Ys, pos, w, R)["Y"][0], Y.detach())
    (Y * dY).sum().backward()
    dw, (drow, _, k2) = ref.combine_backward(dY, Ys, pos, w)
    assert torch.equal(k2, kept)
    close(dw["dw"][0], w.grad)
    got = torch.zeros_like(Ys)
    got[pos[kept].long()] = drow[kept]
    close(got, Ys.grad)


def test_route_gradient_is_that_of_the_softmax():
    M, E, k = 11, 7, 3
    logits = rand(M, E).requires_grad_()
    top, ids = logits.topk(k, 1)
    w = torch.softmax(top, 1)
    dw = rand(M, k, seed=1)
    (w * dw).sum().backward()
    close(ref.route_backward(ids, w, dw, E)["dlogits"][0], logits.grad)


def test_sort_is_stable_and_drops_ids_outside():
    ids = torch.tensor([[2, 0], [-1, 2], [2, 2], [3, 1]])
    pos, off, entries = ref.sort(ids, 3)
    assert off.tolist() == [0, 1, 2, 6] and entries.tolist() == [1, 7, 0, 3, 4, 5]
    assert pos.tolist() == [[2, 0], [-1, 3], [4, 5], [-1, 1]]


def test_e4m3_rounding():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    every = every[torch.isfinite(every)]
    assert torch.equal(ref.to_e4m3(every), every)
    v = torch.cat([rand(4000) * 10 ** torch.linspace(-4, 2.5, 4000, dtype=F64), torch.tensor([0.0, 448.0, 1e6, -1e6, 2.0 ** -10])])
    assert torch.equal(ref.to_e4m3(v), v.clamp(-448, 448).float().to(torch.float8_e4m3fn).double())


@pytest.mark.parametrize("code", ["int4", "e2m1"])
@pytest.mark.parametrize("K,C", [(8, 8), (136, 24), (264, 40)])
def test_packed_layout_round_trip(K, C, code):
    q = torch.randint(0, 16, (K, C), generator=torch.Generator().manual_seed(K)).to(torch.uint8)
    Wq = torch.zeros(-(-C // 16), -(-K // 128), 1024, dtype=torch.uint8)
    assert torch.equal(ref.q4_codes(ref.q4_pack(q, Wq, code), K, C, code), q.long())
    # word (l, j) of a tile holds column l % 16 and k = 32 j + 8 (l / 16) + 0..7
    ct, kt, byte, _ = ref.q4_places(K, C, code)
    word, lane = (byte // 4) % 4, byte // 16
    k, c = torch.arange(K)[:, None].expand(K, C), torch.arange(C)[None, :].expand(K, C)
    assert torch.equal(16 * ct + lane % 16, c) and torch.equal(128 * kt + 32 * word + 8 * (lane // 16) + k % 8, k)


def test_exact_codes():
    """Against rational numbers, at halfway points too."""
    from fractions import Fraction
    g = torch.Generator().manual_seed(5)
    S = torch.randn(6, 40, generator=g).to(torch.bfloat16)
    S[2] = (torch.arange(40) + 1).to(torch.bfloat16) * 0.25       # 448 w / max: halves among them
    S[3] = 0
    S[4, 0] = 28.0                                                # quotients 16 s: every other one a halfway point
    S[4, 1:] = (torch.arange(39) / 16 + 1).to(torch.bfloat16)
    gamma = (1 + 0.3 * torch.randn(40, generator=g)).to(torch.bfloat16)
    every = sorted({float(v) for v in torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()})
    for gm in (gamma, torch.ones_like(gamma)):
        got = ref.q8_codes(S, gm, 0)
        ties = 0
        for i in range(6):
            w = [Fraction(float(a)) * Fraction(float(b)) for a, b in zip(S[i], gm)]
            top = max(abs(v) for v in w)
            for j, v in enumerate(w):
                if top == 0:
                    assert float(got[i, j]) == 0
                    continue
                q = abs(v) * 448 / top
                near = min(abs(Fraction(e) - q) for e in every)
                best = [k for k, e in enumerate(every) if abs(Fraction(e) - q) == near]
                ties += len(best) > 1
                want = every[best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1]]
                assert abs(float(got[i, j])) == want and (want == 0 or float(got[i, j]) * float(v) > 0)
    assert ties > 10
