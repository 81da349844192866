"""Plain fp64 forms of the training operators (SwiGLU backward, layer norm, orthogonalised
update), with bounds on how far a kernel's outputs may be from them.

Rounding to a type moves a value by at most half a step, u = eps / 2 relative to it (bf16 2^-8,
fp32 2^-24); a sum of K terms in fp32, in any order, is off by at most about K 2^-23 of the
sum of the terms' magnitudes (2^-23, not 2^-24: the matrix instructions may truncate)."""
from __future__ import annotations

import torch

U_BF16, U_F32 = 2.0 ** -8, 2.0 ** -24
SUM = 2.0 ** -23            # per term of an fp32 sum, relative to the sum of magnitudes
NS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7


def d(t):
    return t.detach().double().cpu()


def swiglu_backward(X, Wg, Wu, Wd, dY, grad_f32=False):
    """{name: (gradient, bound)} in fp64."""
    X, Wg, Wu, Wd, dY = map(d, (X, Wg, Wu, Wd, dY))
    M, N = X.shape
    O, P = Wd.shape
    a, b, dh = X @ Wg, X @ Wu, dY @ Wd.t()
    s = torch.sigmoid(a)
    t = a * s
    h, da, db = t * b, dh * b * (s + t * (1 - s)), dh * t
    # fp32 sums of a, b and dh, and the activation: silu' <= 1.1 and |silu''| <= 0.5 in
    # magnitude; sigmoid from a hardware exp2 and reciprocal, relative error <= (|a| + 4) 2^-22
    ea, eb = N * SUM * (X.abs() @ Wg.abs()), N * SUM * (X.abs() @ Wu.abs())
    ed = P * SUM * (dY.abs() @ Wd.abs().t())
    es = (a.abs() + 4) * 2.0 ** -22
    act = 2 * es * (s + t.abs())           # error of silu'(a) from that of s
    eh = U_BF16 * h.abs() + 1.1 * ea * b.abs() + t.abs() * (eb + 2 * es * b.abs())
    eda = U_BF16 * da.abs() + 1.1 * (ed * b.abs() + dh.abs() * eb) + dh.abs() * b.abs() * (0.5 * ea + act)
    edb = U_BF16 * db.abs() + ed * t.abs() + dh.abs() * (1.1 * ea + 2 * es * t.abs())
    out = {}

    def put(name, value, err, mags, terms, u):
        # second-order terms: 1 %
        out[name] = (value, 1.01 * (err + terms * SUM * mags + u * value.abs()) + 1e-30)

    u = U_F32 if grad_f32 else U_BF16
    aX = X.abs()
    put("dX", da @ Wg.t() + db @ Wu.t(), eda @ Wg.abs().t() + edb @ Wu.abs().t(),
        da.abs() @ Wg.abs().t() + db.abs() @ Wu.abs().t(), 2 * O, U_BF16)
    put("dWg", X.t() @ da, aX.t() @ eda, aX.t() @ da.abs(), M, u)
    put("dWu", X.t() @ db, aX.t() @ edb, aX.t() @ db.abs(), M, u)
    put("dWd", h.t() @ dY, eh.t() @ dY.abs(), h.abs().t() @ dY.abs(), M, u)
    return out


# additions behind one value of a row sum: 8 per step of a lane (4 steps at most), 6 over the
# wave, 16 over the waves
LN_ADDS = 8 * 4 + 6 + 16


def layernorm_forward(X, gamma, beta, eps):
    u = U_BF16 if X.dtype == torch.bfloat16 else U_F32
    X, gamma, beta = map(d, (X, gamma, beta))
    mean = X.mean(1)
    c = X - mean[:, None]
    var = c.square().mean(1)
    rstd = (var + eps).pow(-0.5)
    y = c * rstd[:, None] * gamma + beta
    emean = LN_ADDS * SUM * X.abs().mean(1)
    ec = emean[:, None] + U_F32 * c.abs()
    evar = (2 * c.abs() * ec).mean(1) + ec.square().mean(1) + (LN_ADDS + 2) * SUM * var
    erstd = rstd * (0.5 * evar / (var + eps) + 4 * SUM)
    ey = gamma.abs() * (ec * rstd[:, None] + c.abs() * erstd[:, None]) + 4 * SUM * (y - beta).abs() \
        + (U_F32 + u) * y.abs()
    return {"Y": (y, 1.01 * ey + 1e-30), "mean": (mean, 1.01 * emean + 1e-30),
            "rstd": (rstd, 1.01 * erstd + 1e-30)}


def layernorm_backward(X, dY, gamma, mean, rstd):
    M, N = X.shape
    u = U_BF16 if X.dtype == torch.bfloat16 else U_F32
    X, dY, gamma, mean, rstd = map(d, (X, dY, gamma, mean, rstd))
    z = (X - mean[:, None]) * rstd[:, None]
    t = dY * gamma
    s1, s2 = t.mean(1, keepdim=True), (t * z).mean(1, keepdim=True)
    dx = rstd[:, None] * (t - s1 - z * s2)
    ez, et = 2 * U_F32 * z.abs(), U_F32 * t.abs()
    e1 = (et + LN_ADDS * SUM * t.abs()).mean(1, keepdim=True)
    e2 = (et * z.abs() + t.abs() * ez + LN_ADDS * SUM * (t * z).abs()).mean(1, keepdim=True)
    mags = t.abs() + s1.abs() + (z * s2).abs()
    edx = rstd[:, None] * (et + e1 + ez * s2.abs() + z.abs() * e2 + 4 * SUM * mags) + u * dx.abs()
    g = dY * z
    rows = M + 16    # terms of a column's sum
    return {"dX": (dx, 1.01 * edx + 1e-30),
            "dgamma": (g.sum(0), 1.01 * (rows * SUM * g.abs().sum(0) + (dY.abs() * ez).sum(0)) + 1e-30),
            "dbeta": (dY.sum(0), 1.01 * rows * SUM * dY.abs().sum(0) + 1e-30)}


def orthogonalize(G, steps=5):
    G = d(G)
    wide = G.shape[0] <= G.shape[1]
    X = G / (torch.linalg.vector_norm(G) + NS_EPS)
    X = X if wide else X.t()
    a, b, c = NS
    for _ in range(steps):
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X if wide else X.t()


# Relative error of an orthogonalised update (Frobenius norm).  The output's bf16 rounding: at
# most 2^-8 per element, spread evenly below that, so 2^-8 / sqrt 3 = 2.3e-3 in the mean.  A
# step's products take fp16 operands, each off by 2^-11 / sqrt 3 = 2.8e-4 in the mean: A's two
# are weighed by |b|, A^2's and the outer product's by 2 |c| + |b| in all, over a result of
# singular values 0.7 and more: 2.8e-4 sqrt 2 (4.8 + 2 * 2.03) / 0.7 = 5.0e-3 where the
# off-diagonals carried everything.  Singular values near 1 contract what earlier steps left.
# sqrt(2.3^2 + 5.0^2) = 5.5e-3; single elements: 8 times that of the matrix's rms, and their
# own rounding.
NS_REL = 5.5e-3


def check(got, ref, what):
    """Every output within its bound, element by element."""
    for name, (value, bound) in ref.items():
        g = d(got[name])
        assert g.shape == value.shape
        assert bool(torch.isfinite(g).all()), f"{what} {name}: not finite"
        over = (g - value).abs() / bound
        worst = float(over.max()) if over.numel() else 0.0
        print(f"  {what} {name}: worst error {worst:.3f} of its bound", flush=True)
        assert worst <= 1.0, f"{what} {name}: {worst:.3f} times its bound"


def check_orthogonalize(U, G, steps, what):
    ref, got = orthogonalize(G, steps), d(U)
    norm = float(torch.linalg.vector_norm(ref))
    rms = norm / ref.numel() ** 0.5
    rel = float(torch.linalg.vector_norm(got - ref)) / norm
    big = float(((got - ref).abs() - U_BF16 * ref.abs()).max()) / rms
    print(f"  {what}: relative error {rel:.2e} (bound {NS_REL:.1e}), largest {big:.2e} rms", flush=True)
    assert rel <= NS_REL and big <= 8 * NS_REL
