"""Plain fp64 forms of the operators around an expert sub-layer (RMS norm, dispatch and combine,
4-bit products), with bounds on how far a kernel's outputs may be from them.

Rounding to a type moves a value by at most half a step, u = eps / 2 relative to it (bf16 2^-8,
fp32 2^-24, e4m3 2^-4); a sum of K terms in fp32, in any order, is off by at most about K 2^-23 of
the sum of the terms' magnitudes (2^-23, not 2^-24: the matrix instructions may truncate)."""
from __future__ import annotations

import math

import torch

from training_ref import LN_ADDS, SUM, U_BF16, U_F32, check, d  # noqa: F401  (check: for the tests)

E4M3_MAX = 448.0
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)


def u_of(dtype):
    return U_BF16 if dtype == torch.bfloat16 else U_F32


# ---------------------------------------------------------------- RMS norm

def _norm(S, gamma, eps):
    """y before any rounding, rstd, and the relative error that fp32 may bring into each."""
    S, gamma = d(S), d(gamma)
    rstd = (S.square().mean(1) + eps).pow(-0.5)
    # squares and their sum: one rounding a square and the sum's, of nonnegative terms, halved by
    # the root; the mean's division, eps, root and reciprocal: 4 more
    e = 0.5 * (LN_ADDS + 2) * SUM + 4 * SUM
    return S * rstd[:, None] * gamma, rstd, e


def rmsnorm_forward(S, gamma, eps):
    """{name: (value, bound)} for the normed sum ``S`` as it was kept."""
    y, rstd, e = _norm(S, gamma, eps)
    return {"Y": (y, 1.01 * (e + 2 * U_F32 + u_of(S.dtype)) * y.abs() + 1e-38),
            "rstd": (rstd, 1.01 * e * rstd)}


def to_e4m3(v):
    """The nearest e4m3 number, ties to the even one, in fp64."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def check_q8(Q, scale, S, gamma, eps, group, what):
    """Scales within fp32's error, and every code that of a value within fp32's error of y / scale."""
    y, _, e = _norm(S, gamma, eps)
    M, N = y.shape
    g = group or N
    pad = torch.nn.functional.pad(y, (0, -N % g)).reshape(M, -1, g)
    want = pad.abs().amax(2).clamp(min=2.0 ** -100) / E4M3_MAX
    got = d(scale)
    assert got.shape == want.shape
    e += 3 * U_F32          # y's products, the scale's division
    off = float(((got - want).abs() / want).max()) if M else 0.0
    print(f"  {what}: scales off by {off:.2e} (bound {e:.2e})", flush=True)
    assert off <= 1.01 * e
    v = (pad / want[:, :, None]).reshape(M, -1)[:, :N]
    e = 2.02 * (e + 2 * U_F32)     # y's and the scale's errors, the reciprocal and the product
    a, b = to_e4m3(v * (1 - e)), to_e4m3(v * (1 + e))
    q = d(Q.cpu().float())
    bad = (q < torch.minimum(a, b)) | (q > torch.maximum(a, b))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} codes are not the nearest"


def q8_codes(S, gamma, group):
    """The codes of bf16 ``S`` and ``gamma`` by the definition, e4m3(448 w / max |w|) with w = s gamma and ties
    to the even code: every number that decides between two codes is exact in fp64 (w: 16 bits, halfway points
    times max |w|: 21 bits)."""
    w = d(S) * d(gamma)
    M, N = w.shape
    pad = torch.nn.functional.pad(w, (0, -N % (group or N))).reshape(M, -1, group or N)
    top = pad.abs().amax(2, keepdim=True)
    mag = pad.abs() * E4M3_MAX
    v = torch.where(top > 0, mag / top, 0.0)
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    k = torch.floor(v / step)
    over = mag - (k + 0.5) * step * top
    q = torch.where(top > 0, (k + ((over > 0) | ((over == 0) & (k % 2 == 1))).double()) * step, 0.0)
    return (q * pad.sign()).reshape(M, -1)[:, :N]


def rmsnorm_backward(S, dY, gamma, rstd, dS=None):
    M, N = S.shape
    u = u_of(S.dtype)
    S, dY, gamma, rstd = map(d, (S, dY, gamma, rstd))
    ds = torch.zeros_like(S) if dS is None else d(dS)
    r = rstd[:, None]
    z, t = S * r, dY * gamma
    s2 = (t * z).mean(1, keepdim=True)
    dx = r * (t - z * s2) + ds
    ez, et = U_F32 * z.abs(), U_F32 * t.abs()
    e2 = (et * z.abs() + t.abs() * ez + (LN_ADDS + 2) * SUM * (t * z).abs()).mean(1, keepdim=True)
    mags = t.abs() + (z * s2).abs()
    edx = r * (et + ez * s2.abs() + z.abs() * e2 + 3 * SUM * mags) + SUM * (ds.abs() + dx.abs()) + u * dx.abs()
    g = dY * z
    return {"dX": (dx, 1.01 * edx + 1e-38),
            "dgamma": (g.sum(0), 1.01 * ((M + 16) * SUM * g.abs().sum(0) + (dY.abs() * ez).sum(0)) + 1e-38)}


# ---------------------------------------------------------------- rows by expert and back

def sort(ids, E):
    """(positions, offsets, entries of the kept places) of expert ids, entry by entry."""
    flat = ids.cpu().reshape(-1).tolist()
    lists = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(i)
    order = [i for x in lists for i in x]
    pos = [-1] * len(flat)
    for p, i in enumerate(order):
        pos[i] = p
    off = [0]
    for x in lists:
        off.append(off[-1] + len(x))
    return (torch.tensor(pos, dtype=torch.int32).reshape(ids.shape), torch.tensor(off, dtype=torch.int32),
            torch.tensor(order, dtype=torch.int32))


def _taken(rows, pos):
    """rows[pos] in fp64, zeros for dropped entries: M x k x N."""
    rows, pos = d(rows), pos.cpu().long()
    kept = (pos >= 0) & (pos < rows.shape[0])
    if rows.shape[0] == 0:
        return torch.zeros(*pos.shape, rows.shape[1], dtype=torch.float64), kept
    return torch.where(kept[:, :, None], rows[torch.where(kept, pos, 0)], 0.0), kept


def combine(rows, pos, w=None, R=None):
    u = u_of(rows.dtype)
    v, kept = _taken(rows, pos)
    w = torch.ones_like(kept, dtype=torch.float64) if w is None else torch.where(kept, d(w), 0.0)
    terms = v * w[:, :, None]
    r = d(R) if R is not None else torch.zeros_like(v[:, 0])
    y = terms.sum(1) + r
    mags = terms.abs().sum(1) + r.abs()
    return {"Y": (y, 1.01 * ((pos.shape[1] + 1) * U_F32 * mags + u * y.abs()) + 1e-38)}


def combine_backward(dY, rows, pos, w=None):
    """dw with its bound, and the expected rows of dYs by entry (M x k x N) with theirs."""
    u = u_of(dY.dtype)
    dy = d(dY)[:, None, :]
    v, kept = _taken(rows, pos)
    w = torch.ones_like(kept, dtype=torch.float64) if w is None else torch.where(kept, d(w), 0.0)
    N = dy.shape[2]
    W = 4 if N > 1024 else 2 if N > 512 else 1
    adds = 8 * -(-N // (512 * W)) + 6 + W
    drow = dy * w[:, :, None]
    return {"dw": ((v * dy).sum(2), 1.01 * (adds + 1) * SUM * (v * dy).abs().sum(2) + 1e-38)}, \
        (drow, 1.01 * (U_F32 + u) * drow.abs() + 1e-38, kept)


def route_backward(ids, w, dw, E):
    M, k = ids.shape
    w, dw, ids = d(w), d(dw), ids.cpu().long()
    mean = (w * dw).sum(1, keepdim=True)
    part = w * (dw - mean)
    mags = w * (dw.abs() + (w * dw).abs().sum(1, keepdim=True))
    out = torch.zeros(M, E + 1, dtype=torch.float64)
    big = torch.zeros(M, E + 1, dtype=torch.float64)
    at = torch.where((ids >= 0) & (ids < E), ids, E)
    out.scatter_add_(1, at, part)
    big.scatter_add_(1, at, mags)
    return {"dlogits": (out[:, :E], 1.01 * (2 * k + 3) * U_F32 * big[:, :E] + 1e-38)}


# ---------------------------------------------------------------- 4-bit products

def q4_places(K, C, code):
    """Where k, c's code lies: (column tile, k tile, byte, upper half), each K x C."""
    k, c = torch.arange(K)[:, None], torch.arange(C)[None, :]
    lane, word, e = 16 * ((k % 32) // 8) + c % 16, (k % 128) // 32, k % 8
    nibble = e if code == "e2m1" else e // 2 + 4 * (e % 2)
    byte = 16 * lane + 4 * word + nibble // 2
    return [x.expand(K, C) for x in (c // 16, k // 128, byte, nibble % 2)]


def q4_codes(Wq, K, C, code):
    ct, kt, byte, upper = q4_places(K, C, code)
    b = Wq.cpu().long()[ct, kt, byte]
    return torch.where(upper == 1, b // 16, b % 16)


def q4_pack(q, Wq, code):
    """Codes (K x C) into a CPU buffer of the packed layout."""
    K, C = q.shape
    ct, kt, byte, upper = q4_places(K, C, code)
    for half in (0, 1):
        on = upper == half
        old = Wq[ct[on], kt[on], byte[on]].long()
        new = q[on].long()
        Wq[ct[on], kt[on], byte[on]] = ((old & 0x0F) | (new << 4) if half else (old & 0xF0) | new).to(torch.uint8)
    return Wq


def q4_groups(s, K, C):
    """Packed scales (or zeros) as K x C values in fp64."""
    k, c = torch.arange(K)[:, None], torch.arange(C)[None, :]
    per = s.shape[-1]
    return d(s)[c // 16, k // 128, c % 16, (k % 128) // (128 // per)]


def q4_weights(Wq, scale, zero, K, C, code):
    """(W, magnitude that a weight's integer form passes through), K x C, fp64."""
    q = q4_codes(Wq, K, C, code)
    s = q4_groups(scale, K, C)
    if code == "e2m1":
        w = E2M1[q] * s
        return w, w.abs()
    z = torch.full_like(s, 8.0) if zero is None else q4_groups(zero, K, C)
    return (q.double() - z) * s, (16.0 + q + (16.0 + z).abs()) * s.abs()


def q4_product(X, Wq, scale, zero, C, code):
    """(a, bound of its fp32 sums): sums of up to 128 terms in a group, then of the groups, the
    waves' sums (16), and the correction's product."""
    X = d(X)
    K = X.shape[1]
    w, m = q4_weights(Wq, scale, zero, K, C, code)
    terms = 128 + 4 * -(-K // 128) + 16 + 4
    return X @ w, terms * SUM * (X.abs() @ m)


def q4_matvec(X, Wq, scale, zero, bias, act, C, code):
    a, ea = q4_product(X, Wq, scale, zero, C, code)
    if bias is not None:
        a = a + d(bias)
        ea = ea + U_F32 * a.abs()
    if act == "relu":
        y, ey = a.clamp(min=0), ea
    elif act == "gelu_tanh":
        t = 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
        y = a * torch.sigmoid(t)
        # |gelu'| <= 1.13; sigmoid from a hardware exp2 and reciprocal
        ey = 1.13 * ea + y.abs() * (t.abs() + 4) * 2.0 ** -22
    else:
        y, ey = a, ea
    return {"Y": (y, 1.01 * (ey + U_BF16 * y.abs()) + 1e-38)}


def q4_swiglu(X, Wg, sg, zg, Wu, su, zu, C, code):
    a, ea = q4_product(X, Wg, sg, zg, C, code)
    b, eb = q4_product(X, Wu, su, zu, C, code)
    t = a * torch.sigmoid(a)
    h = t * b
    # |silu'| <= 1.1; sigmoid from a hardware exp2 and reciprocal
    eh = 1.1 * ea * b.abs() + (t.abs() + 1.1 * ea) * eb + h.abs() * ((a.abs() + 4) * 2.0 ** -22 + U_F32)
    return {"H": (h, 1.01 * (eh + U_BF16 * h.abs()) + 1e-38)}
