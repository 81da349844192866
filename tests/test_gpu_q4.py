"""GPU parity of the products with 4-bit weights, of the quantiser and of the packed layout against
their fp64 forms, within the bounds of sublayer_ref."""
from __future__ import annotations

import pytest

import transformer_ffn_fusion_amd as ffn

import sublayer_ref as ref

pytestmark = pytest.mark.gpu
SHAPES = [(8, 8), (64, 16), (128, 16), (136, 24), (264, 4104), (1992, 1400), (2056, 200), (4096, 48), (4104, 264),
          (520, 32)]     # K, C
KINDS = [("int4", 128, False), ("int4", 64, True), ("int4", 32, False), ("int4", 128, True), ("e2m1", 32, False),
         ("e2m1", 64, False), ("e2m1", 128, False)]


def weight(K, C, kind, seed, experts=None):
    """Random codes, scales of either sign and zero points; NaN in scales that nothing may look at."""
    import torch
    code, group, zero = kind
    g = torch.Generator().manual_seed(seed)
    Wq, s, z = ffn.ffn_q4_empty(K, C, group, zero, experts, device="cpu")
    Wq = torch.randint(0, 256, Wq.shape, generator=g, dtype=torch.uint8)
    s = (torch.exp(0.3 * torch.randn(s.shape, generator=g)) / (4 * K ** 0.5)).to(torch.bfloat16)
    s = torch.where(torch.rand(s.shape, generator=g) < 0.1, -s, s)
    if zero:
        z = torch.randint(0, 16, z.shape, generator=g).to(torch.bfloat16)
    per, kt = 128 // group, -(-K // 128)
    for p in range(per):
        if (kt - 1) * 128 + p * group >= K:
            s[..., kt - 1, :, p] = float("nan")
            if zero:
                z[..., kt - 1, :, p] = float("nan")
    if C % 16:
        s[..., -1, :, C % 16:, :] = float("nan")
    return Wq.cuda(), s.cuda(), None if z is None else z.cuda()


def inputs(M, K, seed):
    import torch
    return torch.randn(M, K, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def empty(M, C):
    import torch
    return torch.full((M, C), float("nan"), dtype=torch.bfloat16, device="cuda")


def cpu(w):
    return [None if t is None else t.cpu() for t in w]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES)
def test_matvec(shape, kind):
    import torch
    K, C = shape
    code = kind[0]
    print(f"case 4-bit product {shape} {kind}", flush=True)
    w = weight(K, C, kind, seed=K + C)
    bias = torch.randn(C, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    for M, act, b in ((1, "none", None), (5, "gelu_tanh", bias), (16, "relu", bias), (13, "none", bias)):
        X, Y = inputs(M, K, M), empty(M, C)
        ffn.ffn_q4_matvec(X, w[0], w[1], Y, zero=w[2], bias=b, act=act, code=code)
        ref.check({"Y": Y}, ref.q4_matvec(X, *cpu(w), b, act, C, code), f"{shape} {kind} {M} rows")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(136, 8712), (648, 12296), (136, 25608), (264, 28664), (72, 40)])
def test_wide_matrices(shape, kind):
    """Several column tiles a wave, the last of them past the matrix."""
    K, C = shape
    print(f"case wide 4-bit product {shape} {kind}", flush=True)
    w = weight(K, C, kind, seed=K + C)
    for M in (1, 6, 16):
        X, Y = inputs(M, K, M), empty(M, C)
        ffn.ffn_q4_matvec(X, w[0], w[1], Y, zero=w[2], code=kind[0])
        ref.check({"Y": Y}, ref.q4_matvec(X, *cpu(w), None, "none", C, kind[0]), f"{shape} {kind} {M} rows")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES)
def test_swiglu(shape, kind):
    K, C = shape
    print(f"case 4-bit gated pair {shape} {kind}", flush=True)
    wg, wu = weight(K, C, kind, 1), weight(K, C, kind, 2)
    for M in (1, 16, 7):
        X, H = inputs(M, K, M), empty(M, C)
        ffn.ffn_q4_swiglu(X, wg[0], wg[1], wu[0], wu[1], H, zero_g=wg[2], zero_u=wu[2], code=kind[0])
        ref.check({"H": H}, ref.q4_swiglu(X, *cpu(wg), *cpu(wu), C, kind[0]), f"{shape} {kind} {M} rows")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(136, 8184), (136, 8200), (264, 20488), (1032, 10248)])
def test_wide(shape, kind):
    """Around the widths at which a wave takes two column tiles and a workgroup four waves."""
    K, C = shape
    print(f"case 4-bit, wide {shape} {kind}", flush=True)
    wg, wu = weight(K, C, kind, 1), weight(K, C, kind, 2)
    for M in (3, 6, 12):      # one, two and four loads of X per tile
        X, Y, H = inputs(M, K, M), empty(M, C), empty(M, C)
        ffn.ffn_q4_matvec(X, wg[0], wg[1], Y, zero=wg[2], code=kind[0])
        ref.check({"Y": Y}, ref.q4_matvec(X, *cpu(wg), None, "none", C, kind[0]), f"{shape} {kind} {M} rows")
        ffn.ffn_q4_swiglu(X, wg[0], wg[1], wu[0], wu[1], H, zero_g=wg[2], zero_u=wu[2], code=kind[0])
        ref.check({"H": H}, ref.q4_swiglu(X, *cpu(wg), *cpu(wu), C, kind[0]), f"{shape} {kind} {M} rows")


# rows per expert: none, one, a full tile, more than one tile, more than two
LISTS = [[1], [0, 0, 3, 0], [1, 0, 16, 17, 2], [5, 40, 0, 33, 1, 0, 16], [0, 0, 0], [i % 7 for i in range(200)]]


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[1], KINDS[4]])
@pytest.mark.parametrize("counts", LISTS)
@pytest.mark.parametrize("shape", [(136, 24), (1032, 200), (512, 64)])
def test_experts(shape, counts, kind):
    import torch
    K, C = shape
    code, E = kind[0], len(counts)
    print(f"case 4-bit experts {shape} {counts} {kind}", flush=True)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    n = int(off[-1])
    X, Y, H = inputs(n + 3, K, 4), empty(n + 3, C), empty(n + 3, C)     # three rows of no expert
    wg, wu = weight(K, C, kind, 1, E), weight(K, C, kind, 2, E)
    bias = torch.randn(E, C, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    Y.fill_(7.0)
    H.fill_(7.0)
    ffn.moe_q4_matvec(X, off, wg[0], wg[1], Y, zero=wg[2], bias=bias, act="gelu_tanh", code=code)
    ffn.moe_q4_swiglu(X, off, wg[0], wg[1], wu[0], wu[1], H, zero_g=wg[2], zero_u=wu[2], code=code)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        g, u = ([None if t is None else t[e].cpu() for t in w] for w in (wg, wu))
        ref.check({"Y": Y[lo:hi]}, ref.q4_matvec(X[lo:hi], *g, bias[e], "gelu_tanh", C, code), f"expert {e}")
        ref.check({"H": H[lo:hi]}, ref.q4_swiglu(X[lo:hi], *g, *u, C, code), f"expert {e}")
    assert bool((Y[n:] == 7.0).all()) and bool((H[n:] == 7.0).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts", [[32, 4, 0, 64, 9], [18, 33, 5, 8, 17, 31], [4093]])
@pytest.mark.parametrize("shape", [(264, 72), (136, 4104)])
def test_experts_of_many_rows(shape, counts, kind):
    """Lists of more than ten rows on average: up to 32 at once."""
    if len(counts) == 1 and shape[1] > 100:
        counts = [100]
    test_experts(shape, counts, kind)


def test_offsets_outside_the_rows():
    """Offsets that decrease or leave the rows: every row that is written belongs to the list as it is
    kept inside the rows."""
    import torch
    K, C, kind = 136, 24, KINDS[0]
    w = weight(K, C, kind, 1, 3)
    X, Y = inputs(20, K, 4), empty(20, C)
    Y.fill_(7.0)
    off = torch.tensor([-5, 4, 2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")    # 0..4, none, 2..20
    ffn.moe_q4_matvec(X, off[:2].clone(), w[0][:1].contiguous(), w[1][:1].contiguous(), Y)
    ref.check({"Y": Y[:4]}, ref.q4_matvec(X[:4], w[0][0].cpu(), w[1][0].cpu(), None, None, "none", C, "int4"), "first")
    assert bool((Y[4:] == 7.0).all())
    Z = empty(20, C)
    Z.fill_(7.0)
    ffn.moe_q4_matvec(X, off[1:].clone(), w[0][1:].contiguous(), w[1][1:].contiguous(), Z)
    ref.check({"Y": Z[2:]}, ref.q4_matvec(X[2:], w[0][2].cpu(), w[1][2].cpu(), None, None, "none", C, "int4"), "last")
    assert bool((Z[:2] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(8, 8), (136, 24), (300 * 8, 72), (520, 200)])
def test_quantize(shape, kind, dtype):
    """Scales, zero points and codes are what the same fp32 steps give on the CPU."""
    import torch
    K, C = shape
    code, group, zero = kind
    print(f"case quantise {shape} {kind} {dtype}", flush=True)
    g = torch.Generator().manual_seed(K)
    W = (torch.randn(K, C, generator=g) * torch.exp(torch.randn(1, C, generator=g))).to(getattr(torch, dtype))
    W[:, 1] = 0
    W[:, 2] = W[:, 2].abs()
    W[:, 3] *= 2.0 ** -120
    Wq, s, z = ffn.ffn_q4_empty(K, C, group, zero)
    ffn.ffn_q4_quantize(W.cuda(), Wq, s, zero=z, code=code)
    G = -(-K // group)
    w = torch.nn.functional.pad(W.float(), (0, 0, 0, G * group - K)).reshape(G, group, C)
    lo, hi = w.amin(1).clamp(max=0), w.amax(1).clamp(min=0)
    top = torch.maximum(-lo, hi)
    want = top / 6 if code == "e2m1" else (hi - lo) / 15 if zero else top / 7
    want = torch.where(top < 2.0 ** -100, 0.0, want).to(torch.bfloat16).float()
    got = ref.q4_groups(s, K, C)[::group].float()
    assert torch.equal(got, want)
    wz = torch.full_like(want, 8.0)
    if zero:
        wz = torch.where(want > 0, torch.round(-lo / want).clamp(0, 15), 8.0)
        assert torch.equal(ref.q4_groups(z, K, C)[::group].float(), wz)
    v = torch.where(want[:, None] > 0, w / want[:, None], 0.0)
    q = ref.q4_codes(Wq, K, C, code)
    if code == "e2m1":
        v = v.reshape(-1, C)[:K].double()
        near = (ref.E2M1[q] - v).abs()
        best = (ref.E2M1[None, None, :8] - v.abs()[:, :, None]).abs().amin(2)
        assert torch.equal(near, best) and bool((ref.E2M1[q] * v >= 0).all())
        tie = ((ref.E2M1[None, None, :8] - v.abs()[:, :, None]).abs() == best[:, :, None]).sum(2) > 1
        assert not bool((q[tie] & 1).any())
    else:
        want_q = (torch.round(v) + wz[:, None]).clamp(0, 15).reshape(-1, C)[:K]
        assert torch.equal(q.float(), want_q)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_quantize_of_the_largest_values(dtype):
    """A group from -2^127 to 2^127 is finite, though its range is not: the scale is 2^128 / 15."""
    import torch
    K, C = 136, 24
    W = (torch.rand(K, C, generator=torch.Generator().manual_seed(1)) - 0.5).mul(2.0 ** 126).to(getattr(torch, dtype))
    W[0], W[1] = 2.0 ** 127, -2.0 ** 127
    Wq, s, z = ffn.ffn_q4_empty(K, C, 128, True)
    ffn.ffn_q4_quantize(W.cuda(), Wq, s, zero=z)
    want = torch.tensor(2.0 ** 128 / 15, dtype=torch.float64).to(torch.bfloat16).double()
    assert torch.equal(ref.q4_groups(s, K, C)[:128], want.expand(128, C))
    zero = torch.round(2.0 ** 127 / want.float()).double()
    assert torch.equal(ref.q4_groups(z, K, C)[:128], zero.expand(128, C))
    back = ref.q4_weights(Wq, s, z, K, C, "int4")[0][:128]
    assert bool(((back - W[:128].double()).abs() <= want).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(8, 8), (136, 24), (520, 200)])
def test_pack(shape, kind):
    import torch
    K, C = shape
    code, group, zero = kind
    g = torch.Generator().manual_seed(K)
    q = torch.randint(0, 16, (K, C), generator=g).to(torch.uint8)
    G = -(-K // group)
    sin = torch.randn(G, C, generator=g).to(torch.bfloat16)
    zin = torch.randint(0, 16, (G, C), generator=g).to(torch.bfloat16) if zero else None
    Wq, s, z = ffn.ffn_q4_empty(K, C, group, zero)
    Wq.fill_(0xFF)
    ffn.ffn_q4_pack(q.cuda() | 0xF0, sin.cuda(), Wq, s, zero_in=None if zin is None else zin.cuda(), zero=z, code=code)
    assert torch.equal(ref.q4_codes(Wq, K, C, code), q.long())
    k = torch.arange(K) // group
    assert torch.equal(ref.q4_groups(s, K, C), sin.double()[k])
    if zero:
        assert torch.equal(ref.q4_groups(z, K, C), zin.double()[k])
    want = ref.q4_pack(q, torch.zeros_like(Wq).cpu(), code)
    assert torch.equal(ref.q4_codes(want, K, C, code), q.long())


def test_rows_with_nan_and_infinity_stay_alone():
    import torch
    K, C = 264, 40
    for kind in (KINDS[1], KINDS[4]):
        w = weight(K, C, kind, 3)
        X, Y, Z = inputs(9, K, 1), empty(9, C), empty(9, C)
        ffn.ffn_q4_matvec(X, w[0], w[1], Y, zero=w[2], code=kind[0])
        X[2, 5], X[8, 263] = float("nan"), float("inf")
        ffn.ffn_q4_matvec(X, w[0], w[1], Z, zero=w[2], code=kind[0])
        keep = [0, 1, 3, 4, 5, 6, 7]
        assert torch.equal(Y[keep], Z[keep])
        assert bool(torch.isnan(Z[2].float()).all()) and not bool(torch.isfinite(Z[8].float()).any())


def test_no_rows_and_repeated_calls():
    import torch
    K, C = 520, 72
    w = weight(K, C, KINDS[0], 3)
    ffn.ffn_q4_matvec(inputs(0, K, 1), w[0], w[1], empty(0, C))
    X, Y = inputs(16, K, 1), empty(16, C)
    ffn.ffn_q4_matvec(X, w[0], w[1], Y)
    for _ in range(20):
        Z = empty(16, C)
        ffn.ffn_q4_matvec(X, w[0], w[1], Z)
        assert torch.equal(Y, Z)
    for m in range(1, 16):         # a row's result does not depend on the rows beside it
        Z = empty(m, C)
        ffn.ffn_q4_matvec(X[:m], w[0], w[1], Z)
        assert torch.equal(Y[:m], Z)


@pytest.mark.parametrize("big", [1e2, 1e4, 1e6, 1e8])
@pytest.mark.parametrize("kind", KINDS[:4])
def test_a_channel_much_larger_than_the_rest(kind, big):
    """Its codes are the zero points, so that it adds nothing: what it leaves is within the stated 2^-10 |x| s."""
    import torch
    _, group, zero = kind
    K, C, M, at = 520, 72, 5, 133
    print(f"case 4-bit, a channel of {big:.0e} {kind}", flush=True)
    g = torch.Generator().manual_seed(int(big))
    G = -(-K // group)
    q = torch.randint(0, 16, (K, C), generator=g).to(torch.uint8)
    z = torch.randint(3, 13, (G, C), generator=g) if zero else torch.full((G, C), 8)
    q[at] = z[at // group].to(torch.uint8)
    s = (0.5 + torch.rand(G, C, generator=g)).to(torch.bfloat16)
    Wq, sp, zp = ffn.ffn_q4_empty(K, C, group, zero)
    ffn.ffn_q4_pack(q.cuda(), s.cuda(), Wq, sp, zero_in=z.to(torch.bfloat16).cuda() if zero else None, zero=zp)
    X, Y = inputs(M, K, 3), empty(M, C)
    X[:, at] = big * torch.tensor([1.0, -1.0, 0.5, 1.0, -0.5], device="cuda")
    ffn.ffn_q4_matvec(X, Wq, sp, Y, zero=zp)
    of = torch.arange(K) // group
    w = (q.double() - z.double()[of]) * s.double()[of]
    x = X.cpu().double()
    y = x @ w
    # of the other channels (|x| <= 5) the same, per group; then the sum of the groups and the rounding
    top = s.double().amax(0)
    off = (Y.cpu().double() - y).abs() - 2.0 ** -10 * (x[:, at:at + 1].abs() * s.double()[at // group] + 5 * G * top)
    off -= 1.01 * ref.U_BF16 * y.abs() + 200 * ref.SUM * (x.abs() @ w.abs())
    print(f"  beyond the bound by {float(off.max()):.3e}", flush=True)
    assert bool((off <= 0).all())
    ref.check({"Y": Y}, ref.q4_matvec(X, *cpu((Wq, sp, zp)), None, "none", C, "int4"), f"{kind} {big:.0e}")


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh"])
@pytest.mark.parametrize("kind", [KINDS[1], KINDS[2], KINDS[4]])
def test_bad_rows_are_seen_through_the_activation(kind, act):
    """NaN, an infinity and sums past fp32 give NaN or infinity; of e2m1, ReLU makes 0 of a negative infinity."""
    import torch
    K, C, E = 264, 40, 2
    w = weight(K, C, kind, 3, E)
    X, Y, Z = inputs(9, K, 1), empty(9, C), empty(9, C)
    off = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    ffn.moe_q4_matvec(X, off, w[0], w[1], Y, zero=w[2], act=act, code=kind[0])
    X[2, 5], X[5, 7], X[8, 263], X[6, 200:203] = float("nan"), float("-inf"), float("inf"), 3e38
    ffn.moe_q4_matvec(X, off, w[0], w[1], Z, zero=w[2], act=act, code=kind[0])
    keep = [0, 1, 3, 4, 7]
    assert torch.equal(Y[keep], Z[keep])
    assert bool(torch.isnan(Z[2].float()).all())
    if kind[0] == "int4":
        assert not bool(torch.isfinite(Z[[5, 6, 8]].float()).any())
    elif act == "none":
        assert not bool(torch.isfinite(Z[[5, 8]].float()).any())
    elif act == "relu":      # a sum of either sign, or NaN where a code is 0
        z, q = Z[[5, 8]].float(), ref.q4_codes(w[0][1], K, C, "e2m1")
        assert bool(((z == 0) | ~torch.isfinite(z)).all())
        assert bool(torch.isnan(z.cpu()[0][(q[7] & 7) == 0]).all())


def check_tiles(got, want, w, X, tiles, C, what):
    """Columns of some column tiles alone: ``want(X, *weights, columns)`` of the weights cut to them."""
    import torch
    at = torch.tensor(tiles)
    col = (16 * at[:, None] + torch.arange(16)).reshape(-1)
    real = col < C
    name, (y, bound) = next(iter(want(X, *[[None if t is None else t.cpu()[at] for t in v] for v in w], 16 * len(tiles)).items()))
    ref.check({name: got[:, col[real].cuda()]}, {name: (y[:, real], bound[:, real])}, what)


def some_tiles(C):
    """The first and last column tiles, and some between."""
    n = -(-C // 16)
    return sorted({*range(min(n, 9)), *range(max(0, n - 9), n), *range(0, n, max(1, n // 12))})


def matvec(code, act="none"):
    return lambda X, w, C: ref.q4_matvec(X, *w, None, act, C, code)


def swiglu(code):
    return lambda X, wg, wu, C: ref.q4_swiglu(X, *wg, *wu, C, code)


@pytest.mark.parametrize("kind", KINDS[:4] + [("int4", 64, False), ("int4", 32, True)])
@pytest.mark.parametrize("K,C", [(2696, 25608)])
def test_four_column_tiles_over_many_k_tiles(K, C, kind):
    """22 k tiles between four waves: a wave's loads and products turn over five times."""
    print(f"case 4-bit, four column tiles {K} x {C} {kind}", flush=True)
    w = weight(K, C, kind, seed=K + C)
    for M in (1, 6, 16):
        X, Y = inputs(M, K, M), empty(M, C)
        ffn.ffn_q4_matvec(X, w[0], w[1], Y, zero=w[2], code=kind[0])
        assert not bool(Y.isnan().any())
        check_tiles(Y, matvec(kind[0]), [w], X, some_tiles(C), C, f"{kind} {M} rows")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K", [1032, 4104])
def test_around_the_rules_of_tiles_and_waves(K, kind):
    """511, 512 and 513 column tiles: one a wave, two in workgroups of eight waves, two in workgroups of four;
    the gated pair at 256 and 257: eight waves, four.  9 and 33 k tiles."""
    print(f"case 4-bit, around the rules, K = {K} {kind}", flush=True)
    for C in (8176, 8192, 8200):
        w = weight(K, C, kind, seed=K + C)
        for M in (1, 6, 16):
            X, Y = inputs(M, K, M), empty(M, C)
            ffn.ffn_q4_matvec(X, w[0], w[1], Y, zero=w[2], code=kind[0])
            assert not bool(Y.isnan().any())
            check_tiles(Y, matvec(kind[0]), [w], X, some_tiles(C), C, f"{C} columns, {M} rows")
    for C in (4096, 4104):
        wg, wu = weight(K, C, kind, 1), weight(K, C, kind, 2)
        for M in (1, 6, 16):
            X, H = inputs(M, K, M), empty(M, C)
            ffn.ffn_q4_swiglu(X, wg[0], wg[1], wu[0], wu[1], H, zero_g=wg[2], zero_u=wu[2], code=kind[0])
            assert not bool(H.isnan().any())
            check_tiles(H, swiglu(kind[0]), [wg, wu], X, some_tiles(C), C, f"pair of {C} columns, {M} rows")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts", [[32, 4, 0, 64, 9], [3, 0, 16, 1, 9]])
@pytest.mark.parametrize("shape", [(2696, 72), (5256, 72), (2696, 4104)])
def test_experts_over_many_k_tiles(shape, counts, kind):
    """Lists of up to 32 and of up to 16 rows at once, 22 k tiles between eight and four waves, 42 between eight."""
    import torch
    K, C = shape
    code, E = kind[0], len(counts)
    print(f"case 4-bit experts over many k tiles {shape} {counts} {kind}", flush=True)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    n = int(off[-1])
    X, Y, H = inputs(n + 3, K, 4), empty(n + 3, C), empty(n + 3, C)     # three rows of no expert
    wg, wu = weight(K, C, kind, 1, E), weight(K, C, kind, 2, E)
    Y.fill_(7.0)
    H.fill_(7.0)
    ffn.moe_q4_matvec(X, off, wg[0], wg[1], Y, zero=wg[2], code=code)
    ffn.moe_q4_swiglu(X, off, wg[0], wg[1], wu[0], wu[1], H, zero_g=wg[2], zero_u=wu[2], code=code)
    assert not bool(Y.isnan().any()) and not bool(H.isnan().any())
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        g, u = ([None if t is None else t[e] for t in w] for w in (wg, wu))
        check_tiles(Y[lo:hi], matvec(code), [g], X[lo:hi], some_tiles(C), C, f"expert {e}")
        check_tiles(H[lo:hi], swiglu(code), [g, u], X[lo:hi], some_tiles(C), C, f"expert {e}")
    assert bool((Y[n:] == 7.0).all()) and bool((H[n:] == 7.0).all())
