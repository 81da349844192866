"""GPU parity of the dispatch of tokens to experts, the combine, their gradients and the routing's
gradient: the sort and the copies bit for bit, sums within the bounds of sublayer_ref."""
from __future__ import annotations

import pytest

import transformer_ffn_fusion_amd as ffn

import sublayer_ref as ref

pytestmark = pytest.mark.gpu
# (M, N, E, k): one token; few tokens; around 1024, 2048 and 12288 entries and 1024 tokens, where the
# kernels change; many entries, more than one turn of a sort workgroup; rows of every width; every k
CASES = [(1, 8, 1, 1), (1, 4096, 8, 2), (16, 4096, 8, 2), (3, 72, 5, 5), (128, 24, 256, 8), (341, 136, 24, 3),
         (342, 136, 24, 3), (513, 264, 7, 2), (1013, 2056, 64, 6), (257, 8200, 100, 4), (4099, 16, 33, 7),
         (40000, 8, 256, 8), (140001, 8, 3, 2), (999, 56, 9, 4), (2001, 256, 16, 8),
         (1024, 136, 24, 2), (1025, 136, 24, 1), (683, 64, 256, 3), (256, 4104, 8, 8), (1536, 136, 16, 8), (1537, 72, 16, 8), (12288, 24, 200, 1)]


def route(M, E, k, seed, drop=0.2):
    import torch
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(M, E, generator=g) + torch.randn(E, generator=g)
    top, ids = logits.topk(k, dim=1)
    ids[torch.rand(M, k, generator=g) < drop] = -1
    return ids.to(torch.int32).cuda(), torch.softmax(top, 1).cuda()


def rows(M, N, dtype, seed):
    import torch
    x = torch.randn(M, N, generator=torch.Generator().manual_seed(seed))
    return (100 * x).clamp(-448, 448).to(dtype).cuda() if dtype == torch.float8_e4m3fn else x.to(dtype).cuda()


def dispatch(X, ids, E, scale=None, ws=None):
    import torch
    M, k = ids.shape
    o = dict(Xs=torch.full((M * k, X.shape[1]), 7.0, device="cuda").to(X.dtype),
             off=torch.full((E + 1,), -9, dtype=torch.int32, device="cuda"),
             entries=torch.full((M * k,), -9, dtype=torch.int32, device="cuda"),
             pos=torch.full((M, k), -9, dtype=torch.int32, device="cuda"),
             scale=None if scale is None else torch.full((M * k, scale.shape[1]), 7.0, device="cuda"))
    ffn.moe_dispatch(X, ids, o["Xs"], o["off"], o["entries"], o["pos"], scale=scale, scale_sorted=o["scale"], ws=ws)
    torch.cuda.synchronize()
    return o


def check_dispatch(o, X, ids, E, scale=None):
    import torch
    k = ids.shape[1]
    pos, off, entries = ref.sort(ids, E)
    n = entries.numel()
    assert torch.equal(o["off"].cpu(), off) and torch.equal(o["pos"].cpu(), pos)
    assert torch.equal(o["entries"][:n].cpu(), entries) and bool((o["entries"][n:] == -9).all())
    bits = torch.int32 if X.dtype == torch.float32 else torch.int16 if X.dtype == torch.bfloat16 else torch.uint8
    got, src = o["Xs"].view(bits), X.view(bits)
    token = (entries // k).long().cuda()
    assert torch.equal(got[:n], src[token])
    assert bool((o["Xs"][n:].float() == 7.0).all()), "rows behind the last kept entry"
    if scale is not None:
        assert torch.equal(o["scale"][:n], scale[token]) and bool((o["scale"][n:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bfloat16", "float32", "float8_e4m3fn"])
@pytest.mark.parametrize("case", CASES)
def test_dispatch(case, dtype):
    import torch
    M, N, E, k = case
    print(f"case dispatch {case} {dtype}", flush=True)
    ids, _ = route(M, E, k, seed=M + N)
    X = rows(M, N, getattr(torch, dtype), seed=M)
    check_dispatch(dispatch(X, ids, E), X, ids, E)
    scale = torch.rand(M, -(-N // 128), device="cuda")
    check_dispatch(dispatch(X, ids, E, scale), X, ids, E, scale)


@pytest.mark.parametrize("M,E,k", [(600000, 256, 8), (1000001, 5, 1), (300001, 9, 7)])
def test_dispatch_of_many_turns(M, E, k):
    """More than 262144 entries: a workgroup ranks its tokens in several turns, whose counts lie in the
    same place.  Against a stable sort."""
    import torch
    print(f"case many turns {M} {E} {k}", flush=True)
    ids = torch.randint(-1, E + 1, (M, k), generator=torch.Generator().manual_seed(M), dtype=torch.int32).cuda()
    X = torch.arange(M, device="cuda").float()[:, None].repeat(1, 8)
    key, order = torch.sort(torch.where((ids < 0) | (ids >= E), E, ids).reshape(-1), stable=True)
    n = int((key < E).sum())
    pos = torch.full((M * k,), -1, dtype=torch.int32, device="cuda")
    pos[order[:n]] = torch.arange(n, dtype=torch.int32, device="cuda")
    off = torch.searchsorted(key, torch.arange(E + 1, dtype=torch.int32, device="cuda"))
    for _ in range(3):
        o = dispatch(X, ids, E)
        assert torch.equal(o["off"].long(), off) and torch.equal(o["pos"].reshape(-1), pos)
        assert torch.equal(o["entries"][:n].long(), order[:n]) and bool((o["entries"][n:] == -9).all())
        assert torch.equal(o["Xs"][:n], X[order[:n] // k]) and bool((o["Xs"][n:] == 7.0).all())


@pytest.mark.parametrize("M", [100, 3000])
def test_dispatch_of_unusual_ids(M):
    """All dropped, all to one expert, the same expert twice in a token, ids far outside."""
    import torch
    E, k = 6, 3
    X = rows(M, 40, torch.bfloat16, seed=M)
    g = torch.Generator().manual_seed(5)
    wild = torch.randint(-2 ** 31, 2 ** 31 - 1, (M, k), generator=g).to(torch.int32)
    wild[::7] = E
    for what, ids in (("none", torch.full((M, k), -1)), ("one", torch.full((M, k), E - 1)),
                      ("any", torch.randint(0, E, (M, k), generator=g)), ("wild", wild),
                      ("both ends", torch.randint(-1, E + 1, (M, k), generator=g))):
        print(f"case dispatch of unusual ids: {what}", flush=True)
        ids = ids.to(torch.int32).cuda()
        check_dispatch(dispatch(X, ids, E), X, ids, E)


def test_dispatch_agrees_with_the_router():
    """On the router's ids the lists are the router's own."""
    import torch
    for M, E, k in ((16, 8, 2), (2000, 32, 4)):
        logits = torch.randn(M, E, generator=torch.Generator().manual_seed(M)).cuda()
        i32 = dict(dtype=torch.int32, device="cuda")
        ids, w = torch.empty(M, k, **i32), torch.empty(M, k, device="cuda")
        off, entries = torch.empty(E + 1, **i32), torch.empty(M * k, **i32)
        ffn.moe_route(logits, k, ids, w, off, entries)
        o = dispatch(rows(M, 16, torch.bfloat16, 1), ids, E)
        assert torch.equal(o["off"], off) and torch.equal(o["entries"], entries)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("case", CASES)
def test_combine_and_gradients(case, dtype):
    import torch
    M, N, E, k = case
    print(f"case combine {case} {dtype}", flush=True)
    dt = getattr(torch, dtype)
    ids, w = route(M, E, k, seed=M + 2 * N)
    pos, _, entries = ref.sort(ids, E)
    n = max(entries.numel(), 1)
    w[pos.cuda() < 0] = float("nan")       # a dropped entry's weight is not looked at
    pos = pos.cuda()
    Ys, R, dY = rows(n, N, dt, 1), rows(M, N, dt, 2), rows(M, N, dt, 3)
    for weights, res in ((w, R), (w, None), (None, R), (None, None)):
        Y = torch.full((M, N), float("nan"), device="cuda", dtype=dt)
        ffn.moe_combine(Ys, pos, Y, topk_w=weights, R=res)
        ref.check({"Y": Y}, ref.combine(Ys, pos, weights, res), f"{case} combine")
    dX = torch.full((M, N), float("nan"), device="cuda", dtype=dt)
    ffn.moe_dispatch_backward(Ys, pos, dX)
    assert torch.equal(dX, Y)
    for weights in (w, None):
        dYs = torch.full((n, N), 7.0, device="cuda", dtype=dt)
        dw = torch.full((M, k), float("nan"), device="cuda")
        ffn.moe_combine_backward(dY, Ys, pos, weights, dYs, dw)
        want, (drow, bound, kept) = ref.combine_backward(dY, Ys, pos, weights)
        ref.check({"dw": dw}, want, f"{case} backward")
        at = torch.where(kept, pos.cpu().long(), 0)
        if bool(kept.any()):
            over = ((ref.d(dYs)[at] - drow).abs() / bound)[kept]
            print(f"  {case} dYs: worst error {float(over.max()):.3f} of its bound", flush=True)
            assert float(over.max()) <= 1.0
        else:
            assert bool((dYs == 7.0).all())
        only = torch.full((n, N), 7.0, device="cuda", dtype=dt)
        ffn.moe_combine_backward(dY, None, pos, weights, only, None)
        assert torch.equal(only, dYs)


def test_positions_outside_the_rows_are_dropped():
    import torch
    M, N, k, n = 50, 72, 4, 60
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (M, k), generator=g).to(torch.int32)
    pos[:, 1] = torch.arange(M)
    pos[3, 2], pos[4, 2] = n, n - 1
    pos = pos.cuda()
    Ys, dY = rows(n, N, torch.float32, 1), rows(M, N, torch.float32, 2)
    w = torch.rand(M, k, generator=g).cuda()
    Y, dYs, dw = torch.empty_like(dY), torch.full_like(Ys, 7.0), torch.empty_like(w)
    ffn.moe_combine(Ys, pos, Y, topk_w=w)
    ffn.moe_combine_backward(dY, Ys, pos, w, dYs, dw)
    ref.check({"Y": Y}, ref.combine(Ys, pos, w), "wild positions")
    ref.check({"dw": dw}, ref.combine_backward(dY, Ys, pos, w)[0], "wild positions")
    untouched = torch.ones(n, dtype=torch.bool)
    untouched[:M] = False
    untouched[n - 1] = False
    assert bool((dYs[untouched.cuda()] == 7.0).all())


def test_in_place():
    import torch
    M, N, E, k = 300, 1032, 12, 3
    ids, w = route(M, E, k, seed=1)
    pos = ref.sort(ids, E)[0].cuda()
    for dt in (torch.bfloat16, torch.float32):
        Ys, R, dY = rows(M * k, N, dt, 1), rows(M, N, dt, 2), rows(M, N, dt, 3)
        Y, dYs, dw = torch.empty_like(R), Ys.clone(), torch.empty_like(w)
        ffn.moe_combine(Ys, pos, Y, topk_w=w, R=R)
        over = R.clone()
        ffn.moe_combine(Ys, pos, over, topk_w=w, R=over)
        assert torch.equal(over, Y)
        ffn.moe_combine_backward(dY, Ys, pos, w, dYs, dw)
        over, dw2 = Ys.clone(), torch.empty_like(dw)
        ffn.moe_combine_backward(dY, over, pos, w, over, dw2)
        assert torch.equal(over, dYs) and torch.equal(dw2, dw)


@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 8, 2), (77, 24, 3), (1013, 256, 8), (20000, 300 - 44, 8)])
def test_route_backward(M, E, k):
    import torch
    print(f"case routing backward {M} {E} {k}", flush=True)
    ids, w = route(M, E, k, seed=M, drop=0.1)
    ids[0, 0] = E                                    # outside: has no logit
    if k > 1:
        ids[-1, 1] = ids[-1, 0]                      # the same expert twice
    dw = torch.randn(M, k, generator=torch.Generator().manual_seed(2)).cuda()
    dl = torch.full((M, E), float("nan"), device="cuda")
    ffn.moe_route_backward(ids, w, dw, dl)
    ref.check({"dlogits": dl}, ref.route_backward(ids, w, dw, E), f"{M} {E} {k}")


def test_no_tokens_and_no_rows():
    import torch
    ids = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    X = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    o = dispatch(X, ids, 5)
    assert not bool(o["off"].any())
    ffn.moe_combine(X, ids, X)
    w = torch.empty(0, 2, device="cuda")
    ffn.moe_combine_backward(X, X, ids, w, X, w)
    ffn.moe_route_backward(ids, w, w, torch.empty(0, 5, device="cuda"))
    pos = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")        # every entry dropped, no rows
    R = rows(4, 64, torch.bfloat16, 1)
    Y = torch.empty_like(R)
    ffn.moe_combine(X, pos, Y, topk_w=torch.ones(4, 2, device="cuda"), R=R)
    assert torch.equal(Y, R)
    dw = torch.full((4, 2), 7.0, device="cuda")
    ffn.moe_combine_backward(R, X, pos, torch.ones(4, 2, device="cuda"), X, dw)
    assert not bool(dw.any())


def test_workspace_contents_do_not_matter():
    import torch
    M, E, k = 5000, 64, 4
    ids, _ = route(M, E, k, seed=9)
    X = rows(M, 24, torch.bfloat16, 1)
    ws = ffn.workspace(ffn.moe_dispatch_workspace_size(M, E, k))
    ws.fill_(0xFF)
    check_dispatch(dispatch(X, ids, E, ws=ws), X, ids, E)


def test_rows_past_32_bit_offsets_and_more_tokens_than_a_launch():
    """9 x 10^9 values a side: 64-bit offsets, and the tokens in two slices of launches.  Checked at both
    ends, around the slices' border and where 2^31 and 2^32 values or bytes end."""
    import torch
    M, N = (1 << 22) + 77, 2048
    print(f"case dispatch and combine of {M} x {N}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, M, 1 << 19):       # (a generator's call on all of it at once would need twice the memory)
        part = X[lo:lo + (1 << 19)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda", dtype=torch.bfloat16))
    ids = torch.randint(-1, 3, (M, 1), generator=g, device="cuda", dtype=torch.int32)
    Xs = torch.zeros_like(X)
    i32 = dict(dtype=torch.int32, device="cuda")
    off, entries, pos = torch.empty(4, **i32), torch.empty(M, **i32), torch.empty(M, 1, **i32)
    ffn.moe_dispatch(X, ids, Xs, off, entries, pos)
    w = torch.rand(M, 1, generator=g, device="cuda")
    at = torch.cat([torch.arange(b - 200, b + 200) for b in (200, 1 << 19, 1 << 20, 1 << 21, 1 << 22)] +
                   [torch.arange(M - 300, M)]).unique()
    at = at[at < M].cuda()
    kept = pos[at, 0] >= 0
    assert torch.equal(kept, ids[at, 0] >= 0)
    p = pos[at, 0].clamp(min=0).long()
    assert torch.equal(Xs[p][kept], X[at][kept])
    n = int(off[-1])
    assert n == int((ids >= 0).sum()) and not bool(Xs[n:].any())
    Y = torch.empty_like(X)
    ffn.moe_combine(Xs, pos, Y, topk_w=w, R=X)
    ref.check({"Y": Y[at]}, ref.combine(Xs[p], torch.where(kept, torch.arange(len(at), device="cuda"), -1)[:, None], w[at], X[at]),
              "combine")
    dw = torch.full_like(w, float("nan"))
    ffn.moe_combine_backward(X, Xs, pos, w, Xs, dw)        # in place
    want = (X[at].float() * w[at]).to(torch.bfloat16)
    assert torch.equal(Xs[p][kept], want[kept])
    ref.check({"dw": dw[at]}, ref.combine_backward(X[at], X[at], torch.where(kept, torch.arange(len(at), device="cuda"), -1)[:, None],
                                                   w[at])[0], "combine's gradients")


@pytest.mark.parametrize("M,N,E,k,dtype", [(150, 72, 9, 3, "bfloat16"), (61, 520, 24, 8, "float32")])
def test_routing_gradient_where_entries_are_dropped_after_the_router(M, N, E, k, dtype):
    """The router's own ids, and the dispatch's with dropped entries at -1: the logits' gradient is that of the
    combined rows by differentiation, dropped choices (which still stand in the softmax) among them."""
    import torch
    dt = getattr(torch, dtype)
    print(f"case routing gradient with dropped entries {M} {E} {k} {dtype}", flush=True)
    g = torch.Generator().manual_seed(M)
    logits = torch.randn(M, E, generator=g).cuda()
    ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
    w = torch.empty(M, k, device="cuda")
    ffn.moe_route(logits, k, topk_ids=ids, topk_w=w)
    kept = torch.where(torch.rand(M, k, generator=g).cuda() < 0.3, -1, ids)
    kept[0] = -1
    o = dispatch(rows(M, N, dt, 1), kept, E)
    Ys, dY = rows(M * k, N, dt, 2), rows(M, N, dt, 3)
    dw, dYs, dl = torch.empty_like(w), torch.empty_like(Ys), torch.full((M, E), float("nan"), device="cuda")
    ffn.moe_combine_backward(dY, Ys, o["pos"], w, dYs, dw)
    ffn.moe_route_backward(ids, w, dw, dl)
    x = ref.d(logits).requires_grad_()
    v, on = ref._taken(Ys, o["pos"])
    p = torch.softmax(x.gather(1, ids.cpu().long()), 1)
    ((v * (p * on)[:, :, None]).sum(1) * ref.d(dY)).sum().backward()
    # the fp32 weights are within e of the softmax's, and the gradient is linear in products of two of them
    want, off = ref.combine_backward(dY, Ys, o["pos"], w)[0]["dw"]
    e = float((ref.d(w) / p.detach() - 1).abs().max())
    assert e < 1e-5
    far = ref.route_backward(ids, w, want, E)["dlogits"][1]
    wd = ref.d(w)
    far.scatter_add_(1, ids.cpu().long(), wd * (off + (wd * off).sum(1, keepdim=True)))
    far.scatter_add_(1, ids.cpu().long(), 3 * e * wd * (want.abs() + (wd * want.abs()).sum(1, keepdim=True)))
    ref.check({"dlogits": dl}, {"dlogits": (x.grad, 1.01 * far + 1e-30)}, f"{M} {E} {k}")
    gone = (kept < 0).cpu() & (wd > 0.01)
    assert bool(gone[1:].any()) and bool((x.grad.gather(1, ids.cpu().long())[1:][gone[1:]] != 0).any())
