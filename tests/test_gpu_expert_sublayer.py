"""The operators around an expert sub-layer as they are used together: a training step (norm, routing,
dispatch, the experts' gated blocks, combine, and all gradients back to the input), a decode step with
4-bit experts, and a prompt whose rows are dispatched in 8 bits -- eagerly, on side streams, two at
once, captured and replayed."""
from __future__ import annotations

import pytest

import transformer_ffn_fusion_amd as ffn

import sublayer_ref as ref
import training_ref

pytestmark = pytest.mark.gpu


def rand(g, *shape, scale=1.0, dtype=None):
    import torch
    return (scale * torch.randn(*shape, generator=g)).to(dtype or torch.bfloat16).cuda()


def hole(*shape, dtype=None):
    import torch
    t = torch.zeros(*shape, dtype=dtype or torch.bfloat16, device="cuda")
    return t.fill_(float("nan")) if t.is_floating_point() and dtype != torch.float8_e4m3fn else t.fill_(0)


class Steps:
    """What the chains share: outputs by name, cleared and taken."""

    def clear(self):
        import torch
        for t in self.out.values():
            t.view(torch.uint8).fill_(0xFF) if t.dtype == torch.float8_e4m3fn else \
                t.fill_(float("nan") if t.is_floating_point() else -7)

    def take(self):
        import torch
        torch.cuda.synchronize()
        return {k: v.clone() for k, v in self.out.items()}


def same(a, b):
    """Names of outputs that differ (bits; NaN in untouched rows on both sides)."""
    import torch
    return [k for k in a if not torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8))]


class Training(Steps):
    """Pre-norm expert sub-layer, S = x + r, out = S + sum_s w_s expert(norm(S)), and its gradients."""

    def __init__(self, M, N, O, E, k, seed):
        import torch
        g = torch.Generator().manual_seed(seed)
        f32, i32 = torch.float32, torch.int32
        self.shape = M, N, O, E, k
        self.x, self.r, self.dout = rand(g, M, N), rand(g, M, N), rand(g, M, N)
        self.gamma, self.logits = 1 + rand(g, N, scale=0.2), rand(g, M, E, dtype=f32)
        self.w = [rand(g, E, N, O, scale=N ** -0.5), rand(g, E, N, O, scale=N ** -0.5), rand(g, E, O, N, scale=O ** -0.5)]
        R = M * k
        self.out = dict(S=hole(M, N), n=hole(M, N), rstd=hole(M, dtype=f32), ids=hole(M, k, dtype=i32),
                        w=hole(M, k, dtype=f32), xs=hole(R, N), off=hole(E + 1, dtype=i32), entries=hole(R, dtype=i32),
                        pos=hole(M, k, dtype=i32), ys=hole(R, N), y=hole(M, N), dys=hole(R, N), dw=hole(M, k, dtype=f32),
                        dxs=hole(R, N), dn=hole(M, N), dl=hole(M, E, dtype=f32), dx=hole(M, N), dgamma=hole(N, dtype=f32))
        self.grads = [hole(E, N, O), hole(E, N, O), hole(E, O, N)]
        self.ws = dict(route=ffn.workspace(ffn.moe_workspace_size(M, E, k, 8, 8, 8)),
                       sort=ffn.workspace(ffn.moe_dispatch_workspace_size(M, E, k)),
                       fwd=ffn.workspace(ffn.ffn_swiglu_workspace_size(R, N, O, N)),
                       bwd=ffn.workspace(ffn.ffn_swiglu_backward_workspace_size(R, N, O, N)),
                       norm=ffn.workspace(ffn.ffn_rmsnorm_backward_workspace_size(M, N)))
        torch.cuda.synchronize()

    def run(self):
        o, ws, k = self.out, self.ws, self.shape[4]
        ffn.ffn_rmsnorm_forward(self.x, self.gamma, o["n"], R=self.r, S=o["S"], rstd=o["rstd"])
        ffn.moe_route(self.logits, k, topk_ids=o["ids"], topk_w=o["w"], ws=ws["route"])
        ffn.moe_dispatch(o["n"], o["ids"], o["xs"], o["off"], o["entries"], o["pos"], ws=ws["sort"])
        off = o["off"].tolist()
        lists = [(e, off[e], off[e + 1]) for e in range(self.shape[3]) if off[e] < off[e + 1]]
        for e, lo, hi in lists:
            ffn.ffn_swiglu_forward(o["xs"][lo:hi], *(w[e] for w in self.w), o["ys"][lo:hi], ws=ws["fwd"])
        ffn.moe_combine(o["ys"], o["pos"], o["y"], topk_w=o["w"], R=o["S"])
        ffn.moe_combine_backward(self.dout, o["ys"], o["pos"], o["w"], o["dys"], o["dw"])
        for e, lo, hi in lists:
            ffn.ffn_swiglu_backward(o["xs"][lo:hi], *(w[e] for w in self.w), o["dys"][lo:hi], o["dxs"][lo:hi],
                                    *(d[e] for d in self.grads), ws=ws["bwd"])
        ffn.moe_dispatch_backward(o["dxs"], o["pos"], o["dn"])
        ffn.moe_route_backward(o["ids"], o["w"], o["dw"], o["dl"])
        ffn.ffn_rmsnorm_backward(o["S"], o["dn"], self.gamma, o["rstd"], o["dx"], o["dgamma"], dS=self.dout, ws=ws["norm"])


@pytest.mark.parametrize("shape", [(70, 72, 136, 5, 2), (300, 520, 264, 8, 3)])
def test_training_step_stage_by_stage(shape):
    """Every stage on what the stage before it wrote, within that stage's own bounds."""
    import torch
    print(f"case expert sub-layer training step {shape}", flush=True)
    M, N, O, E, k = shape
    s = Training(*shape, seed=1)
    s.run()
    o = s.take()
    assert torch.equal(o["S"].cpu(), (s.x.cpu().float() + s.r.cpu().float()).bfloat16())
    ref.check({"Y": o["n"], "rstd": o["rstd"]}, ref.rmsnorm_forward(o["S"], s.gamma, 1e-5), "norm")
    pos, off, entries = ref.sort(o["ids"], E)
    assert torch.equal(o["pos"].cpu(), pos) and torch.equal(o["off"].cpu(), off) and torch.equal(o["entries"].cpu(), entries)
    assert torch.equal(o["xs"], o["n"][(entries // k).long().cuda()])
    ref.check({"Y": o["y"]}, ref.combine(o["ys"], pos, o["w"], o["S"]), "combine")
    dw, (drow, bound, kept) = ref.combine_backward(s.dout, o["ys"], pos, o["w"])
    ref.check({"dw": o["dw"]}, dw, "combine's gradients")
    assert bool(((ref.d(o["dys"])[pos.long()] - drow).abs() <= bound).all()) and bool(kept.all())
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo < hi:
            names = ("dX", "dWg", "dWu", "dWd")
            got = dict(zip(names, (o["dxs"][lo:hi], *(d[e] for d in s.grads))))
            training_ref.check(got, training_ref.swiglu_backward(o["xs"][lo:hi], *(w[e] for w in s.w), o["dys"][lo:hi]),
                               f"expert {e}")
    ref.check({"Y": o["dn"]}, ref.combine(o["dxs"], pos), "dispatch's gradient")
    ref.check({"dlogits": o["dl"]}, ref.route_backward(o["ids"], o["w"], o["dw"], E), "routing's gradient")
    ref.check({"dX": o["dx"], "dgamma": o["dgamma"]},
              ref.rmsnorm_backward(o["S"], o["dn"], s.gamma, o["rstd"], s.dout), "norm's gradients")


class Decode(Steps):
    """A few tokens through the sub-layer with 4-bit experts: no host step between the calls."""

    def __init__(self, M, N, O, E, k, seed, code="int4", group=128, zero=False):
        import torch
        g = torch.Generator().manual_seed(seed)
        f32, i32 = torch.float32, torch.int32
        self.shape, self.code = (M, N, O, E, k), code
        self.x, self.r, self.gamma = rand(g, M, N), rand(g, M, N), 1 + rand(g, N, scale=0.2)
        self.wr = rand(g, N, E, scale=N ** -0.5)
        self.packed = {}
        for name, K, C in (("g", N, O), ("u", N, O), ("d", O, N)):
            W, sc, z = ffn.ffn_q4_empty(K, C, group, zero, experts=E)
            for e in range(E):
                ffn.ffn_q4_quantize(rand(g, K, C, scale=K ** -0.5), W[e], sc[e], zero=None if z is None else z[e], code=code)
            self.packed[name] = W, sc, z
        R = M * k
        self.out = dict(S=hole(M, N), n=hole(M, N), logits=hole(M, E, dtype=f32), ids=hole(M, k, dtype=i32),
                        w=hole(M, k, dtype=f32), xs=hole(R, N), off=hole(E + 1, dtype=i32), entries=hole(R, dtype=i32),
                        pos=hole(M, k, dtype=i32), h=hole(R, O), ys=hole(R, N), y=hole(M, N))
        self.ws = [ffn.workspace(ffn.moe_workspace_size(M, E, k, N, 8, 8)), ffn.workspace(ffn.moe_dispatch_workspace_size(M, E, k))]
        torch.cuda.synchronize()

    def run(self, stream=None):
        o, k = self.out, self.shape[4]
        (g, sg, zg), (u, su, zu), (d, sd, zd) = (self.packed[n] for n in "gud")
        ffn.ffn_rmsnorm_forward(self.x, self.gamma, o["n"], R=self.r, S=o["S"], stream=stream)
        ffn.moe_router(o["n"], self.wr, None, k, logits_out=o["logits"], topk_ids=o["ids"], topk_w=o["w"], ws=self.ws[0],
                       stream=stream)
        ffn.moe_dispatch(o["n"], o["ids"], o["xs"], o["off"], o["entries"], o["pos"], ws=self.ws[1], stream=stream)
        ffn.moe_q4_swiglu(o["xs"], o["off"], g, sg, u, su, o["h"], zero_g=zg, zero_u=zu, code=self.code, stream=stream)
        ffn.moe_q4_matvec(o["h"], o["off"], d, sd, o["ys"], zero=zd, code=self.code, stream=stream)
        ffn.moe_combine(o["ys"], o["pos"], o["y"], topk_w=o["w"], R=o["S"], stream=stream)


DECODE = [(1, 264, 136, 8, 2), (16, 520, 264, 8, 2), (13, 136, 1032, 16, 4)]


@pytest.mark.parametrize("code,group,zero", [("int4", 128, False), ("int4", 32, True), ("e2m1", 32, False)])
@pytest.mark.parametrize("shape", DECODE)
def test_decode_step_stage_by_stage(shape, code, group, zero):
    import torch
    print(f"case expert sub-layer decode step {shape} {code} {group}", flush=True)
    M, N, O, E, k = shape
    s = Decode(*shape, seed=2, code=code, group=group, zero=zero)
    s.run()
    o = s.take()
    ref.check({"Y": o["n"]}, {"Y": ref.rmsnorm_forward(o["S"], s.gamma, 1e-5)["Y"]}, "norm")
    pos, off, entries = ref.sort(o["ids"], E)
    assert torch.equal(o["pos"].cpu(), pos) and torch.equal(o["off"].cpu(), off)
    assert torch.equal(o["xs"], o["n"][(entries // k).long().cuda()])
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        g, u, d = ([None if t is None else t[e].cpu() for t in s.packed[n]] for n in "gud")
        ref.check({"H": o["h"][lo:hi]}, ref.q4_swiglu(o["xs"][lo:hi], *g, *u, O, code), f"expert {e}, pair")
        ref.check({"Y": o["ys"][lo:hi]}, ref.q4_matvec(o["h"][lo:hi], *d, None, "none", N, code), f"expert {e}, down")
    ref.check({"Y": o["y"]}, ref.combine(o["ys"], pos, o["w"], o["S"]), "combine")


@pytest.mark.parametrize("shape", DECODE)
def test_decode_captured_and_replayed(shape):
    """The step in a graph, replayed on new inputs (and so new routes) with eager work in between."""
    import torch
    s = Decode(*shape, seed=3)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for i in range(5):
        s.x.copy_(torch.randn(s.x.shape, generator=torch.Generator().manual_seed(60 + i)).to(s.x))
        s.clear()
        graph.replay()
        got = s.take()
        s.clear()
        for w in s.ws:
            w.fill_(0x5A)
        s.run()
        assert same(s.take(), got) == [], f"replay {i}"


def test_decode_on_side_streams_and_two_at_once():
    import torch
    a, b = Decode(*DECODE[1], seed=4), Decode(*DECODE[2], seed=5, code="e2m1", group=64)
    a.run()
    b.run()
    want = a.take(), b.take()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for explicit in (False, True):
        a.clear()
        b.clear()
        torch.cuda.synchronize()
        for _ in range(3):
            if explicit:
                a.run(stream=sa.cuda_stream)
                b.run(stream=sb.cuda_stream)
            else:
                with torch.cuda.stream(sa):
                    a.run()
                with torch.cuda.stream(sb):
                    b.run()
        assert same(a.take(), want[0]) == [] and same(b.take(), want[1]) == []


class Gradients(Steps):
    """The training calls without a host step: captured, and beside others on other streams."""

    def __init__(self, M, N, E, k, seed):
        import torch
        g = torch.Generator().manual_seed(seed)
        f32, i32 = torch.float32, torch.int32
        self.k = k
        self.x, self.r, self.dout = rand(g, M, N), rand(g, M, N), rand(g, M, N)
        self.gamma, self.ids = 1 + rand(g, N, scale=0.2), torch.randint(-1, E, (M, k), generator=g).to(i32).cuda()
        self.w = torch.rand(M, k, generator=g).cuda()
        R = M * k
        self.out = dict(S=hole(M, N), n=hole(M, N), rstd=hole(M, dtype=f32), xs=hole(R, N), off=hole(E + 1, dtype=i32),
                        entries=hole(R, dtype=i32), pos=hole(M, k, dtype=i32), y=hole(M, N), dys=hole(R, N),
                        dw=hole(M, k, dtype=f32), dn=hole(M, N), dl=hole(M, E, dtype=f32), dx=hole(M, N),
                        dgamma=hole(N, dtype=f32), q=hole(M, N, dtype=torch.float8_e4m3fn), qs=hole(M, -(-N // 128), dtype=f32),
                        xq=hole(R, N, dtype=torch.float8_e4m3fn), xqs=hole(R, -(-N // 128), dtype=f32))
        self.ws = dict(sort=ffn.workspace(ffn.moe_dispatch_workspace_size(M, E, k)),
                       norm=ffn.workspace(ffn.ffn_rmsnorm_backward_workspace_size(M, N)))
        torch.cuda.synchronize()

    def run(self, stream=None, own_ws=False):
        o, st = self.out, dict(stream=stream)
        sort, norm = (None, None) if own_ws else (self.ws["sort"], self.ws["norm"])
        ffn.ffn_rmsnorm_forward(self.x, self.gamma, o["n"], R=self.r, S=o["S"], rstd=o["rstd"], **st)
        ffn.moe_dispatch(o["n"], self.ids, o["xs"], o["off"], o["entries"], o["pos"], ws=sort, **st)
        ffn.moe_combine(o["xs"], o["pos"], o["y"], topk_w=self.w, R=o["S"], **st)
        ffn.moe_combine_backward(self.dout, o["xs"], o["pos"], self.w, o["dys"], o["dw"], **st)
        ffn.moe_dispatch_backward(o["dys"], o["pos"], o["dn"], **st)
        ffn.moe_route_backward(self.ids, self.w, o["dw"], o["dl"], **st)
        ffn.ffn_rmsnorm_backward(o["S"], o["dn"], self.gamma, o["rstd"], o["dx"], o["dgamma"], dS=self.dout, ws=norm, **st)
        ffn.ffn_rmsnorm_q8_forward(o["S"], self.gamma, o["q"], o["qs"], **st)
        ffn.moe_dispatch(o["q"], self.ids, o["xq"], o["off"], o["entries"], o["pos"], scale=o["qs"],
                         scale_sorted=o["xqs"], ws=sort, **st)


GRADS = [(40, 72, 5, 2), (700, 520, 24, 3), (3000, 264, 64, 4)]    # one sort launch, one with the rows, three


@pytest.mark.parametrize("shape", GRADS)
def test_8_bit_rows_travel_with_their_scales(shape):
    import torch
    s = Gradients(*shape, seed=6)
    s.run()
    o = s.take()
    n = int(o["off"][-1])
    token = (o["entries"][:n] // s.k).long()
    assert torch.equal(o["xq"].view(torch.uint8)[:n], o["q"].view(torch.uint8)[token])
    assert torch.equal(o["xqs"][:n], o["qs"][token])
    ref.check_q8(o["q"], o["qs"], o["S"], s.gamma, 1e-5, 128, f"{shape}")


@pytest.mark.parametrize("shape", GRADS)
def test_gradients_captured_replayed_and_on_other_streams(shape):
    import torch
    a, b = Gradients(*shape, seed=7), Gradients(*shape, seed=8)
    a.clear()
    b.clear()
    a.run()
    b.run()
    want = a.take(), b.take()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    a.clear()
    b.clear()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(sa):
            a.run()
        b.run(stream=sb.cuda_stream)
    assert same(a.take(), want[0]) == [] and same(b.take(), want[1]) == []
    b.clear()
    torch.cuda.synchronize()
    torch.cuda._sleep(100000)          # the current stream is busy; the workspaces are the call's own
    b.run(stream=sb.cuda_stream, own_ws=True)
    other = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    assert same(b.take(), want[1]) == []
    del other
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    again = torch.cuda.CUDAGraph()     # a second graph on the same buffers and workspaces
    with torch.cuda.graph(again):
        a.run()
    for i in range(4):
        a.ids.copy_(torch.roll(a.ids, 1, 0))
        a.x.mul_(-0.5)
        a.clear()
        (graph if i % 2 else again).replay()
        got = a.take()
        a.clear()
        for w in a.ws.values():
            w.fill_(0x5A)
        a.run()
        assert same(a.take(), got) == [], f"replay {i}"


def test_stream_given_as_a_ctypes_handle():
    import ctypes
    import torch
    s = Gradients(*GRADS[1], seed=9)
    s.clear()
    s.run()
    want = s.take()
    st = torch.cuda.Stream()
    for handle in (ctypes.c_void_p(st.cuda_stream), ctypes.c_void_p(None), ctypes.c_void_p(0)):
        for own in (False, True):
            s.clear()
            torch.cuda.synchronize()
            s.run(stream=handle, own_ws=own)
            assert same(s.take(), want) == []
