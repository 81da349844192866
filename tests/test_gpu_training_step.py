"""The training operators as a training step of the gated sub-layer uses them: layer norm, the SwiGLU
block, its gradients, the norm's gradients, the three matrices' updates -- eagerly, on a side stream,
captured into a graph and replayed, and two at once."""
from __future__ import annotations

import pytest

import transformer_ffn_fusion_amd as ffn

import training_ref as ref

pytestmark = pytest.mark.gpu


class Step:
    """One sub-layer's inputs, buffers and workspaces."""

    def __init__(self, M, N, O, P, seed):
        import torch
        g = torch.Generator().manual_seed(seed)
        bf, f32 = torch.bfloat16, torch.float32

        def r(*s, scale=1.0):
            return (scale * torch.randn(*s, generator=g)).to(bf).cuda()

        def e(*s, dtype=bf):
            return torch.full(s, float("nan"), dtype=dtype, device="cuda")
        self.shape = M, N, O, P
        self.x, self.dy = r(M, N), r(M, P)
        self.gamma, self.beta = 1 + r(N, scale=0.2), r(N, scale=0.2)
        self.w = [r(N, O, scale=N ** -0.5), r(N, O, scale=N ** -0.5), r(O, P, scale=O ** -0.5)]
        self.out = dict(n=e(M, N), mean=e(M, dtype=f32), rstd=e(M, dtype=f32), y=e(M, P), dn=e(M, N),
                        dWg=e(N, O), dWu=e(N, O), dWd=e(O, P), dx=e(M, N), dgamma=e(N, dtype=f32),
                        dbeta=e(N, dtype=f32), Ug=e(N, O), Uu=e(N, O), Ud=e(O, P))
        self.ws = dict(
            fwd=ffn.workspace(ffn.ffn_swiglu_workspace_size(M, N, O, P)),
            bwd=ffn.workspace(ffn.ffn_swiglu_backward_workspace_size(M, N, O, P)),
            norm=ffn.workspace(ffn.ffn_layernorm_backward_workspace_size(M, N)),
            up=ffn.workspace(max(ffn.ffn_orthogonalize_workspace_size(1, N, O),
                                 ffn.ffn_orthogonalize_workspace_size(1, O, P))))
        torch.cuda.synchronize()

    def run(self):
        o, ws = self.out, self.ws
        ffn.ffn_layernorm_forward(self.x, self.gamma, self.beta, o["n"], o["mean"], o["rstd"])
        ffn.ffn_swiglu_forward(o["n"], *self.w, o["y"], ws=ws["fwd"])
        ffn.ffn_swiglu_backward(o["n"], *self.w, self.dy, o["dn"], o["dWg"], o["dWu"], o["dWd"], ws=ws["bwd"])
        ffn.ffn_layernorm_backward(self.x, o["dn"], self.gamma, o["mean"], o["rstd"], o["dx"], o["dgamma"],
                                   o["dbeta"], ws=ws["norm"])
        for d, u in (("dWg", "Ug"), ("dWu", "Uu"), ("dWd", "Ud")):
            ffn.ffn_orthogonalize(o[d], o[u], ws=ws["up"])

    def clear(self):
        for t in self.out.values():
            t.fill_(float("nan"))

    def take(self):
        import torch
        torch.cuda.synchronize()
        return {k: v.clone() for k, v in self.out.items()}


def same(a, b):
    import torch
    return [k for k in a if not torch.equal(a[k], b[k])]


SHAPES = [(70, 72, 136, 104), (300, 520, 264, 392)]


@pytest.mark.parametrize("shape", SHAPES)
def test_each_stage_against_fp64(shape):
    """Every stage on what the stage before it wrote, within that stage's own bounds."""
    print(f"case training step {shape}", flush=True)
    s = Step(*shape, seed=1)
    s.run()
    o = s.take()
    ref.check({"Y": o["n"], "mean": o["mean"], "rstd": o["rstd"]},
              ref.layernorm_forward(s.x, s.gamma, s.beta, 1e-5), "norm")
    ref.check({"dX": o["dn"], "dWg": o["dWg"], "dWu": o["dWu"], "dWd": o["dWd"]},
              ref.swiglu_backward(o["n"], *s.w, s.dy), "block")
    ref.check({"dX": o["dx"], "dgamma": o["dgamma"], "dbeta": o["dbeta"]},
              ref.layernorm_backward(s.x, o["dn"], s.gamma, o["mean"], o["rstd"]), "norm's gradients")
    for d, u in (("dWg", "Ug"), ("dWu", "Uu"), ("dWd", "Ud")):
        ref.check_orthogonalize(o[u], o[d], 5, u)


@pytest.mark.parametrize("shape", SHAPES)
def test_side_stream_and_two_at_once(shape):
    import torch
    a, b = Step(*shape, seed=2), Step(*shape, seed=3)
    a.run()
    b.run()
    want = a.take(), b.take()
    for s in (a, b):
        s.clear()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):      # each with its own workspaces, neither waits for the other
        with torch.cuda.stream(sa):
            a.run()
        with torch.cuda.stream(sb):
            b.run()
    assert same(a.take(), want[0]) == [] and same(b.take(), want[1]) == []


def test_explicit_stream_argument():
    import torch
    s = Step(*SHAPES[0], seed=4)
    s.run()
    want = s.take()
    st = torch.cuda.Stream()
    n = torch.empty_like(want["n"])
    U = torch.empty_like(want["Ug"])
    torch.cuda.synchronize()
    ffn.ffn_layernorm_forward(s.x, s.gamma, s.beta, n, stream=st.cuda_stream)
    ffn.ffn_orthogonalize(want["dWg"], U, ws=s.ws["up"], stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(n, want["n"]) and torch.equal(U, want["Ug"])


def test_explicit_stream_brings_its_own_workspace():
    """A call on another stream than the current one, with no workspace given, while the current
    stream is busy: the workspace is filled on the call's stream, not behind that work."""
    import torch
    M, N, O = 1024, 2048, 1536
    g = torch.Generator(device="cuda").manual_seed(8)

    def rand(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") / shape[-1] ** 0.5).bfloat16()

    args = [rand(M, N), rand(N, O), rand(N, O), rand(O, N), rand(M, N)]

    def grads():
        return [torch.empty_like(args[k]) for k in (0, 1, 2, 3)]
    want = grads()
    ffn.ffn_swiglu_backward(*args, *want)
    G = torch.randn(512, 1024, generator=g, device="cuda")
    wantU = torch.empty(512, 1024, dtype=torch.bfloat16, device="cuda")
    ffn.ffn_orthogonalize(G, wantU)
    st = torch.cuda.Stream()
    for sleep in (0, 20000, 60000, 120000, 200000, 400000):
        got, U = grads(), torch.empty_like(wantU)
        torch.cuda.synchronize()
        torch.cuda._sleep(sleep)    # (clocks; the calls take 0.1 to 0.3 ms)
        ffn.ffn_swiglu_backward(*args, *got, stream=st.cuda_stream)
        ffn.ffn_orthogonalize(G, U, stream=st.cuda_stream)
        other = [torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(U, wantU), sleep
        del other


@pytest.mark.parametrize("shape", SHAPES)
def test_captured_and_replayed(shape):
    """The whole step in a graph, replayed on new inputs with eager work between the replays."""
    import torch
    s = Step(*shape, seed=5)
    s.run()                     # (loads the kernels)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for k in range(4):
        s.x.copy_(torch.randn(s.x.shape, generator=torch.Generator().manual_seed(50 + k)).to(s.x))
        s.clear()
        graph.replay()
        got = s.take()
        s.clear()
        for w in s.ws.values():     # eager work of the program's own in between, on the same workspaces
            w.fill_(0x5A)
        s.run()
        assert same(s.take(), got) == [], f"replay {k}"


def test_shapes_with_joined_splits_repeat_bitwise():
    """Sums split over the depth and joined by whichever workgroup comes last: the same bits always."""
    import torch
    for M, N, O, P in [(8, 128, 512, 128), (1013, 2056, 1400, 1992), (40, 1024, 1536, 2048)]:
        s = Step(M, N, O, P, seed=6)
        first = None
        for _ in range(12):
            s.clear()
            ffn.ffn_swiglu_backward(s.x, *s.w, s.dy, s.out["dn"], s.out["dWg"], s.out["dWu"], s.out["dWd"],
                                    ws=s.ws["bwd"])
            got = {k: v for k, v in s.take().items() if k in ("dn", "dWg", "dWu", "dWd")}
            first = first or got
            assert same(got, first) == [], (M, N, O, P)
    G = torch.randn(2, 264, 2048, generator=torch.Generator().manual_seed(7)).cuda()
    U = torch.empty(2, 264, 2048, dtype=torch.bfloat16, device="cuda")
    ws = ffn.workspace(ffn.ffn_orthogonalize_workspace_size(2, 264, 2048))
    first = None
    for _ in range(12):
        ffn.ffn_orthogonalize(G, U, ws=ws)
        torch.cuda.synchronize()
        first = U.clone() if first is None else first
        assert torch.equal(U, first)


def test_stream_given_as_a_ctypes_handle():
    """A handle as C programs pass it around, with and without a workspace of the caller's."""
    import ctypes
    import torch
    M, N, O, P = 40, 72, 136, 104
    s = Step(M, N, O, P, seed=9)
    s.run()
    want = s.take()
    st = torch.cuda.Stream()
    for handle in (ctypes.c_void_p(st.cuda_stream), ctypes.c_void_p(None), ctypes.c_void_p(0)):
        for ws in (None, s.ws):
            y, dn = torch.full_like(want["y"], float("nan")), torch.full_like(want["dn"], float("nan"))
            torch.cuda.synchronize()
            ffn.ffn_swiglu_forward(want["n"], *s.w, y, ws=ws and ws["fwd"], stream=handle)
            ffn.ffn_swiglu_backward(want["n"], *s.w, s.dy, dn, s.out["dWg"], s.out["dWu"], s.out["dWd"],
                                    ws=ws and ws["bwd"], stream=handle)
            torch.cuda.synchronize()
            assert torch.equal(y, want["y"]) and torch.equal(dn, want["dn"])
