"""The decode stream in a program that uses several streams: the first workgroup of a launch on the
default stream is then dealt to another XCD than the first, and the calls have to stay right."""
from __future__ import annotations

import pytest

import transformer_ffn_fusion_amd as ffn

pytestmark = pytest.mark.gpu


def _operands(M, N, O, P, gated):
    import torch
    g = torch.Generator().manual_seed(M + O)

    def r(*s):
        return torch.randn(*s, generator=g).bfloat16().cuda()
    W = [(r(N, O) / N ** 0.5) for _ in range(2 if gated else 1)]
    return r(M, N), W, r(O, P) / O ** 0.5


@pytest.mark.parametrize("gated", [False, True])
def test_decode_stream_after_side_streams(gated):
    import torch
    M, N, O, P = 4, 4096, 512, 4096
    X, W, Wd = _operands(M, N, O, P, gated)

    def call(stream=None):
        Y = torch.full((M, P), float("nan"), dtype=torch.bfloat16, device="cuda")
        if gated:
            ffn.ffn_swiglu_forward(X, *W, Wd, Y, variant=ffn.VARIANT_DECODE, stream=stream)
        else:
            ffn.ffn_forward_ex(X, W[0], None, Wd, None, Y, variant=ffn.VARIANT_DECODE, stream=stream)
        torch.cuda.synchronize()
        return Y
    first = call()
    for k in range(1, 6):     # one workgroup each on streams of their own: the deal moves on
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            torch.zeros(8, device="cuda")
        torch.cuda.synchronize()
        Y = call()
        print(f"  after {k} side streams: {int(torch.isnan(Y).sum())} NaN", flush=True)
        assert torch.equal(Y, first)
        assert torch.equal(call(st.cuda_stream), first)
    assert not bool(torch.isnan(first).any())


@pytest.mark.parametrize("gated", [False, True])
def test_decode_stream_after_side_streams_ordered(gated):
    """Y's fill has ended before a call on another stream than the current one begins."""
    import torch
    M, N, O, P = 4, 4096, 512, 4096
    X, W, Wd = _operands(M, N, O, P, gated)

    def call(stream=None):
        Y = torch.full((M, P), float("nan"), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        if gated:
            ffn.ffn_swiglu_forward(X, *W, Wd, Y, variant=ffn.VARIANT_DECODE, stream=stream)
        else:
            ffn.ffn_forward_ex(X, W[0], None, Wd, None, Y, variant=ffn.VARIANT_DECODE, stream=stream)
        torch.cuda.synchronize()
        return Y
    first = call()
    assert not bool(torch.isnan(first).any())
    for k in range(1, 6):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            torch.zeros(8, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(call(), first), k
        assert torch.equal(call(st.cuda_stream), first), k
