"""Refusals of the operators around an expert sub-layer (RMS norm, dispatch and combine, 4-bit
products), on the CPU: the binding's checks of tensors, the C ABI's checks of pointers, sizes and
workspaces (no call reaches a launch)."""
from __future__ import annotations

import pytest
import torch

import transformer_ffn_fusion_amd as ffn

BF, F32, F8, I32, U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32, torch.uint8
E_INVAL, E_WS, E_UNSUP, E_ALIGN = -1, -2, -3, -4
M, N, E, K = 32, 264, 6, 2
TOP = 2 ** 63 - 1


def meta(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


def at(i):      # never dereferenced device pointers, far enough apart
    return (i + 1) << 22


# ---------------------------------------------------------------- the binding

def rms(dt=BF):
    return dict(X=meta(M, N, dtype=dt), gamma=meta(N, dtype=dt), Y=meta(M, N, dtype=dt), R=meta(M, N, dtype=dt),
                S=meta(M, N, dtype=dt), rstd=meta(M, dtype=F32))


def rms_q8():
    a = rms()
    del a["Y"]
    return dict(a, Q=meta(M, N, dtype=F8), scale=meta(M, 3, dtype=F32))


def rms_bwd():
    return dict(S=meta(M, N), dY=meta(M, N), gamma=meta(N), rstd=meta(M, dtype=F32), dX=meta(M, N),
                dgamma=meta(N, dtype=F32), dS=meta(M, N))


def dispatch():
    return dict(X=meta(M, N), topk_ids=meta(M, K, dtype=I32), Xs=meta(M * K, N), expert_offsets=meta(E + 1, dtype=I32),
                sorted_entries=meta(M * K, dtype=I32), positions=meta(M, K, dtype=I32), scale=meta(M, 3, dtype=F32),
                scale_sorted=meta(M * K, 3, dtype=F32))


def dispatch_bwd():
    return dict(dXs=meta(40, N), positions=meta(M, K, dtype=I32), dX=meta(M, N))


def combine():
    return dict(Ys=meta(40, N), positions=meta(M, K, dtype=I32), Y=meta(M, N), topk_w=meta(M, K, dtype=F32),
                R=meta(M, N))


def combine_bwd():
    return dict(dY=meta(M, N), Ys=meta(40, N), positions=meta(M, K, dtype=I32), topk_w=meta(M, K, dtype=F32),
                dYs=meta(40, N), dw=meta(M, K, dtype=F32))


def route_bwd():
    return dict(topk_ids=meta(M, K, dtype=I32), topk_w=meta(M, K, dtype=F32), dw=meta(M, K, dtype=F32),
                dlogits=meta(M, E, dtype=F32))


def weight(*lead, per=1):
    return meta(*lead, 17, 3, 1024, dtype=U8), meta(*lead, 17, 3, 16, per)      # 264 x 264


def q4():
    w, s = weight()
    return dict(X=meta(4, N), Wq=w, scale=s, Y=meta(4, N), zero=meta(*s.shape), bias=meta(N))


def q4_swiglu():
    w, s = weight(per=4)
    return dict(X=meta(4, N), Wg=w, scale_g=s, Wu=w, scale_u=s, H=meta(4, N), zero_g=meta(*s.shape),
                zero_u=meta(*s.shape))


def moe_q4():
    w, s = weight(E)
    return dict(X=meta(40, N), expert_offsets=meta(E + 1, dtype=I32), Wq=w, scale=s, Y=meta(40, N),
                zero=meta(*s.shape), bias=meta(E, N))


def moe_q4_swiglu():
    w, s = weight(E, per=2)
    return dict(X=meta(40, N), expert_offsets=meta(E + 1, dtype=I32), Wg=w, scale_g=s, Wu=w, scale_u=s,
                H=meta(40, N))


def quantize():
    w, s = weight()
    return dict(W=meta(N, N), Wq=w, scale=s, zero=meta(*s.shape))


def pack():
    w, s = weight(per=2)
    return dict(codes=meta(N, N, dtype=U8), scale_in=meta(5, N), Wq=w, scale=s, zero_in=meta(5, N), zero=meta(*s.shape))


CALLS = {ffn.ffn_rmsnorm_forward: rms, ffn.ffn_rmsnorm_q8_forward: rms_q8, ffn.ffn_rmsnorm_backward: rms_bwd,
         ffn.moe_dispatch: dispatch, ffn.moe_dispatch_backward: dispatch_bwd, ffn.moe_combine: combine,
         ffn.moe_combine_backward: combine_bwd, ffn.moe_route_backward: route_bwd, ffn.ffn_q4_matvec: q4,
         ffn.ffn_q4_swiglu: q4_swiglu, ffn.moe_q4_matvec: moe_q4, ffn.moe_q4_swiglu: moe_q4_swiglu,
         ffn.ffn_q4_quantize: quantize, ffn.ffn_q4_pack: pack}


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_binding_needs_gpu_tensors(call):
    with pytest.raises(ValueError, match="on the GPU"):
        call(**CALLS[call]())


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_binding_refuses_each_tensor_of_another_shape_type_or_layout(call):
    """Every tensor in turn: one row more, another type, a transposed or strided view."""
    for name, good in CALLS[call]().items():
        taller = (good.shape[0] + 1, *good.shape[1:])
        deeper = (*good.shape, 1)
        # (the first dimension of X, dX and the like is what the others are measured by)
        for bad in (meta(*taller, dtype=good.dtype), meta(*deeper, dtype=good.dtype),
                    meta(*good.shape, dtype=torch.float16),
                    meta(*good.shape[:-1], 2 * good.shape[-1], dtype=good.dtype)[..., ::2]):
            if bad.is_contiguous() and bad.shape == good.shape and bad.dtype == good.dtype:
                continue
            with pytest.raises((ValueError, TypeError)) as e:
                call(**{**CALLS[call](), name: bad})
            assert "on the GPU" not in str(e.value) or bad.shape == taller, (name, tuple(bad.shape), str(e.value))


@pytest.mark.parametrize("call,change,msg", [
    (ffn.ffn_rmsnorm_forward, dict(S=None), "both or neither"),
    (ffn.ffn_rmsnorm_forward, dict(R=None), "both or neither"),
    (ffn.ffn_rmsnorm_forward, dict(gamma=None), "None"),
    (ffn.ffn_rmsnorm_q8_forward, dict(group=64), "group"),
    (ffn.ffn_rmsnorm_q8_forward, dict(group=0), "shape"),
    (ffn.ffn_rmsnorm_q8_forward, dict(Q=meta(M, N, dtype=U8)), "dtype"),
    (ffn.ffn_rmsnorm_backward, dict(dgamma=None), "None"),
    (ffn.ffn_rmsnorm_backward, dict(ws=meta(64, dtype=F32)), "uint8"),
    (ffn.moe_dispatch, dict(scale=None), "together"),
    (ffn.moe_dispatch, dict(scale_sorted=None), "together"),
    (ffn.moe_dispatch, dict(scale=meta(M, 0, dtype=F32)), "columns"),
    (ffn.moe_dispatch, dict(positions=None), "None"),
    (ffn.moe_dispatch, dict(topk_ids=meta(M, K, dtype=torch.int64)), "dtype"),
    (ffn.moe_combine, dict(Y=meta(M, N, dtype=F8)), "dtype"),
    (ffn.moe_combine_backward, dict(dw=None), "both or neither"),
    (ffn.moe_combine_backward, dict(Ys=None), "both or neither"),
    (ffn.ffn_q4_matvec, dict(scale=meta(17, 3, 16, 3)), "groups"),
    (ffn.ffn_q4_matvec, dict(scale=None), "None"),
    (ffn.ffn_q4_swiglu, dict(zero_u=None), "both zero points"),
    (ffn.ffn_q4_swiglu, dict(scale_u=meta(17, 3, 16, 2), zero_u=meta(17, 3, 16, 2)), "same group"),
    (ffn.ffn_q4_pack, dict(zero_in=None), "together"),
])
def test_binding_refuses(call, change, msg):
    with pytest.raises((ValueError, TypeError), match=msg):
        call(**{**CALLS[call](), **change})


def test_binding_refuses_unknown_names():
    for call in (ffn.ffn_q4_matvec, ffn.moe_q4_swiglu, ffn.ffn_q4_quantize):
        a = CALLS[call]()
        with pytest.raises(ValueError):
            call(**a, code="int3")
    with pytest.raises(ValueError, match="group"):
        ffn.ffn_q4_empty(264, 40, 48, device="cpu")
    assert [tuple(t.shape) for t in ffn.ffn_q4_empty(264, 40, 32, True, device="cpu")] == \
        [(3, 3, 1024), (3, 3, 16, 4), (3, 3, 16, 4)]
    assert ffn.ffn_q4_empty(264, 40, experts=5, device="cpu")[0].shape == (5, 3, 3, 1024)


# ---------------------------------------------------------------- the C ABI

class Abi:
    """One entry point: its arguments by name, pointers far apart, sizes small."""

    def __init__(self, entry, order, **values):
        self.entry, self.order, self.values = entry, order.split(), values
        self.pointers = [n for n in self.order if n not in values and n != "stream"]

    def __call__(self, **kw):
        v = {n: at(i) for i, n in enumerate(self.pointers)} | {"stream": None} | self.values | kw
        return getattr(ffn.lib(), self.entry)(*[v[n] for n in self.order])


SIZES = dict(M=32, N=264, dtype=ffn.BF16)
RMS = Abi("ffn_rmsnorm_forward", "X R gamma S Y rstd M N dtype eps stream", **SIZES, eps=1e-5)
RMS_Q8 = Abi("ffn_rmsnorm_q8_forward", "X R gamma S Q scale rstd M N dtype group eps stream", **SIZES, group=128, eps=1e-5)
RMS_BWD = Abi("ffn_rmsnorm_backward", "S dY dS gamma rstd dX dgamma M N dtype ws wsb stream", **SIZES, wsb=1 << 20)
DISPATCH = Abi("moe_dispatch", "X ids scale M N E k dtype cols Xs scale_sorted offsets entries positions ws wsb stream",
               **SIZES, E=6, k=2, cols=3, wsb=1 << 20)
DISPATCH_BWD = Abi("moe_dispatch_backward", "dXs positions dX M N k rows dtype stream", **SIZES, k=2, rows=40)
COMBINE = Abi("moe_combine", "Ys positions w R Y M N k rows dtype stream", **SIZES, k=2, rows=40)
COMBINE_BWD = Abi("moe_combine_backward", "dY Ys positions w dYs dw M N k rows dtype stream", **SIZES, k=2, rows=40)
ROUTE_BWD = Abi("moe_route_backward", "ids w dw dlogits M E k stream", M=32, E=6, k=2)
Q4 = dict(K=264, C=136, code=0, group=128)
MATVEC = Abi("ffn_q4_matvec", "X W s z bias Y M K C code group act stream", M=4, act=0, **Q4)
SWIGLU = Abi("ffn_q4_swiglu", "X Wg sg zg Wu su zu H M K C code group stream", M=4, **Q4)
MOE_MATVEC = Abi("moe_q4_matvec", "X off W s z bias Y rows E K C code group act stream", rows=40, E=6, act=0, **Q4)
MOE_SWIGLU = Abi("moe_q4_swiglu", "X off Wg sg zg Wu su zu H rows E K C code group stream", rows=40, E=6, **Q4)
QUANTIZE = Abi("ffn_q4_quantize", "W Wq s z K C dtype code group stream", dtype=ffn.F32, **Q4)
PACK = Abi("ffn_q4_pack", "codes s_in z_in Wq s z K C code group stream", **Q4)
ENTRIES = [RMS, RMS_Q8, RMS_BWD, DISPATCH, DISPATCH_BWD, COMBINE, COMBINE_BWD, ROUTE_BWD, MATVEC, SWIGLU, MOE_MATVEC,
           MOE_SWIGLU, QUANTIZE, PACK]
# pointers that may be NULL by themselves (others of theirs then too are checked below)
MAY = {RMS: {"rstd"}, RMS_Q8: {"rstd"}, RMS_BWD: {"dS"}, COMBINE: {"w", "R"}, COMBINE_BWD: {"w"},
       MATVEC: {"z", "bias"}, MOE_MATVEC: {"z", "bias"}, QUANTIZE: {"z"}}


@pytest.mark.parametrize("e", ENTRIES, ids=lambda e: e.entry)
def test_null_and_misaligned_pointers(e):
    for n in e.pointers:
        if n not in MAY.get(e, ()):
            assert e(**{n: None}) == E_INVAL and "NULL" in ffn.ffn_last_error() or "both" in ffn.ffn_last_error() \
                or "together" in ffn.ffn_last_error(), n
        assert e(**{n: at(50) + 8}) == E_ALIGN and "aligned" in ffn.ffn_last_error(), n


@pytest.mark.parametrize("e,kw,code", [
    (RMS, dict(M=-1), E_INVAL), (RMS, dict(N=0), E_INVAL), (RMS, dict(N=20), E_UNSUP), (RMS, dict(N=16392), E_UNSUP),
    (RMS, dict(M=1 << 31), E_UNSUP), (RMS, dict(M=TOP), E_UNSUP), (RMS, dict(dtype=2), E_INVAL),
    (RMS, dict(eps=0.0), E_INVAL), (RMS, dict(eps=-1.0), E_INVAL), (RMS, dict(eps=float("nan")), E_INVAL),
    (RMS, dict(R=None), E_INVAL), (RMS, dict(S=None), E_INVAL),
    (RMS_Q8, dict(group=64), E_UNSUP), (RMS_Q8, dict(group=-128), E_UNSUP), (RMS_Q8, dict(N=12), E_UNSUP),
    (RMS_BWD, dict(N=16392), E_UNSUP), (RMS_BWD, dict(dtype=7), E_INVAL), (RMS_BWD, dict(ws=at(9) + 16), E_ALIGN),
    (RMS_BWD, dict(wsb=ffn.ffn_rmsnorm_backward_workspace_size(32, 264) - 1), E_WS),
    (DISPATCH, dict(E=0), E_UNSUP), (DISPATCH, dict(E=257), E_UNSUP), (DISPATCH, dict(k=0), E_UNSUP),
    (DISPATCH, dict(k=9), E_UNSUP), (DISPATCH, dict(N=12), E_UNSUP), (DISPATCH, dict(N=1 << 23), E_UNSUP),
    (DISPATCH, dict(M=1 << 30), E_UNSUP), (DISPATCH, dict(M=TOP), E_UNSUP), (DISPATCH, dict(M=-1), E_INVAL),
    (DISPATCH, dict(dtype=3), E_INVAL), (DISPATCH, dict(cols=-1), E_INVAL), (DISPATCH, dict(cols=0), E_INVAL),
    (DISPATCH, dict(scale=None, scale_sorted=None), E_INVAL), (DISPATCH, dict(ws=at(20) + 64), E_ALIGN),
    (DISPATCH, dict(M=4096, wsb=ffn.moe_dispatch_workspace_size(4096, 6, 2) - 1), E_WS),
    (COMBINE, dict(dtype=ffn.E4M3), E_UNSUP), (COMBINE, dict(rows=-1), E_INVAL), (COMBINE, dict(rows=1 << 31), E_UNSUP),
    (COMBINE, dict(k=9), E_UNSUP), (COMBINE, dict(N=4), E_UNSUP), (DISPATCH_BWD, dict(rows=TOP), E_UNSUP),
    (COMBINE_BWD, dict(Ys=None), E_INVAL), (COMBINE_BWD, dict(dw=None), E_INVAL), (COMBINE_BWD, dict(N=0), E_INVAL),
    (ROUTE_BWD, dict(E=300), E_UNSUP), (ROUTE_BWD, dict(k=0), E_UNSUP), (ROUTE_BWD, dict(M=-5), E_INVAL),
    (MATVEC, dict(M=17), E_UNSUP), (MATVEC, dict(M=-1), E_INVAL), (MATVEC, dict(K=4), E_UNSUP),
    (MATVEC, dict(C=0), E_INVAL), (MATVEC, dict(K=1 << 22), E_UNSUP), (MATVEC, dict(K=65536, C=65536), E_UNSUP),
    (MATVEC, dict(code=2), E_INVAL), (MATVEC, dict(group=16), E_UNSUP), (MATVEC, dict(group=0), E_UNSUP),
    (MATVEC, dict(act=5), E_INVAL), (MATVEC, dict(code=1), E_INVAL),
    (SWIGLU, dict(zg=None), E_INVAL), (SWIGLU, dict(zu=None), E_INVAL), (SWIGLU, dict(code=1, zg=None, zu=None, M=99), E_UNSUP),
    (MOE_MATVEC, dict(rows=4097), E_UNSUP), (MOE_MATVEC, dict(E=0), E_UNSUP), (MOE_MATVEC, dict(E=257), E_UNSUP),
    (MOE_SWIGLU, dict(rows=-1), E_INVAL), (MOE_SWIGLU, dict(C=20), E_UNSUP),
    (QUANTIZE, dict(dtype=ffn.E4M3), E_INVAL), (QUANTIZE, dict(code=1), E_INVAL), (QUANTIZE, dict(K=12), E_UNSUP),
    (PACK, dict(z=None), E_INVAL), (PACK, dict(z_in=None), E_INVAL), (PACK, dict(code=1), E_INVAL),
])
def test_abi_refuses(e, kw, code):
    assert e(**kw) == code and ffn.ffn_last_error() != ""


# what may be the very array of what
SAME = {RMS: {("S", "X"), ("S", "R")}, RMS_Q8: {("S", "X"), ("S", "R")},
        RMS_BWD: {("dX", "S"), ("dX", "dY"), ("dX", "dS")}, COMBINE: {("Y", "R")}, COMBINE_BWD: {("dYs", "Ys")}}
OUTPUTS = {RMS: "S Y rstd", RMS_Q8: "S Q scale rstd", RMS_BWD: "dX dgamma ws",
           DISPATCH: "Xs scale_sorted offsets entries positions ws", DISPATCH_BWD: "dX", COMBINE: "Y",
           COMBINE_BWD: "dYs dw", ROUTE_BWD: "dlogits", MATVEC: "Y", SWIGLU: "H", MOE_MATVEC: "Y", MOE_SWIGLU: "H",
           QUANTIZE: "Wq s z", PACK: "Wq s z"}


@pytest.mark.parametrize("e", ENTRIES, ids=lambda e: e.entry)
def test_overlapping_arrays_are_refused(e):
    """Every output on every other array: at its very place, and one alignment before and behind it."""
    outs = OUTPUTS[e].split()
    base = {n: at(i) for i, n in enumerate(e.pointers)}
    for out in outs:
        for other in e.pointers:
            if other == out:
                continue
            for shift in (0,) if out == "ws" else (0, 16, -16):    # (a workspace lies at multiples of 256)
                if shift == 0 and (out, other) in SAME.get(e, ()):
                    continue
                rc = e(**{out: base[other] + shift})
                assert rc == E_INVAL and "overlap" in ffn.ffn_last_error(), (out, other, shift, ffn.ffn_last_error())


def test_no_rows_need_no_pointers():
    none = dict.fromkeys
    assert RMS(M=0, **none(["X", "R", "S", "Y", "rstd"])) == 0
    assert RMS_Q8(M=0, **none(["X", "R", "S", "Q", "scale", "rstd"])) == 0
    assert COMBINE(M=0, rows=0, **none(["Ys", "positions", "w", "R", "Y"])) == 0
    assert COMBINE_BWD(M=0, rows=0, **none(["dY", "Ys", "positions", "w", "dYs", "dw"])) == 0
    assert ROUTE_BWD(M=0, **none(["ids", "w", "dw", "dlogits"])) == 0
    assert MATVEC(M=0, X=None, Y=None) == 0 and MOE_SWIGLU(rows=0, X=None, H=None) == 0
    # what is not per row is still checked
    assert RMS(M=0, gamma=None) == E_INVAL and MATVEC(M=0, X=None, Y=None, W=None) == E_INVAL


def test_sizes():
    assert ffn.ffn_rmsnorm_backward_workspace_size(4, 12) == 0 and ffn.ffn_rmsnorm_backward_workspace_size(-1, 64) == 0
    assert ffn.ffn_rmsnorm_backward_workspace_size(0, 64) == 256
    for m in (1, 255, 256, 257, 1 << 30):
        assert ffn.ffn_rmsnorm_backward_workspace_size(m, 8192) >= 4 * 8192 * min(m, 256)
    assert ffn.moe_dispatch_workspace_size(4, 300, 2) == 0 and ffn.moe_dispatch_workspace_size(4, 8, 9) == 0
    for m in (0, 1, 512):
        assert ffn.moe_dispatch_workspace_size(m, 8, 2) >= 256
    for m in (513, 6145, 1 << 20, 1 << 29):      # (up to 12288 entries need none)
        assert ffn.moe_dispatch_workspace_size(m, 64, 2) >= 4 * 64 * min(256, -(-2 * m // 1024)) // 2
        assert ffn.moe_dispatch_workspace_size(m, 64, 2) <= 4 * 64 * 256
    assert ffn.ffn_q4_bytes(264, 40) == 3 * 3 * 1024 and ffn.ffn_q4_bytes(8, 8) == 1024
    assert ffn.ffn_q4_bytes(264, 42) == 0 and ffn.ffn_q4_bytes(1 << 22, 8) == 0
