"""Refusals of the gated linear recurrence and the norms, without a GPU: every call here fails
validation (or computes nothing), so no kernel is launched and no pointer dereferenced."""
import ctypes
import math

import pytest
import torch

FAKE = 1 << 20


@pytest.fixture(scope="module")
def ssd():
    from selective_state_space_10_b200 import build
    build.build()
    from selective_state_space_10_b200 import ssd as mod
    return mod


def _p(v):
    return None if v is None else ctypes.c_void_p(v)


def _glr(ssd, which, dims=(2, 8, 64, 64, 64), dtype=1, ws=FAKE, ws_bytes=1 << 40, **ptr):
    d = None if dims is None else ctypes.byref(ssd.GlrDims(*dims))
    p = dict.fromkeys(("x", "r", "i", "A", "init", "h", "final", "state", "dh", "dfinal", "dx", "dr", "di", "dA",
                       "dinit"), FAKE)
    p.update(ptr)
    p = {k: _p(v) for k, v in p.items()}
    if which == "prefill":
        return ssd.lib.ssd_glr_prefill(d, dtype, p["x"], p["r"], p["i"], p["A"], p["init"], p["h"], p["final"], None)
    if which == "step":
        return ssd.lib.ssd_glr_decode_step(d, dtype, p["state"], p["x"], p["r"], p["i"], p["A"], p["h"], None)
    return ssd.lib.ssd_glr_backward(d, dtype, p["x"], p["r"], p["i"], p["A"], p["init"], p["h"], p["dh"], p["dfinal"],
                                    p["dx"], p["dr"], p["di"], p["dA"], p["dinit"], _p(ws), ws_bytes, None)


BAD_SIZES = [dict(dims=None), dict(dtype=2), dict(dims=(-1, 8, 64, 64, 64)), dict(dims=(2, 8, 0, 64, 64)),
             dict(dims=(2, 8, 64, 63, 64)), dict(dims=(1 << 31, 8, 64, 64, 64)), dict(dims=(1 << 29, 8, 64, 64, 64)),
             dict(dims=(2, 8, 64, 1 << 42, 64)), dict(x=None), dict(r=None), dict(i=None), dict(A=None), dict(h=None),
             dict(x=FAKE + 1), dict(r=FAKE + 1), dict(A=FAKE + 2), dict(h=FAKE + 1), dict(dtype=0, x=FAKE + 2)]


@pytest.mark.parametrize("which", ["prefill", "step", "backward"])
@pytest.mark.parametrize("case", BAD_SIZES, ids=str)
def test_glr_rejects_invalid(ssd, which, case):
    assert _glr(ssd, which, **case) == ssd.ERR_INVALID_ARG


@pytest.mark.parametrize("which,case", [
    ("prefill", dict(dims=(2, -1, 64, 64, 64))), ("prefill", dict(init=FAKE + 2)), ("prefill", dict(final=None)),
    ("prefill", dict(final=FAKE + 1)), ("prefill", dict(dims=(2, 0, 64, 64, 64), final=None)),
    ("prefill", dict(dims=(1 << 20, 1 << 20, 64, 64, 64))),
    ("step", dict(state=None)), ("step", dict(state=FAKE + 2)),
    ("backward", dict(dims=(2, 8, 64, 64, 63))), ("backward", dict(dh=None)), ("backward", dict(dx=None)),
    ("backward", dict(dr=FAKE + 1)), ("backward", dict(di=None)), ("backward", dict(dA=None)),
    ("backward", dict(dfinal=FAKE + 1)), ("backward", dict(dinit=FAKE + 2)), ("backward", dict(init=FAKE + 2)),
], ids=str)
def test_glr_rejects_invalid_of_each_call(ssd, which, case):
    assert _glr(ssd, which, **case) == ssd.ERR_INVALID_ARG


def test_glr_workspace(ssd):
    d = ssd.GlrDims(2, 8, 64, 64, 64)
    need = ssd.lib.ssd_glr_backward_workspace_size(ctypes.byref(d), 1)
    assert need >= 2 * 64 * 4
    for bad in (dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=need - 1)):
        assert _glr(ssd, "backward", **bad) == ssd.ERR_WORKSPACE
    for dims in ((0, 8, 64, 64, 64), (2, 0, 64, 64, 64), (2, 8, 64, 60, 64)):
        assert ssd.lib.ssd_glr_backward_workspace_size(ctypes.byref(ssd.GlrDims(*dims)), 1) == 0


def test_glr_of_nothing_is_a_no_op(ssd):
    none = dict.fromkeys(("x", "r", "i", "A", "init", "h", "final", "state"))
    assert _glr(ssd, "prefill", dims=(0, 8, 64, 64, 64), **none) == ssd.OK
    assert _glr(ssd, "step", dims=(0, 8, 64, 64, 64), **none) == ssd.OK
    # no tokens and the state updated in place: nothing to copy
    assert _glr(ssd, "prefill", dims=(2, 0, 64, 64, 64), init=FAKE, final=FAKE) == ssd.OK


def _norm(ssd, which, dims=(4, 64, 2, 64, 64), dtype=1, wdt=0, eps=1e-5, gate_first=1, ws=FAKE, ws_bytes=1 << 40, **ptr):
    d = None if dims is None else ctypes.byref(ssd.NormDims(*dims))
    p = dict.fromkeys(("x", "scale", "wide", "w", "wide_out", "out", "dout", "dwide", "dx", "dw", "dscale"), FAKE)
    p.update(ptr)
    p = {k: _p(v) for k, v in p.items()}
    if which == "residual":
        return ssd.lib.ssd_residual_norm(d, dtype, wdt, p["x"], p["scale"], p["wide"], p["w"], eps, p["wide_out"],
                                         p["out"], None)
    if which == "residual_backward":
        return ssd.lib.ssd_residual_norm_backward(d, dtype, wdt, p["x"], p["scale"], p["wide"], p["w"], eps, p["dout"],
                                                  p["dwide"], p["dx"], p["wide_out"], p["dw"], p["dscale"], _p(ws),
                                                  ws_bytes, None)
    if which == "gated":
        return ssd.lib.ssd_gated_norm(d, dtype, wdt, gate_first, p["wide"], p["x"], p["w"], eps, p["out"], None)
    return ssd.lib.ssd_gated_norm_backward(d, dtype, wdt, gate_first, p["wide"], p["x"], p["w"], eps, p["dout"],
                                           p["wide_out"], p["dx"], p["dw"], _p(ws), ws_bytes, None)


ALL = ["residual", "residual_backward", "gated", "gated_backward"]


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("case", [
    dict(dims=None), dict(dtype=2), dict(wdt=-1), dict(dims=(-1, 64, 1, 64, 64)), dict(dims=(4, 0, 1, 64, 64)),
    dict(dims=(1 << 31, 64, 1, 64, 64)), dict(eps=0.0), dict(eps=-1e-5), dict(eps=math.nan), dict(eps=math.inf),
    dict(w=None), dict(w=FAKE + 2), dict(x=FAKE + 1), dict(wide_out=FAKE + 2)], ids=str)
def test_norms_reject_invalid(ssd, which, case):
    if which == "gated" and "wide_out" in case:
        case = dict(out=FAKE + 1)
    assert _norm(ssd, which, **case) == ssd.ERR_INVALID_ARG


@pytest.mark.parametrize("which,case", [
    ("residual", dict(x=None)), ("residual", dict(out=None)), ("residual", dict(out=FAKE + 1)),
    ("residual", dict(scale=FAKE + 2)),
    ("residual_backward", dict(wide=None)), ("residual_backward", dict(dout=None)), ("residual_backward", dict(x=None)),
    ("residual_backward", dict(dx=FAKE + 1)), ("residual_backward", dict(dw=FAKE + 1)),
    ("residual_backward", dict(dscale=FAKE + 1)), ("residual_backward", dict(dwide=FAKE + 2)),
    ("gated", dict(wide=None)), ("gated", dict(x=None)), ("gated", dict(out=None)), ("gated", dict(dims=(4, 64, 3, 64, 64))),
    ("gated", dict(dims=(4, 64, 0, 64, 64))), ("gated", dict(dims=(4, 64, 1, 63, 64))),
    ("gated", dict(dims=(1 << 30, 64, 64, 64, 64))), ("gated", dict(dims=(4, 64, 1, 1 << 41, 64))),
    ("gated_backward", dict(dims=(4, 64, 1, 64, 63))), ("gated_backward", dict(dout=None)),
    ("gated_backward", dict(dx=FAKE + 1)), ("gated_backward", dict(dw=FAKE + 1)),
], ids=str)
def test_norms_reject_invalid_of_each_call(ssd, which, case):
    assert _norm(ssd, which, **case) == ssd.ERR_INVALID_ARG


@pytest.mark.parametrize("which", ALL)
def test_norms_refuse_a_narrow_stream_beside_fp32(ssd, which):
    assert _norm(ssd, which, dtype=0, wdt=1) == ssd.ERR_UNSUPPORTED


@pytest.mark.parametrize("which", ["residual_backward", "gated_backward"])
def test_norm_workspace(ssd, which):
    need = ssd.lib.ssd_norm_backward_workspace_size(ctypes.byref(ssd.NormDims(4, 64, 1, 64, 64)))
    assert need >= 2 * 64 * 4
    for bad in (dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=need - 1)):
        assert _norm(ssd, which, **bad) == ssd.ERR_WORKSPACE
    assert ssd.lib.ssd_norm_backward_workspace_size(ctypes.byref(ssd.NormDims(0, 64, 1, 64, 64))) == 0


@pytest.mark.parametrize("which", ALL)
def test_norms_of_no_rows_are_no_ops(ssd, which):
    none = dict.fromkeys(("x", "scale", "wide_out", "out", "dout", "dwide", "dx", "w", "dw", "dscale"))
    assert _norm(ssd, which, dims=(0, 64, 1, 64, 64), **none) == ssd.OK


def test_binding_refuses_bad_tensors(ssd):
    """The binding's own checks come before any call: CPU tensors, types, shapes, strides."""
    t = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        ssd.glr_prefill(t, t, t, torch.zeros(8))
    with pytest.raises(ValueError, match="unsupported x dtype"):
        ssd.residual_norm(t.half(), torch.zeros(8))
    with pytest.raises(ValueError, match="must be \\[b,L,D\\]"):
        ssd.glr_prefill(t[0], t[0], t[0], torch.zeros(8))
    dev, f = -1, torch.float32  # a CPU tensor's get_device()
    row = lambda v: ssd._row_stride(v, "z", v.shape, f, dev)
    assert row(torch.zeros(2, 3, 24)[..., 8:16]) == 24
    assert row(torch.zeros(2, 1, 24)[..., 8:16]) == 24
    assert row(torch.zeros(4, 9)[:1, 1:6]) == 5 or row(torch.zeros(4, 9)[:1, 1:6]) == 9
    assert row(torch.zeros(2, 3, 8)) == 8 and row(torch.zeros(0, 8)) == 8
    for bad in (torch.zeros(8, 3).t(), torch.zeros(1, 8).expand(3, 8), torch.zeros(2, 6, 8)[:, ::2][:, :2],
                torch.zeros(4, 16)[:, ::2]):
        with pytest.raises(ValueError, match="rows must be"):
            row(bad)
    a, b = torch.zeros(3, 24)[:, :8], torch.zeros(3, 16)[:, :8]
    with pytest.raises(ValueError, match="same row stride"):
        ssd._same_stride(("x", "r", "i"), a, b, a, a.shape, f, dev)
    with pytest.raises(ValueError, match="shape"):
        ssd._row_stride(a, "z", (3, 9), f, dev)
