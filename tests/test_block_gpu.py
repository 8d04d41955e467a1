"""GPU parity of the gated linear recurrence and the norms with the fp64 oracle
(oracle/block.py), within the error bounds that the oracle carries for fp32 arithmetic plus
one rounding to the output's type (at most eps / 2 of the value)."""
import os
import subprocess
import sys
import zlib

import numpy as np
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu
EPS = 1e-5
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ssd():
    from selective_state_space_10_b200 import ssd as mod
    return mod


def _rand(gen, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).to(dtype).cuda()


def _gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(got, ref, bound, what):
    """|got - ref| <= bound + half a step of got's type (1e-36: results below the normal range may be flushed)."""
    half = torch.finfo(got.dtype).eps / 2
    g = _np(got)
    assert g.shape == ref.shape, what
    assert np.isfinite(g).all(), f"{what}: not finite"
    tol = bound + half * (np.abs(ref) + bound) + 1e-36
    over = np.abs(g - ref) / tol
    assert over.size == 0 or over.max() <= 1, f"{what}: {over.max():.2f} times its bound at {np.unravel_index(over.argmax(), over.shape)}"


def _wide(gen, b, L, D, dtype, layout):
    """x, r, i [b, L, D]: contiguous, slices of one [b, L, 3D], or odd-offset slices (no wide loads)."""
    if layout == "own":
        return [_rand(gen, b, L, D, dtype=dtype, std=1.5) for _ in range(3)]
    pad = 0 if layout == "sliced" else 1
    return list(_rand(gen, b, L, 3 * D + pad, dtype=dtype, std=1.5)[..., pad:].split(D, dim=2))


def _decays(gen, D):
    A = -torch.exp(torch.empty(D).uniform_(np.log(2e-3), np.log(3.0), generator=gen))
    return A.cuda()


SHAPES = [(1, 1, 1), (1, 1, 8), (2, 5, 3), (3, 64, 64), (1, 65, 72), (2, 127, 130), (1, 700, 8), (1, 2100, 200),
          (4, 33, 520), (1, 4097, 64), (5, 2, 1000),
          (700, 3, 64), (40, 100, 1024)]


@pytest.mark.parametrize("layout", ["own", "sliced", "odd"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("b,L,D", SHAPES + [(2, 300, 74)])
def test_glr_prefill_and_backward(ssd, b, L, D, dtype, layout):
    gen = _gen(b, L, D, layout)
    x, r, i = _wide(gen, b, L, D, dtype, layout)
    A = _decays(gen, D)
    init = layout != "own"
    h0 = _rand(gen, b, D) if init else None
    h, last = ssd.glr_prefill(x, r, i, A, initial_state=h0)
    args = [_np(v) for v in (x, r, i, A)]
    ref, rlast, bound = block.glr(*args, _np(h0))
    check(h, ref, bound, "h")
    check(last, rlast, bound[:, -1], "final state")
    dh = _rand(gen, b, L, D, dtype=dtype)
    dfinal = _rand(gen, b, D) if init else None
    if layout == "own":
        out = ssd.glr_backward(x, r, i, A, h, dh, h0, dfinal)
    else:  # gradients into slices of one array; what surrounds them stays
        buf = torch.full((b, L, 3 * D + 8), 7.0, dtype=dtype, device="cuda")
        dx, dr, di = buf[..., 5:5 + 3 * D].split(D, dim=2) if layout == "odd" else buf[..., 8:].split(D, dim=2)
        out = ssd.glr_backward(x, r, i, A, h, dh, h0, dfinal, dx=dx, dr=dr, di=di)
        edge = torch.cat([buf[..., :5], buf[..., 5 + 3 * D:]], -1) if layout == "odd" else buf[..., :8]
        assert (edge == 7).all()
    want, tol = block.glr_backward(*args, _np(h), _np(dh), _np(h0), _np(dfinal))
    for got, name in zip(out, ("dx", "dr", "di", "dA", "dh0")):
        check(got, want[name], tol[name], name)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("b,D,layout", [(1, 1, "own"), (3, 8, "sliced"), (7, 131, "own"), (2, 520, "odd"), (256, 72, "sliced")])
def test_glr_decode_step(ssd, b, D, layout, dtype):
    gen = _gen(b, D, layout)
    x, r, i = (v[:, 0] for v in _wide(gen, b, 1, D, dtype, layout))
    A, state = _decays(gen, D), _rand(gen, b, D)
    ref, _, bound = block.glr(_np(x)[:, None], _np(r)[:, None], _np(i)[:, None], _np(A), _np(state))
    h = ssd.glr_decode_step(state, x, r, i, A)
    check(h, ref[:, 0], bound[:, 0], "h")
    check(state, ref[:, 0], bound[:, 0], "state")


def test_glr_extreme_gates_and_decays(ssd):
    """Saturated and infinite logits, decays of 1 and next to it, and to nothing in one step."""
    vals = torch.tensor([-float("inf"), -200.0, -90.0, -30.0, -1.0, 0.0, 1.0, 30.0, 90.0, 200.0, float("inf")])
    A = torch.tensor([0.0, -1e-30, -1e-9, -1e-4, -0.499, -0.5, -0.501, -2.0, -50.0, -3e4]).cuda()
    L, D = len(vals) ** 2, len(A)
    r = vals.repeat_interleave(len(vals))[None, :, None].expand(1, L, D).contiguous().cuda()
    i = vals.repeat(len(vals))[None, :, None].expand(1, L, D).contiguous().cuda()
    gen = _gen(7)
    x, dh, h0 = _rand(gen, 1, L, D), _rand(gen, 1, L, D), _rand(gen, 1, D)
    h, last = ssd.glr_prefill(x, r, i, A, initial_state=h0)
    args = [_np(v) for v in (x, r, i, A)]
    with np.errstate(over="ignore"):
        ref, rlast, bound = block.glr(*args, _np(h0))
        want, tol = block.glr_backward(*args, _np(h), _np(dh), _np(h0))
    # a sigmoid below the normal range (1e-38) is flushed to 0: its term of the sum is at most sqrt(2e-38 * 3e4) |x|
    floor = 1e-16 * np.abs(_np(x)).max() * L
    check(h, ref, bound + floor, "h")
    # the same flush in the slope a^2 / beta of the decay: the term it multiplies is off by as little
    for got, name in zip(ssd.glr_backward(x, r, i, A, h, dh, h0), ("dx", "dr", "di", "dA", "dh0")):
        check(got, want[name], tol[name] + 100 * floor, name)


def test_glr_nan_stays_in_its_channel(ssd):
    gen = _gen(8)
    x, r, i = (_rand(gen, 1, 300, 16) for _ in range(3))
    A = _decays(gen, 16)
    clean, _ = ssd.glr_prefill(x, r, i, A)
    x[0, 100, 3] = float("nan")
    h, last = ssd.glr_prefill(x, r, i, A)
    other = [c for c in range(16) if c != 3]
    assert torch.equal(h[..., other], clean[..., other]) and torch.equal(h[:, :100], clean[:, :100])
    assert torch.isnan(h[0, 100:, 3]).all() and torch.isnan(last[0, 3])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_glr_pieces_and_steps_continue_one_another(ssd, dtype):
    """A prompt in pieces (state in place), then single tokens, against the oracle over all of it."""
    b, L, D = 3, 400, 136
    gen = _gen(9)
    x, r, i = _wide(gen, b, L, D, dtype, "own")
    A = _decays(gen, D)
    state, parts = torch.zeros(b, D, device="cuda"), []
    for lo, hi in ((0, 1), (1, 130), (130, 390)):
        v = [t[:, lo:hi].contiguous() for t in (x, r, i)]
        h, same = ssd.glr_prefill(*v, A, initial_state=state, final_state=state)
        assert same is state
        parts.append(h)
    for t in range(390, L):
        parts.append(ssd.glr_decode_step(state, x[:, t], r[:, t], i[:, t], A)[:, None])
    ref, last, bound = block.glr(_np(x), _np(r), _np(i), _np(A))
    check(torch.cat(parts, 1), ref, bound, "h")
    check(state, last, bound[:, -1], "state")


def test_glr_of_no_tokens(ssd):
    z = torch.empty(2, 0, 8, device="cuda")
    A, h0, df = -torch.ones(8, device="cuda"), torch.randn(2, 8, device="cuda"), torch.randn(2, 8, device="cuda")
    h, last = ssd.glr_prefill(z, z, z, A, initial_state=h0)
    assert h.shape == (2, 0, 8) and torch.equal(last, h0)
    assert torch.equal(ssd.glr_prefill(z, z, z, A)[1], torch.zeros_like(h0))
    dx, dr, di, dA, dh0 = ssd.glr_backward(z, z, z, A, h, z, h0, df)
    assert torch.equal(dA, torch.zeros_like(A)) and torch.equal(dh0, df)
    assert torch.equal(ssd.glr_backward(z, z, z, A, h, z)[4], torch.zeros_like(h0))
    e = torch.empty(0, 5, 8, device="cuda")
    assert ssd.glr_prefill(e, e, e, A)[0].shape == e.shape
    assert torch.equal(ssd.glr_backward(e, e, e, A, e, e)[3], torch.zeros_like(A))


WIDTHS = [(1, 1), (3, 8), (5, 7), (4, 64), (33, 520), (2, 768), (7, 1001), (300, 2560), (3, 5120), (2, 9000), (1, 33000),
          (700, 24)]


@pytest.mark.parametrize("types", [(F32, F32), (BF, F32), (BF, BF)], ids=["f32", "bf16-f32", "bf16"])
@pytest.mark.parametrize("rows,D", WIDTHS)
def test_residual_norm(ssd, rows, D, types):
    tx, tr = types
    gen = _gen(rows, D)
    x, w, scale = _rand(gen, rows, D, dtype=tx), 1 + _rand(gen, D, std=0.2), _rand(gen, D)
    res, dres, dout = _rand(gen, rows, D, dtype=tr, std=2), _rand(gen, rows, D, dtype=tr), _rand(gen, rows, D, dtype=tx)
    for sc, rs in ((scale, res), (None, res), (scale, None), (None, None)):
        out, s = ssd.residual_norm(x, w, residual=rs, scale=sc, residual_dtype=tr, eps=EPS)
        ro, rsum, bo, bs = block.residual_norm(_np(x), _np(sc), _np(rs), _np(w), EPS)
        check(out, ro, bo, "out")
        check(s, rsum, bs, "residual_out")
        dr = dres if rs is not None else None
        got = ssd.residual_norm_backward(dout, s, w, x=x, scale=sc, dresidual_out=dr, eps=EPS)
        want, tol = block.residual_norm_backward(_np(x), _np(sc), _np(s), _np(w), EPS, _np(dout), _np(dr))
        for g, name in zip(got, ("dx", "dres", "dw", "dscale")):
            if name in want:
                check(g, want[name], tol[name], name)
            else:
                assert g is None


GATED = [(1, 1, 1), (3, 8, 1), (5, 21, 3), (4, 64, 8), (33, 520, 1), (2, 1536, 24), (7, 1001, 7), (300, 2560, 2), (3, 5120, 1),
         (2, 9000, 1), (1, 33000, 1), (130, 1536, 1), (700, 48, 2)]


@pytest.mark.parametrize("gate_first", [True, False], ids=["gate_first", "norm_first"])
@pytest.mark.parametrize("types", [(F32, F32), (BF, F32), (BF, BF)], ids=["f32", "bf16-f32", "bf16"])
@pytest.mark.parametrize("rows,D,G", GATED)
def test_gated_norm(ssd, rows, D, G, types, gate_first):
    tx, ty = types
    gen = _gen(rows, D, G)
    y, w, dout = _rand(gen, rows, D, dtype=ty), 1 + _rand(gen, D, std=0.2), _rand(gen, rows, D, dtype=tx)
    for lo, pad in ((0, 0), (0, 16), (3, 7)):  # own rows, wide-load slices, odd slices
        z = _rand(gen, rows, D + pad, dtype=tx, std=2)[:, lo:lo + D]
        out = ssd.gated_norm(y, z, w, ngroups=G, gate_first=gate_first, eps=EPS)
        ref, bound = block.gated_norm(_np(y), _np(z), _np(w), G, gate_first, EPS)
        check(out, ref, bound, "out")
        dzs = torch.full((rows, D + pad), 7.0, dtype=tx, device="cuda")
        got = ssd.gated_norm_backward(dout, y, z, w, ngroups=G, gate_first=gate_first, eps=EPS, dz=dzs[:, lo:lo + D])
        want, tol = block.gated_norm_backward(_np(y), _np(z), _np(w), G, gate_first, EPS, _np(dout))
        for g, name in zip(got, ("dy", "dz", "dw")):
            check(g, want[name], tol[name], name)
        assert (dzs[:, :lo] == 7).all() and (dzs[:, lo + D:] == 7).all()


def test_norms_of_zero_and_tiny_and_large_rows(ssd):
    x = torch.zeros(4, 64, device="cuda")
    x[1], x[2], x[3] = 1e-20, 1e15, -1e-3
    w = torch.ones(64, device="cuda")
    out, s = ssd.residual_norm(x, w, eps=EPS)
    ref, _, bound, _ = block.residual_norm(_np(x), None, None, _np(w), EPS)
    check(out, ref, bound, "out")
    assert (out[0] == 0).all() and torch.equal(s, x)
    z = torch.full_like(x, -200.0)  # silu(-200) vanishes: a row whose gate leaves nothing
    for first in (True, False):
        assert (ssd.gated_norm(torch.ones_like(x), z, w, gate_first=first).abs() < 1e-30).all()
        for g in ssd.gated_norm_backward(torch.ones_like(x), torch.ones_like(x), z, w, gate_first=first):
            assert torch.isfinite(g).all()
    for inf in (float("inf"), -float("inf"), float("nan")):  # an outlier ends in its own row
        y = torch.ones(3, 64, device="cuda")
        y[1, 5] = inf
        got = ssd.gated_norm(y, torch.ones_like(y), w)
        assert torch.isfinite(got[[0, 2]]).all() and not torch.isfinite(got[1]).all()


def test_first_gradient_of_a_process():
    """A kernel's shared memory is asked for before its first launch, not left from a larger call: 1536 fp32 channels
    take 48 KB of it beside the kernel's own."""
    code = ("import torch; from selective_state_space_10_b200 import ssd; y = torch.ones(9, 1536, device='cuda'); "
            "w = torch.ones(1536, device='cuda'); ssd.gated_norm_backward(y, y, y, w); torch.cuda.synchronize()")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_norms_of_no_rows(ssd):
    e, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    assert ssd.residual_norm(e, w, residual=e, scale=w)[0].shape == e.shape
    assert ssd.gated_norm(e, e, w).shape == e.shape
    dw, ds = ssd.residual_norm_backward(e, e, w, x=e, scale=w)[2:]
    assert (dw == 0).all() and (ds == 0).all()
    assert (ssd.gated_norm_backward(e, e, e, w)[2] == 0).all()


def test_in_place_forms(ssd):
    gen = _gen(11)
    x, res, w = _rand(gen, 37, 1536, dtype=BF), _rand(gen, 37, 1536), 1 + _rand(gen, 1536, std=0.1)
    out, s = ssd.residual_norm(x, w, residual=res)
    kept = res.clone()
    out2, s2 = ssd.residual_norm(x, w, residual=kept, residual_out=kept)
    assert s2 is kept and torch.equal(out, out2) and torch.equal(s, kept)
    d = _rand(gen, 37, 1536)
    a = ssd.residual_norm_backward(x, s, w, dresidual_out=d)
    b = ssd.residual_norm_backward(x, s, w, dresidual_out=d, dresidual=d)
    assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3])) and b[1] is d
    y, z = _rand(gen, 37, 1536, dtype=BF), _rand(gen, 37, 1536, dtype=BF)
    for target in (1, 2):
        first = ssd.gated_norm(y, z, w, ngroups=3)
        yz = [y.clone(), z.clone()]
        assert torch.equal(ssd.gated_norm(*yz, w, ngroups=3, out=yz[target - 1]), first)
    A, h0, df = _decays(gen, 136), _rand(gen, 2, 136), _rand(gen, 2, 136)
    xri = _wide(gen, 2, 300, 136, BF, "own")
    h, last = ssd.glr_prefill(*xri, A, initial_state=h0)
    a = ssd.glr_backward(*xri, A, h, h, h0, df)
    b = ssd.glr_backward(*xri, A, h, h, h0, df, dinitial_state=df)
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and b[4] is df


def _everything(ssd, t):
    h, last = ssd.glr_prefill(t["x"], t["r"], t["i"], t["A"], initial_state=t["h0"])
    g = ssd.glr_backward(t["x"], t["r"], t["i"], t["A"], h, t["dh"], t["h0"], t["h0"])
    out, s = ssd.residual_norm(t["x"], t["w"], residual=t["dh"], scale=t["sc"])
    rb = ssd.residual_norm_backward(t["dh"], s, t["w"], x=t["x"], scale=t["sc"], dresidual_out=t["x"])
    n = ssd.gated_norm(h, t["r"], t["w"], ngroups=2)
    gb = ssd.gated_norm_backward(t["dh"], h, t["r"], t["w"], ngroups=2, gate_first=False)
    return [h, last, out, s, n, *g, *rb, *gb]


def _inputs(seed, b=2, L=600, D=272, dtype=BF):
    gen = _gen(seed)
    x, r, i, dh = (_rand(gen, b, L, D, dtype=dtype) for _ in range(4))
    return dict(x=x, r=r, i=i, dh=dh, A=_decays(gen, D), h0=_rand(gen, b, D), w=1 + _rand(gen, D, std=0.1),
                sc=_rand(gen, D))


def test_repeatable_bit_for_bit(ssd):
    t = _inputs(12)
    for a, b in zip(_everything(ssd, t), _everything(ssd, t)):
        assert torch.equal(a, b)


def test_on_a_side_stream_and_in_graphs(ssd):
    """On another stream, and captured: two graphs, each with its own workspaces, replayed in turn with new
    inputs, give what eager calls give."""
    t, u = _inputs(13), _inputs(14)
    want = {id(t): _everything(ssd, t), id(u): _everything(ssd, u)}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _everything(ssd, t)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[id(t)]))
    held = [{k: v.clone() for k, v in t.items()} for _ in range(2)]
    graphs, outs = [torch.cuda.CUDAGraph() for _ in held], []
    for g, v in zip(graphs, held):
        with torch.cuda.graph(g):
            outs.append(_everything(ssd, v))
    for order in ((t, u), (u, t)):
        for v, new in zip(held, order):
            for k in v:
                v[k].copy_(new[k])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out, new in zip(outs, order):
            assert all(torch.equal(a, b) for a, b in zip(out, want[id(new)]))


def test_first_calls_of_a_process_may_be_captured():
    """No call needs an eager one before it: launch set-up and queries are allowed during capture."""
    code = """
import torch
from selective_state_space_10_b200 import ssd
x = torch.randn(2, 700, 128, device='cuda', dtype=torch.bfloat16); y = torch.randn(2, 700, 128, device='cuda')
w = torch.ones(128, device='cuda')
def run():
    h, s = ssd.glr_prefill(x, x, x, -w)
    g = ssd.glr_backward(x, x, x, -w, h, x, None, s)
    out, r = ssd.residual_norm(x, w, residual=y, scale=w)
    b = ssd.residual_norm_backward(x, r, w, x=x, scale=w)
    return [h, s, out, r, ssd.gated_norm(y, x, w), ssd.glr_decode_step(s.clone(), x[:, 0], x[:, 1], x[:, 2], -w), *g, *b,
            *ssd.gated_norm_backward(x, y, x, w)]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_outputs_not_wanted(ssd):
    """NULL for an optional array of the C calls leaves the others as they are with it."""
    gen, null = _gen(19), None
    rows, D = 37, 512
    x, y, dout, res = (_rand(gen, rows, D) for _ in range(4))
    w, sc = 1 + _rand(gen, D, std=0.1), _rand(gen, D)
    st = torch.cuda.current_stream().cuda_stream
    dims = ssd.NormDims(rows, D, 2, D, D)
    out, s = ssd.residual_norm(x, w, residual=res, scale=sc)
    only = torch.empty_like(out)
    assert ssd.lib.ssd_residual_norm(dims, 0, 0, x.data_ptr(), sc.data_ptr(), res.data_ptr(), w.data_ptr(), EPS, null,
                                     only.data_ptr(), st) == ssd.OK
    assert torch.equal(only, out)
    need = ssd.lib.ssd_norm_backward_workspace_size(dims)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = ssd.residual_norm_backward(dout, s, w, x=x, scale=sc, dresidual_out=res)
    gates = ssd.gated_norm_backward(dout, y, x, w, ngroups=2)
    for k in range(4):
        got = [torch.full_like(t, 7.0) for t in want]
        p = [null if j == k else t.data_ptr() for j, t in enumerate(got)]
        assert ssd.lib.ssd_residual_norm_backward(dims, 0, 0, x.data_ptr() if k != 3 else null, sc.data_ptr(),
                                                  s.data_ptr(), w.data_ptr(), EPS, dout.data_ptr(), res.data_ptr(), *p,
                                                  ws.data_ptr(), need, st) == ssd.OK
        for j, t in enumerate(got):
            assert (t == 7).all() if j == k else torch.equal(t, want[j])
        if k < 3:
            got = [torch.full_like(t, 7.0) for t in gates]
            p = [null if j == k else t.data_ptr() for j, t in enumerate(got)]
            assert ssd.lib.ssd_gated_norm_backward(dims, 0, 0, 1, y.data_ptr(), x.data_ptr(), w.data_ptr(), EPS,
                                                   dout.data_ptr(), *p, ws.data_ptr(), need, st) == ssd.OK
            for j, t in enumerate(got):
                assert (t == 7).all() if j == k else torch.equal(t, gates[j])
    v = [t[None] for t in (x, y, dout)]
    h, _ = ssd.glr_prefill(*v, -w.abs())
    want = ssd.glr_backward(*v, -w.abs(), h, v[0])
    got = [torch.empty_like(t) for t in want[:4]]
    gd = ssd.GlrDims(1, rows, D, D, D)
    need = ssd.lib.ssd_glr_backward_workspace_size(gd, 0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    A = -w.abs()
    assert ssd.lib.ssd_glr_backward(gd, 0, *(t.data_ptr() for t in v), A.data_ptr(), null, h.data_ptr(), v[0].data_ptr(),
                                    null, *(t.data_ptr() for t in got), null, ws.data_ptr(), need, st) == ssd.OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("shift", [4, 8, 2, 1])
def test_norms_at_every_alignment(ssd, shift):
    """Arrays and workspaces `shift` fp32 (4: 16 bytes, but not 32) from an aligned address give the aligned ones' bits
    where the same path runs, and the oracle's values anyway."""
    gen, rows, D = _gen(21), 70, 512

    def moved(t):
        base = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")[shift:]
        return base.view(t.shape).copy_(t)

    x, dout = _rand(gen, rows, D, dtype=BF), _rand(gen, rows, D, dtype=BF)
    y, res, w, sc = _rand(gen, rows, D), _rand(gen, rows, D), 1 + _rand(gen, D, std=0.1), _rand(gen, D)
    nbytes = 1 << 22
    ws = torch.empty(nbytes + 16, dtype=torch.uint8, device="cuda")[16:]
    m = [moved(t) for t in (x, dout, y, res, w, sc)]
    for a in ((x, dout, y, res, w, sc), m, (x, dout, moved(y), res, moved(w), moved(sc))):
        X, U, Y, R, Wt, S = a
        so = moved(R)
        out, s = ssd.residual_norm(X, Wt, residual=R, scale=S, residual_out=so, eps=EPS)
        ro, rsum, bo, bs = block.residual_norm(_np(x), _np(sc), _np(res), _np(w), EPS)
        check(out, ro, bo, "out")
        check(s, rsum, bs, "residual_out")
        got = ssd.residual_norm_backward(U, s, Wt, x=X, scale=S, dresidual_out=Y, eps=EPS, dresidual=moved(Y), workspace=ws)
        want, tol = block.residual_norm_backward(_np(x), _np(sc), _np(s), _np(w), EPS, _np(dout), _np(y))
        for g, name in zip(got, ("dx", "dres", "dw", "dscale")):
            check(g, want[name], tol[name], name)
        got = ssd.gated_norm_backward(U, Y, X, Wt, ngroups=2, eps=EPS, dy=moved(Y), dz=moved(X), workspace=ws)
        want, tol = block.gated_norm_backward(_np(y), _np(x), _np(w), 2, True, EPS, _np(dout))
        for g, name in zip(got, ("dy", "dz", "dw")):
            check(g, want[name], tol[name], name)
        check(ssd.gated_norm(Y, X, Wt, ngroups=2, eps=EPS, out=moved(X)),
              *block.gated_norm(_np(y), _np(x), _np(w), 2, True, EPS), "gated")


def test_explicit_stream_argument(ssd):
    t = _inputs(15, b=1, L=200)
    want = ssd.glr_prefill(t["x"], t["r"], t["i"], t["A"])[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        h = ssd.glr_prefill(t["x"], t["r"], t["i"], t["A"], stream=stream)[0]
        side.synchronize()
        assert torch.equal(h, want)


def test_memory_of_a_call_on_another_stream_is_not_reused(ssd):
    """Workspaces that a call allocates live until its stream has used them: while the side stream is held back, the
    current one allocates and overwrites blocks of their size."""
    t = _inputs(20, b=2, L=600)
    dout, s = t["dh"], t["x"].float()
    calls = [lambda **k: ssd.glr_backward(t["x"], t["r"], t["i"], t["A"], t["x"], t["dh"], t["h0"], **k),
             lambda **k: ssd.residual_norm_backward(dout, s, t["w"], x=t["x"], scale=t["sc"], **k),
             lambda **k: ssd.gated_norm_backward(dout, s, t["x"], t["w"], **k)]
    want = [c() for c in calls]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call, ref in zip(calls, want):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about 10 ms
        got = call(stream=side)
        for n in (1 << 12, 1 << 16, 600 * 2 * 272 * 2, 1 << 20, 4 << 20):
            for _ in range(4):
                torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_offsets_beyond_32_bits(ssd):
    """Rows of a projection 2^30 + 8 elements apart (the gate, x, r and i), and their gradients likewise."""
    far, D = (1 << 30) + 8, 24
    gen = _gen(16)
    buf = torch.zeros(2 * far + 4 * D, dtype=BF, device="cuda")
    rows = buf.as_strided((1, 3, 4 * D), (0, far, 1))
    rows.copy_(_rand(gen, 1, 3, 4 * D, dtype=BF))
    x, r, i, z = rows.split(D, dim=2)
    A, w = _decays(gen, D), 1 + _rand(gen, D, std=0.1)
    h, last = ssd.glr_prefill(x, r, i, A)
    near = [v.contiguous() for v in (x, r, i, z)]
    h2, last2 = ssd.glr_prefill(*near[:3], A)
    assert torch.equal(h, h2) and torch.equal(last, last2)
    want = ssd.glr_backward(*near[:3], A, h, h)
    n = ssd.gated_norm(h[0], z[0], w)
    assert torch.equal(n, ssd.gated_norm(h[0], near[3][0], w))
    wz = ssd.gated_norm_backward(n, h[0], near[3][0], w)
    grads = torch.zeros_like(buf).as_strided((1, 3, 4 * D), (0, far, 1))
    dx, dr, di, dz = grads.split(D, dim=2)
    got = ssd.glr_backward(x, r, i, A, h, h, dx=dx, dr=dr, di=di)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = ssd.gated_norm_backward(n, h[0], z[0], w, dz=dz[0])
    assert all(torch.equal(a, b) for a, b in zip(got, wz))


def test_behind_the_ssd_prefill(ssd):
    """The SSD layer's fp32 y and a gate sliced from the in-projection, through the gated norm and the next
    block's residual norm, for a prompt and for one more token."""
    from selective_state_space_10_b200 import inputs
    from helpers import decode_args, to_device
    b, L, H, P, N = 1, 300, 4, 64, 128
    full = inputs.sequence(b, L + 1, H, P, N, 1, "bf16", seed=5)
    gen = _gen(17)
    w, w2 = 1 + _rand(gen, H * P, std=0.1), 1 + _rand(gen, H * P, std=0.1)
    z = _rand(gen, b, L + 1, 3 * H * P + H, dtype=BF)[..., :H * P]
    stream = _rand(gen, b, L + 1, H * P)
    y, state = ssd.prefill(**to_device(full.token_slice(0, L)), chunk=128)
    y1 = ssd.decode_step(state, **decode_args(to_device(full.token_slice(L, L + 1))))
    for ys, zs, res in ((y.flatten(2), z[:, :L], stream[:, :L]), (y1.flatten(1), z[:, L], stream[:, L])):
        out = ssd.gated_norm(ys, zs, w)
        flat = lambda v: _np(v).reshape(-1, H * P)
        ref, bound = block.gated_norm(flat(ys), flat(zs), _np(w), 1, True, EPS)
        check(out.reshape(-1, H * P), ref, bound, "gated norm")
        nxt, s = ssd.residual_norm(out, w2, residual=res.contiguous())
        ro, rsum, bo, bs = block.residual_norm(flat(out), None, flat(res), _np(w2), EPS)
        check(nxt.reshape(-1, H * P), ro, bo, "residual norm")
        check(s.reshape(-1, H * P), rsum, bs, "residual")


def _block_plain(p, d):
    """The block in fp64 with autograd: residual norm, projection, recurrence, gated norm, out-projection."""
    s = p["res"] + p["x"] * p["scale"]
    n = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS) * p["w"]
    v, r, i, z = (n @ p["W"]).split(d, dim=2)
    a = torch.exp(p["A"] * torch.sigmoid(r))
    u = torch.sqrt(1 - a * a) * torch.sigmoid(i) * v
    h, hs = p["h0"], []
    for t in range(v.shape[1]):
        h = a[:, t] * h + u[:, t]
        hs.append(h)
    y = torch.stack(hs, 1) * z * torch.sigmoid(z)
    o = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * p["w2"]
    return o @ p["V"], s, h


def test_a_trained_block(ssd):
    """A whole block as a program trains it, forward and backward through the library, against fp64 autograd.
    Every stage is within (GATE + STEP / (1 - a)) roundings of its terms (1 - a >= 0.1 here: 80 U = 5e-6), the
    products' fp32 sums of 48 to 96 terms add 100 U; ten such stages in a row make 1e-4 of the result's norm."""
    b, L, D, d = 2, 90, 48, 24
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    p = dict(x=rnd(b, L, D), res=rnd(b, L, D), scale=rnd(D), w=1 + 0.1 * rnd(D), W=rnd(D, 4 * d) / D ** 0.5,
             A=-0.3 - rnd(d).abs(), h0=rnd(b, d), w2=1 + 0.1 * rnd(d), V=rnd(d, D) / d ** 0.5)
    p = {k: v.float().double().requires_grad_() for k, v in p.items()}
    out, s, last = _block_plain(p, d)
    dout, ds, dlast = rnd(*out.shape).float(), rnd(*s.shape).float(), rnd(*last.shape).float()
    ((out * dout).sum() + (s * ds).sum() + (last * dlast).sum()).backward()
    q = {k: v.detach().float().cuda() for k, v in p.items()}
    dout, ds, dlast = dout.cuda(), ds.cuda(), dlast.cuda()

    n, s2 = ssd.residual_norm(q["x"], q["w"], residual=q["res"], scale=q["scale"])
    proj = n @ q["W"]
    v, r, i, z = proj.split(d, dim=2)
    h, last2 = ssd.glr_prefill(v, r, i, q["A"], initial_state=q["h0"])
    o = ssd.gated_norm(h, z, q["w2"])
    out2 = o @ q["V"]
    g = {"V": o.flatten(0, 1).t() @ dout.flatten(0, 1)}
    dproj = torch.empty_like(proj)
    dv, dr, di, dz = dproj.split(d, dim=2)
    dh, _, g["w2"] = ssd.gated_norm_backward(dout @ q["V"].t(), h, z, q["w2"], dz=dz)
    _, _, _, g["A"], g["h0"] = ssd.glr_backward(v, r, i, q["A"], h, dh, q["h0"], dlast, dx=dv, dr=dr, di=di)
    g["W"] = n.flatten(0, 1).t() @ dproj.flatten(0, 1)
    g["x"], g["res"], g["w"], g["scale"] = ssd.residual_norm_backward(dproj @ q["W"].t(), s2, q["w"], x=q["x"],
                                                                      scale=q["scale"], dresidual_out=ds)
    for name, got, ref in [("out", out2, out), ("s", s2, s), ("last", last2, last)] + [(k, g[k], p[k].grad) for k in p]:
        err = (got.double().cpu() - ref).norm() / ref.norm()
        assert err < 1e-4, (name, float(err))


def test_calls_back_to_back_wait_for_one_another(ssd):
    """Each kernel may be launched before the last one ends, and reads nothing of it before that: a chain through both
    mixers and all norms, each call on the outputs of the one before and outputs reused from turn to turn, gives the
    bits of the same chain with the GPU idle between calls."""
    from selective_state_space_10_b200 import inputs
    from helpers import to_device
    b, L, H, P = 1, 512, 8, 64
    D = H * P
    seq = to_device(inputs.sequence(b, L, H, P, 128, 1, "bf16", seed=7))
    gen = _gen(22)
    x0, z, w, sc = _rand(gen, b, L, D, dtype=BF), _rand(gen, b, L, D, dtype=BF), 1 + _rand(gen, D, std=0.1), _rand(gen, D)
    A = _decays(gen, D)

    def chain(idle):
        x, res, state = x0.clone(), torch.zeros(b, L, D, device="cuda"), torch.zeros(b, D, device="cuda")
        n, g, h = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        sync = torch.cuda.synchronize if idle else lambda: None
        kept = []
        for turn in range(12):
            ssd.residual_norm(x, w, residual=res, scale=sc, residual_out=res, out=n); sync()
            ssd.glr_prefill(n, z, n, A, initial_state=state, h=h, final_state=state); sync()
            y, _ = ssd.prefill(h.view(b, L, H, P), seq["dt"], seq["A"], seq["B"], seq["C"], seq["D"], chunk=256); sync()
            ssd.gated_norm(y.view(b, L, D), z, w, ngroups=4, out=g); sync()
            ssd.glr_decode_step(state, g[:, 0].contiguous(), z[:, 0].contiguous(), n[:, 0].contiguous(), A); sync()
            grads = ssd.glr_backward(n, z, n, A, h, g, state); sync()
            dy, dz, dw = ssd.gated_norm_backward(grads[0], y.view(b, L, D), z, w, ngroups=4); sync()
            out = ssd.residual_norm_backward(dz, res, w, x=x, scale=sc, dresidual_out=dy); sync()
            x.copy_(g); sync()
            kept += [t.clone() for t in (n, h, g, state, *grads, dy, dz, dw, *out)]; sync()
        torch.cuda.synchronize()
        return kept

    apart = chain(True)
    for _ in range(3):
        assert all(torch.equal(a, c) for a, c in zip(chain(False), apart))


def test_binding_refusals_on_the_gpu(ssd):
    t = _inputs(18, L=8)
    with pytest.raises(ValueError, match="dtype"):
        ssd.glr_prefill(t["x"], t["r"].float(), t["i"], t["A"])
    with pytest.raises(ValueError, match="shape"):
        ssd.glr_prefill(t["x"], t["r"], t["i"], t["A"][:-1])
    with pytest.raises(ValueError, match="expected cuda"):
        ssd.gated_norm(t["x"], t["r"], t["w"].cpu())
    with pytest.raises(ValueError, match="needs x"):
        ssd.residual_norm_backward(t["x"], t["x"], t["w"], scale=t["sc"])
    with pytest.raises(ssd.SSDError) as e:
        ssd.gated_norm(t["x"], t["r"], t["w"], ngroups=7)
    assert e.value.status == ssd.ERR_INVALID_ARG
    with pytest.raises(ssd.SSDError) as e:
        ssd.residual_norm(t["x"], t["w"], eps=0.0)
    assert e.value.status == ssd.ERR_INVALID_ARG
    with pytest.raises(ssd.SSDError) as e:
        ssd.gated_norm(t["x"], t["r"].float(), t["w"])  # bf16 y beside an fp32 gate
    assert e.value.status == ssd.ERR_UNSUPPORTED
    with pytest.raises(ssd.SSDError) as e:
        ssd.glr_backward(t["x"], t["r"], t["i"], t["A"], t["x"], t["dh"],
                         workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == ssd.ERR_WORKSPACE
