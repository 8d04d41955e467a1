"""GPU tests of the gated linear recurrence and the norms at the limits of what their calls allow: the widest rows, calls
from several host threads, calls after a failed one, the strongest decays and nearly shut gates."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import block
from test_block_gpu import BF, EPS, F32, _decays, _gen, _np, _rand, check

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ssd():
    from selective_state_space_10_b200 import ssd as mod
    return mod


def _residual_gradient(ssd, rows, D, types, scaled):
    tx, tr = types
    gen = _gen(rows, D, scaled)
    x, w = _rand(gen, rows, D, dtype=tx), 1 + _rand(gen, D, std=0.2)
    scale = _rand(gen, D) if scaled else None
    s, dres, dout = _rand(gen, rows, D, dtype=tr, std=2), _rand(gen, rows, D, dtype=tr), _rand(gen, rows, D, dtype=tx)
    got = ssd.residual_norm_backward(dout, s, w, x=x, scale=scale, dresidual_out=dres, eps=EPS)
    want, tol = block.residual_norm_backward(_np(x), _np(scale), _np(s), _np(w), EPS, _np(dout), _np(dres))
    for g, name in zip(got, ("dx", "dres", "dw", "dscale")):
        if name in want:
            check(g, want[name], tol[name], name)


WIDE = [6144, 6152, 7168, 8192, 9216, 9220, 10240, 11264, 11268, 11272, 12288, 12292, 12296, 12300, 16384]


@pytest.mark.parametrize("scaled", [True, False], ids=["scale", "plain"])
@pytest.mark.parametrize("types", [(F32, F32), (BF, F32), (BF, BF)], ids=["f32", "bf16-f32", "bf16"])
@pytest.mark.parametrize("D", WIDE)
def test_residual_gradient_of_wide_rows(ssd, D, types, scaled):
    """Around the widths at which a row's share of shared memory passes what a CTA may have."""
    _residual_gradient(ssd, 5, D, types, scaled)


@pytest.mark.parametrize("types", [(F32, F32), (BF, F32), (BF, BF)], ids=["f32", "bf16-f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(310, 10240), (700, 12288)])
def test_residual_gradient_of_many_wide_rows(ssd, rows, D, types):
    """More rows than CTAs of either kernel: each CTA takes several."""
    _residual_gradient(ssd, rows, D, types, True)


@pytest.mark.parametrize("gate_first", [True, False], ids=["gate_first", "norm_first"])
@pytest.mark.parametrize("types", [(F32, F32), (BF, F32), (BF, BF)], ids=["f32", "bf16-f32", "bf16"])
@pytest.mark.parametrize("D,G", [(6152, 1), (10240, 1), (12288, 1), (12296, 1), (24576, 2)])
def test_gated_gradient_of_wide_rows(ssd, D, G, types, gate_first):
    tx, ty = types
    rows, gen = 5, _gen(D, G)
    y, w, dout = _rand(gen, rows, D, dtype=ty), 1 + _rand(gen, D, std=0.2), _rand(gen, rows, D, dtype=tx)
    z = _rand(gen, rows, D, dtype=tx, std=2)
    got = ssd.gated_norm_backward(dout, y, z, w, ngroups=G, gate_first=gate_first, eps=EPS)
    want, tol = block.gated_norm_backward(_np(y), _np(z), _np(w), G, gate_first, EPS, _np(dout))
    for g, name in zip(got, ("dy", "dz", "dw")):
        check(g, want[name], tol[name], name)


def test_a_failed_call_is_reported_once():
    """A launch that the runtime refuses is reported by the call that made it, and the next good call in the thread
    answers for itself.  The refused launches go to the legacy stream while this thread captures another, blocking
    stream, which the runtime forbids; nothing of them reaches the GPU."""
    code = """
import torch
from cuda.bindings import runtime as rt
from selective_state_space_10_b200 import ssd
f = lambda *s: torch.randn(*s, device='cuda')
y, w, A = f(9, 256), f(256), -f(256).abs()
h, st = f(9, 256), f(2, 4, 64, 16)
x4, B4, dt, a4, o4 = f(2, 4, 64), f(2, 1, 16), f(2, 4).abs(), -f(4).abs(), torch.empty(2, 4, 64, device='cuda')
out = torch.empty_like(y)
nd, gd, sd = ssd.NormDims(9, 256, 1, 256, 256), ssd.GlrDims(1, 9, 256, 256, 256), ssd.Dims(2, 1, 4, 64, 16, 1)
wide = f(3, 40000)
ww, wo, wd = f(40000), torch.empty_like(wide), ssd.NormDims(3, 40000, 1, 40000, 40000)
last = torch.empty(1, 256, device='cuda')
p = lambda t: t.data_ptr()
fails = dict(
    norm=lambda s: ssd.lib.ssd_gated_norm(nd, 0, 0, 1, p(y), p(h), p(w), 1e-5, p(out), s),
    long_norm=lambda s: ssd.lib.ssd_gated_norm(wd, 0, 0, 1, p(wide), p(wide), p(ww), 1e-5, p(wo), s),
    scan=lambda s: ssd.lib.ssd_glr_prefill(gd, 0, p(y), p(h), p(y), p(A), None, p(out), p(last), s),
    step=lambda s: ssd.lib.ssd_glr_decode_step(ssd.GlrDims(1, 1, 256, 256, 256), 0, p(last), p(y), p(h), p(y), p(A), p(out), s))
good = dict(
    decode=lambda s: ssd.lib.ssd_decode_step(sd, 0, p(st), p(x4), p(dt), p(a4), p(B4), p(B4), p(a4), p(o4), s),
    long_norm=fails['long_norm'])
for fn in list(fails.values()) + list(good.values()):
    assert fn(torch.cuda.current_stream().cuda_stream) == ssd.OK
torch.cuda.synchronize()
def do(r):
    assert r[0] == rt.cudaError_t.cudaSuccess, r
    return r[1] if len(r) == 2 else None
for name, bad in fails.items():
    for after, fn in good.items():
        s = do(rt.cudaStreamCreate())
        do(rt.cudaStreamBeginCapture(s, rt.cudaStreamCaptureMode.cudaStreamCaptureModeGlobal))
        first = bad(None)
        rt.cudaStreamEndCapture(s)  # the refused launch has invalidated it
        rt.cudaGetLastError()
        assert first == ssd.ERR_CUDA, (name, first)
        assert fn(torch.cuda.current_stream().cuda_stream) == ssd.OK, (name, after)
        torch.cuda.synchronize()
        do(rt.cudaStreamDestroy(s))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


class _Job(ctypes.Structure):  # `job` of call_in_threads.c
    _fields_ = ([("fn", ctypes.c_void_p)] + [(k, ctypes.c_int64) for k in ("scan", "rows", "dim")] +
                [(k, ctypes.c_void_p) for k in ("input", "weight", "out", "vec", "workspace", "stream")] +
                [(k, ctypes.c_int64) for k in ("workspace_bytes", "calls", "failed")] + [("thread", ctypes.c_ulong)])


def test_host_threads_with_calls_of_different_sizes(ssd, tmp_path):
    """No call depends on the sizes of another thread's: threads that call the same kernels with little and with much
    shared memory, all at once, each get what the same call gives alone."""
    here = os.path.dirname(os.path.abspath(__file__))
    lib = str(tmp_path / "threads.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-I" + os.path.join(os.path.dirname(here), "include"),
                    os.path.join(here, "call_in_threads.c"), "-o", lib, "-lpthread"], check=True)
    run = ctypes.CDLL(lib).call_in_threads
    sizes = [(0, 9, 512), (0, 9, 5120), (0, 9, 4096), (0, 9, 8192), (1, 9, 64), (1, 900, 64), (1, 100, 64), (1, 2000, 64)]
    jobs, held = (_Job * len(sizes))(), []
    for job, (scan, rows, dim) in zip(jobs, sizes):
        gen = _gen(rows, dim)
        x, w = _rand(gen, rows, dim), -_rand(gen, dim).abs()
        out, vec, side = torch.zeros(2, rows, dim, device="cuda"), torch.zeros(dim, device="cuda"), torch.cuda.Stream()
        need = ssd.lib.ssd_norm_backward_workspace_size(ssd.NormDims(rows, dim, 1, dim, dim))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        if scan:
            want = [t.clone() for t in ssd.glr_prefill(x[None], x[None], x[None], w)]
        else:
            want = [t.clone() for t in ssd.gated_norm_backward(x, x, x, w)]
        fn = ssd.lib.ssd_glr_prefill if scan else ssd.lib.ssd_gated_norm_backward
        job.fn, job.scan, job.rows, job.dim = ctypes.cast(fn, ctypes.c_void_p), scan, rows, dim
        job.input, job.weight, job.out, job.vec = (t.data_ptr() for t in (x, w, out, vec))
        job.workspace, job.workspace_bytes, job.stream, job.calls = ws.data_ptr(), need, side.cuda_stream, 3000
        held.append((x, w, ws, side, out, vec, want))
    torch.cuda.synchronize()
    assert run(jobs, len(sizes)) == 1
    torch.cuda.synchronize()
    assert [j.failed for j in jobs] == [0] * len(sizes)
    for (scan, rows, dim), (*_, out, vec, want) in zip(sizes, held):
        got = [out[0][None], vec[None]] if scan else [out[0], out[1], vec]
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (scan, rows, dim)


def _kept(ssd, L, D, dtype, gen, strong):
    """Shut input gates (nothing comes in), so that h = a_1 ... a_t h_0 alone: the recurrence gate is shut too (a = 1)
    but for the tokens `strong`.  A from -0.01 to -20: decays from 0.99 down to 1e-9 a token."""
    A = -torch.logspace(-2, np.log10(20.0), D).cuda()
    r = torch.full((1, L, D), -float("inf"))
    for t in strong:
        r[0, t] = torch.randn(D, generator=gen) * 1.5
    r = r.to(dtype).cuda()
    i, x = torch.full_like(r, -float("inf")), torch.full_like(r, 3.0)
    h0 = (0.5 + torch.rand(1, D, generator=gen)).cuda()
    logs = _np(A) * block.sigmoid(_np(r))
    ref = _np(h0)[:, None] * np.exp(np.cumsum(logs, axis=1))
    # a token's decay: its sigmoid within 24 U, the product with A, the range reduction's constant and sum within 2 U of
    # L, all relative to L; the polynomial, 2^n and 1 - p within 4 U of a, and 2 products (into a tile's update, and of
    # that with the state) within U each.  At a = 1 nothing is rounded.
    steps = np.where(logs < 0, 26 * U * np.abs(logs) + 6 * U, 0)
    return (x, r, i, A, h0), ref, np.abs(ref) * np.expm1(np.cumsum(steps, axis=1)) * 1.01


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("L,strong", [(5, (0, 1, 3)), (1, (0,)), (900, (0, 63, 64, 301, 899))])
def test_a_small_decay_keeps_its_precision(ssd, L, strong, dtype):
    """What a token forgets to 1e-9 is that, to the precision of fp32: the decay's own, not 1 - a's."""
    args, ref, bound = _kept(ssd, L, 120, dtype, _gen(L, 41), strong)
    x, r, i, A, h0 = args
    h, last = ssd.glr_prefill(x, r, i, A, initial_state=h0)
    check(h, ref, bound, "h")
    check(last, ref[:, -1], bound[:, -1], "final state")


@pytest.mark.parametrize("D", [120, 119])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_a_small_decay_of_a_step_keeps_its_precision(ssd, D, dtype):
    (x, r, i, A, state), ref, bound = _kept(ssd, 1, D, dtype, _gen(D, 42), (0,))
    h = ssd.glr_decode_step(state, x[:, 0], r[:, 0], i[:, 0], A)
    check(h, ref[:, 0], bound[:, 0], "h")
    check(state, ref[:, 0], bound[:, 0], "state")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 62, 63])
def test_a_nearly_shut_input_gate_lets_in_what_it_should(ssd, D, dtype):
    """sigmoid(i) down to the end of the normal range, 1e-38, and nothing at all where the decay is exactly 1."""
    i = torch.linspace(-86.0, -30.0, D).expand(1, 3, D).to(dtype).cuda().contiguous()
    x = torch.full_like(i, 5120.0)
    r = torch.full_like(i, 1.0)
    r[0, 1] = -float("inf")  # a = 1: the state stays as it is, bit for bit
    A = -torch.logspace(-3, 0, D).cuda()
    args = [_np(v) for v in (x, r, i, A)]
    ref, rlast, _ = block.glr(*args)
    # exp(-i): its exponent is rounded at a magnitude of |i| log2 e and its factor is within U / 4 of log2 e, together
    # 1.25 |i| U of the result; the other gate, the root and the decay of the state as GATE each.  1e-36 (in check): what
    # lies below the normal range is flushed
    rel = U * (110 + 3 * block.GATE)
    h, last = ssd.glr_prefill(x, r, i, A)
    check(h, ref, rel * np.abs(ref), "h")
    check(last, rlast, rel * np.abs(rlast), "final state")
    assert torch.equal(h[:, 1], h[:, 0])
    state, one = torch.zeros(1, D, device="cuda"), []
    for t in range(3):
        one.append(ssd.glr_decode_step(state, x[:, t], r[:, t], i[:, t], A))
    check(torch.stack(one, 1), ref, rel * np.abs(ref), "step")
    check(state, rlast, rel * np.abs(rlast), "state")
    assert torch.equal(one[1], one[0])
    big = torch.full_like(x, 1e30)
    assert (ssd.glr_prefill(big, torch.full_like(r, -float("inf")), torch.zeros_like(i), A)[0] == 0).all()
    assert (ssd.glr_prefill(big, r, torch.zeros_like(i), torch.zeros_like(A))[0] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("b,L,D", [(1, 1000, 64), (2, 37, 131), (40, 100, 70)])
def test_nearly_shut_gates_among_open_ones(ssd, b, L, D, dtype):
    """In the same tile and in neighbouring channels, in lone CTAs and in clusters."""
    gen = _gen(b, L, D, 51)
    x, r, i = (_rand(gen, b, L, D, dtype=dtype, std=1.5) for _ in range(3))
    shut = torch.rand(b, L, D, generator=gen).cuda()
    i[shut < 0.05] = -60.0
    i[shut < 0.02] = -float("inf")
    r[shut < 0.01] = -float("inf")
    A, h0 = _decays(gen, D), _rand(gen, b, D)
    h, last = ssd.glr_prefill(x, r, i, A, initial_state=h0)
    ref, rlast, bound = block.glr(*(_np(v) for v in (x, r, i, A, h0)))
    check(h, ref, bound, "h")
    check(last, rlast, bound[:, -1], "final state")


@pytest.mark.parametrize("ranks", [2, 5, 8])
def test_a_scan_whose_waits_hold(ssd, ranks):
    """The self-test without a late rank, and with one that is late but within the limit: the sums of ones."""
    want = torch.arange(2.0, 2 + 6 * ranks * 4, device="cuda").view(6, ranks, 4, 1).expand(6, ranks, 4, 64)
    assert torch.equal(ssd.glr_wait_selftest(ranks, 6), want)
    assert torch.equal(ssd.glr_wait_selftest(ranks, 6, late_rank=1, late_tile=2, delay_ns=2_000_000), want)


@pytest.mark.parametrize("ranks,late_rank", [(2, 0), (2, 1), (5, 0), (5, 3), (8, 7)])
@pytest.mark.parametrize("late_tile", [0, 1, 2, 4, 5])
def test_a_scan_whose_wait_expires_leaves_nothing_wrong(ssd, ranks, late_rank, late_tile):
    """A rank late by ten times the limit: before its round all is right; in that round its own states are, which wait for
    ranks that came in time, and those of the ranks that gave up on it are NaN; after it everything is NaN, the last
    rank's state included."""
    want = torch.arange(2.0, 2 + 6 * ranks * 4, device="cuda").view(6, ranks, 4, 1).repeat(1, 1, 1, 64)
    got = ssd.glr_wait_selftest(ranks, 6, late_rank, late_tile, delay_ns=40_000_000, limit_ns=4_000_000)
    others = [k for k in range(ranks) if k != late_rank]
    assert torch.equal(got[:late_tile], want[:late_tile])
    assert torch.equal(got[late_tile, late_rank], want[late_tile, late_rank])
    assert torch.isnan(got[late_tile, others]).all() and torch.isnan(got[late_tile + 1:]).all()
    assert torch.equal(ssd.glr_wait_selftest(ranks, 6), torch.arange(2.0, 2 + 6 * ranks * 4, device="cuda").view(
        6, ranks, 4, 1).expand(6, ranks, 4, 64))  # the next call is not touched by it


@pytest.mark.parametrize("mask", [-1e4, -float("inf"), "lowest"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("b,L,D", [(1, 1000, 64), (3, 50, 74), (2, 21, 33)])
def test_masked_tokens_leave_the_state_as_it_is(ssd, b, L, D, dtype, mask):
    """Both gates masked at single tokens and at a padded end: every token gets what it gets in a sequence without the
    masked ones, a masked one what the last token before it got.  (Not bit for bit: the state that enters a warp's tokens
    is a sum grouped otherwise than the steps before it, so both are within the last token's bound.  Before the first
    token, and in single steps, nothing is rounded.)"""
    gen = _gen(b, L, D, 61)
    x, r, i = (_rand(gen, b, L, D, dtype=dtype, std=1.5) for _ in range(3))
    off = torch.rand(L, generator=gen) < 0.3
    off[L - L // 4:] = True
    low = torch.finfo(dtype).min if mask == "lowest" else mask
    r[:, off.cuda()], i[:, off.cuda()] = low, low
    A, h0 = _decays(gen, D), _rand(gen, b, D)
    h, last = ssd.glr_prefill(x, r, i, A, initial_state=h0)
    on = (~off).nonzero()[:, 0].cuda()
    ref, rlast, bound = block.glr(*(_np(v[:, on]) for v in (x, r, i)), _np(A), _np(h0))
    seen = np.cumsum(~off.numpy())  # tokens up to and with each one that are not masked; 0: the initial state
    ref, bound = np.concatenate([_np(h0)[:, None], ref], 1), np.concatenate([0 * _np(h0)[:, None], bound], 1)
    check(h, ref[:, seen], bound[:, seen], "h")
    check(last, rlast, bound[:, -1], "final state")
    state = h0.clone()
    for t in off.nonzero()[:3, 0].tolist():
        out = ssd.glr_decode_step(state, x[:, t], r[:, t], i[:, t], A)
        assert torch.equal(state, h0) and torch.equal(out, h0.to(dtype))
