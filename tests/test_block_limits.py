"""Refusals of the gated linear recurrence and the norms at the limits of their calls, without a GPU."""
import ctypes
import os
import re
import subprocess
from types import SimpleNamespace

import numpy as np
import pytest
import torch

FAKE = 1 << 20


@pytest.fixture(scope="module")
def ssd():
    from selective_state_space_10_b200 import build
    build.build()
    from selective_state_space_10_b200 import ssd as mod
    return mod


@pytest.mark.parametrize("bad", [dict(out=None), dict(out=FAKE + 4), dict(nbytes=6 * 4 * 4 * 64 * 4 - 1), dict(ranks=1),
                                 dict(ranks=9), dict(tiles=0), dict(tiles=65), dict(late_rank=4), dict(late_rank=-2),
                                 dict(late_tile=6), dict(late_tile=-1), dict(delay=100_000_001), dict(limit=0),
                                 dict(limit=100_000_001)], ids=str)
def test_wait_selftest_refusals(ssd, bad):
    a = dict(out=FAKE, nbytes=1 << 30, ranks=4, tiles=6, late_rank=-1, late_tile=0, delay=0, limit=1000)
    a.update(bad)
    out = None if a["out"] is None else ctypes.c_void_p(a["out"])
    assert ssd.lib.ssd_glr_wait_selftest(out, a["nbytes"], a["ranks"], a["tiles"], a["late_rank"], a["late_tile"],
                                         a["delay"], a["limit"], None) == ssd.ERR_INVALID_ARG


@pytest.mark.parametrize("view", [torch.empty(1, dtype=torch.uint8).expand(1 << 20), torch.empty(64, 64)[:, :32],
                                  torch.empty(64, dtype=torch.uint8)[::2]], ids=["expanded", "columns", "strided"])
def test_scratch_that_is_a_view_with_gaps_is_refused(ssd, view):
    """Its bytes are not where the call would write them."""
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        ssd._workspace(view, 16, torch.empty(1))
    with pytest.raises(ValueError, match="device_buffer must be contiguous"):
        ssd._scratch_bytes(view, "device_buffer")


def test_scratch_that_is_whole_is_taken(ssd):
    for t in (torch.empty(64, dtype=torch.uint8)[16:], torch.empty(4, 4), torch.empty(0, dtype=torch.uint8)):
        got, nbytes = ssd._workspace(t, 16, torch.empty(1))
        assert got is t and nbytes == t.numel() * t.element_size()


def test_a_stream_of_another_device_is_refused(ssd):
    """The call would have run on the current stream of the tensors' device, not on the one given."""
    ran = []
    on0 = SimpleNamespace(is_cuda=True, device=torch.device("cuda", 0))
    stream1 = SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream is on cuda:1, expected cuda:0"):
        ssd._on(stream1, on0, ran.append, 1)
    t = torch.zeros(1, 3, 8)
    for stream in (0, stream1):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            ssd.glr_prefill(t, t, t, torch.zeros(8), stream=stream)
    assert not ran


def test_what_the_runtime_says_is_kept_by_kernel_and_device(tmp_path):
    here = os.path.dirname(os.path.abspath(__file__))
    csrc = os.path.join(os.path.dirname(here), "selective_state_space_10_b200", "csrc")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc"))), "include")
    exe = str(tmp_path / "per_device_test")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I" + csrc, "-I" + cuda, os.path.join(here, "per_device_test.cpp"), "-o", exe],
                   check=True)
    done = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0, done.stdout


def test_kernels_that_start_early_promise_nothing_of_their_memory():
    """A kernel that waits for the one before it may not have __restrict__ pointers: the memory behind them changes until
    the wait, and the qualifier allows loads before it."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_10_b200", "csrc")
    early = []
    for name in ("glr.cu", "norm.cu"):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        for kernel in re.split(r"(?=__global__ void)", text)[1:]:
            head, body = kernel.split("{", 1)
            body = body[:body.index("\n}")]
            if "grid_dep_wait" in body:
                early.append(re.search(r"(k_\w+)\(", head).group(1))
                assert "__restrict__" not in head, early[-1]
    assert sorted(early) == ["k_glr_backward", "k_glr_decode", "k_glr_prefill", "k_norm_backward_rows", "k_norm_rows",
                             "k_row_sums"]


def test_the_polynomial_of_the_decay():
    """1 - exp(f) over |f| <= ln 2 / 2, from the coefficients in the kernel's source: as close as its comment says; and
    the decay a and 1 - a that the fp32 steps around it make, each within a few roundings of its own size."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_10_b200", "csrc")
    with open(os.path.join(csrc, "glr.cu")) as f:
        text = f.read()
    body = text[text.index("void decay("):]
    numbers = [float(v) for v in re.findall(r"both\((-?[0-9.e-]+)f\)", body[:body.index("\n}")])]
    magic, back, ln2 = numbers[:3]
    coefficients = numbers[3:9]
    assert (magic, back) == (12582912.0, -12582912.0) and coefficients[4:] == [-0.5, -1.0]
    f32 = np.float32

    def fma(a, b, c):  # of fp32 values: the product is exact in fp64
        return (np.float64(a) * np.float64(b) + np.float64(c)).astype(f32)

    f = np.linspace(-0.5, 0.5, 200001) * np.log(2)
    f = f[np.abs(f) > 1e-8]
    p = np.zeros_like(f)
    for k in coefficients:
        p = p * f + np.float64(f32(k))
    assert np.abs(p * f / -np.expm1(f) - 1).max() < 1.85e-8
    L = -np.concatenate([np.geomspace(1e-30, 86.9, 200001), np.linspace(0, 3, 100001)[1:]]).astype(f32)
    t = fma(L, f32(1.4426950408889634), f32(magic))
    n = t + f32(back)
    f = fma(n, f32(ln2), L)
    p = np.full_like(f, f32(coefficients[0]))
    for k in coefficients[1:]:
        p = fma(p, f, f32(k))
    p = p * f
    two_n = np.exp2(n.astype(np.float64)).astype(f32)
    v, a = fma(two_n, p, fma(two_n, f32(-1), f32(1))), two_n * fma(p, f32(-1), f32(1))
    true = np.exp(L.astype(np.float64)), -np.expm1(L.astype(np.float64))
    U = 2.0 ** -24
    # f: its sum is rounded once, within U / 2 of ln 2 / 2 at n != 0, and the constant is U / 20 of |L| off; p adds four
    # roundings that shrink with f, its own and the last product's; then 1 - p and 2^n
    assert (np.abs(a / true[0] - 1) <= U * (4 + np.abs(L) / 16)).all()
    # 1 - a: the same, but 2^n p may cancel half of 1 - 2^n, which is exact or rounded to 1
    assert (np.abs(v / true[1] - 1) <= U * 8).all()
