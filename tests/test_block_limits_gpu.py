"""GPU tests of the gated linear recurrence and the norms at the limits of what their calls allow: the widest rows, calls
from several host threads, calls after a failed one, the strongest decays and nearly shut gates."""

import pytest
import torch

from oracle import block
from test_block_gpu import BF, EPS, F32, _gen, _np, _rand, check

pytestmark = pytest.mark.gpu


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
