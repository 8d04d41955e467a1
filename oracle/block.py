"""fp64 oracle of the gated linear recurrence and of the norms around a mixer, with their
gradients (test infrastructure only).  Plain definitions in float64, token by token:

    L_t = A sigmoid(r_t);  a_t = exp(L_t);  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t
    s = residual + scale x;  out = s / sqrt(mean(s^2) + eps) weight
    v = y silu(z);  out = v / sqrt(mean_g(v^2) + eps) weight          (gate first)
    out = y / sqrt(mean_g(y^2) + eps) weight silu(z)                  (norm first)

The gradients are the formulas obtained from these by hand; tests/test_block_pins.py holds
them against central differences of the forward functions.

Every function also returns an error bound for fp32 arithmetic, element by element: the
sizes of the terms that are added up (before they cancel), carried through the recurrences
with the decays, times U = 2^-24 and a count of roundings.  A sigmoid costs at most 24 U
(its exponent is rounded at a magnitude of |v| log2 e, up to 12 for the inputs of the tests,
then ex2.approx, an add and rcp.approx, each within 2 ulp), a gate built from it at most 40.
"""
import numpy as np

U = 2.0 ** -24
GATE = 40.0  # roundings in a gate: one sigmoid, expm1 or its exponential, a root, three products
STEP = 4.0   # roundings of one link of a chain: the decay, its product, the sum, the chunked regrouping


def _f64(v):
    return None if v is None else np.asarray(v, dtype=np.float64)


def sigmoid(v):
    v = np.asarray(v, dtype=np.float64)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def _gates(x, r, i, A):
    sr, si = sigmoid(r), sigmoid(i)
    L = A * sr
    u = np.expm1(L)
    return sr, si, L, u, 1.0 + u, np.sqrt(-u * (2.0 + u))


def glr(x, r, i, A, h0=None):
    """(h [b, L, D], final state [b, D], bound of h)."""
    x, r, i, A, h0 = map(_f64, (x, r, i, A, h0))
    b, L, D = x.shape
    _, si, _, u, a, beta = _gates(x, r, i, A)
    v = beta * si * x
    h, bound = np.zeros((b, L, D)), np.zeros((b, L, D))
    last = np.zeros((b, D)) if h0 is None else h0.copy()
    err = np.zeros((b, D))
    for t in range(L):
        before = last
        last = a[:, t] * before + v[:, t]
        err = a[:, t] * err + U * (GATE * (np.abs(u[:, t] * before) + np.abs(v[:, t])) +
                                   STEP * (np.abs(a[:, t] * before) + np.abs(v[:, t])))
        h[:, t], bound[:, t] = last, err
    return h, last.copy(), bound


def glr_backward(x, r, i, A, h, dh, h0=None, dfinal=None):
    """({dx, dr, di, dA, dh0}, the same of bounds), from the h that the forward returned."""
    x, r, i, A, h, dh, h0, dfinal = map(_f64, (x, r, i, A, h, dh, h0, dfinal))
    b, L, D = x.shape
    sr, si, Lg, u, a, beta = _gates(x, r, i, A)
    with np.errstate(divide="ignore"):
        inv = np.where(beta > 0, 1.0 / beta, 0.0)
    c = np.zeros((b, D)) if dfinal is None else dfinal.copy()
    err = np.zeros((b, D))
    dx, dr, di, dA = np.zeros((b, L, D)), np.zeros((b, L, D)), np.zeros((b, L, D)), np.zeros(D)
    bx, br, bi, bA = np.zeros((b, L, D)), np.zeros((b, L, D)), np.zeros((b, L, D)), np.zeros(D)
    for t in range(L - 1, -1, -1):
        before = h[:, t - 1] if t else (np.zeros((b, D)) if h0 is None else h0)
        after = c
        g = dh[:, t] + after
        gerr = err + U * STEP * np.abs(g)
        p, q = a[:, t] * before, a[:, t] ** 2 * inv[:, t] * si[:, t] * x[:, t]
        dL = g * (p - q)
        lerr = gerr * np.abs(p - q) + U * GATE * np.abs(g) * (np.abs(p) + np.abs(q))
        dx[:, t] = g * beta[:, t] * si[:, t]
        di[:, t] = dx[:, t] * x[:, t] * (1 - si[:, t])
        dr[:, t] = dL * Lg[:, t] * (1 - sr[:, t])
        dA += (dL * sr[:, t]).sum(0)
        bx[:, t] = gerr * beta[:, t] * si[:, t] + U * GATE * np.abs(dx[:, t])
        bi[:, t] = bx[:, t] * np.abs(x[:, t]) * (1 - si[:, t]) + U * GATE * np.abs(di[:, t])
        br[:, t] = lerr * np.abs(Lg[:, t]) * (1 - sr[:, t]) + U * GATE * np.abs(dr[:, t])
        bA += (lerr * sr[:, t] + U * (GATE + L + 8 * b) * np.abs(dL * sr[:, t])).sum(0)
        c = a[:, t] * g
        # a link of the chain is a_t c_{t+1} + a_t dh_t, regrouped over tiles (A c + C): its products are rounded
        # one by one, each within U of its own size, before the sum may cancel
        err = a[:, t] * gerr + U * (GATE * np.abs(u[:, t] * g) + STEP * a[:, t] * (np.abs(after) + np.abs(dh[:, t])))
    return (dict(dx=dx, dr=dr, di=di, dA=dA, dh0=c),
            dict(dx=bx, dr=br, di=bi, dA=bA, dh0=err))


def _rms(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps)


def _depth(n):
    return 16 + n / 32.0  # longest chain of adds over n values: at least 32 lanes add them in turn, then a tree


def residual_norm(x, scale, residual, weight, eps):
    """(out, s, bound of out, bound of s)."""
    x, scale, residual, weight = map(_f64, (x, scale, residual, weight))
    v = x if scale is None else x * scale
    s = v if residual is None else v + residual
    size = np.abs(v) + (0 if residual is None else np.abs(residual))
    out = s * _rms(s, eps) * weight
    return out, s, U * ((8 + _depth(s.shape[-1])) * np.abs(out) + 4 * size * _rms(s, eps) * np.abs(weight)), U * 2 * size


def _norm_backward(v, un, weight, eps):
    """Gradient of v -> v / rms(v) weight over the last axis; its bound; n."""
    W = v.shape[-1]
    rstd = _rms(v, eps)
    n = v * rstd
    uw = un * weight
    mean = np.mean(uw * n, axis=-1, keepdims=True)
    size = np.mean(np.abs(uw * n), axis=-1, keepdims=True)
    dv = rstd * (uw - n * mean)
    return dv, U * (8 + _depth(W)) * rstd * (np.abs(uw) + np.abs(n) * (np.abs(mean) + size)), n


def _rows(n):
    return 24 + n  # a sum over n rows, however it is split


def residual_norm_backward(x, scale, s, weight, eps, dout, dres=None):
    """({dx, dres, dw, dscale}, the same of bounds)."""
    x, scale, s, weight, dout, dres = map(_f64, (x, scale, s, weight, dout, dres))
    k = s.shape[0]
    dv, err, n = _norm_backward(s, dout, weight, eps)
    ds = dv if dres is None else dv + dres
    err = err + U * np.abs(ds)
    g = dict(dx=ds if scale is None else ds * scale, dres=ds, dw=(dout * n).sum(0))
    e = dict(dx=err if scale is None else err * np.abs(scale) + U * np.abs(ds * scale), dres=err,
             dw=U * (_rows(k) + _depth(s.shape[-1])) * np.abs(dout * n).sum(0))
    if scale is not None:
        g["dscale"] = (ds * x).sum(0)
        e["dscale"] = (err * np.abs(x)).sum(0) + U * _rows(k) * np.abs(ds * x).sum(0)
    return g, e


def _gate(z):
    sg = sigmoid(z)
    return z * sg, sg * (1 + z * (1 - sg)), sg * (1 + np.abs(z) * (1 - sg))


def gated_norm(y, z, weight, groups, gate_first, eps):
    """(out, bound)."""
    y, z, weight = map(_f64, (y, z, weight))
    rows, D = y.shape
    gate = _gate(z)[0]
    v = (y * gate if gate_first else y).reshape(rows, groups, -1)
    out = (v * _rms(v, eps)).reshape(rows, D) * weight
    out = out if gate_first else out * gate
    return out, U * (GATE + _depth(D // groups)) * np.abs(out)


def gated_norm_backward(y, z, weight, groups, gate_first, eps, dout):
    """({dy, dz, dw}, the same of bounds)."""
    y, z, weight, dout = map(_f64, (y, z, weight, dout))
    rows, D = y.shape
    gate, slope, steep = _gate(z)
    split = lambda a: a.reshape(rows, groups, -1)
    un = dout if gate_first else dout * gate
    w = np.broadcast_to(weight, (rows, D))
    dv, err, n = (a.reshape(rows, D) for a in
                  _norm_backward(split(y * gate if gate_first else y), split(un), split(w), eps))
    err = err * GATE / 8  # its inputs carry a gate's error
    dw = (un * n).sum(0)
    bw = U * (_rows(rows) + GATE + _depth(D // groups)) * np.abs(un * n).sum(0)
    if gate_first:
        g = dict(dy=dv * gate, dz=dv * y * slope, dw=dw)
        e = dict(dy=err * np.abs(gate) + U * GATE * np.abs(dv * gate),
                 dz=err * np.abs(y) * steep + U * GATE * np.abs(dv * y) * steep, dw=bw)
    else:
        g = dict(dy=dv, dz=dout * n * weight * slope, dw=dw)
        e = dict(dy=err, dz=U * (GATE + _depth(D // groups)) * np.abs(dout * n * weight) * steep, dw=bw)
    return g, e
