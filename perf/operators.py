"""The gated linear recurrence and the norms around a mixer: what is timed, their plain forms and their definitions.

Each case names one operator and one direction.  `run` computes it in elementary torch operations in fp32 (`own` false)
or through the library's binding (`own` true); `exact` is the definition in fp64, token by token where there is a
recurrence.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5


def listed():
    return [
        # the mixer of the 2.7B-shaped layer (80 heads x 64 channels), x and both gates sliced from one projection
        dict(name="glr_prefill_d5120_l4096", op="glr_prefill", b=1, L=4096, D=5120, dtype="bf16", sliced=True, init=False),
        # a ragged piece of a longer prompt, continued from a state, odd width, fp32
        dict(name="glr_prefill_f32_odd", op="glr_prefill", b=3, L=1021, D=771, dtype="f32", sliced=False, init=True),
        # one token of 256 sequences, the serving step
        dict(name="glr_decode_b256_d5120", op="glr_decode", b=256, L=1, D=5120, dtype="bf16", sliced=True, init=True),
        # training on the long-context layer (24 heads x 64 channels): the largest case
        dict(name="glr_backward_b4_l16384", op="glr_backward", b=4, L=16384, D=1536, dtype="bf16", sliced=True, init=False),
        # truncated backpropagation over a short odd piece, gradients into the state that it began from
        dict(name="glr_backward_f32_odd", op="glr_backward", b=2, L=577, D=1100, dtype="f32", sliced=False, init=True),
        # before a block of the 2.7B-shaped layer: fp32 residual stream, a learned scale of the branch
        dict(name="residual_norm_d2560", op="residual_norm", rows=4096, D=2560, dtype="bf16", aux="f32", scale=True, res=True),
        # before a block while decoding a small batch: the smallest call
        dict(name="residual_norm_decode", op="residual_norm", rows=16, D=768, dtype="bf16", aux="bf16", scale=False, res=True),
        # its gradient over the long-context batch
        dict(name="residual_norm_backward_b4_l16384", op="residual_norm_backward", rows=65536, D=768, dtype="bf16", aux="f32",
             scale=True, res=True),
        # behind the 2.7B-shaped SSD prefill: y in fp32, z a slice of the in-projection (z | x B C | dt)
        dict(name="gated_norm_d5120", op="gated_norm", rows=4096, D=5120, G=1, dtype="bf16", aux="f32", gate_first=True,
             zs=5120 + 5376 + 80),
        # a norm of its own for each head of 64, gate after the norm, odd number of rows
        dict(name="gated_norm_heads_odd", op="gated_norm", rows=2049, D=1536, G=24, dtype="bf16", aux="bf16", gate_first=False,
             zs=0),
        # the gradient behind the 2.7B-shaped prefill
        dict(name="gated_norm_backward_d5120", op="gated_norm_backward", rows=4096, D=5120, G=1, dtype="bf16", aux="f32",
             gate_first=True, zs=5120 + 5376 + 80),
        # a ragged training batch in fp32, two groups of an odd width
        dict(name="gated_norm_backward_f32_odd", op="gated_norm_backward", rows=997, D=2 * 385, G=2, dtype="f32", aux="f32",
             gate_first=False, zs=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glr_prefill", "glr_decode", "glr_backward", "residual_norm", "residual_norm_backward", "gated_norm",
                     "gated_norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    width = _log(rng, 64, 6000)
    if rng.random() < 0.6:
        width = max(8, width // 8 * 8)
    most = 1 << 25  # elements
    if op == "glr_decode":
        return dict(op=op, b=_log(rng, 1, 512), L=1, D=width, dtype=dtype, sliced=rng.random() < 0.5, init=True)
    if op.startswith("glr"):
        b = rng.choice([1, 1, 2, 3, 5])
        length = max(1, min(_log(rng, 1, 20000), most // (b * width)))
        return dict(op=op, b=b, L=length, D=width, dtype=dtype, sliced=rng.random() < 0.5, init=rng.random() < 0.5)
    rows = max(1, min(_log(rng, 1, 70000), most // width))
    aux = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
    if op.startswith("residual"):
        back = op.endswith("backward")
        return dict(op=op, rows=rows, D=width, dtype=dtype, aux=aux, scale=rng.random() < 0.6, res=back or rng.random() < 0.8)
    groups = rng.choice([1, 1, 2, 3, 8])
    width = max(1, width // groups) * groups
    zs = width + rng.randrange(0, 600) if rng.random() < 0.5 else 0
    return dict(op=op, rows=rows, D=width, G=groups, dtype=dtype, aux=aux, gate_first=rng.random() < 0.5, zs=zs)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, op, D = _T[case["dtype"]], case["op"], case["D"]

    def normal(*shape, std=1.0, of=None):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(of or dtype)

    s = dict(op=op)
    if op.startswith("glr"):
        b, L = case["b"], case["L"]
        if case["sliced"]:  # one projection gives x, r and i side by side
            x, r, i = normal(b, L, 3 * D).split(D, dim=2)
        else:
            x, r, i = (normal(b, L, D) for _ in range(3))
        # decays at an open gate from 0.43 to 0.99 a token
        A = 8.0 * torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device="cuda"))
        s.update(x=x, r=r, i=i, A=A, h0=normal(b, D, std=0.7, of=torch.float32) if case["init"] else None)
        if op == "glr_decode":
            s.update(x=x[:, 0], r=r[:, 0], i=i[:, 0], state=s["h0"])
        if op == "glr_backward":
            s["h"] = _glr_prefill(x, r, i, A, s["h0"])[0]
            s["dh"] = normal(b, L, D)
            s["dfinal"] = normal(b, D, of=torch.float32)
        return s
    rows, aux = case["rows"], _T[case["aux"]]
    s["w"] = 1 + normal(D, std=0.1, of=torch.float32)
    if op.startswith("residual"):
        s["x"] = normal(rows, D)
        s["scale"] = normal(D, std=0.3, of=torch.float32) if case["scale"] else None
        s["res"] = normal(rows, D, std=2.0, of=aux) if case["res"] else None
        s["aux"] = aux
        if op.endswith("backward"):
            s["sum"] = _residual_norm(s["x"], s["scale"], s["res"], s["w"], aux)[1]
            s["dout"], s["dres"] = normal(rows, D), normal(rows, D, of=aux)
        return s
    s["y"] = normal(rows, D, of=aux)
    s["z"] = normal(rows, case["zs"])[:, :D] if case["zs"] else normal(rows, D)
    s["G"], s["gate_first"] = case["G"], case["gate_first"]
    if op.endswith("backward"):
        s["dout"] = normal(rows, D)
    return s


# plain forms: fp32 whatever the inputs' type, rounded once at the end

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from zero, by doubling."""
    k = 1
    while k < a.shape[1]:
        b = torch.cat([b[:, :k], a[:, k:] * b[:, :-k] + b[:, k:]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _gates(r, i, A):
    sr, si = torch.sigmoid(r.float()), torch.sigmoid(i.float())
    logs = A * sr
    return sr, si, logs, torch.exp(logs), torch.sqrt(-torch.expm1(2 * logs))


def _glr_prefill(x, r, i, A, h0):
    _, si, _, a, beta = _gates(r, i, A)
    b = beta * si * x.float()
    if h0 is not None:
        b[:, 0] += a[:, 0] * h0
    h = _scan(a, b)
    return h.to(x.dtype), h[:, -1].contiguous()


def _glr_decode(x, r, i, A, state):
    _, si, _, a, beta = _gates(r, i, A)
    h = a * state + beta * si * x.float()
    state.copy_(h)
    return h.to(x.dtype), state


def _glr_backward(x, r, i, A, h, dh, h0, dfinal):
    sr, si, logs, a, beta = _gates(r, i, A)
    x, h, dh = x.float(), h.float(), dh.to(torch.float32, copy=True)
    dh[:, -1] += dfinal
    c = _scan(a.flip(1), (a * dh).flip(1)).flip(1)  # c_t = a_t g_t
    g = dh + torch.cat([c[:, 1:], torch.zeros_like(c[:, :1])], 1)
    first = (h0 if h0 is not None else torch.zeros_like(dfinal))[:, None]
    before = torch.cat([first, h[:, :-1]], 1)
    inv = torch.where(beta > 0, 1 / beta, torch.zeros_like(beta))
    dx = g * beta * si
    dlog = g * (a * before - a * a * inv * si * x)
    return dx, dlog * logs * (1 - sr), dx * x * (1 - si), (dlog * sr).sum((0, 1)), c[:, 0].contiguous()


def _residual_norm(x, scale, res, w, aux):
    s = x.float() if scale is None else x.float() * scale
    if res is not None:
        s = s + res.float()
    out = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + _EPS) * w
    return out.to(x.dtype), s.to(aux)


def _residual_norm_backward(x, scale, s, w, dout, dres, aux):
    s, u = s.float(), dout.float()
    rstd = torch.rsqrt(s.square().mean(-1, keepdim=True) + _EPS)
    n = s * rstd
    uw = u * w
    ds = rstd * (uw - n * (uw * n).mean(-1, keepdim=True)) + dres.float()
    dx = ds if scale is None else ds * scale
    dscale = None if scale is None else (ds * x.float()).sum(0)
    return dx.to(x.dtype), ds.to(aux), (u * n).sum(0), dscale


def _gated_norm(y, z, w, groups, gate_first):
    rows, D = y.shape
    gate = z.float() * torch.sigmoid(z.float())
    v = (y.float() * gate if gate_first else y.float()).view(rows, groups, -1)
    n = (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + _EPS)).view(rows, D) * w
    return (n if gate_first else n * gate).to(z.dtype)


def _gated_norm_backward(y, z, w, dout, groups, gate_first):
    rows, D = y.shape
    y32, z32, u = y.float(), z.float(), dout.float()
    sig = torch.sigmoid(z32)
    gate, slope = z32 * sig, sig * (1 + z32 * (1 - sig))
    v = (y32 * gate if gate_first else y32).view(rows, groups, -1)
    rstd = torch.rsqrt(v.square().mean(-1, keepdim=True) + _EPS)
    n = v * rstd
    un = u if gate_first else u * gate
    uw = (un * w).view(rows, groups, -1)
    dv = (rstd * (uw - n * (uw * n).mean(-1, keepdim=True))).view(rows, D)
    n = n.view(rows, D)
    dw = (un * n).sum(0)
    if gate_first:
        return (dv * gate).to(y.dtype), (dv * y32 * slope).to(z.dtype), dw
    return dv.to(y.dtype), (u * n * w * slope).to(z.dtype), dw


def run(s):
    op = s["op"]
    if own:
        from selective_state_space_10_b200 import ssd
        if op == "glr_prefill":
            return ssd.glr_prefill(s["x"], s["r"], s["i"], s["A"], initial_state=s["h0"])
        if op == "glr_decode":
            return ssd.glr_decode_step(s["state"], s["x"], s["r"], s["i"], s["A"]), s["state"]
        if op == "glr_backward":
            return ssd.glr_backward(s["x"], s["r"], s["i"], s["A"], s["h"], s["dh"], initial_state=s["h0"],
                                    dfinal_state=s["dfinal"])
        if op == "residual_norm":
            return ssd.residual_norm(s["x"], s["w"], residual=s["res"], scale=s["scale"], residual_dtype=s["aux"], eps=_EPS)
        if op == "residual_norm_backward":
            return ssd.residual_norm_backward(s["dout"], s["sum"], s["w"], x=s["x"], scale=s["scale"],
                                              dresidual_out=s["dres"], eps=_EPS)
        if op == "gated_norm":
            return ssd.gated_norm(s["y"], s["z"], s["w"], ngroups=s["G"], gate_first=s["gate_first"], eps=_EPS)
        return ssd.gated_norm_backward(s["dout"], s["y"], s["z"], s["w"], ngroups=s["G"], gate_first=s["gate_first"],
                                       eps=_EPS)
    if op == "glr_prefill":
        return _glr_prefill(s["x"], s["r"], s["i"], s["A"], s["h0"])
    if op == "glr_decode":
        return _glr_decode(s["x"], s["r"], s["i"], s["A"], s["state"])
    if op == "glr_backward":
        dx, dr, di, dA, dh0 = _glr_backward(s["x"], s["r"], s["i"], s["A"], s["h"], s["dh"], s["h0"], s["dfinal"])
        t = s["x"].dtype
        return dx.to(t), dr.to(t), di.to(t), dA, dh0
    if op == "residual_norm":
        return _residual_norm(s["x"], s["scale"], s["res"], s["w"], s["aux"])
    if op == "residual_norm_backward":
        return _residual_norm_backward(s["x"], s["scale"], s["sum"], s["w"], s["dout"], s["dres"], s["aux"])
    if op == "gated_norm":
        return _gated_norm(s["y"], s["z"], s["w"], s["G"], s["gate_first"])
    return _gated_norm_backward(s["y"], s["z"], s["w"], s["dout"], s["G"], s["gate_first"])


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, D = case["op"], case["D"]
    if op.startswith("glr"):
        n, state = case["b"] * case["L"] * D, case["b"] * D * 4
        if op == "glr_prefill":  # x, r, i in, h out
            return dict(bytes=n * 4 * e + 4 * D + state * (2 if case["init"] else 1), flops=28 * n)
        if op == "glr_decode":
            return dict(bytes=n * 4 * e + 4 * D + 2 * state, flops=28 * n)
        return dict(bytes=n * 8 * e + 8 * D + state * (3 if case["init"] else 2), flops=50 * n)
    n, f = case["rows"] * D, 2 if case["aux"] == "bf16" else 4
    if op == "residual_norm":  # x, residual in, residual and normed out
        return dict(bytes=n * (2 * e + f * (2 if case["res"] else 1)) + 4 * D * (2 if case["scale"] else 1), flops=6 * n)
    if op == "residual_norm_backward":  # dout, the sum, its gradient (and x, for the scale's) in; dx, dresidual out
        return dict(bytes=n * (2 * e + 3 * f + (e if case["scale"] else 0)) + 4 * D * (4 if case["scale"] else 2), flops=14 * n)
    if op == "gated_norm":
        return dict(bytes=n * (2 * e + f) + 4 * D, flops=12 * n)
    return dict(bytes=n * (3 * e + 2 * f) + 8 * D, flops=28 * n)


# the definitions in fp64

def _exact_glr(s):
    d = torch.float64
    x, r, i, A = (s[k].to(d) for k in ("x", "r", "i", "A"))
    sr, si = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-i))
    logs = A * sr
    return x, sr, si, logs, torch.exp(logs), torch.sqrt(-torch.expm1(2 * logs))


def exact(case, seed):
    s = prepare(case, seed)
    op, d = s["op"], torch.float64
    if op == "glr_decode":
        x, _, si, _, a, beta = _exact_glr(s)
        h = a * s["state"].to(d) + beta * si * x
        return h, h
    if op == "glr_prefill":
        x, _, si, _, a, beta = _exact_glr(s)
        v = beta * si * x
        h = torch.empty_like(v)
        last = torch.zeros_like(v[:, 0]) if s["h0"] is None else s["h0"].to(d)
        for t in range(v.shape[1]):
            last = torch.addcmul(v[:, t], a[:, t], last, out=h[:, t])
        return h, last.clone()
    if op == "glr_backward":
        x, sr, si, logs, a, beta = _exact_glr(s)
        g = s["dh"].to(d)
        carry = s["dfinal"].to(d)
        for t in range(g.shape[1] - 1, -1, -1):
            g[:, t] += carry
            carry = a[:, t] * g[:, t]
        before = torch.zeros_like(g)
        before[:, 1:] = s["h"][:, :-1].to(d)
        if s["h0"] is not None:
            before[:, 0] = s["h0"].to(d)
        dlog = g * (a * before - torch.where(beta > 0, a * a / beta, torch.zeros_like(beta)) * si * x)
        return g * beta * si, dlog * logs * (1 - sr), g * beta * x * si * (1 - si), (dlog * sr).sum((0, 1)), carry
    w = s["w"].to(d)
    D = w.numel()
    if op.startswith("residual"):
        scale = torch.ones_like(w) if s["scale"] is None else s["scale"].to(d)
        x = s["x"].to(d)
        if op == "residual_norm":
            v = scale * x + (0 if s["res"] is None else s["res"].to(d))
            return v / torch.sqrt((v * v).sum(-1, keepdim=True) / D + _EPS) * w, v
        v, u = s["sum"].to(d), s["dout"].to(d)
        root = torch.sqrt((v * v).sum(-1, keepdim=True) / D + _EPS)
        ds = u * w / root - v * (u * w * v).sum(-1, keepdim=True) / (D * root ** 3) + s["dres"].to(d)
        return ds * scale, ds, (u * v / root).sum(0), None if s["scale"] is None else (ds * x).sum(0)
    rows, G = s["y"].shape[0], s["G"]
    y, z = s["y"].to(d).view(rows, G, -1), s["z"].to(d).reshape(rows, G, -1)
    n, w = D // G, w.view(G, -1)
    gate = z / (1 + torch.exp(-z))
    v = y * gate if s["gate_first"] else y
    root = torch.sqrt((v * v).sum(-1, keepdim=True) / n + _EPS)
    if op == "gated_norm":
        return (v / root * w * (1 if s["gate_first"] else gate)).view(rows, D)
    u = s["dout"].to(d).view(rows, G, -1)
    slope = (1 + torch.exp(-z) * (1 + z)) / (1 + torch.exp(-z)) ** 2  # of z sigma(z)
    un = u if s["gate_first"] else u * gate
    dv = un * w / root - v * (un * w * v).sum(-1, keepdim=True) / (n * root ** 3)
    dw = (un * v / root).sum(0).view(D)
    if s["gate_first"]:
        return (dv * gate).view(rows, D), (dv * y * slope).view(rows, D), dw
    return dv.view(rows, D), (u * v / root * w * slope).view(rows, D), dw
