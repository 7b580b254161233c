"""Plain 64-bit forms of the operators in include/based_ops.h, row by row on the CPU, with bounds on
the error a float32 evaluation that rounds once to the output's type may have.

Bounds: an output of type t may be off by half a step, eps(t) / 2 relative, plus the float32 error.
exp(x) is good to 2^-22 and |x| 2^-24 relative, the logistic function made of it (one addition, a
reciprocal to 2^-23, one product) to 2^-21 where x is small and so a decay is far from 0, and
every float32 operation adds 2^-24; DELTA = 2^-20 per row covers
the decay, the increment, the row's own multiply-add and its share of the products that join
stretches of rows. Sums over a group or over rows add at most their depth times 2^-24 relative to
the sum of magnitudes.
"""
import torch

DELTA = 2.0 ** -20
# arguments of the logistic function below -87 count as -87: an absolute error of at most exp(-87)
CLAMP = 2e-38


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """The absolute error of a rounding below the type's smallest normal number."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def decay(mode, g, x):
    """a, 1 - a (1 for log decays) and u in 64 bits."""
    if mode == "log":
        return torch.exp(g), torch.ones_like(g), x
    rest = torch.sigmoid(-g)
    return torch.sigmoid(g), rest, rest * x


def scan(gate, x, mode, state=None, lengths=None, dy=None, dfinal=None):
    """Values and error bounds of the recurrence and its gradients: two dicts of 64-bit tensors."""
    dtype = x.dtype
    gate, x = gate.detach().cpu().double(), x.detach().cpu().double()
    B, T, D = x.shape
    lens = torch.full((B,), T) if lengths is None else lengths.cpu().long().clamp(0, T)
    live = (torch.arange(T)[None] < lens[:, None])[..., None]
    gate, x = torch.where(live, gate, 0.0), torch.where(live, x, 0.0)
    a, rest, u = decay(mode, gate, x)
    a, rest, u = torch.where(live, a, 1.0), torch.where(live, rest, 0.0), torch.where(live, u, 0.0)
    first = torch.zeros(B, D, dtype=torch.float64) if state is None else state.detach().cpu().double()

    def run(start, add, reverse=False):
        out, h = torch.empty_like(add), start
        for t in (range(T - 1, -1, -1) if reverse else range(T)):
            if reverse:  # lam_t = add_t + (what comes back from the row after)
                out[:, t] = add[:, t] + h
                h = a[:, t] * out[:, t]
            else:
                h = out[:, t] = a[:, t] * h + add[:, t]
        return out, h

    h, last = run(first, u)
    # error: e_t = a e_{t-1} + DELTA (a |h|_{t-1} + |u_t|), with |h| the sum of magnitudes
    mag, mag_last = run(first.abs(), u.abs())
    err, err_last = run(torch.zeros_like(first), torch.where(live, DELTA * mag, 0.0))
    half = half_step(dtype)
    y = torch.where(live, h, 0.0)
    val = {"y": y, "final": last}
    bound = {"y": half * y.abs() + err + tiny(dtype), "final": err_last + 2.0 ** -24 * last.abs()}
    if dy is not None:
        d = torch.where(live, dy.detach().cpu().double(), 0.0)
        end = torch.zeros(B, D, dtype=torch.float64) if dfinal is None else dfinal.detach().cpu().double()
        lam, back = run(end, d, reverse=True)
        lmag, _ = run(end.abs(), d.abs(), reverse=True)
        lerr, berr = run(torch.zeros_like(end), DELTA * lmag, reverse=True)
        before = torch.cat([first[:, None], h[:, :-1]], 1)
        berr_h = torch.cat([torch.zeros_like(first)[:, None], err[:, :-1]], 1)
        if mode == "log":
            diff, slope, dx = before, a, lam
            mags = before.abs()
        else:
            diff, slope, dx = before - x, a * rest, rest * lam
            mags = before.abs() + x.abs()
        dg = slope * diff * lam
        dge = slope * ((berr_h + DELTA * mags) * lam.abs() + diff.abs() * (lerr + DELTA * lmag))
        dxe = (lerr + DELTA * lmag) * (1.0 if mode == "log" else rest)
        dge = dge + CLAMP * mags * lmag
        zero = lambda v: torch.where(live, v, 0.0)  # noqa: E731
        val.update(dgate=zero(dg), dx=zero(dx), dstate=back)
        bound.update(dgate=half * zero(dg).abs() + zero(dge) + tiny(dtype),
                     dx=half * zero(dx).abs() + zero(dxe) + tiny(dtype),
                     dstate=berr + DELTA * back.abs() + tiny(torch.float32))
    return val, bound


def activation(act, v):
    if act == "none":
        return v, torch.ones_like(v)
    p = torch.sigmoid(v)
    if act == "sigmoid":
        return p, p * (1 - p)
    return v * p, p + v * p * (1 - p)


def norm(x, groups, weight=None, bias=None, gate=None, act="silu", eps=1e-5, dy=None, out_dtype=None):
    """Values and error bounds of the group norm and its gradients."""
    C = x.shape[-1]
    n = C // groups
    dtype = gate.dtype if gate is not None else out_dtype if out_dtype is not None else x.dtype
    xd = x.detach().cpu().double().reshape(-1, groups, n)
    R = xd.shape[0]
    one = torch.ones(C, dtype=torch.float64)
    w = one if weight is None else weight.detach().cpu().double()
    b = 0 * one if bias is None else bias.detach().cpu().double()
    wg, bg = w.view(groups, n), b.view(groups, n)
    # depth of the sums over a group: 8 in a thread, then at most 9 halvings and 16 warps
    d = 33 * 2.0 ** -24
    mean = xd.mean(-1, keepdim=True)
    dev = xd - mean
    rstd = 1 / torch.sqrt((dev * dev).mean(-1, keepdim=True) + eps)
    hat = dev * rstd
    # the mean is off by d mean|x|; that shifts every deviation, and the variance by its square and
    # by a relative d; the deviations round once more
    me = d * xd.abs().mean(-1, keepdim=True)
    rel_r = d + 4 * 2.0 ** -24 + 0.5 * (2 * me * dev.abs().mean(-1, keepdim=True) + me * me) * rstd * rstd
    he = (me + 2.0 ** -24 * dev.abs()) * rstd + hat.abs() * rel_r
    v = hat * wg + bg
    ve = he * wg.abs() + 2.0 ** -23 * ((hat * wg).abs() + v.abs())
    z = v if gate is None else gate.detach().cpu().double().reshape(-1, groups, n)
    f, df = activation(act, z)
    sig = 2.0 ** -20 if act != "none" else 0.0  # relative error of the activation's factors
    if gate is None:
        y, ye = f, 1.1 * ve + sig * (f.abs() + 2.0 ** -24)
    else:
        y, ye = v * f, ve * f.abs() + sig * (v * f).abs() + 2.0 ** -24 * (v * f).abs()
    far = CLAMP * (1 + z.abs()) if act != "none" else 0.0  # of act(z) and act'(z), see CLAMP
    ye = ye + far * (1 if gate is None else v.abs() + ve)
    half = half_step(dtype)
    shape = lambda t: t.reshape(x.shape)  # noqa: E731
    val, bound = {"y": shape(y)}, {"y": shape(half * y.abs() + ye + tiny(dtype))}
    if dy is not None:
        dyd = dy.detach().cpu().double().reshape(-1, groups, n)
        slope_mag = df.abs() + (z.abs() if act == "silu" else 0) * 2  # what df is the difference of, at most
        if gate is None:
            dv = dyd * df
            # |act''| <= 1/2 for both activations
            dve = dyd.abs() * ((0.5 * ve if act != "none" else 0 * ve) + sig * slope_mag + 2.0 ** -23 * df.abs())
        else:
            dv = dyd * f
            dve = dyd.abs() * f.abs() * (sig + 2.0 ** -23)
            dg = dyd * v * df
            dge = dyd.abs() * (ve * df.abs() + v.abs() * (sig * slope_mag + 2.0 ** -22 * df.abs()))
            val["dgate"] = shape(dg)
            bound["dgate"] = shape(half * dg.abs() + dge + tiny(dtype))
        dve = dve + dyd.abs() * far
        if gate is not None:
            bound["dgate"] = bound["dgate"] + shape(dyd.abs() * (v.abs() + ve) * far)
        q, qe = dv * wg, dve * wg.abs() + 2.0 ** -24 * (dv * wg).abs()
        avg = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
        m0, m1 = avg(q), avg(q * hat)
        m0e = avg(qe) + d * avg(q.abs())
        m1e = avg(qe * hat.abs() + q.abs() * he) + d * avg((q * hat).abs())
        dx = rstd * (q - m0 - hat * m1)
        inner = qe + m0e + he * m1.abs() + hat.abs() * m1e + 2.0 ** -22 * (q.abs() + m0.abs() + (hat * m1).abs())
        dxe = rstd * inner + rel_r * dx.abs()
        val["dx"] = shape(dx)
        bound["dx"] = shape(half_step(x.dtype) * dx.abs() + dxe + tiny(x.dtype))
        # sums over rows: any order is within R additions
        ds = R * 2.0 ** -24
        for name, t, te, par in (("dweight", dv * hat, dve * hat.abs() + dv.abs() * he, weight), ("dbias", dv, dve, bias)):
            if par is not None:
                s = t.sum(0).reshape(-1)
                e = (te + (ds + 2.0 ** -23) * t.abs()).sum(0).reshape(-1)
                val[name], bound[name] = s, half_step(par.dtype) * s.abs() + e + tiny(par.dtype)
    return val, bound


def embed_grad(ids, dy, rows, scale, dtype):
    D = dy.shape[-1]
    ids, dy = ids.cpu().reshape(-1).long(), dy.detach().cpu().double().reshape(-1, D)
    live = (ids >= 0) & (ids < rows)
    zero = torch.zeros(rows, D, dtype=torch.float64)
    val = zero.index_add(0, ids[live], dy[live]) * scale
    mag = zero.index_add(0, ids[live], dy[live].abs()) * abs(scale)
    count = torch.zeros(rows, 1, dtype=torch.float64).index_add(0, ids[live], torch.ones(int(live.sum()), 1, dtype=torch.float64))
    return val, half_step(dtype) * val.abs() + (count + 2) * 2.0 ** -24 * mag + tiny(dtype)


def assert_within(got, val, bound, what):
    g = got.detach().cpu().double()
    assert g.shape == val.shape, (what, g.shape, val.shape)
    assert torch.isfinite(g).all(), what
    over = (g - val).abs() - bound
    assert over.max() <= 0, (what, "off by", float((g - val).abs().flatten()[over.argmax()]), "allowed",
                             float(bound.flatten()[over.argmax()]), "at", int(over.argmax()))
