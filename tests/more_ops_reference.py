"""Plain 64-bit forms of the delta rule, the residual stream's norm and sampling (include/based_ops.h), on the CPU, with bounds on
the error that the kernels may have.

Delta rule: values row by row; bounds from the chunks' matrices. A product of float16 pairs leaves out lo lo (2^-22 of
the operands' largest), splits to 2^-23, and sums up to 128 products of three terms on tensor cores, whose sums are off by at most 2^-23 a step of 16
products: PAIR = 2^-18 of the sum of magnitudes covers them with the roundings around them. A state takes one such error a chunk, and errors of a state
are carried on by whole (1 - ...), which does not enlarge them where beta |k|^2 <= 2: after n chunks they are n times
the largest. Sums of magnitudes of products with states are bounded by norms (Cauchy and Schwarz). Results that are rounded to bfloat16 take single
float16 terms (2^-12 of an operand, three operands in a row): SINGLE = 2^-10.
"""
import math

import torch

PAIR, SINGLE = 2.0 ** -18, 2.0 ** -10
CHUNK = 64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def delta_rows(q, k, v, beta, gate, scale, state, lengths, do=None, dfinal=None):
    """Values of the delta rule and its gradients in 64 bits, row by row: a dict. q, k (B,T,HK,K), v (B,T,H,V)."""
    B, T, H, V = v.shape
    HK, K = q.shape[2:]
    group = H // HK
    cpu = lambda t: t.detach().cpu().double()  # noqa: E731
    q, k = (cpu(t).repeat_interleave(group, 2) for t in (q, k))
    v, beta = cpu(v), cpu(beta)
    gated = gate is not None
    gate = cpu(gate) if gated else torch.zeros(B, T, H, dtype=torch.float64)
    scale = K ** -0.5 if scale is None else scale
    lens = torch.full((B,), T) if lengths is None else lengths.cpu().long().clamp(0, T)
    live = torch.arange(T)[None] < lens[:, None]
    m4, m3 = live[..., None, None], live[..., None]
    q, k, v = (torch.where(m4, t, 0.0) for t in (q, k, v))
    beta, gate = torch.where(m3, beta, 0.0), torch.where(m3, gate, 0.0)
    a = torch.exp(gate)
    S = torch.zeros(B, H, K, V, dtype=torch.float64) if state is None else cpu(state)
    first, o, rows = S, torch.zeros_like(v), []
    for t in range(T):
        P = S * a[:, t, :, None, None]
        e = v[:, t] - torch.einsum("bhkv,bhk->bhv", P, k[:, t])
        u = beta[:, t, :, None] * e
        S = P + k[:, t, :, :, None] * u[:, :, None, :]
        o[:, t] = scale * torch.einsum("bhkv,bhk->bhv", S, q[:, t])
        rows.append((P, e, u, S))
    out = {"o": o, "final": S}
    if do is not None:
        do = torch.where(m4, cpu(do), 0.0)
        G = torch.zeros_like(first) if dfinal is None else cpu(dfinal)
        dq, dk, dv, dbeta, dgate = (torch.zeros_like(t) for t in (q, k, v, beta, gate))
        for t in range(T - 1, -1, -1):
            P, e, u, S = rows[t]
            dq[:, t] = scale * torch.einsum("bhkv,bhv->bhk", S, do[:, t])
            G = G + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
            du = torch.einsum("bhkv,bhk->bhv", G, k[:, t])
            de = beta[:, t, :, None] * du
            dv[:, t], dbeta[:, t] = de, (du * e).sum(-1)
            dk[:, t] = torch.einsum("bhkv,bhv->bhk", G, u) - torch.einsum("bhkv,bhv->bhk", P, de)
            G = G - k[:, t, :, :, None] * de[:, :, None, :]
            dgate[:, t] = (G * P).sum((-1, -2))
            G = G * a[:, t, :, None, None]
        shared = lambda t: t.unflatten(2, (HK, group)).sum(3)  # noqa: E731
        out.update(dq=shared(dq), dk=shared(dk), dv=dv, dbeta=torch.where(m3, dbeta, 0.0), dstate=G)
        if gated:
            out["dgate"] = torch.where(m3, dgate, 0.0)
    return out


def delta_bounds(val, q, k, v, beta, gate, scale, state, lengths, do=None, dfinal=None):
    """Bounds for the values of delta_rows, from norms of the chunks' quantities."""
    dtype = v.dtype
    B, T, H, V = v.shape
    HK, K = q.shape[2:]
    group, n = H // HK, -(-T // CHUNK)
    scale = K ** -0.5 if scale is None else abs(scale)
    lens = torch.full((B,), T) if lengths is None else lengths.cpu().long().clamp(0, T)
    live = (torch.arange(T)[None] < lens[:, None])[..., None]
    cpu = lambda t: t.detach().cpu().double()  # noqa: E731

    def cut(t, width):  # (B,T,H,...) -> (B,H,n,64,...)
        t = torch.where(live.reshape(B, T, *[1] * (t.dim() - 2)), t, 0.0)
        t = torch.cat([t, t.new_zeros(B, n * CHUNK - T, *t.shape[2:])], 1)
        return t.unflatten(1, (n, CHUNK)).movedim(3, 1)

    q, k = (cut(cpu(t).repeat_interleave(group, 2), 2) for t in (q, k))
    v, beta = cut(cpu(v), 2), cut(cpu(beta), 1)
    g = torch.zeros_like(beta) if gate is None else cut(cpu(gate), 1)
    b = g.clamp(min=-1e5).cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool).tril()
    D = torch.where(lower, torch.exp(torch.where(lower, b[..., :, None] - b[..., None, :], 0.0)), 0.0)
    grow, rest, whole = torch.exp(b), torch.exp(b[..., -1:] - b), torch.exp(b[..., -1])
    strict = lower.tril(-1)
    # A score is a sum of K products, off by PAIR |q| |k| however small it comes out (Cauchy and Schwarz again): q_i k_i of unit
    # vectors is 1 / sqrt(K) on average, and its relative error that much larger.
    kk = k.norm(dim=-1)[..., :, None] * k.norm(dim=-1)[..., None, :]
    qk = q.norm(dim=-1)[..., :, None] * k.norm(dim=-1)[..., None, :]
    A = torch.where(strict, beta[..., None] * D * (k @ k.mT), 0.0)
    inv = torch.linalg.inv(torch.eye(CHUNK, dtype=torch.float64) + A)  # (1 + A)^-1; diag(beta) (1 + L)^-1 = (1 + A)^-1 diag(beta)
    Y = torch.where(strict, D * (k @ k.mT) * beta[..., None, :], 0.0)
    inv_e = torch.linalg.inv(torch.eye(CHUNK, dtype=torch.float64) + Y).abs()
    # the inverses are computed by substitution from entries off by PAIR: |inv| |A| |inv| more
    inv_e = inv_e + inv_e @ torch.where(strict, D * kk * beta[..., None, :].abs(), 0.0) @ inv_e
    inv_r = inv.abs() + inv.abs() @ torch.where(strict, beta[..., None].abs() * D * kk, 0.0) @ inv.abs()
    P = scale * D * qk
    nk, nq = k.norm(dim=-1), q.norm(dim=-1)
    S = torch.zeros(B, H, K, V, dtype=torch.float64) if state is None else cpu(state)
    before, X = [], []
    for i in range(n):  # states, by the chunks' products in 64 bits
        before.append(S)
        x = v[:, :, i] - grow[:, :, i, :, None] * (k[:, :, i] @ S)
        X.append(v[:, :, i].abs() + (grow[:, :, i] * nk[:, :, i])[..., None] * S.norm(dim=-2)[:, :, None])
        u = inv[:, :, i] @ (beta[:, :, i, :, None] * x)
        S = whole[:, :, i, None, None] * S + (rest[:, :, i, :, None] * k[:, :, i]).mT @ u
    before, X = torch.stack(before, 2), torch.stack(X, 2)
    E = inv_e @ X                       # magnitudes of E as they are summed up
    U = beta.abs()[..., None] * E
    # one chunk's error of a state, by columns: PAIR of everything that is added up
    per = whole[..., None] * before.norm(dim=-2) + ((rest * nk)[..., None] * U).sum(-2)
    state_err = (n + 2) * PAIR * per.amax(2)                        # (B,H,V)
    fine = SINGLE if dtype == torch.bfloat16 else PAIR
    half = half_step(dtype)

    def rows(t):
        return t.movedim(1, 3).flatten(1, 2)[:, :T]

    mag_o = scale * (grow * nq)[..., None] * before.norm(dim=-2)[..., None, :] + P @ U
    err = {"o": rows(fine * mag_o + (scale * (grow * nq)[..., None] * state_err[:, :, None, None])
                     + P @ (beta.abs()[..., None] * (inv_e @ ((grow * nk)[..., None] * state_err[:, :, None, None] + PAIR * X)))),
           "final": state_err[:, :, None].expand(B, H, K, V)}
    if do is not None:
        d = cut(cpu(do), 2)
        G = torch.zeros_like(S) if dfinal is None else cpu(dfinal)
        after, dU = [None] * n, [None] * n
        for i in reversed(range(n)):
            after[i] = G
            pt = (scale * D * (q @ k.mT))[:, :, i].mT
            du = pt @ d[:, :, i] + rest[:, :, i, :, None] * (k[:, :, i] @ G)
            dU[i] = P[:, :, i].mT @ d[:, :, i].abs() + (rest[:, :, i] * nk[:, :, i])[..., None] * G.norm(dim=-2)[:, :, None]
            dr = inv[:, :, i].mT @ du
            G = (whole[:, :, i, None, None] * G + (scale * grow[:, :, i, :, None] * q[:, :, i]).mT @ d[:, :, i]
                 - ((beta * grow)[:, :, i, :, None] * k[:, :, i]).mT @ dr)
        after, dU = torch.stack(after, 2), torch.stack(dU, 2)
        R = inv_r.mT @ dU
        per = (whole[..., None] * after.norm(dim=-2) + (scale * (grow * nq)[..., None] * d.abs()).sum(-2)
               + ((beta.abs() * grow * nk)[..., None] * R).sum(-2))
        grad_err = (n + 2) * PAIR * per.amax(2)
        r_err = inv_r.mT @ (PAIR * dU + (rest * nk)[..., None] * grad_err[:, :, None, None]) + PAIR * R
        e_err = inv_e @ ((grow * nk)[..., None] * state_err[:, :, None, None] + PAIR * X) + PAIR * E
        # relative errors of what the last products take in: their own, and what came before
        norm_s, norm_g = (t.flatten(-2).norm(dim=-1)[..., None, None] for t in (before, after))
        dn, Rn, En, Un = (t.norm(dim=-1, keepdim=True) for t in (d, R, E, U))
        ds, dg = state_err.norm(dim=-1)[:, :, None, None, None], grad_err.norm(dim=-1)[:, :, None, None, None]
        re, ee = r_err.norm(dim=-1, keepdim=True), e_err.norm(dim=-1, keepdim=True)
        bt = beta.abs()[..., None]
        dP, dA = dn * (bt * En).mT, Rn * (bt * En).mT
        dPe, dAe = fine * dP + dn * (bt * ee).mT, fine * dA + Rn * (bt * ee).mT + re * (bt * En).mT
        gr, rs = grow[..., None], rest[..., None]
        pd, ad = scale * D, torch.where(strict, bt * D, 0.0)
        mq = fine * (scale * gr * dn * norm_s) + scale * gr * dn * ds + (pd * (2 * fine * dP + dPe)) @ nk[..., None]
        mk = (bt * gr * (fine * Rn * norm_s + Rn * ds + re * norm_s) + rs * (fine * Un * norm_g + Un * dg + bt * ee * norm_g)
              + (pd * (2 * fine * dP + dPe)).mT @ nq[..., None] + (ad * (2 * fine * dA + dAe)) @ nk[..., None]
              + (ad * (2 * fine * dA + dAe)).mT @ nk[..., None])
        shared = lambda t: t.unflatten(2, (HK, group)).sum(3)  # noqa: E731
        err["dq"], err["dk"] = (shared(rows(t)).expand(B, T, HK, K) for t in (mq, mk))
        err["dv"] = rows(bt * r_err)
        err["dbeta"] = rows((fine * Rn * En + re * En + Rn * ee)[..., 0])
        err["dstate"] = grad_err[:, :, None].expand(B, H, K, V)
        if gate is not None:
            w = whole[..., None, None]
            pairs = P / scale * scale * dPe + fine * P * dP + ad * kk * (dAe + fine * dA)
            db = (nq[..., None] * mq + nk[..., None] * mk).squeeze(-1) + pairs.sum(-1) + pairs.sum(-2)
            end = (w * (fine * norm_s * norm_g + ds * norm_g + norm_s * dg)).flatten(-2).sum(-1)
            end = end + (rs * nk[..., None] * (fine * Un * norm_g + Un * dg + bt * ee * norm_g)).flatten(-2).sum(-1)
            err["dgate"] = rows(db.flip(-1).cumsum(-1).flip(-1) + end[..., None])
    types = {"final": torch.float32, "dstate": torch.float32}
    # (the bounds of dq, dk and dgate add up worst cases over 64 rows; assert_near holds them to what roundings come to)
    return {name: half_step(types.get(name, dtype)) * val[name].abs() + err[name] + tiny(types.get(name, dtype)) for name in val}


def rms(x, weight, residual, eps, dy=None, dsum=None, quantize=False):
    """Values and bounds of the residual stream's norm: sums over a row are within 40 roundings of 2^-24 (32 in a thread, then halvings), the
    reciprocal square root 2^-22, and each float32 operation 2^-24: 2^-18 in all, relative to magnitudes."""
    d = lambda t: t.detach().cpu().double()  # noqa: E731
    stream = x.dtype if residual is None else residual.dtype
    s = x.detach().cpu() if residual is None else (x.detach().cpu().float() + residual.detach().cpu().float()).to(stream)
    val, bound = {}, {}
    if residual is not None:
        val["sum"] = d(s)
        bound["sum"] = torch.zeros_like(val["sum"])  # float32's sum, rounded once: the same bits
    s = d(s)
    w = torch.ones(s.shape[-1], dtype=torch.float64) if weight is None else d(weight)
    r = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    y = s * r * w
    if quantize:
        top = y.abs().amax(-1, keepdim=True)
        scale = torch.where(top > 0, top / 448, 1.0)
        val["scale"], bound["scale"] = scale[..., 0], scale[..., 0] * 2.0 ** -18
        # e4m3: half a step of 2^-3 relative, 2^-10 below its smallest normal number 2^-6
        val["y"] = y / scale
        bound["y"] = (2.0 ** -4 + 2.0 ** -16) * (y / scale).abs() + 2.0 ** -10
        return val, bound
    val["y"], bound["y"] = y, (half_step(x.dtype) + 2.0 ** -18) * y.abs() + tiny(x.dtype)
    if dy is not None:
        g, extra = d(dy), 0.0 if dsum is None else d(dsum)
        t = g * w
        mean = (t * s).mean(-1, keepdim=True)
        val["ds"] = r * (t - s * r * r * mean) + extra
        mags = r * (t.abs() + s.abs() * r * r * (t * s).abs().mean(-1, keepdim=True)) + (0.0 if dsum is None else extra.abs())
        bound["ds"] = half_step(stream) * val["ds"].abs() + 2.0 ** -18 * mags + tiny(stream)
        if stream != x.dtype:
            val["dx"], bound["dx"] = val["ds"], half_step(x.dtype) * val["ds"].abs() + 2.0 ** -18 * mags + tiny(x.dtype)
        if weight is not None:
            rows = g.flatten(0, -2) if g.dim() > 1 else g[None]
            hat = (s * r).reshape(rows.shape)
            val["dweight"] = (rows * hat).sum(0)
            # any order of R additions
            e = (2.0 ** -18 + rows.shape[0] * 2.0 ** -24) * (rows * hat).abs().sum(0)
            bound["dweight"] = half_step(weight.dtype) * val["dweight"].abs() + e + tiny(weight.dtype)
    return val, bound


def sample_order(logits, temperature, top_k, top_p, min_p):
    """What a row of logits keeps: (indices in rising order, their probabilities among the kept), by the definition in 64 bits."""
    x = logits.detach().cpu().double()
    x = torch.where(x.isnan(), -math.inf, x)
    order = torch.argsort(x, descending=True, stable=True)
    order = order[x[order] > -math.inf]
    m = torch.exp((x[order] - x[order[0]]) / temperature)
    if top_k is not None and 0 < top_k < order.numel():
        order, m = order[:top_k], m[:top_k]
    if top_p is not None and top_p < 1:
        c = m.cumsum(0)
        n = 1 if top_p <= 0 else 1 + int((c < top_p * c[-1]).sum())
        order, m = order[:n], m[:n]
    if min_p is not None and min_p > 0:
        keep = m >= min(min_p, 1.0)
        order, m = order[keep], m[keep]
    order, by = torch.sort(order)
    m = m[by]
    return order, m / m.sum()


def assert_within(got, val, bound, what):
    g = got.detach().cpu().double()
    assert g.shape == val.shape, (what, g.shape, val.shape)
    assert torch.isfinite(g).all(), what
    over = (g - val).abs() - bound
    if over.numel():
        assert over.max() <= 0, (what, "off by", float((g - val).abs().flatten()[over.argmax()]), "allowed",
                                 float(bound.flatten()[over.argmax()]), "at", int(over.argmax()))


def assert_near(got, val, dtype, what, rows=16):
    """A tighter bound of a whole than assert_within's of its worst element: roundings are independent of one another, so that the root mean square
    of 16 rows' errors is that of a rounding of the result (half a step at most), and of the terms in it: 2^-12 an operand of SINGLE's, 2^-22 of
    PAIR's, times 8 (three operands one after the other, and sums whose terms cancel to a third). Rows whose values are small count as the
    average one does."""
    g = got.detach().cpu().double()
    tol = half_step(dtype) + 8 * (2.0 ** -12 if dtype == torch.bfloat16 else 2.0 ** -22 * 8)
    cut = lambda t: torch.stack([b.square().flatten(1).mean(1) for b in t.split(rows, 1)]).sqrt()  # noqa: E731
    err, size = cut(g - val), cut(val).clamp(min=float(val.square().mean().sqrt()))
    assert (err <= tol * size + tiny(dtype)).all(), (what, float((err / size).max()), tol)
