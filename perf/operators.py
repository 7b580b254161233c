"""The language-model operators beside the Based forward pass, as cases that can be timed.

Three operators: the gated linear recurrence (``based_scan_*``), the per-token group norm with an
activation (``based_norm_*``) and the scaled embedding with its gradient (``based_embed_*``). Each
case runs either in plain torch (``own`` false) or through the package's entry points (``own``
true) on the same inputs.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------
def _scan(name, b, t, d, mode, dtype, way, ragged=False, packed=False):
    return {"name": name, "op": "scan", "way": way, "b": b, "t": t, "d": d, "mode": mode, "dtype": dtype,
            "ragged": ragged, "packed": packed}


def _step(name, n, slots, d, mode, dtype):
    return {"name": name, "op": "step", "n": n, "slots": slots, "d": d, "mode": mode, "dtype": dtype}


def _norm(name, rows, c, groups, x_dtype, dtype, params, act, gated, way):
    return {"name": name, "op": "norm", "way": way, "rows": rows, "c": c, "groups": groups, "x_dtype": x_dtype,
            "dtype": dtype, "params": params, "act": act, "gated": gated}


def _embed(name, n, vocab, d, dtype, grad, way, padded=False):
    return {"name": name, "op": "embed", "way": way, "n": n, "vocab": vocab, "d": d, "dtype": dtype, "grad": grad,
            "padded": padded}


def listed():
    return [
        # one sequence that generates: one token through one layer's recurrence (16 heads x 64)
        _step("step of one sequence", 1, 1, 1024, "sigmoid", "bfloat16"),
        # a full serving batch: every running sequence advances by one token, in a pool of states
        _step("step of 256 sequences", 256, 512, 4096, "log", "bfloat16"),
        # prefill of one long prompt (the long workload's width and length); gate and x are the two
        # halves of one projection's output
        _scan("prefill of a long prompt", 1, 16384, 2048, "sigmoid", "bfloat16", "forward", packed=True),
        # a training step on right-padded sequences (the ragged workload's sizes)
        _scan("training on padded sequences", 8, 3000, 1536, "sigmoid", "bfloat16", "train", ragged=True),
        # a small model trained in float32, with sizes that no tile divides
        _scan("training in float32, odd sizes", 2, 2047, 777, "log", "float32", "train"),
        # a large training batch of long sequences
        _scan("training on long sequences", 8, 16384, 2048, "log", "bfloat16", "train", packed=True),
        # the norm of one decoding step
        _norm("norm of a decoding step", 16, 2048, 32, "bfloat16", "bfloat16", "bfloat16", "silu", True, "forward"),
        # norm and gate on the float32 output of the headline Based call (16 heads x 64)
        _norm("norm of the headline output", 16384, 1024, 16, "float32", "bfloat16", "float32", "silu", True, "forward"),
        # a training step at the ragged workload's sizes (12 heads x 128)
        _norm("norm in training", 24000, 1536, 12, "bfloat16", "bfloat16", "float32", "silu", True, "train"),
        # groups of 125 channels, activation on the normalised value itself, no gate
        _norm("norm in training, odd groups", 4099, 1000, 8, "float16", "float16", "float32", "silu", False, "train"),
        # a small training batch on a small vocabulary
        _embed("embedding, small batch", 512, 8192, 512, "float16", "float32", "train"),
        # a training batch with padding on a large vocabulary
        _embed("embedding, large batch", 32768, 50000, 1024, "bfloat16", "float32", "train", padded=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    kind = rng.choice(["step", "scan", "scan", "scan", "norm", "norm", "norm", "embed", "embed"])
    if kind == "step":
        n = _log_uniform(rng, 1, 512)
        d = _log_uniform(rng, 128, 8192)
        return _step("", n, n + rng.randrange(0, 64), d - d % 8 if rng.random() < 0.7 else d, rng.choice(["log", "sigmoid"]),
                     dtype)
    if kind == "scan":
        d = _log_uniform(rng, 64, 4096)
        return _scan("", _log_uniform(rng, 1, 16), _log_uniform(rng, 16, 20000), d - d % 8 if rng.random() < 0.7 else d,
                     rng.choice(["log", "sigmoid"]), dtype, rng.choice(["forward", "train", "train"]),
                     ragged=rng.random() < 0.4, packed=rng.random() < 0.5)
    if kind == "norm":
        groups = rng.choice([1, 2, 4, 8, 12, 16, 32])
        size = rng.choice([32, 64, 64, 128, 128, 256, rng.randrange(17, 300)])
        x_dtype = "float32" if rng.random() < 0.3 else dtype
        return _norm("", _log_uniform(rng, 1, 100000), groups * size, groups, x_dtype, dtype, rng.choice(["float32", dtype]),
                     rng.choice(["silu", "sigmoid", "none"]), rng.random() < 0.7, rng.choice(["forward", "train", "train"]))
    d = _log_uniform(rng, 64, 4096)
    return _embed("", _log_uniform(rng, 1, 65536), _log_uniform(rng, 1000, 100000), d - d % 8 if rng.random() < 0.8 else d,
                  dtype, rng.choice(["float32", dtype]), rng.choice(["forward", "train", "train"]), padded=rng.random() < 0.4)


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        case = _draw(rng)
        if work(case)["bytes"] <= most:
            del case["name"]
            return case


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def gates(mode, *shape):
        # forget-gate logits with a positive bias (memories of a few to some hundred tokens), or
        # log decays -softplus(.) / 4 of about the same memories
        f = normal(*shape) * 1.5 + 2.5
        return f if mode == "sigmoid" else torch.nn.functional.logsigmoid(f) * 0.5

    op, s = case["op"], {"case": case}
    dtype = DTYPES[case["dtype"]]
    if op == "step":
        s["gate"] = gates(case["mode"], case["n"], case["d"]).to(dtype)
        s["x"] = normal(case["n"], case["d"]).to(dtype)
        s["pool"] = normal(case["slots"], case["d"])
        s["slots"] = torch.randperm(case["slots"], generator=gen, device=DEV)[: case["n"]].to(torch.int32)
    elif op == "scan":
        b, t, d = case["b"], case["t"], case["d"]
        if case["packed"]:  # one projection's output, split in two
            both = torch.empty(b, t, 2 * d, device=DEV, dtype=dtype)
            both[..., :d] = gates(case["mode"], b, t, d)
            both[..., d:] = normal(b, t, d)
            s["gate"], s["x"] = both[..., :d], both[..., d:]
        else:
            s["gate"], s["x"] = gates(case["mode"], b, t, d).to(dtype), normal(b, t, d).to(dtype)
        s["state"] = normal(b, d) * 0.5
        s["lengths"] = None
        if case["ragged"]:
            s["lengths"] = torch.randint(0, t + 1, (b,), generator=gen, device=DEV, dtype=torch.int32)
            s["lengths"][0] = t
        if case["way"] == "train":
            s["dy"], s["dfinal"] = normal(b, t, d).to(dtype), normal(b, d)
    elif op == "norm":
        rows, c = case["rows"], case["c"]
        s["x"] = (normal(rows, c) * 0.7 + 0.2).to(DTYPES[case["x_dtype"]])
        s["gate"] = normal(rows, c).to(dtype) if case["gated"] else None
        s["weight"] = (1 + 0.2 * normal(c)).to(DTYPES[case["params"]])
        s["bias"] = (0.2 * normal(c)).to(DTYPES[case["params"]])
        if case["way"] == "train":
            s["dy"] = normal(rows, c).to(dtype)
    else:
        n, vocab, d = case["n"], case["vocab"], case["d"]
        # token frequencies fall with the rank (about 1 / rank), as in text
        u = torch.rand(n, generator=gen, device=DEV, dtype=torch.float64)
        rank = torch.exp(u * math.log(vocab + 1.0)).to(torch.int64) - 1
        s["ids"] = torch.randperm(vocab, generator=gen, device=DEV)[rank.clamp(0, vocab - 1)].to(torch.int32)
        if case["padded"]:
            s["ids"][torch.rand(n, generator=gen, device=DEV) < 0.1] = -1
        s["table"] = (normal(vocab, d) * d ** -0.5).to(dtype)
        s["scale"] = float(d) ** 0.5
        if case["way"] == "train":
            s["dy"] = normal(n, d).to(dtype)
    return s


# ------------------------------------------------------------------------------------------------
# The plain forms: float32 throughout, one rounding at the end
# ------------------------------------------------------------------------------------------------
def _decay(mode, gate, x):
    g, x = gate.float(), x.float()
    if mode == "log":
        return torch.exp(g), x
    return torch.sigmoid(g), torch.sigmoid(-g) * x


def _prefix(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1, from h = 0, by doubling: after k steps (a, u) at t hold the
    composition of the 2^k affine maps that end at t."""
    s, t = 1, a.shape[1]
    while s < t:
        u = torch.cat([u[:, :s], u[:, s:] + a[:, s:] * u[:, :-s]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return u


def _plain_scan(s):
    c = s["case"]
    b, t, d = c["b"], c["t"], c["d"]
    dtype = s["x"].dtype
    a, u = _decay(c["mode"], s["gate"], s["x"])
    live = None
    if s["lengths"] is not None:  # rows past a sequence's length keep its state
        live = (torch.arange(t, device=DEV) < s["lengths"][:, None])[..., None]
        a, u = torch.where(live, a, 1.0), torch.where(live, u, 0.0)
    h = _prefix(a, torch.cat([u[:, :1] + a[:, :1] * s["state"][:, None], u[:, 1:]], 1))
    y = h if live is None else torch.where(live, h, 0.0)
    out = {"y": y.to(dtype), "final": h[:, -1].contiguous()}
    if c["way"] == "train":
        dy = s["dy"].float() if live is None else torch.where(live, s["dy"].float(), 0.0)
        dy = torch.cat([dy[:, :-1], dy[:, -1:] + s["dfinal"][:, None]], 1)
        # lam_t = dy_t + a_{t+1} lam_{t+1}: the same prefix over reversed time
        nxt = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
        lam = _prefix(nxt.flip(1), dy.flip(1)).flip(1)
        before = torch.cat([s["state"][:, None], h[:, :-1]], 1)
        if c["mode"] == "log":
            dg, dx = a * before * lam, lam
        else:
            rest = torch.sigmoid(-s["gate"].float())
            dg, dx = a * rest * (before - s["x"].float()) * lam, rest * lam
        if live is not None:
            dg, dx = torch.where(live, dg, 0.0), torch.where(live, dx, 0.0)
        out.update(dgate=dg.to(dtype), dx=dx.to(dtype), dstate=a[:, 0] * lam[:, 0])
    return out


def _plain_step(s):
    a, u = _decay(s["case"]["mode"], s["gate"], s["x"])
    at = s["slots"].long()
    h = a * s["pool"][at] + u
    s["pool"][at] = h
    return {"y": h.to(s["x"].dtype), "pool": s["pool"]}


def _act(kind, v):
    """act(v) and its derivative."""
    if kind == "none":
        return v, torch.ones_like(v)
    p = torch.sigmoid(v)
    if kind == "sigmoid":
        return p, p * (1 - p)
    return v * p, p * (1 + v * (1 - p))


def _plain_norm(s):
    c = s["case"]
    rows, n, g = c["rows"], c["c"], c["groups"]
    x = s["x"].float().view(rows, g, n // g)
    x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)
    hat = (x * rstd).view(rows, n)
    w, b = s["weight"].float(), s["bias"].float()
    v = hat * w + b
    gate = None if s["gate"] is None else s["gate"].float()
    f, df = _act(c["act"], v if gate is None else gate)
    dtype = DTYPES[c["dtype"]]
    out = {"y": (f if gate is None else v * f).to(dtype)}
    if c["way"] == "train":
        dy = s["dy"].float()
        dv = dy * (df if gate is None else f)
        if gate is not None:
            out["dgate"] = (dy * v * df).to(dtype)
        out["dweight"] = (dv * hat).sum(0).to(s["weight"].dtype)
        out["dbias"] = dv.sum(0).to(s["bias"].dtype)
        dh, hat = (dv * w).view(rows, g, n // g), hat.view(rows, g, n // g)
        dx = rstd * (dh - dh.mean(-1, keepdim=True) - hat * (dh * hat).mean(-1, keepdim=True))
        out["dx"] = dx.view(rows, n).to(s["x"].dtype)
    return out


def _plain_embed(s):
    c = s["case"]
    live = ((s["ids"] >= 0) & (s["ids"] < c["vocab"]))[:, None]
    at = s["ids"].clamp(0, c["vocab"] - 1).long()
    out = {"y": torch.where(live, s["table"][at].float() * s["scale"], 0.0).to(s["table"].dtype)}
    if c["way"] == "train":
        dy = torch.where(live, s["dy"].float(), 0.0)
        dt = torch.zeros(c["vocab"], c["d"], device=DEV).index_add_(0, at, dy)
        out["dtable"] = (dt * s["scale"]).to(DTYPES[c["grad"]])
    return out


# ------------------------------------------------------------------------------------------------
# The package's operators
# ------------------------------------------------------------------------------------------------
def _own_scan(s):
    from linear_attention_gb300 import based_scan_bwd, based_scan_fwd

    mode, train = s["case"]["mode"], s["case"]["way"] == "train"
    y, final, saved = based_scan_fwd(s["gate"], s["x"], mode=mode, state=s["state"], lengths=s["lengths"], save=train)
    out = {"y": y, "final": final}
    if train:
        out["dgate"], out["dx"], out["dstate"] = based_scan_bwd(s["gate"], s["x"], s["dy"], saved, mode=mode,
                                                                dfinal=s["dfinal"], lengths=s["lengths"])
    return out


def _own_step(s):
    from linear_attention_gb300 import based_scan_step

    return {"y": based_scan_step(s["gate"], s["x"], s["pool"], mode=s["case"]["mode"], slots=s["slots"]), "pool": s["pool"]}


def _own_norm(s):
    from linear_attention_gb300 import based_norm_bwd, based_norm_fwd

    c = s["case"]
    args = dict(groups=c["groups"], weight=s["weight"], bias=s["bias"], gate=s["gate"], act=c["act"], eps=1e-5)
    out = {"y": based_norm_fwd(s["x"], out_dtype=DTYPES[c["dtype"]], **args)}
    if c["way"] == "train":
        dx, dgate, dweight, dbias = based_norm_bwd(s["dy"], s["x"], **args)
        out.update(dx=dx, dweight=dweight, dbias=dbias)
        if dgate is not None:
            out["dgate"] = dgate
    return out


def _own_embed(s):
    from linear_attention_gb300 import based_embed_bwd, based_embed_fwd

    c = s["case"]
    out = {"y": based_embed_fwd(s["ids"], s["table"], scale=s["scale"])}
    if c["way"] == "train":
        out["dtable"] = based_embed_bwd(s["ids"], s["dy"], c["vocab"], scale=s["scale"], dtype=DTYPES[c["grad"]])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"scan": _own_scan, "step": _own_step, "norm": _own_norm, "embed": _own_embed}[op](state)
    return {"scan": _plain_scan, "step": _plain_step, "norm": _plain_norm, "embed": _plain_embed}[op](state)


# ------------------------------------------------------------------------------------------------
# What a pass cannot do without: each input read once, each output written once
# ------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    es = 4 if case["dtype"] == "float32" else 2
    if op == "step":
        n = case["n"] * case["d"]
        return {"bytes": n * (3 * es + 8) + 4 * case["n"], "flops": 10 * n}
    if op == "scan":
        n, rows = case["b"] * case["t"] * case["d"], case["b"] * case["d"]
        if case["way"] == "forward":
            return {"bytes": n * 3 * es + rows * 8, "flops": 10 * n}
        return {"bytes": n * 6 * es + rows * 16, "flops": 25 * n}
    if op == "norm":
        n, xs = case["rows"] * case["c"], 4 if case["x_dtype"] == "float32" else 2
        ps = 4 if case["params"] == "float32" else 2
        if case["way"] == "forward":
            return {"bytes": n * (xs + es + (es if case["gated"] else 0)) + 2 * ps * case["c"], "flops": 15 * n}
        return {"bytes": n * (2 * xs + 2 * es + (2 * es if case["gated"] else 0)) + 4 * ps * case["c"], "flops": 45 * n}
    n = case["n"] * case["d"]
    # a table row is read once however often its token occurs: at most one row per token, or the table
    table = min(case["n"], case["vocab"]) * case["d"]
    total = table * es + n * es + 4 * case["n"]
    if case["way"] == "train":
        total += n * es + case["vocab"] * case["d"] * (4 if case["grad"] == "float32" else 2)
    return {"bytes": total, "flops": (1 if case["way"] == "forward" else 3) * n}


# ------------------------------------------------------------------------------------------------
# The definitions in 64 bits, row by row
# ------------------------------------------------------------------------------------------------
def _exact_scan(s):
    c = s["case"]
    b, t = c["b"], c["t"]
    # time first, so that one step reads one block
    g, x = (s[k].double().transpose(0, 1).contiguous() for k in ("gate", "x"))
    a = torch.exp(g) if c["mode"] == "log" else 1 / (1 + torch.exp(-g))
    rest = None if c["mode"] == "log" else 1 / (1 + torch.exp(g))
    del g
    u = x if rest is None else rest * x
    lens = torch.full((b,), t, device=DEV) if s["lengths"] is None else s["lengths"].long()
    whole = s["lengths"] is None
    h = torch.empty_like(x)
    now = s["state"].double()
    for i in range(t):
        nxt = a[i] * now + u[i]
        now = nxt if whole else torch.where((lens > i)[:, None], nxt, now)
        h[i] = now

    def back(v):  # (t, b, d) -> (b, t, d), zero past the lengths
        if not whole:
            v = v * (torch.arange(t, device=DEV)[:, None] < lens[None])[..., None]
        return v.transpose(0, 1)

    out = {"y": back(h), "final": now}
    if c["way"] == "train":
        dy = s["dy"].double().transpose(0, 1).contiguous()
        first, later = s["state"].double(), s["dfinal"].double()  # later: d loss / d h_i from the rows after i
        dg, dx = torch.empty_like(x), torch.empty_like(x)
        for i in range(t - 1, -1, -1):
            lam = later + dy[i]
            before = h[i - 1] if i else first
            if rest is None:
                dg[i], dx[i] = a[i] * before * lam, lam
            else:
                dg[i], dx[i] = a[i] * rest[i] * (before - x[i]) * lam, rest[i] * lam
            lam = a[i] * lam
            later = lam if whole else torch.where((lens > i)[:, None], lam, later)
        out.update(dgate=back(dg), dx=back(dx), dstate=later)
    return out


def _exact_step(s):
    g, x, at = s["gate"].double(), s["x"].double(), s["slots"].long()
    a = torch.exp(g) if s["case"]["mode"] == "log" else 1 / (1 + torch.exp(-g))
    u = x if s["case"]["mode"] == "log" else x / (1 + torch.exp(g))
    pool = s["pool"].double()
    pool[at] = a * pool[at] + u
    return {"y": pool[at], "pool": pool}


def _exact_norm(s):
    c = s["case"]
    x = s["x"].double().unflatten(1, (c["groups"], -1))
    mean, var = x.mean(2), x.var(2, unbiased=False)
    sd = (var + 1e-5).sqrt()
    hat = ((x - mean[..., None]) / sd[..., None]).flatten(1)
    v = hat * s["weight"].double() + s["bias"].double()
    z = v if s["gate"] is None else s["gate"].double()
    p = 1 / (1 + torch.exp(-z))
    f = {"none": z, "sigmoid": p, "silu": z * p}[c["act"]]
    slope = {"none": torch.ones_like(p), "sigmoid": p * (1 - p), "silu": p + z * p * (1 - p)}[c["act"]]
    out = {"y": f if s["gate"] is None else f * v}
    if c["way"] == "train":
        dy = s["dy"].double()
        dv = dy * (slope if s["gate"] is None else f)
        if s["gate"] is not None:
            out["dgate"] = dy * slope * v
        out["dweight"], out["dbias"] = torch.einsum("rc,rc->c", dv, hat), torch.einsum("rc->c", dv)
        # through hat = (x - mean) / sd: d hat_j / d x_i = (delta_ij - 1/n - hat_i hat_j / n) / sd
        q, k = (dv * s["weight"].double()).unflatten(1, (c["groups"], -1)), hat.unflatten(1, (c["groups"], -1))
        n = q.shape[2]
        dx = q - q.sum(2, keepdim=True) / n - k * torch.einsum("rgi,rgi->rg", q, k)[..., None] / n
        out["dx"] = (dx / sd[..., None]).flatten(1)
    return out


def _exact_embed(s):
    c = s["case"]
    ids = s["ids"].long()
    live = (ids >= 0) & (ids < c["vocab"])
    y = torch.zeros(c["n"], c["d"], device=DEV, dtype=torch.float64)
    y[live] = s["table"][ids[live]].double() * s["scale"]
    out = {"y": y}
    if c["way"] == "train":
        grad = torch.zeros(c["vocab"], c["d"], device=DEV, dtype=torch.float64)
        grad.index_put_((ids[live],), s["dy"][live].double() * s["scale"], accumulate=True)
        out["dtable"] = grad
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"scan": _exact_scan, "step": _exact_step, "norm": _exact_norm, "embed": _exact_embed}[case["op"]](s)
