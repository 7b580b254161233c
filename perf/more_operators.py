"""More language-model operators beside the Based forward pass, as cases that can be timed.

Three operators: the gated delta rule, a linear attention whose state forgets and corrects itself
(``based_delta_*``), the root-mean-square norm of a residual stream with the addition in front of it
and an output in 8 bits (``based_rms_*``), and the choice of the next token (``based_sample``). Each
case runs either in plain torch (``own`` false) or through the package's entry points (``own`` true)
on the same inputs.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
CHUNK = 64  # rows that the plain form of the delta rule takes at once
RMS_EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------
def _delta(name, b, t, h, hk, k, v, dtype, way, gated=True, ragged=False):
    return {"name": name, "op": "delta", "way": way, "b": b, "t": t, "h": h, "hk": hk, "k": k, "v": v, "dtype": dtype,
            "gated": gated, "ragged": ragged}


def _step(name, n, slots, h, hk, k, v, dtype):
    return {"name": name, "op": "delta_step", "n": n, "slots": slots, "h": h, "hk": hk, "k": k, "v": v, "dtype": dtype}


def _rms(name, rows, c, dtype, stream, way, residual=True, quantize=False):
    return {"name": name, "op": "rms", "way": way, "rows": rows, "c": c, "dtype": dtype, "stream": stream, "residual": residual,
            "quantize": quantize}


def _sample(name, n, vocab, dtype, top_k, top_p, min_p):
    return {"name": name, "op": "sample", "n": n, "vocab": vocab, "dtype": dtype, "top_k": top_k, "top_p": top_p, "min_p": min_p}


def listed():
    return [
        # one sequence that generates: one token through one layer's delta rule
        _step("delta step, one sequence", 1, 1, 16, 16, 64, 64, "bfloat16"),
        # a full serving batch: every running sequence advances by one token, in a pool of states; pairs of
        # value heads share their queries and keys
        _step("delta step, 256 sequences", 256, 320, 16, 8, 128, 128, "bfloat16"),
        # prefill of one long prompt (the long workload's length, heads and value size)
        _delta("delta prefill, long prompt", 1, 16384, 16, 16, 128, 128, "bfloat16", "forward"),
        # a training step on right-padded sequences (the ragged workload's sizes), shared query and key heads
        _delta("delta training, padded", 8, 3000, 12, 6, 64, 128, "bfloat16", "train", ragged=True),
        # a small model trained in float32, with sizes that no tile divides, without decays
        _delta("delta training, float32, odd", 2, 777, 3, 3, 40, 75, "float32", "train", gated=False),
        # a large training batch (the headline's length and heads at twice its batch)
        _delta("delta training, large batch", 8, 4096, 16, 16, 128, 128, "bfloat16", "train"),
        # addition and norm of one decoding step
        _rms("rms of a decoding step", 16, 2048, "bfloat16", "bfloat16", "forward"),
        # prefill in front of an 8-bit matrix product: a float32 residual stream, an output in e4m3
        _rms("rms of a prompt, 8 bits out", 16384, 4096, "bfloat16", "float32", "forward", quantize=True),
        # a training step at the ragged workload's sizes
        _rms("rms in training", 24000, 1536, "bfloat16", "bfloat16", "train"),
        # the next token of one sequence
        _sample("sampling, one sequence", 1, 50000, "float32", 0, 0.95, 0.0),
        # a serving batch in which each request brings its own limits
        _sample("sampling, 256 sequences", 256, 50000, "bfloat16", 64, 0.9, 0.02),
        # a large vocabulary of odd size
        _sample("sampling, large vocabulary", 61, 130001, "float32", 0, 0.9, 0.0),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    kind = rng.choice(["delta", "delta", "delta", "step", "rms", "rms", "sample", "sample"])
    if kind in ("delta", "step"):
        hk = _log_uniform(rng, 1, 16)
        h = hk * rng.choice([1, 1, 2, 4])
        k = rng.choice([16, 32, 64, 64, 128, 128, rng.randrange(8, 129)])
        v = rng.choice([32, 64, 64, 128, 128, 256, rng.randrange(8, 257)])
        if kind == "step":
            n = _log_uniform(rng, 1, 384)
            return _step("", n, n + rng.randrange(0, 64), h, hk, k, v, dtype)
        return _delta("", _log_uniform(rng, 1, 12), _log_uniform(rng, 8, 8192), h, hk, k, v, dtype,
                      rng.choice(["forward", "train", "train"]), gated=rng.random() < 0.8, ragged=rng.random() < 0.3)
    if kind == "rms":
        c = _log_uniform(rng, 64, 8192)
        quantize = rng.random() < 0.3
        return _rms("", _log_uniform(rng, 1, 50000), c - c % 8 if rng.random() < 0.7 else c, dtype, rng.choice([dtype, "float32"]),
                    "forward" if quantize else rng.choice(["forward", "train", "train"]), residual=rng.random() < 0.8,
                    quantize=quantize)
    return _sample("", _log_uniform(rng, 1, 384), _log_uniform(rng, 1000, 200000), dtype, rng.choice([0, 1, 20, 64, 1000]),
                   rng.choice([1.0, 0.95, 0.9, 0.5]), rng.choice([0.0, 0.0, 0.02, 0.1]))


def draw(rng):
    # a drawn case costs at most what the largest listed one of its operator does
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], 0), w["bytes"] + w["flops"] / 100)
    while True:
        case = _draw(rng)
        w = work(case)
        if w["bytes"] + w["flops"] / 100 <= most[case["op"]]:
            del case["name"]
            return case


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    def direction(*shape):  # queries and keys of length 1, as the delta rule's layers make them
        x = normal(*shape)
        return x / (x * x).sum(-1, keepdim=True).sqrt()

    op, s, dtype = case["op"], {"case": case}, DTYPES[case["dtype"]]
    if op in ("delta", "delta_step"):
        lead = (case["b"], case["t"]) if op == "delta" else (case["n"],)
        h, hk, k, v = case["h"], case["hk"], case["k"], case["v"]
        s["q"], s["k"] = direction(*lead, hk, k).to(dtype), direction(*lead, hk, k).to(dtype)
        s["v"] = normal(*lead, h, v).to(dtype)
        s["beta"] = torch.sigmoid(normal(*lead, h)).to(dtype)
        # log decays with memories of a few to some hundred tokens
        f = normal(*lead, h) * 1.5 + 2.5
        s["gate"] = (-0.5 * torch.log1p(torch.exp(-f))).to(dtype) if case.get("gated", True) else None
        if op == "delta_step":
            s["pool"] = normal(case["slots"], h, k, v) * 0.3
            s["slots"] = torch.randperm(case["slots"], generator=gen, device=DEV)[: case["n"]].to(torch.int32)
            return s
        s["state"] = normal(case["b"], h, k, v) * 0.3
        s["lengths"] = None
        if case["ragged"]:
            s["lengths"] = torch.randint(0, case["t"] + 1, (case["b"],), generator=gen, device=DEV, dtype=torch.int32)
            s["lengths"][0] = case["t"]
        if case["way"] == "train":
            s["do"] = normal(*lead, h, v).to(dtype)
            s["dfinal"] = normal(case["b"], h, k, v) * 0.3
    elif op == "rms":
        rows, c, stream = case["rows"], case["c"], DTYPES[case["stream"]]
        s["residual"] = (normal(rows, c) * 2.0).to(stream) if case["residual"] else None
        s["x"] = normal(rows, c).to(dtype)
        s["weight"] = (1 + 0.2 * normal(c)).to(dtype)
        if case["way"] == "train":
            s["dy"] = normal(rows, c).to(dtype)
            s["dsum"] = normal(rows, c).to(stream if case["residual"] else dtype)
    else:
        n, vocab = case["n"], case["vocab"]
        # logits of a trained model: most of the mass in some tokens, a long tail
        s["logits"] = (normal(n, vocab) * 2.0 + 4.0 * uniform(n, vocab) ** 8).to(dtype)
        s["u"] = uniform(n)
        # requests of a batch bring their own limits around the case's
        s["temperature"] = 0.5 + uniform(n)
        s["top_k"] = None
        if case["top_k"]:
            s["top_k"] = (1 + uniform(n) * (2 * case["top_k"] - 1)).to(torch.int32)
        s["top_p"] = None
        if case["top_p"] < 1:
            s["top_p"] = 1 - (1 - case["top_p"]) * 2 * uniform(n)
        s["min_p"] = None
        if case["min_p"] > 0:
            s["min_p"] = case["min_p"] * 2 * uniform(n)
    return s


# ------------------------------------------------------------------------------------------------
# The plain forms: float32 throughout (sums of log decays and the order of tokens' masses in 64 bits), one
# rounding at the end
# ------------------------------------------------------------------------------------------------
def _chunks(x, n):
    """(B,T,H,...) -> (B,H,n,CHUNK,...) in float32, with zeros behind the last row."""
    x = x.float()
    pad = n * CHUNK - x.shape[1]
    x = torch.cat([x, x.new_zeros(x.shape[0], pad, *x.shape[2:])], 1)
    return x.unflatten(1, (n, CHUNK)).movedim(3, 1)


def _rows(x, t):
    """(B,H,n,CHUNK,...) -> (B,T,H,...)."""
    return x.movedim(1, 3).flatten(1, 2)[:, :t]


def _plain_delta(s):
    c = s["case"]
    t, h, hk, dtype = c["t"], c["h"], c["hk"], s["v"].dtype
    n, group, scale = -(-t // CHUNK), h // hk, c["k"] ** -0.5
    q, k, v = s["q"].repeat_interleave(group, 2), s["k"].repeat_interleave(group, 2), s["v"]
    beta, gate = s["beta"], s["gate"]
    live = None
    if s["lengths"] is not None:  # rows past a sequence's length change nothing
        live = (torch.arange(t, device=DEV) < s["lengths"][:, None])[..., None]
        q, k, v = (torch.where(live[..., None], x, 0) for x in (q, k, v))
        beta, gate = torch.where(live, beta, 0), gate if gate is None else torch.where(live, gate, 0)
    q, k, v, beta = (_chunks(x, n) for x in (q, k, v, beta))
    b = torch.zeros_like(beta, dtype=torch.float64) if gate is None else _chunks(gate, n).double().cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, device=DEV, dtype=torch.bool).tril()
    strict = lower.tril(-1)
    decay = torch.where(lower, torch.exp(torch.where(lower, b[..., :, None] - b[..., None, :], 0.0)), 0.0).float()
    grow, rest = torch.exp(b).float()[..., None], torch.exp(b[..., -1:] - b).float()[..., None]
    whole = grow[..., -1:, :]
    y = torch.where(strict, decay * (k @ k.transpose(-1, -2)), 0.0)
    p = scale * decay * (q @ k.transpose(-1, -2))
    a = beta[..., None] * y
    inv = torch.eye(CHUNK, device=DEV).expand_as(a).clone()  # (1 + a)^-1, row by row
    for i in range(1, CHUNK):
        inv[..., i, :i] = -(a[..., i:i + 1, :i] @ inv[..., :i, :i])[..., 0, :]
    state = s["state"].float()
    before, x, u = [], torch.empty_like(v), torch.empty_like(v)
    for i in range(n):
        before.append(state)
        x[:, :, i] = v[:, :, i] - grow[:, :, i] * (k[:, :, i] @ state)
        u[:, :, i] = inv[:, :, i] @ (beta[:, :, i, :, None] * x[:, :, i])
        state = whole[:, :, i] * state + (rest[:, :, i] * k[:, :, i]).transpose(-1, -2) @ u[:, :, i]
    before = torch.stack(before, 2)
    o = _rows(scale * grow * (q @ before) + p @ u, t)
    out = {"o": (o if live is None else torch.where(live[..., None], o, 0.0)).to(dtype), "final": state}
    if c["way"] != "train":
        return out
    do = s["do"] if live is None else torch.where(live[..., None], s["do"], 0)
    do = _chunks(do, n)
    later, dr, after = s["dfinal"].float(), torch.empty_like(v), [None] * n
    for i in reversed(range(n)):
        after[i] = later
        du = p[:, :, i].transpose(-1, -2) @ do[:, :, i] + rest[:, :, i] * (k[:, :, i] @ later)
        dr[:, :, i] = inv[:, :, i].transpose(-1, -2) @ du
        later = (whole[:, :, i] * later + (scale * grow[:, :, i] * q[:, :, i]).transpose(-1, -2) @ do[:, :, i]
                 - (beta[:, :, i, :, None] * grow[:, :, i] * k[:, :, i]).transpose(-1, -2) @ dr[:, :, i])
    after = torch.stack(after, 2)
    dp, da = do @ u.transpose(-1, -2), -(dr @ u.transpose(-1, -2))
    dq_state, dk_state = scale * grow * (do @ before.transpose(-1, -2)), -beta[..., None] * grow * (dr @ before.transpose(-1, -2))
    dk_next = rest * (u @ after.transpose(-1, -2))
    dpd, dad = scale * decay * dp, torch.where(strict, beta[..., None] * decay * da, 0.0)
    dq = dq_state + dpd @ k
    dk = dk_state + dk_next + dpd.transpose(-1, -2) @ q + (dad + dad.transpose(-1, -2)) @ k
    dbeta = (dr * x).sum(-1) + (da * y).sum(-1)
    out["dq"], out["dk"] = (_rows(d, t).unflatten(2, (hk, group)).sum(3).to(dtype) for d in (dq, dk))
    out["dv"], out["dbeta"], out["dstate"] = _rows(beta[..., None] * dr, t).to(dtype), _rows(dbeta, t).to(dtype), later
    if live is not None:
        out["dbeta"] = torch.where(live, out["dbeta"], 0)
    if s["gate"] is not None:
        # by the sums of log decays: where row i reads what row j wrote, +1 at i and -1 at j
        pairs = dp * p + da * a
        next_ = (k * dk_next).sum(-1)
        db = (q * dq_state + k * dk_state).sum(-1) - next_ + pairs.sum(-1) - pairs.sum(-2)
        end = (whole[..., 0] * (before * after).sum(-1, keepdim=True).sum(-2)) + next_.sum(-1, keepdim=True)
        db = torch.cat([db[..., :-1], db[..., -1:] + end], -1)
        dgate = _rows(db.double().flip(-1).cumsum(-1).flip(-1).float(), t)
        out["dgate"] = (dgate if live is None else torch.where(live, dgate, 0.0)).to(dtype)
    return out


def _plain_step(s):
    c = s["case"]
    group, at = c["h"] // c["hk"], s["slots"].long()
    q, k = (s[x].float().repeat_interleave(group, 1) for x in ("q", "k"))
    state = s["pool"][at] * torch.exp(s["gate"].float())[..., None, None]
    u = s["beta"].float()[..., None] * (s["v"].float() - (state * k[..., None]).sum(-2))
    state = state + k[..., None] * u[..., None, :]
    s["pool"][at] = state
    return {"o": ((state * q[..., None]).sum(-2) * c["k"] ** -0.5).to(s["v"].dtype), "pool": s["pool"]}


def _plain_rms(s):
    c = s["case"]
    x = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    f, w = x.float(), s["weight"].float()
    r = 1 / torch.sqrt((f * f).mean(-1, keepdim=True) + RMS_EPS)
    y = f * r * w
    out = {} if s["residual"] is None else {"sum": x}
    if c["quantize"]:
        top = y.abs().amax(-1, keepdim=True)
        scale = torch.where(top > 0, top / E4M3_MAX, 1.0)
        out["y"], out["scale"] = (y / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale[..., 0]
        return out
    out["y"] = y.to(s["x"].dtype)
    if c["way"] == "train":
        dy = s["dy"].float()
        d = dy * w
        ds = r * d - f * (r * r * r) * (d * f).mean(-1, keepdim=True) + s["dsum"].float()
        out["ds"], out["dweight"] = ds.to(x.dtype), (dy * f * r).sum(0).to(s["weight"].dtype)
        if x.dtype != s["x"].dtype:
            out["dx"] = ds.to(s["x"].dtype)
    return out


def _plain_sample(s):
    x = s["logits"].double()
    n, vocab = x.shape
    x, order = torch.sort(x, dim=-1, descending=True, stable=True)  # equal ones by their index
    m = torch.exp((x - x[:, :1]) / s["temperature"].double()[:, None])
    rank = torch.arange(vocab, device=DEV)
    keep = torch.ones(n, vocab, device=DEV, dtype=torch.bool)
    if s["top_k"] is not None:
        keep = rank < s["top_k"][:, None]
    m = torch.where(keep, m, 0.0)
    if s["top_p"] is not None:  # the fewest of the largest that reach the share
        c = m.cumsum(-1)
        keep = c - m < s["top_p"].double()[:, None] * c[:, -1:]
        m = torch.where(keep, m, 0.0)
    if s["min_p"] is not None:
        m = torch.where(m >= s["min_p"].double()[:, None], m, 0.0)
    m = torch.zeros_like(m).scatter_(1, order, m)  # back in the tokens' order
    c = m.cumsum(-1)
    token = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(-1)
    last = (m > 0).double().mul(rank + 1).amax(-1).long() - 1
    token = torch.minimum(token, last)
    prob = m.gather(1, token[:, None])[:, 0] / c[:, -1]
    return {"token": token.to(torch.int32), "prob": prob.float()}


# ------------------------------------------------------------------------------------------------
# The package's operators
# ------------------------------------------------------------------------------------------------
def _own_delta(s):
    from linear_attention_gb300 import based_delta_bwd, based_delta_fwd

    train = s["case"]["way"] == "train"
    args = s["q"], s["k"], s["v"], s["beta"], s["gate"]
    o, final, saved = based_delta_fwd(*args, state=s["state"], lengths=s["lengths"], save=train)
    out = {"o": o, "final": final}
    if train:
        dq, dk, dv, dbeta, dgate, dstate = based_delta_bwd(*args, s["do"], saved, dfinal=s["dfinal"], lengths=s["lengths"])
        out.update(dq=dq, dk=dk, dv=dv, dbeta=dbeta, dstate=dstate)
        if dgate is not None:
            out["dgate"] = dgate
    return out


def _own_step(s):
    from linear_attention_gb300 import based_delta_step

    return {"o": based_delta_step(s["q"], s["k"], s["v"], s["beta"], s["gate"], s["pool"], slots=s["slots"]), "pool": s["pool"]}


def _own_rms(s):
    from linear_attention_gb300 import based_rms_bwd, based_rms_fwd

    c = s["case"]
    y, total, scale = based_rms_fwd(s["x"], s["weight"], residual=s["residual"], eps=RMS_EPS, quantize=c["quantize"])
    out = {"y": y}
    if s["residual"] is not None:
        out["sum"] = total
    if c["quantize"]:
        out["scale"] = scale
    if c["way"] == "train":
        ds, dx, dweight = based_rms_bwd(s["dy"], total, s["weight"], dsum=s["dsum"], eps=RMS_EPS)
        out.update(ds=ds, dweight=dweight)
        if dx is not ds:
            out["dx"] = dx
    return out


def _own_sample(s):
    from linear_attention_gb300 import based_sample

    token, prob = based_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                               min_p=s["min_p"])
    return {"token": token, "prob": prob}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"delta": _own_delta, "delta_step": _own_step, "rms": _own_rms, "sample": _own_sample}[op](state)
    return {"delta": _plain_delta, "delta_step": _plain_step, "rms": _plain_rms, "sample": _plain_sample}[op](state)


# ------------------------------------------------------------------------------------------------
# What a pass cannot do without: each input read once, each output written once
# ------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    es = 4 if case["dtype"] == "float32" else 2
    if op in ("delta", "delta_step"):
        h, hk, k, v = case["h"], case["hk"], case["k"], case["v"]
        rows = case["b"] * case["t"] if op == "delta" else case["n"]
        seqs = case["b"] if op == "delta" else case["n"]
        scalars = 2 if case.get("gated", True) else 1
        qk, vs, states = 2 * hk * k, h * v, 4 * seqs * h * k * v
        once = rows * es * (qk + 2 * vs + scalars * h) + 2 * states
        if op == "delta_step" or case["way"] == "forward":
            return {"bytes": once, "flops": 6 * rows * h * k * v}
        # forward, and backward: q, k, v, do and the scalars read, their gradients written, with the states'
        return {"bytes": once + rows * es * (2 * qk + 3 * vs + 2 * scalars * h) + 2 * states, "flops": 18 * rows * h * k * v}
    if op == "rms":
        n, rs = case["rows"] * case["c"], 4 if case["stream"] == "float32" else 2
        streams = 2 * rs if case["residual"] else 0
        out = 1 if case["quantize"] else es
        total = n * (es + streams + out) + es * case["c"] + (4 * case["rows"] if case["quantize"] else 0)
        if case["way"] == "train":
            rs = rs if case["residual"] else es
            # dy, the sum and its gradient read, the gradient (in both types where they differ) written
            total += n * (es + 3 * rs + (es if rs != es else 0)) + 2 * es * case["c"]
        return {"bytes": total, "flops": (5 if case["way"] == "forward" else 15) * n}
    n = case["n"] * case["vocab"]
    return {"bytes": n * es + 28 * case["n"], "flops": 8 * n}


# ------------------------------------------------------------------------------------------------
# The definitions in 64 bits, token by token
# ------------------------------------------------------------------------------------------------
def _exact_delta(s):
    c = s["case"]
    t, h, hk, scale = c["t"], c["h"], c["hk"], c["k"] ** -0.5
    group = h // hk
    q, k = (s[x].double().transpose(0, 1).repeat_interleave(group, 2) for x in ("q", "k"))
    v, beta = (s[x].double().transpose(0, 1) for x in ("v", "beta"))
    a = torch.ones_like(beta) if s["gate"] is None else torch.exp(s["gate"].double().transpose(0, 1))
    if s["lengths"] is not None:  # a row behind the last of its sequence: no decay, nothing written
        live = torch.arange(t, device=DEV)[:, None] < s["lengths"][None].long()
        a, beta = torch.where(live[..., None], a, 1.0), torch.where(live[..., None], beta, 0.0)
        q, do_mask = torch.where(live[..., None, None], q, 0.0), live[..., None, None]
        k, v = torch.where(do_mask, k, 0.0), torch.where(do_mask, v, 0.0)
    row = lambda m, x: torch.einsum("bhkv,bhk->bhv", m, x)  # noqa: E731

    def ahead(m, i):
        m = m * a[i][..., None, None]
        e = v[i] - row(m, k[i])
        return m, e, m + k[i][..., None] * (beta[i][..., None] * e)[..., None, :]

    m = s["state"].double()
    o, marks = torch.empty_like(v), []
    for i in range(t):
        if i % CHUNK == 0:
            marks.append(m)
        m = ahead(m, i)[2]
        o[i] = scale * row(m, q[i])
    back = lambda x: x.transpose(0, 1)  # noqa: E731
    out = {"o": back(o), "final": m}
    if c["way"] != "train":
        return out
    do = s["do"].double().transpose(0, 1)
    if s["lengths"] is not None:
        do = torch.where(do_mask, do, 0.0)
    col = lambda g, x: torch.einsum("bhkv,bhv->bhk", g, x)  # noqa: E731
    dq, dk, dv, dbeta, dgate = (torch.empty_like(x) for x in (q, k, v, beta, a))
    g = s["dfinal"].double()
    for first in reversed(range(0, t, CHUNK)):
        m, steps = marks[first // CHUNK], []
        for i in range(first, min(first + CHUNK, t)):
            steps.append(ahead(m, i))
            m = steps[-1][2]
        for i in reversed(range(first, min(first + CHUNK, t))):
            decayed, e, new = steps[i - first]
            dq[i] = scale * col(new, do[i])
            g = g + scale * q[i][..., None] * do[i][..., None, :]
            du = row(g, k[i])
            de = beta[i][..., None] * du
            dv[i], dbeta[i] = de, (du * e).sum(-1)
            dk[i] = col(g, beta[i][..., None] * e) - col(decayed, de)
            g = g - k[i][..., None] * de[..., None, :]
            dgate[i] = (g * decayed).sum((-1, -2))
            g = g * a[i][..., None, None]
    if s["lengths"] is not None:
        dbeta, dgate = torch.where(live[..., None], dbeta, 0.0), torch.where(live[..., None], dgate, 0.0)
    out["dq"], out["dk"] = (back(x.unflatten(2, (hk, group)).sum(3)) for x in (dq, dk))
    out.update(dv=back(dv), dbeta=back(dbeta), dstate=g)
    if s["gate"] is not None:
        out["dgate"] = back(dgate)
    return out


def _exact_step(s):
    c = s["case"]
    group, at, pool = c["h"] // c["hk"], s["slots"].long(), s["pool"].double()
    q, k = (s[x].double().repeat_interleave(group, 1) for x in ("q", "k"))
    m = pool[at] * torch.exp(s["gate"].double())[..., None, None]
    u = s["beta"].double()[..., None] * (s["v"].double() - torch.einsum("nhkv,nhk->nhv", m, k))
    m = m + torch.einsum("nhk,nhv->nhkv", k, u)
    pool[at] = m
    return {"o": torch.einsum("nhkv,nhk->nhv", m, q) / math.sqrt(c["k"]), "pool": pool}


def _exact_rms(s):
    c, w = s["case"], s["weight"].double()
    x = s["x"].double()
    out = {}
    if s["residual"] is not None:  # the norm is that of the sum as it is written
        x = (x + s["residual"].double()).to(s["residual"].dtype).double()
        out["sum"] = s["x"].double() + s["residual"].double()
    n = x.shape[1]
    size = (torch.einsum("rc,rc->r", x, x) / n + RMS_EPS).sqrt()[:, None]
    y = x / size * w
    if c["quantize"]:
        out["scale"] = y.abs().amax(1) / E4M3_MAX
        out["y"] = y / out["scale"][:, None]
        return out
    out["y"] = y
    if c["way"] == "train":
        dy, hat = s["dy"].double(), x / size
        d = dy * w
        ds = (d - hat * (torch.einsum("rc,rc->r", d, hat) / n)[:, None]) / size + s["dsum"].double()
        out["ds"], out["dweight"] = ds, torch.einsum("rc,rc->c", dy, hat)
        if s["residual"] is not None and s["residual"].dtype != s["x"].dtype:
            out["dx"] = ds
    return out


def _exact_sample(s):
    """Row by row, from the largest logit down."""
    tokens, probs = [], []
    for i in range(s["logits"].shape[0]):
        x = s["logits"][i].double() / s["temperature"][i].double()
        m = torch.exp(x - x.max())
        order = torch.argsort(s["logits"][i].float(), descending=True, stable=True)
        if s["top_k"] is not None:
            order = order[: max(1, int(s["top_k"][i]))]
        if s["top_p"] is not None:
            c = m[order].cumsum(0)
            order = order[: 1 + int((c < s["top_p"][i].double() * c[-1]).sum())]
        if s["min_p"] is not None:
            order = order[m[order] >= s["min_p"][i].double()]
        kept = torch.sort(order)[0]
        c = m[kept].cumsum(0)
        at = min(int((c <= s["u"][i].double() * c[-1]).sum()), kept.numel() - 1)
        tokens.append(int(kept[at]))
        probs.append(float(m[kept[at]] / c[-1]))
    return {"token": torch.tensor(tokens, dtype=torch.int32), "prob": torch.tensor(probs, dtype=torch.float64)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "delta_step": _exact_step, "rms": _exact_rms, "sample": _exact_sample}[case["op"]](s)
