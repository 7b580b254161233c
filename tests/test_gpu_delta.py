"""The gated delta rule on the GPU against the 64-bit recurrence, row by row."""
import math

import pytest
import torch

import more_ops_reference as ref
from linear_attention_gb300 import based_delta_bwd, based_delta_fwd, based_delta_step, ops
from linear_attention_gb300.autograd import delta_rule
from linear_attention_gb300.based import BasedError

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def inputs(B, T, H, HK, K, V, dtype, seed=0, gated=True, lengths=None, state=True):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    s = dict(q=unit(rand(B, T, HK, K)), k=unit(rand(B, T, HK, K)), v=rand(B, T, H, V), beta=torch.sigmoid(rand(B, T, H)),
             gate=-0.3 * torch.rand(B, T, H, generator=gen) if gated else None)
    s = {n: None if t is None else t.to(dtype).cuda() for n, t in s.items()}
    more = dict(state=(rand(B, H, K, V) * 0.3).cuda() if state else None,
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda())
    return s, more, rand(B, T, H, V).to(dtype).cuda(), (rand(B, H, K, V) * 0.3).cuda()


def check(s, more, do, dfinal, scale=None, near=True):
    o, final, saved = based_delta_fwd(**s, **more, scale=scale, save=True)
    names = "dq dk dv dbeta dgate dstate".split()
    got = dict(o=o, final=final, **dict(zip(names, based_delta_bwd(s["q"], s["k"], s["v"], s["beta"], s["gate"], do, saved, scale=scale,
                                                                   dfinal=dfinal, lengths=more["lengths"]))))
    args = s["q"], s["k"], s["v"], s["beta"], s["gate"], scale, more["state"], more["lengths"], do, dfinal
    val = ref.delta_rows(*args)
    bound = ref.delta_bounds(val, *args)
    for name in val:
        ref.assert_within(got[name], val[name], bound[name], name)
        if near and name not in ("final", "dstate"):
            ref.assert_near(got[name], val[name], s["v"].dtype, name)
    if s["gate"] is None:
        assert got["dgate"] is None
    return got


CASES = [
    # B, T, H, HK, K, V, dtype, options
    (1, 1, 1, 1, 1, 1, F32, {}),
    (2, 1, 2, 1, 17, 5, F16, {}),
    (1, 63, 2, 2, 64, 16, F32, {}),
    (1, 64, 2, 1, 64, 64, BF16, {}),
    (2, 65, 4, 2, 128, 33, F32, dict(gated=False)),
    (1, 200, 3, 3, 128, 128, BF16, {}),
    (2, 130, 4, 1, 40, 75, F32, {}),
    (3, 129, 2, 2, 65, 20, F16, dict(lengths=[129, 0, 70])),
    (2, 192, 4, 4, 128, 48, BF16, dict(lengths=[64, 191], gated=False)),
    (1, 140, 2, 1, 96, 260, F16, dict(state=False)),
    (2, 70, 6, 2, 16, 32, F32, dict(lengths=[-3, 1000])),
]


@pytest.mark.parametrize("B,T,H,HK,K,V,dtype,opt", CASES)
def test_values_and_gradients(cuda_device, B, T, H, HK, K, V, dtype, opt):
    check(*inputs(B, T, H, HK, K, V, dtype, **opt))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_slices_of_many_heads(cuda_device, dtype):
    """More than 32 slices of a head (the gradients' factors come in groups of 32), and several to a CTA."""
    check(*inputs(2, 66, 2, 2, 24, 600, dtype))
    check(*inputs(40, 66, 8, 4, 64, 64, dtype))


@pytest.mark.parametrize("scale", [0.05, 3.0])
def test_scale(cuda_device, scale):
    check(*inputs(1, 90, 2, 2, 32, 32, F32), scale=scale)


def test_strided_inputs(cuda_device):
    """Views of one projection, transposed heads, and rows on no 16-byte word."""
    gen = torch.Generator().manual_seed(3)
    B, T, H, K = 2, 100, 2, 32
    p = (torch.randn(B, T, 3 * H * K + 5, generator=gen) * K ** -0.5).to(BF16).cuda()
    q, k, v = (p[..., 1 + i * H * K:1 + (i + 1) * H * K].unflatten(-1, (H, K)) for i in range(3))
    beta = torch.rand(B, 2 * T, H, generator=gen).to(BF16).cuda()[:, ::2]
    gate = -torch.rand(T, B, H, generator=gen).to(BF16).cuda().transpose(0, 1)
    do = torch.randn(B, H, T, K, generator=gen).to(BF16).cuda().transpose(1, 2)
    check(dict(q=q, k=k, v=v, beta=beta, gate=gate), dict(state=None, lengths=None), do, None)
    one = torch.randn(1, 1, 1, K, generator=gen).to(BF16).cuda() * 0.1
    check(dict(q=one.expand(B, T, H, K), k=one.expand(B, T, H, K), v=v, beta=beta, gate=gate), dict(state=None, lengths=None), do, None)


def test_heavy_and_cleared_decays(cuda_device):
    """Log decays whose sum is large, a type's lowest value and -inf: rows behind a cleared state do not see what was in front."""
    s, more, do, dfinal = inputs(1, 150, 2, 2, 64, 32, F32, seed=5)
    s["gate"][:, 20] = -300.0
    s["gate"][:, 70] = torch.finfo(F32).min
    s["gate"][:, 100] = -math.inf
    got = check(s, more, do, dfinal)
    other = dict(more, state=more["state"] * 5)
    o, final, _ = based_delta_fwd(**s, **other)
    assert torch.equal(o[:, 100:], got["o"][:, 100:]) and torch.equal(final, got["final"])
    assert (got["dgate"][:, 70] == 0).all() and (got["dgate"][:, 100] == 0).all()


def test_no_steps_and_large_steps(cuda_device):
    """beta of 0 (nothing is written) and up to 2 (reflections), zero keys, magnitudes far from 1."""
    s, more, do, dfinal = inputs(1, 130, 2, 2, 64, 32, F32, seed=6)
    s["beta"][:, ::3] = 0.0
    s["beta"][:, 1::3] = 2.0
    s["k"][:, 5:9] = 0.0
    check(s, more, do, dfinal, near=False)
    for c in (1e-6, 1e6):
        t = dict(s, v=s["v"] * c)
        check(t, dict(more, state=more["state"] * c), do, dfinal, near=False)


def test_equal_keys(cuda_device):
    """The same key in all rows: every row corrects the one before; the inverse's entries alternate."""
    s, more, do, dfinal = inputs(1, 128, 1, 1, 32, 16, F32, seed=7, gated=False)
    s["k"] = s["k"][:, :1].expand(-1, 128, -1, -1).contiguous()
    s["beta"].fill_(1.0)
    check(s, more, do, dfinal, near=False)


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
def test_padding_is_not_read(cuda_device, poison):
    s, more, do, dfinal = inputs(2, 150, 2, 1, 64, 32, BF16, lengths=[90, 0])
    want = check(s, more, do, dfinal)
    for b, n in enumerate((90, 0)):
        for name in s:
            s[name][b, n:] = poison
        do[b, n:] = poison
    o, final, saved = based_delta_fwd(**s, **more, save=True)
    got = based_delta_bwd(s["q"], s["k"], s["v"], s["beta"], s["gate"], do, saved, dfinal=dfinal, lengths=more["lengths"])
    for name, t in dict(o=o, final=final, **dict(zip("dq dk dv dbeta dgate dstate".split(), got))).items():
        assert torch.equal(t, want[name]), name


def test_nan_stays_in_its_sequence_and_head(cuda_device):
    s, more, _, _ = inputs(2, 100, 2, 2, 32, 32, F32)
    o, final, _ = based_delta_fwd(**s, **more)
    s["v"][1, 30, 1] = math.nan
    p, last, _ = based_delta_fwd(**s, **more)
    assert torch.equal(p[0], o[0]) and torch.equal(p[1, :, 0], o[1, :, 0]) and torch.equal(last[0], final[0])
    assert p[1, 31:, 1].isnan().all() and last[1, 1].isnan().all()


def test_chunks_of_a_sequence_one_after_the_other(cuda_device):
    """A prompt in parts, each from the state behind the one before, in place, and then single tokens."""
    s, more, _, _ = inputs(2, 150, 4, 2, 64, 40, F32)
    val = ref.delta_rows(*(s[n] for n in ("q", "k", "v", "beta", "gate")), None, more["state"], None)
    bound = ref.delta_bounds(val, *(s[n] for n in ("q", "k", "v", "beta", "gate")), None, more["state"], None)
    state, o = more["state"].clone(), []
    for a, b in ((0, 64), (64, 65), (65, 140)):
        part = {n: t[:, a:b] for n, t in s.items()}
        y, final, _ = based_delta_fwd(**part, state=state, final_state=state)
        assert final is state or final.data_ptr() == state.data_ptr()
        o.append(y)
    pool = torch.zeros(5, 4, 64, 40, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    for t in range(140, 150):
        o.append(based_delta_step(*(s[n][:, t] for n in ("q", "k", "v", "beta", "gate")), pool, slots=slots)[:, None])
    # three calls and ten rows: as many chunks more
    ref.assert_within(torch.cat(o, 1), val["o"], 5 * bound["o"], "o")
    ref.assert_within(pool[slots.long()], val["final"], 5 * bound["final"], "final")
    assert (pool[[0, 2, 4]] == 0).all()


@pytest.mark.parametrize("N,S,H,HK,K,V,dtype", [(1, 1, 1, 1, 1, 1, F32), (3, 7, 4, 2, 128, 64, BF16), (5, 5, 2, 2, 37, 75, F16),
                                              (2, 9, 3, 1, 128, 33, F32), (3, 7, 4, 2, 32, 226, BF16), (2, 4, 2, 2, 20, 131, F32),
                                              (4, 6, 2, 1, 64, 36, F16), (2, 3, 2, 1, 33, 130, F32), (3, 4, 2, 2, 32, 128, BF16),
                                              (2, 5, 2, 1, 64, 97, F32)])
def test_step(cuda_device, N, S, H, HK, K, V, dtype):
    s, _, _, _ = inputs(N, 1, H, HK, K, V, dtype, seed=N)
    gen = torch.Generator().manual_seed(1)
    pool = torch.randn(S, H, K, V, generator=gen).cuda()
    slots = torch.randperm(S, generator=gen)[:N].to(torch.int32).cuda()
    val = ref.delta_rows(*(s[n] for n in ("q", "k", "v", "beta", "gate")), None, pool[slots.long()], None)
    bound = ref.delta_bounds(val, *(s[n] for n in ("q", "k", "v", "beta", "gate")), None, pool[slots.long()], None)
    rows = {n: t[:, 0] for n, t in s.items()}
    rows["q"] = rows["q"].clone().transpose(0, 1).contiguous().transpose(0, 1)  # other strides
    before = pool.clone()
    o = based_delta_step(**rows, pool=pool, slots=slots)
    ref.assert_within(o[:, None], val["o"], bound["o"], "o")
    ref.assert_within(pool[slots.long()], val["final"], bound["final"], "pool")
    idle = torch.ones(S, dtype=torch.bool)
    idle[slots.cpu().long()] = False
    assert torch.equal(pool[idle], before[idle])
    # idle sequences
    slots[0] = -1 if N % 2 else S
    again = pool.clone()
    o = based_delta_step(**rows, pool=pool, slots=slots)
    assert (o[0] == 0).all()
    if N == 1:
        assert torch.equal(pool, again)


def test_results_repeat_and_do_not_depend_on_the_batch(cuda_device):
    """The same bits again, for a sequence alone (another number of slices to a CTA), and on a side stream."""
    s, more, do, dfinal = inputs(24, 140, 8, 4, 64, 64, BF16)
    o, final, saved = based_delta_fwd(**s, **more, save=True)
    grads = based_delta_bwd(s["q"], s["k"], s["v"], s["beta"], s["gate"], do, saved, dfinal=dfinal)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, final2, saved2 = based_delta_fwd(**s, **more, save=True, stream=side)
    grads2 = based_delta_bwd(s["q"], s["k"], s["v"], s["beta"], s["gate"], do, saved2, dfinal=dfinal, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o2) and torch.equal(final, final2)
    assert all(torch.equal(a, b) for a, b in zip(grads, grads2))
    one = {n: t[7:8].contiguous() for n, t in s.items()}
    o3, final3, saved3 = based_delta_fwd(**one, state=more["state"][7:8], save=True)
    grads3 = based_delta_bwd(one["q"], one["k"], one["v"], one["beta"], one["gate"], do[7:8], saved3, dfinal=dfinal[7:8])
    assert torch.equal(o[7:8], o3) and torch.equal(final[7:8], final3)
    assert all(torch.equal(a[7:8], b) for a, b in zip(grads, grads3))


def test_capture_and_replay(cuda_device):
    """Two captured calls of other sizes with workspaces of their own, replayed in turn on new inputs."""
    sets = [inputs(2, 100, 2, 1, 64, 32, BF16, seed=1), inputs(1, 70, 4, 4, 128, 64, BF16, seed=2)]
    side, graphs, outs = torch.cuda.Stream(), [], []
    for s, more, do, dfinal in sets:
        def call():
            o, final, saved = based_delta_fwd(**s, **more, save=True)
            return o, final, *based_delta_bwd(s["q"], s["k"], s["v"], s["beta"], s["gate"], do, saved, dfinal=dfinal)
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(call())
        graphs.append(g)
    for r in range(2):
        for s, more, do, dfinal in sets:
            s["v"].mul_(0.5), do.mul_(-1.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (s, more, do, dfinal), got in zip(sets, outs):
            o, final, saved = based_delta_fwd(**s, **more, save=True)
            want = (o, final, *based_delta_bwd(s["q"], s["k"], s["v"], s["beta"], s["gate"], do, saved, dfinal=dfinal))
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_passed_outputs_and_workspaces(cuda_device):
    s, more, do, dfinal = inputs(2, 100, 4, 2, 64, 32, BF16)
    want = based_delta_fwd(**s, **more, save=True)
    sizes = (2, 100, 4, 2, 64, 32, BF16)
    ws = torch.full((ops.delta_workspace_size(*sizes),), 255, dtype=torch.uint8, device="cuda")
    out, last = torch.empty_like(want[0]), torch.empty_like(want[1])
    got = based_delta_fwd(**s, **more, save=True, out=out, final_state=last, workspace=ws)
    assert got[0].data_ptr() == out.data_ptr() and torch.equal(out, want[0]) and torch.equal(last, want[1])
    args = s["q"], s["k"], s["v"], s["beta"], s["gate"], do
    ws2 = torch.full((ops.delta_workspace_size(*sizes, backward=True),), 255, dtype=torch.uint8, device="cuda")
    a = based_delta_bwd(*args, want[2], dfinal=dfinal)
    b = based_delta_bwd(*args, got[2], dfinal=dfinal, workspace=ws2)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(BasedError):
        based_delta_fwd(**s, **more, workspace=ws[:-64])
    with pytest.raises(BasedError):
        based_delta_fwd(**s, **more, out=s["v"])


def test_autograd(cuda_device):
    """Gradients of a loss through the differentiable function: the kernel's own, absent and broadcast ones, and differences."""
    s, more, do, dfinal = inputs(2, 80, 4, 2, 32, 24, F32, seed=9)
    leaves = {n: t.clone().requires_grad_() for n, t in s.items()}
    state = more["state"].clone().requires_grad_()
    o, final = delta_rule(**leaves, state=state)
    ((o * do).sum() + (final * dfinal).sum()).backward()
    val = ref.delta_rows(*(s[n] for n in ("q", "k", "v", "beta", "gate")), None, more["state"], None, do, dfinal)
    bound = ref.delta_bounds(val, *(s[n] for n in ("q", "k", "v", "beta", "gate")), None, more["state"], None, do, dfinal)
    for n, t in leaves.items():
        ref.assert_within(t.grad, val["d" + n], bound["d" + n], n)
    ref.assert_within(state.grad, val["dstate"], bound["dstate"], "state")
    # only the last state, and a gradient that is a broadcast number
    for use in (lambda o, f: f.sum(), lambda o, f: o.sum()):
        t = {n: x.clone().requires_grad_() for n, x in s.items()}
        use(*delta_rule(**t)).backward()
        assert all(x.grad is not None and x.grad.isfinite().all() for x in t.values())
    with torch.no_grad():
        p, _ = delta_rule(**s, state=more["state"])
    assert torch.equal(p, o)


def test_empty_batches(cuda_device):
    s, more, do, dfinal = inputs(2, 4, 2, 1, 8, 8, F32)
    for cut in (slice(0, 0), slice(0, 2)):
        part = {n: t[cut] if cut.stop == 0 else t[:, :0] for n, t in s.items()}
        st = more["state"][cut]
        o, final, saved = based_delta_fwd(**part, state=st, save=True)
        assert o.shape == part["v"].shape and torch.equal(final, st)
        grads = based_delta_bwd(part["q"], part["k"], part["v"], part["beta"], part["gate"], torch.empty_like(part["v"]), saved, dfinal=dfinal[cut])
        assert torch.equal(grads[-1], dfinal[cut]) and all(g.numel() == 0 for g in grads[:-1])
    none = {n: t[:0, 0] for n, t in s.items()}
    assert based_delta_step(**none, pool=more["state"]).shape == (0, 2, 8)


def test_more_sequences_than_a_grid_holds(cuda_device):
    """Above 65535 sequences a CTA goes through several, of different lengths: they give what a call of their own gives, bit for bit."""
    B, T, H, K, V = 66000, 65, 1, 8, 70  # five slices: a CTA of four and one of one with three idle
    gen = torch.Generator(device="cuda").manual_seed(9)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF16)  # noqa: E731
    q, k, v, do = rand(B, T, H, K), rand(B, T, H, K) * 0.3, rand(B, T, H, V), rand(B, T, H, V)
    beta, gate = torch.rand(B, T, H, generator=gen, device="cuda").to(BF16), -torch.rand(B, T, H, generator=gen, device="cuda").to(BF16)
    state = torch.randn(B, H, K, V, generator=gen, device="cuda")
    lengths = torch.randint(-1, T + 2, (B,), generator=gen, device="cuda").to(torch.int32)

    def run(at):
        s = [t[at] for t in (q, k, v, beta, gate)]
        o, final, saved = based_delta_fwd(*s, state=state[at], lengths=lengths[at], save=True)
        return o, final, *based_delta_bwd(*s, do[at], saved, dfinal=state[at], lengths=lengths[at])

    whole = run(slice(0, B))
    for at in (slice(0, 600), slice(B - 65535 - 100, B - 65535 + 100), slice(B - 600, B)):
        assert all(torch.equal(a[at], b) for a, b in zip(whole, run(at)))
