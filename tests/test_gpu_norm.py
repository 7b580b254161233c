"""The group norm with an activation on the GPU against its 64-bit form (tests/ops_reference.py)."""
import pytest
import torch

import ops_reference as ref
from linear_attention_gb300.based import BasedError
from linear_attention_gb300.ops import based_norm_bwd, based_norm_fwd, norm_bwd_workspace_size

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
PAIRS = [(F32, F32), (BF16, BF16), (F16, F16), (F32, BF16), (F32, F16)]


def draw(R, C, xt, yt, pt, gated, seed):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = (rand(R, C) * 0.8 + 0.3).to(xt).cuda()
    gate = (rand(R, C) * 2).to(yt).cuda() if gated else None
    w, b = (1 + 0.3 * rand(C)).to(pt).cuda(), (0.3 * rand(C)).to(pt).cuda()
    return x, gate, w, b, rand(R, C).to(yt).cuda()


def check(x, gate, w, b, dy, groups, act, eps=1e-5, what=""):
    y = based_norm_fwd(x, groups, w, b, gate, act, eps, out_dtype=None if gate is not None else dy.dtype)
    dx, dgate, dw, db = based_norm_bwd(dy, x, groups, w, b, gate, act, eps)
    torch.cuda.synchronize()
    val, bound = ref.norm(x, groups, w, b, gate, act, eps, dy, out_dtype=dy.dtype)
    for name, got in dict(y=y, dx=dx, dgate=dgate, dweight=dw, dbias=db).items():
        assert (got is None) == (name not in val), name
        if got is not None:
            ref.assert_within(got, val[name], bound[name], (what, name))


@pytest.mark.parametrize("xt,yt", PAIRS, ids=[f"{str(a)[6:]}-{str(b)[6:]}" for a, b in PAIRS])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
def test_types_and_activations(xt, yt, act, gated, cuda_device):
    check(*draw(37, 256, xt, yt, F32, gated, 1), 4, act)
    check(*draw(9, 100, xt, yt, yt, gated, 2), 4, act)


GROUPS = [(1, 1), (3, 3), (8, 1), (16, 4), (24, 3), (20, 4), (33, 1), (64, 1), (96, 1), (1536, 12), (2048, 32), (255, 1),
          (256, 1), (257, 1), (520, 2), (512, 1), (1000, 8), (1024, 1), (1032, 1), (2048, 1), (3 * 1000, 3), (4096, 1), (4095, 1),
          (8192, 2), (8192, 64), (768, 256)]


@pytest.mark.parametrize("C,G", GROUPS)
def test_group_sizes(C, G, cuda_device):
    # a group of one channel is zero before weight and bias: its variance is 0 and eps keeps it finite
    for R in (1, 5):
        check(*draw(R, C, BF16, BF16, F32, True, C + R), G, "silu", what=R)
    check(*draw(3, C, F32, F32, F32, False, C), G, "silu", what="float32")


@pytest.mark.parametrize("R", [1, 2, 3, 31, 64, 1000, 5003])
def test_rows(R, cuda_device):
    check(*draw(R, 192, BF16, BF16, F32, True, R), 3, "silu")
    check(*draw(R, 50, F32, BF16, BF16, True, R), 2, "sigmoid")


def test_strides_alignment_and_leading_axes(cuda_device):
    for C in (64, 66):
        x, gate, w, b, dy = draw(24, 2 * C, BF16, BF16, F32, True, C)
        check(x[:, :C], gate[:, C:], w[:C], b[C:], dy[:, :C], 2, "silu", what="halves")
        check(x[:, 1:C + 1], gate[:, 3:C + 3], w[1:C + 1], b[3:C + 3], dy[:, 1:C + 1], 2, "silu", what="odd starts")
        check(x[:1, :C].expand(24, C), gate[:, :C], w[:C], b[:C], dy[:1, :C].expand(24, C), 2, "silu", what="broadcast")
        x3, g3, d3 = (t[:, :C].unflatten(0, (2, 3, 4)) for t in (x, gate, dy))
        y = based_norm_fwd(x3, 2, w[:C], b[:C], g3)
        assert y.shape == (2, 3, 4, C) and torch.equal(y.reshape(24, C), based_norm_fwd(x[:, :C], 2, w[:C], b[:C], gate[:, :C]))
        got = based_norm_bwd(d3, x3, 2, w[:C], b[:C], g3)
        want = based_norm_bwd(dy[:, :C], x[:, :C], 2, w[:C], b[:C], gate[:, :C])
        assert all(torch.equal(p.reshape(q.shape), q) for p, q in zip(got, want))
    with pytest.raises(ValueError):
        based_norm_fwd(torch.zeros(4, 6, 64, device="cuda").transpose(0, 1), 2)


def test_parts_left_out(cuda_device):
    x, gate, w, b, dy = draw(40, 128, BF16, BF16, F32, True, 3)
    check(x, gate, None, None, dy, 2, "silu", what="no weight, no bias")
    check(x, gate, w, None, dy, 2, "silu", what="no bias")
    check(x, None, None, b, dy, 2, "silu", what="no weight")


def test_in_place(cuda_device):
    x, gate, w, b, _ = draw(40, 128, BF16, BF16, F32, True, 4)
    want = based_norm_fwd(x, 2, w, b, gate)
    assert torch.equal(based_norm_fwd(x, 2, w, b, gate, out=gate), want)
    x, gate, w, b, _ = draw(40, 128, BF16, BF16, F32, True, 4)
    assert torch.equal(based_norm_fwd(x, 2, w, b, gate, out=x), want)


def test_large_mean_and_constant_rows(cuda_device):
    # a mean 1000 times the deviation, in float32: the bound follows it; a constant group gives the bias
    x, gate, w, b, dy = draw(20, 128, F32, F32, F32, True, 5)
    check(x * 0.1 + 100, gate, w, b, dy, 2, "silu")
    y = based_norm_fwd(torch.full((3, 128), 2.5, device="cuda"), 2, w, b, act="none")
    assert torch.equal(y, b.expand(3, 128))
    z = torch.zeros(3, 128, device="cuda")
    assert torch.equal(based_norm_fwd(z, 2, w, b, act="none"), b.expand(3, 128))


def test_extreme_gates_and_nan(cuda_device):
    inf = float("inf")
    x, gate, w, b, dy = draw(4, 128, BF16, BF16, F32, True, 6)
    gate[1, :64], gate[1, 64:] = -300.0, 300.0
    check(x, gate, w, b, dy, 2, "silu")
    check(x, gate, w, b, dy, 2, "sigmoid")
    want = based_norm_fwd(x, 2, w, b, gate)
    x2 = x.clone()
    x2[0, 3], x2[2, 100] = float("nan"), inf
    got = based_norm_fwd(x2, 2, w, b, gate)
    bad = torch.zeros(4, 128, dtype=torch.bool, device="cuda")
    bad[0, :64], bad[2, 64:] = True, True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("xt,yt", PAIRS, ids=[f"{str(a)[6:]}-{str(b)[6:]}" for a, b in PAIRS])
def test_groups_that_end_inside_a_word(xt, yt, cuda_device):
    # groups of odd size: what a neighbour's channels hold is in the same word and stays out
    inf = float("inf")
    for C, G in ((6, 2), (20, 4), (50, 2), (250, 2), (1000, 8), (1026, 2)):
        n = C // G
        x, gate, w, b, dy = draw(37, C, xt, yt, F32, True, C)
        check(x, gate, w, b, dy, G, "silu", what=(C, G))
        check(x[1:], gate[1:], w, b, dy[1:], G, "none", what=(C, G))
        check(x, None, w, b, dy, G, "sigmoid", what=(C, G))
        want = based_norm_fwd(x, G, w, b, gate), *based_norm_bwd(dy, x, G, w, b, gate)
        bad = torch.zeros(C, dtype=torch.bool, device="cuda")
        bad[n:2 * n] = True
        for k, t in enumerate((x, gate, dy)):
            t = t.clone()
            t[3, n], t[3, 2 * n - 1], t[36, n:2 * n] = inf, float("nan"), float("nan")
            args = [t if k == j else o for j, o in enumerate((x, gate, dy))]
            got = based_norm_fwd(args[0], G, w, b, args[1]), *based_norm_bwd(args[2], args[0], G, w, b, args[1])
            for p, q in zip(got, want):
                assert torch.equal(p[..., ~bad], q[..., ~bad]), (C, G, k)
        if xt == yt:
            y = want[0]
            assert torch.equal(based_norm_fwd(x, G, w, b, gate, out=gate.clone()), y)
            for into in (x.clone(), gate.clone()):
                first = into.data_ptr()
                same = based_norm_fwd(into if torch.equal(into, x) else x, G, w, b, into if torch.equal(into, gate) else gate, out=into)
                assert same.data_ptr() == first and torch.equal(same, y), (C, G)


def test_determinism_streams_graphs_and_workspace(cuda_device):
    x, gate, w, b, dy = draw(3000, 512, BF16, BF16, BF16, True, 7)
    want = (based_norm_fwd(x, 8, w, b, gate), *based_norm_bwd(dy, x, 8, w, b, gate))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (based_norm_fwd(x, 8, w, b, gate, stream=side), *based_norm_bwd(dy, x, 8, w, b, gate, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    n = norm_bwd_workspace_size(3000, 512, 8)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns: contents are ignored
    assert all(torch.equal(p, q) for p, q in zip(want[1:], based_norm_bwd(dy, x, 8, w, b, gate, workspace=ws[:n])))
    assert (ws[n:] == 255).all()
    with pytest.raises(BasedError):
        based_norm_bwd(dy, x, 8, w, b, gate, workspace=ws[:n - 4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = (based_norm_fwd(x, 8, w, b, gate), *based_norm_bwd(dy, x, 8, w, b, gate))
    x.copy_(x.flip(0))
    want = (based_norm_fwd(x, 8, w, b, gate), *based_norm_bwd(dy, x, 8, w, b, gate))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, cap))


def test_gradient_against_differences(cuda_device):
    # central differences of the kernel's forward pass in float32; a step of 2^-6 leaves about
    # (2^-6)^2 of curvature and 2^-19 / 2^-6 of rounding
    for gated in (True, False):
        x, gate, w, b, dy = draw(3, 24, F32, F32, F32, gated, 8)
        grads = dict(zip("xgwb", based_norm_bwd(dy, x, 2, w, b, gate)))
        args = dict(x=x, g=gate, w=w, b=b)

        def loss(**kw):
            a = {**args, **kw}
            return float((based_norm_fwd(a["x"], 2, a["w"], a["b"], a["g"]).double() * dy.double()).sum())

        for name, t in args.items():
            for i in range(0, 0 if t is None else t.numel(), 5):
                vals = []
                for sign in (1, -1):
                    moved = t.clone()
                    moved.view(-1)[i] += sign * 2.0 ** -6
                    vals.append(loss(**{name: moved}))
                diff, got = (vals[0] - vals[1]) / 2.0 ** -5, float(grads[name].reshape(-1)[i])
                assert abs(diff - got) <= 5e-3 * max(1.0, float(grads[name].abs().max())), (gated, name, i, diff, got)


def test_nothing_is_written_past_the_outputs(cuda_device):
    for C, G in ((96, 2), (50, 2), (257, 1)):
        x, gate, w, b, _ = draw(13, C, BF16, BF16, F32, True, 9)
        buf = torch.full((13 * C + 512,), 7.0, dtype=BF16, device="cuda")
        based_norm_fwd(x, G, w, b, gate, out=buf[:13 * C].view(13, C))
        assert (buf[13 * C:] == 7).all()


def test_offsets_past_32_bits(cuda_device):
    C, R = 1024, (1 << 21) + 3  # more than 2^31 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(8, C, generator=g, device="cuda").to(BF16)
    big = x.repeat((R + 7) // 8, 1)[:R]
    y = based_norm_fwd(big, 8, act="silu")
    want = based_norm_fwd(x, 8, act="silu")
    assert torch.equal(y[-3:], want[[(R - 3) % 8, (R - 2) % 8, (R - 1) % 8]]) and torch.equal(y[:8], want)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gates_of_the_lowest_value(dtype, act, cuda_device):
    # what masks a gate: its activation and its slope are 0 for every type, and nothing else of the row changes
    for C in (128, 50):
        x, gate, w, b, dy = draw(6, C, dtype, dtype, F32, True, C)
        low = torch.rand(6, C, generator=torch.Generator().manual_seed(C)).cuda() < 0.3
        for value in (torch.finfo(dtype).min, -1e4):
            gate[low] = value
            y = based_norm_fwd(x, 2, w, b, gate, act)
            dx, dgate, dw, db = based_norm_bwd(dy, x, 2, w, b, gate, act)
            assert y[low].abs().max() <= 1e-30 and dgate[low].abs().max() <= 1e-30
            far = gate.clone()
            far[low] = -120.0
            want = based_norm_fwd(x, 2, w, b, far, act), *based_norm_bwd(dy, x, 2, w, b, far, act)
            for p, q in zip((y, dx, dgate, dw, db), want):
                assert torch.equal(torch.where(p.abs() > 1e-30, p, 0), torch.where(q.abs() > 1e-30, q, 0))
        # without a gate, v itself: a bias of the lowest value
        bias = torch.full((C,), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        assert based_norm_fwd(x, 2, None, bias, act=act).abs().max() <= 1e-30


def test_infinite_gates_in_sums_over_rows(cuda_device):
    # rows that do not come out even over the CTAs: threads without a row in the last turn keep an earlier one's values
    inf = float("inf")
    for R, C, G in ((5003, 192, 3), (3, 192, 3), (2999, 50, 2), (700, 512, 1)):
        x, gate, w, b, dy = draw(R, C, BF16, BF16, F32, True, R)
        gate[:, 7], dy[:, 7], gate[:, 9], dy[:, 9] = inf, 1, -inf, 1
        for act, want in (("silu", (inf, 0)), ("none", (inf, -inf)), ("sigmoid", (R, 0))):
            _, _, dw, db = based_norm_bwd(dy, x, G, w, b, gate, act)
            assert float(db[7]) == want[0] and (abs(float(db[9])) <= 1e-30 if want[1] == 0 else float(db[9]) == want[1])
            rest = torch.tensor([c not in (7, 9) for c in range(C)], device="cuda")
            assert torch.isfinite(dw[rest]).all() and torch.isfinite(db[rest]).all()


def test_workspace_sizes_at_the_limits(cuda_device):
    big = 1 << 20
    for R, C, G in ((4, 2 * big, big), (1 << 40, 64, 4), (4, 8192, 1), (0, 64, 4), (4, 64, 5)):
        assert norm_bwd_workspace_size(R, C, G) == 0, (R, C, G)
    for R, C, G in ((4, big, big), ((1 << 40) - 1, 64, 4), (4, 4096, 1)):
        assert norm_bwd_workspace_size(R, C, G) > 0, (R, C, G)
