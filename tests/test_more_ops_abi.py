"""Refusals of the delta rule, the residual stream's norm and sampling without a GPU, and the 64-bit form of the delta rule's
gradients against differences."""
import ctypes

import pytest
import torch

import more_ops_reference as ref
from linear_attention_gb300 import build as lbuild

NULL, TYPE, SIZE, STRIDE, ALIGN, ALIAS, WS, ARG = -1, -13, -14, -15, -5, -6, -7, -11
MB = 1 << 20
BASE = 1 << 40
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    from linear_attention_gb300 import ops
    return ops._load()


def at(i):
    """The i-th of a row of fake, aligned device addresses 64 MiB apart."""
    return BASE + i * 64 * MB


def f(x):
    return ctypes.c_float(x)


def delta_fwd(lib, **kw):
    # B 2, T 100, H 4, HK 2, K 64, V 32
    a = dict(q=at(0), qb=12800, qt=128, qh=64, k=at(1), kb=12800, kt=128, kh=64, v=at(2), vb=12800, vt=128, vh=32, beta=at(3), bb=400, bt=4,
             gate=at(4), gb=400, gt=4, B=2, T=100, H=4, HK=2, K=64, V=32, dtype=1, scale=f(0.0), state=at(5), lengths=at(6), o=at(7),
             final=at(8), saved=at(9), ws=at(10), n=32 * MB)
    a.update(kw)
    return lib.based_delta_fwd(*a.values(), None)


def delta_bwd(lib, **kw):
    a = dict(q=at(0), qb=12800, qt=128, qh=64, k=at(1), kb=12800, kt=128, kh=64, v=at(2), vb=12800, vt=128, vh=32, beta=at(3), bb=400, bt=4,
             gate=at(4), gb=400, gt=4, do=at(5), db=12800, dt=128, dh=32, saved=at(6), B=2, T=100, H=4, HK=2, K=64, V=32, dtype=1, scale=f(0.0),
             dfinal=at(7), lengths=at(8), dq=at(9), dk=at(10), dv=at(11), dbeta=at(12), dgate=at(13), dstate=at(14), ws=at(15), n=32 * MB)
    a.update(kw)
    return lib.based_delta_bwd(*a.values(), None)


def delta_step(lib, **kw):
    a = dict(q=at(0), qn=128, qh=64, k=at(1), kn=128, kh=64, v=at(2), vn=128, vh=32, beta=at(3), bn=4, gate=at(4), gn=4, N=3, H=4, HK=2, K=64,
             V=32, S=5, dtype=1, scale=f(0.0), pool=at(5), slots=at(6), o=at(7))
    a.update(kw)
    return lib.based_delta_step(*a.values(), None)


def rms_fwd(lib, **kw):
    a = dict(x=at(0), xs=64, res=at(1), rs=64, st=0, w=at(2), pt=1, R=7, C=64, eps=f(1e-6), sum=at(3), y=at(4), dt=1, scales=None)
    a.update(kw)
    return lib.based_rms_fwd(*a.values(), None)


def rms_bwd(lib, **kw):
    a = dict(dy=at(0), ds_=64, s=at(1), ss=64, st=0, w=at(2), pt=1, dsum=at(3), dss=64, R=7, C=64, eps=f(1e-6), ds=at(4), dx=at(5), dw=at(6),
             dt=1, ws=at(7), n=MB)
    a.update(kw)
    return lib.based_rms_bwd(*a.values(), None)


def sample(lib, **kw):
    a = dict(x=at(0), xs=1000, dt=0, N=4, V=1000, u=at(1), t=at(2), ta=f(1.0), k=at(3), ka=0, p=at(4), pa=f(1.0), m=at(5), ma=f(0.0), out=at(6),
             probs=at(7))
    a.update(kw)
    return lib.based_sample(*a.values(), None)


REFUSALS = [
    *[(delta_fwd, {n: None}, NULL) for n in ("q", "k", "v", "beta", "o")], (delta_fwd, dict(ws=None), WS), (delta_fwd, dict(n=64), WS),
    (delta_fwd, dict(ws=at(10) + 8), WS), (delta_fwd, dict(dtype=3), TYPE), (delta_fwd, dict(scale=f(NAN)), ARG),
    *[(delta_fwd, {n: 0}, SIZE) for n in ("B", "T", "H", "HK", "K", "V")], (delta_fwd, dict(K=129), SIZE), (delta_fwd, dict(HK=3), SIZE),
    (delta_fwd, dict(V=(1 << 16) + 1), SIZE), (delta_fwd, dict(H=1 << 17, HK=1), SIZE), (delta_fwd, dict(B=1 << 20, T=1 << 20), SIZE),
    (delta_fwd, dict(B=1 << 15, T=1 << 15, H=1 << 10, HK=1), SIZE),
    *[(delta_fwd, {n: -1}, STRIDE) for n in ("qb", "qt", "qh", "kb", "vt", "vh", "bb", "bt", "gb", "gt")],
    *[(delta_fwd, {n: at(i) + 1}, ALIGN) for i, n in ((0, "q"), (2, "v"), (4, "gate"), (5, "state"), (6, "lengths"), (8, "final"))],
    (delta_fwd, dict(saved=at(9) + 8), ALIGN),
    (delta_fwd, dict(o=at(2)), ALIAS), (delta_fwd, dict(o=at(0) + 2 * 12800 * 2 - 2), ALIAS), (delta_fwd, dict(final=at(5) + 4), ALIAS),
    (delta_fwd, dict(saved=at(7)), ALIAS), (delta_fwd, dict(ws=at(3)), ALIAS), (delta_fwd, dict(ws=at(9)), ALIAS), (delta_fwd, dict(o=at(6)), ALIAS),
    *[(delta_bwd, {n: None}, NULL) for n in ("do", "saved", "dq", "dk", "dv", "dbeta", "dgate", "gate")], (delta_bwd, dict(n=64), WS),
    (delta_bwd, dict(dk=at(9)), ALIAS), (delta_bwd, dict(dv=at(5)), ALIAS), (delta_bwd, dict(dstate=at(6)), ALIAS),
    (delta_bwd, dict(dgate=at(12)), ALIAS), (delta_bwd, dict(dh=-1), STRIDE), (delta_bwd, dict(dq=at(9) + 2), ALIGN),
    *[(delta_step, {n: None}, NULL) for n in ("q", "k", "v", "beta", "pool", "o")], (delta_step, dict(slots=None, N=6), SIZE),
    (delta_step, dict(S=0), SIZE), (delta_step, dict(S=1 << 20, H=65532, K=128, V=1 << 16), SIZE), (delta_step, dict(K=130), SIZE), (delta_step, dict(HK=3), SIZE), (delta_step, dict(vn=-1), STRIDE),
    (delta_step, dict(pool=at(5) + 2), ALIGN), (delta_step, dict(o=at(5)), ALIAS), (delta_step, dict(pool=at(1)), ALIAS),
    (delta_step, dict(dtype=-1), TYPE), (delta_step, dict(scale=f(NAN)), ARG),
    *[(rms_fwd, {n: None}, NULL) for n in ("x", "y", "res", "sum")], (rms_fwd, dict(st=2), TYPE), (rms_fwd, dict(dt=3), TYPE),
    (rms_fwd, dict(pt=2), TYPE), (rms_fwd, dict(eps=f(-1.0)), ARG), (rms_fwd, dict(eps=f(NAN)), ARG), (rms_fwd, dict(R=0), SIZE),
    (rms_fwd, dict(C=0), SIZE), (rms_fwd, dict(C=16385), SIZE), (rms_fwd, dict(R=1 << 42), SIZE), (rms_fwd, dict(xs=-1), STRIDE),
    (rms_fwd, dict(res=at(1) + 2), ALIGN), (rms_fwd, dict(sum=at(0)), ALIAS), (rms_fwd, dict(y=at(3)), ALIAS), (rms_fwd, dict(sum=at(1) + 256), ALIAS),
    (rms_fwd, dict(sum=at(1), rs=128), ALIAS), (rms_fwd, dict(scales=at(4)), ALIAS), (rms_fwd, dict(scales=at(5) + 2), ALIGN),
    *[(rms_bwd, {n: None}, NULL) for n in ("dy", "s", "ds", "dx", "w")], (rms_bwd, dict(st=1), NULL), (rms_bwd, dict(ws=None), WS),
    (rms_bwd, dict(n=64), WS), (rms_bwd, dict(dx=at(4)), ALIAS), (rms_bwd, dict(ds=at(1)), ALIAS), (rms_bwd, dict(dw=at(2)), ALIAS),
    (rms_bwd, dict(ds=at(3), dss=65), ALIAS), (rms_bwd, dict(dss=-1), STRIDE), (rms_bwd, dict(C=1 << 15), SIZE), (rms_bwd, dict(ws=at(0)), ALIAS),
    *[(sample, {n: None}, NULL) for n in ("x", "u", "out")], (sample, dict(dt=4), TYPE), (sample, dict(N=0), SIZE), (sample, dict(V=0), SIZE),
    (sample, dict(V=(1 << 22) + 1), SIZE), (sample, dict(N=(1 << 26) + 1), SIZE), (sample, dict(xs=-1), STRIDE), (sample, dict(x=at(0) + 2), ALIGN),
    (sample, dict(u=at(1) + 2), ALIGN), (sample, dict(out=at(1)), ALIAS), (sample, dict(probs=at(6)), ALIAS), (sample, dict(probs=at(0) + 12000), ALIAS),
]


@pytest.mark.parametrize("call,change,code", REFUSALS,
                         ids=[f"{c.__name__}-{'-'.join(d)}-{i}" for i, (c, d, _) in enumerate(REFUSALS)])
def test_refused_before_any_cuda_call(lib, call, change, code):
    assert call(lib, **change) == code


def test_sizes_are_zero_where_calls_are_refused(lib):
    for B, T, H, HK, K, V in ((0, 1, 1, 1, 1, 1), (1, 0, 1, 1, 1, 1), (1, 1, 3, 2, 1, 1), (1, 1, 1, 1, 129, 1), (1 << 20, 1 << 20, 1, 1, 1, 1)):
        assert delta_fwd(lib, B=B, T=T, H=H, HK=HK, K=K, V=V) == SIZE
        assert lib.based_delta_workspace_size(B, T, H, HK, K, V, 1, 0) == lib.based_delta_workspace_size(B, T, H, HK, K, V, 1, 1) == 0
    assert lib.based_delta_workspace_size(1, 1, 1, 1, 1, 1, 5, 0) == lib.based_delta_saved_size(1, 1, 1, 1, 1, 5) == 0
    assert 0 < lib.based_delta_workspace_size(2, 100, 4, 2, 64, 32, 1, 0) < lib.based_delta_workspace_size(2, 100, 4, 2, 64, 32, 1, 1)
    # a chunk's state and rows in 16 bits
    assert lib.based_delta_saved_size(1, 64, 1, 64, 16, 1) >= 2 * (64 * 16 + 64 * 16)
    assert lib.based_rms_bwd_workspace_size(0, 4) == lib.based_rms_bwd_workspace_size(4, 1 << 15) == 0
    assert lib.based_rms_bwd_workspace_size(3, 8) == 3 * 8 * 4


def test_binding_refuses_host_tensors_types_and_shapes():
    from linear_attention_gb300 import ops
    q, v, b = torch.zeros(2, 5, 2, 8), torch.zeros(2, 5, 2, 8), torch.zeros(2, 5, 2)
    for call in (lambda: ops.based_delta_fwd(q, q, v, b), lambda: ops.based_delta_fwd(q[0], q[0], v[0], b[0]),
                 lambda: ops.based_delta_bwd(q, q, v, b, None, v, None), lambda: ops.based_delta_step(q[0], q[0], v[0], b[0], None, q),
                 lambda: ops.based_delta_step(q[0], q[0], v[0], b[0], None, q[0]), lambda: ops.based_rms_fwd(v), lambda: ops.based_rms_bwd(v, v),
                 lambda: ops.based_sample(b[0], b[0, :, 0]), lambda: ops.based_sample(b, b)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ops.based_delta_fwd(q, q, v.double(), b), lambda: ops.based_rms_fwd(v.int()), lambda: ops.based_sample(b[0].double(), b[0, :, 0]),
                 lambda: ops.based_rms_fwd(3), lambda: ops.based_delta_fwd(q, q, v, None)):
        with pytest.raises(TypeError):
            call()


def test_reference_gradients_against_differences():
    """The 64-bit gradients themselves, along a direction: central differences, off by h^2."""
    gen = torch.Generator().manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    B, T, H, HK, K, V = 2, 9, 4, 2, 5, 3
    x = [rand(B, T, HK, K) * 0.4, rand(B, T, HK, K) * 0.4, rand(B, T, H, V), torch.rand(B, T, H, generator=gen).double(),
         -torch.rand(B, T, H, generator=gen).double()]
    state, do, dfinal = rand(B, H, K, V), rand(B, T, H, V), rand(B, H, K, V)
    lengths = torch.tensor([9, 4])
    val = ref.delta_rows(*x, 0.7, state, lengths, do, dfinal)
    way, way_s = [rand(*t.shape) for t in x], rand(*state.shape)

    def loss(h):
        out = ref.delta_rows(*(t + h * d for t, d in zip(x, way)), 0.7, state + h * way_s, lengths)
        return (out["o"] * do).sum() + (out["final"] * dfinal).sum()

    h = 1e-5
    want = sum((val["d" + n] * d).sum() for n, d in zip("q k v beta gate".split(), way)) + (val["dstate"] * way_s).sum()
    assert abs((loss(h) - loss(-h)) / (2 * h) - want) < 1e-6 * abs(want) + 1e-7
