"""Refusals of the operators in include/based_ops.h, without a GPU: the C functions check their
arguments before any CUDA call, and the binding checks tensors before the C functions."""
import ctypes
import os
import re

import pytest
import torch

from linear_attention_gb300 import build as lbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, TYPE, SIZE, STRIDE, ALIGN, ALIAS, WS, ARG = -1, -13, -14, -15, -5, -6, -7, -11
MB = 1 << 20
BASE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    from linear_attention_gb300 import ops
    return ops._load()


def at(i):
    """The i-th of a row of fake, aligned device addresses 64 MiB apart."""
    return BASE + i * 64 * MB


def test_every_declared_operator_is_exported(lib):
    src = open(os.path.join(ROOT, "include", "based_ops.h")).read()
    names = set(re.findall(r"BASED_API\s+[\w\s\*]+?\b(based_\w+)\s*\(", src))
    assert {"based_scan_fwd", "based_scan_bwd", "based_scan_step", "based_norm_fwd", "based_norm_bwd",
            "based_embed_fwd", "based_embed_bwd"} <= names
    for n in names:
        assert hasattr(lib, n), n
    for code in (TYPE, SIZE, STRIDE):
        assert lib.based_fwd_strerror(code).decode() != "unknown error code"


def scan_fwd(lib, **kw):
    a = dict(gate=at(0), gsb=640, gst=64, x=at(1), xsb=640, xst=64, B=2, T=10, D=64, dtype=1, mode=1, state=at(2),
             lengths=at(3), y=at(4), final=at(5), saved=at(6))
    a.update(kw)
    return lib.based_scan_fwd(*a.values(), None)


def scan_bwd(lib, **kw):
    a = dict(gate=at(0), gsb=640, gst=64, x=at(1), xsb=640, xst=64, dy=at(2), dsb=640, dst=64, saved=at(3), B=2, T=10,
             D=64, dtype=1, mode=1, dfinal=at(4), lengths=at(5), dgate=at(6), dx=at(7), dstate=at(8))
    a.update(kw)
    return lib.based_scan_bwd(*a.values(), None)


def step(lib, **kw):
    a = dict(gate=at(0), gs=64, x=at(1), xs=64, N=3, D=64, S=5, dtype=1, mode=1, pool=at(2), slots=at(3), y=at(4))
    a.update(kw)
    return lib.based_scan_step(*a.values(), None)


def norm_fwd(lib, **kw):
    a = dict(x=at(0), xs=64, xt=1, gate=at(1), gs=64, w=at(2), b=at(3), pt=0, R=7, C=64, G=4, eps=ctypes.c_float(1e-5),
             act=1, y=at(4), dt=1)
    a.update(kw)
    return lib.based_norm_fwd(*a.values(), None)


def norm_bwd(lib, **kw):
    a = dict(dy=at(0), ds=64, x=at(1), xs=64, xt=1, gate=at(2), gs=64, w=at(3), b=at(4), pt=0, R=7, C=64, G=4,
             eps=ctypes.c_float(1e-5), act=1, dx=at(5), dgate=at(6), dw=at(7), db=at(8), dt=1, ws=at(9), n=MB)
    a.update(kw)
    return lib.based_norm_bwd(*a.values(), None)


def embed_fwd(lib, **kw):
    a = dict(ids=at(0), w=0, table=at(1), ts=64, N=9, V=100, D=64, dt=1, scale=ctypes.c_float(2.0), y=at(2))
    a.update(kw)
    return lib.based_embed_fwd(*a.values(), None)


def embed_bwd(lib, **kw):
    a = dict(ids=at(0), w=0, dy=at(1), ds=64, N=9, V=100, D=64, dt=1, scale=ctypes.c_float(2.0), out=at(2), gt=0,
             ws=at(3), n=MB)
    a.update(kw)
    return lib.based_embed_bwd(*a.values(), None)


REFUSALS = [
    (scan_fwd, dict(gate=None), NULL), (scan_fwd, dict(x=None), NULL), (scan_fwd, dict(y=None), NULL),
    (scan_fwd, dict(dtype=3), TYPE), (scan_fwd, dict(dtype=-1), TYPE), (scan_fwd, dict(mode=2), ARG),
    (scan_fwd, dict(B=0), SIZE), (scan_fwd, dict(T=0), SIZE), (scan_fwd, dict(D=-1), SIZE),
    (scan_fwd, dict(B=1 << 16, D=1 << 15), SIZE), (scan_fwd, dict(T=(1 << 30) + 1), SIZE),
    (scan_fwd, dict(B=1, D=(1 << 20) + 1), SIZE), (scan_fwd, dict(gst=-64), STRIDE), (scan_fwd, dict(xsb=-1), STRIDE),
    (scan_fwd, dict(x=at(1) + 1), ALIGN), (scan_fwd, dict(state=at(2) + 2), ALIGN), (scan_fwd, dict(lengths=at(3) + 2), ALIGN),
    (scan_fwd, dict(y=at(0)), ALIAS), (scan_fwd, dict(y=at(1) + 2 * 1279), ALIAS), (scan_fwd, dict(final=at(4)), ALIAS),
    (scan_fwd, dict(saved=at(5) + 256), ALIAS), (scan_fwd, dict(final=at(2) + 4), ALIAS), (scan_fwd, dict(y=at(3)), ALIAS),
    (scan_bwd, dict(dy=None), NULL), (scan_bwd, dict(saved=None), NULL), (scan_bwd, dict(dx=None), NULL),
    (scan_bwd, dict(dgate=at(0)), ALIAS), (scan_bwd, dict(dx=at(6)), ALIAS), (scan_bwd, dict(dstate=at(3)), ALIAS),
    (scan_bwd, dict(dstate=at(4)), ALIAS), (scan_bwd, dict(dst=-1), STRIDE), (scan_bwd, dict(dy=at(2) + 1), ALIGN), (scan_bwd, dict(dtype=7), TYPE),
    (step, dict(pool=None), NULL), (step, dict(N=0), SIZE), (step, dict(slots=None, N=6), SIZE), (step, dict(S=0), SIZE),
    (step, dict(gs=-1), STRIDE), (step, dict(pool=at(2) + 2), ALIGN), (step, dict(y=at(2)), ALIAS),
    (step, dict(pool=at(0)), ALIAS), (step, dict(mode=-1), ARG), (step, dict(dtype=9), TYPE),
    (norm_fwd, dict(x=None), NULL), (norm_fwd, dict(y=None), NULL), (norm_fwd, dict(xt=1, dt=2), TYPE),
    (norm_fwd, dict(xt=1, dt=0), TYPE), (norm_fwd, dict(pt=5), TYPE), (norm_fwd, dict(act=3), ARG),
    (norm_fwd, dict(eps=ctypes.c_float(-1.0)), ARG), (norm_fwd, dict(eps=ctypes.c_float(float("nan"))), ARG),
    (norm_fwd, dict(G=5), SIZE), (norm_fwd, dict(R=0), SIZE), (norm_fwd, dict(G=0), SIZE),
    (norm_fwd, dict(C=8192, xs=8192, gs=8192, G=1), SIZE), (norm_fwd, dict(C=1 << 21, G=1 << 20), SIZE),
    (norm_fwd, dict(xs=-64), STRIDE), (norm_fwd, dict(gate=at(1) + 1), ALIGN), (norm_fwd, dict(w=at(2) + 2), ALIGN),
    (norm_fwd, dict(y=at(0) + 128), ALIAS), (norm_fwd, dict(y=at(2)), ALIAS), (norm_fwd, dict(y=at(0), xs=128), ALIAS),
    (norm_fwd, dict(y=at(0), xt=0), ALIAS),
    (norm_bwd, dict(dy=None), NULL), (norm_bwd, dict(dgate=None), NULL), (norm_bwd, dict(gate=None), NULL),
    (norm_bwd, dict(dx=at(1)), ALIAS), (norm_bwd, dict(dw=at(8)), ALIAS), (norm_bwd, dict(dx=at(5) + 1), ALIGN),
    (embed_fwd, dict(ids=None), NULL), (embed_fwd, dict(dt=3), TYPE), (embed_fwd, dict(N=0), SIZE), (embed_fwd, dict(V=0), SIZE),
    (embed_fwd, dict(ts=-1), STRIDE), (embed_fwd, dict(ids=at(0) + 4, w=1), ALIGN), (embed_fwd, dict(y=at(1) + 128), ALIAS),
    (embed_bwd, dict(out=None), NULL), (embed_bwd, dict(dt=1, gt=2), TYPE), (embed_bwd, dict(N=1 << 30), SIZE),
    (embed_bwd, dict(D=0), SIZE), (embed_bwd, dict(ds=-2), STRIDE), (embed_bwd, dict(out=at(2) + 2), ALIGN),
    (embed_bwd, dict(out=at(1)), ALIAS), (embed_bwd, dict(ws=None), WS), (embed_bwd, dict(n=64), WS),
    (embed_bwd, dict(ws=at(3) + 8), WS), (embed_bwd, dict(ws=at(1)), ALIAS), (embed_bwd, dict(ws=at(2) + 256), ALIAS),
]


@pytest.mark.parametrize("call,change,code", REFUSALS,
                         ids=[f"{c.__name__}-{'-'.join(d)}-{i}" for i, (c, d, _) in enumerate(REFUSALS)])
def test_refused_before_any_cuda_call(lib, call, change, code):
    assert call(lib, **change) == code


def test_workspace_sizes_of_refused_shapes_are_zero(lib):
    assert lib.based_embed_bwd_workspace_size(0, 10, 10) == 0
    assert lib.based_embed_bwd_workspace_size(10, 0, 10) == 0
    assert lib.based_norm_bwd_workspace_size(4, 10, 3) == 0
    # two keys and two positions a token, two partial rows a tile
    assert lib.based_embed_bwd_workspace_size(32, 1000, 16) >= 4 * 32 * 4 + 2 * 16 * 4


def test_binding_refuses_host_tensors_types_and_shapes():
    from linear_attention_gb300 import ops
    g = torch.zeros(2, 5, 8)
    with pytest.raises(ValueError):
        ops.based_scan_fwd(g, g)
    with pytest.raises(TypeError):
        ops.based_scan_fwd(g.double(), g.double())
    with pytest.raises(ValueError):
        ops.based_scan_fwd(g[0], g[0])
    with pytest.raises(ValueError):
        ops.based_scan_step(g[0], g[0], g[0])
    with pytest.raises(ValueError):
        ops.based_norm_fwd(g, 2)
    with pytest.raises(ValueError):
        ops.based_norm_bwd(g, g, 2)
    with pytest.raises(TypeError):
        ops.based_embed_fwd(torch.zeros(3), g[0])
    with pytest.raises(ValueError):
        ops.based_embed_fwd(torch.zeros(3, dtype=torch.int32), g[0])
    with pytest.raises(ValueError):
        ops.based_embed_bwd(torch.zeros(3, dtype=torch.int32), g[0, :3], 10)


def run_copy(tmp_path, code):
    """Runs `code` beside a copy of the package's Python files: a checkout in which nothing is built."""
    import shutil
    import subprocess
    import sys
    shutil.copytree(os.path.join(ROOT, "linear_attention_gb300"), tmp_path / "linear_attention_gb300",
                    ignore=shutil.ignore_patterns("_lib", "__pycache__"))
    return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300)


def test_import_before_the_build_and_a_call_that_says_so(tmp_path):
    out = run_copy(tmp_path, """
import torch
from linear_attention_gb300 import autograd, based, based_scan_fwd, ops
assert ops.__file__.startswith(%r), ops.__file__
for call in (lambda: based_scan_fwd(torch.zeros(1, 1, 1), torch.zeros(1, 1, 1)), ops.library):
    try:
        call()
    except based.BasedError as e:
        assert "not built" in str(e)
    else:
        raise SystemExit("no error")
print("refused")
""" % str(tmp_path))
    assert out.returncode == 0 and out.stdout.strip() == "refused", out.stderr[-2000:]


def test_a_binding_of_another_torch_is_not_taken(lib, monkeypatch):
    path = lbuild.binding_path()
    assert os.path.exists(path)
    monkeypatch.setattr(torch, "__version__", "0.0.1/x")
    other = lbuild.binding_path()
    assert other != path and os.path.dirname(other) == os.path.dirname(path) and not os.path.exists(other)


def test_the_library_is_built_where_the_binding_cannot_be(lib, monkeypatch):
    built = []
    monkeypatch.setattr(lbuild, "build_library", lambda *a: built.append(a))

    def broken(*a):
        raise RuntimeError("no headers")

    monkeypatch.setattr(lbuild, "_binding_commands", broken)
    with pytest.raises(RuntimeError):
        lbuild.build()
    assert built


def test_workspace_sizes_at_the_limits(lib):
    """The sizes are 0 exactly where the calls refuse theirs."""
    big = 1 << 20
    for N, V, D in ((9, 100, big), (9, 100, big + 1), ((1 << 30) - 1, 5, 1), (1 << 30, 5, 1), (9, 100, -1), (9, -1, 4)):
        refused = embed_bwd(lib, N=N, V=V, D=D, ds=max(D, 0), n=64) == SIZE
        assert (lib.based_embed_bwd_workspace_size(N, V, D) == 0) == refused, (N, V, D)
    # (the norm's sizes depend on the GPU; without one all are 0)
    for R, C, G in ((4, 2 * big, big), (1 << 40, 64, 4), (4, 8192, 1), (0, 64, 4), (4, 64, -4)):
        assert norm_bwd(lib, R=R, C=C, G=G, xs=C, ds=C, gs=C) == SIZE
        assert lib.based_norm_bwd_workspace_size(R, C, G) == 0
