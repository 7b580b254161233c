"""The residual stream's root-mean-square norm on the GPU against its 64-bit form."""
import math

import pytest
import torch

import more_ops_reference as ref
from linear_attention_gb300 import based_rms_bwd, based_rms_fwd, ops
from linear_attention_gb300.autograd import rms_norm
from linear_attention_gb300.based import BasedError

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
E4M3 = torch.float8_e4m3fn


def inputs(shape, dtype, stream, seed=0, residual=True, weight=None):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    s = dict(x=rand(*shape).to(dtype).cuda(), residual=(2 * rand(*shape)).to(stream).cuda() if residual else None,
             weight=None if weight == "none" else (1 + 0.3 * rand(shape[-1])).to(weight or dtype).cuda())
    return s, rand(*shape).to(dtype).cuda(), rand(*shape).to(stream if residual else dtype).cuda()


def check(s, dy, dsum, eps=1e-6):
    y, total, scales = based_rms_fwd(s["x"], s["weight"], residual=s["residual"], eps=eps)
    assert scales is None and (s["residual"] is not None or total is s["x"])
    ds, dx, dweight = based_rms_bwd(dy, total, s["weight"], dsum=dsum, eps=eps)
    val, bound = ref.rms(s["x"], s["weight"], s["residual"], eps, dy, dsum)
    got = dict(y=y, ds=ds, dweight=dweight, sum=total)
    assert (dx is ds) == (total.dtype == s["x"].dtype)
    if dx is not ds:
        got["dx"] = dx
    for name in val:
        ref.assert_within(got[name], val[name], bound[name], name)
    assert (dweight is None) == (s["weight"] is None)
    return got


# channels on both sides of every change of the threads of a row, and of other than whole words
WIDTHS = [1, 7, 8, 64, 65, 72, 256, 264, 512, 520, 777, 1024, 1032, 1536, 1544, 2048, 3080, 4096, 4104, 6144, 8192, 8200, 16384, 16383]


@pytest.mark.parametrize("C", WIDTHS)
def test_every_width(cuda_device, C):
    for dtype, stream in ((BF16, F32), (F32, F32), (F16, F16)):
        check(*inputs((5, C), dtype, stream, seed=C))


@pytest.mark.parametrize("rows", [1, 3, 33, 700, 5000])
@pytest.mark.parametrize("C", [40, 520, 1536])
def test_rows(cuda_device, rows, C):
    check(*inputs((rows, C), BF16, BF16, seed=rows))
    check(*inputs((rows, C), F16, F32, seed=rows, residual=False))


@pytest.mark.parametrize("weight", ["none", F32, None])
def test_weights_and_absent_gradients(cuda_device, weight):
    s, dy, _ = inputs((3, 4, 96), BF16, F32, weight=weight)
    check(s, dy, None)
    check(*inputs((3, 4, 96), BF16, BF16, weight=weight, residual=False))


@pytest.mark.parametrize("C", [16, 500, 520, 4096, 16384])
@pytest.mark.parametrize("dtype,stream", [(BF16, F32), (F16, F16), (F32, F32)])
def test_eight_bits(cuda_device, C, dtype, stream):
    s, _, _ = inputs((9, C), dtype, stream, seed=C)
    s["x"][3] = 0
    s["residual"][3] = 0
    y, total, scales = based_rms_fwd(s["x"], s["weight"], residual=s["residual"], quantize=True)
    assert y.dtype == E4M3 and scales.shape == (9,) and scales[3] == 1 and (y[3].float() == 0).all()
    val, bound = ref.rms(s["x"], s["weight"], s["residual"], 1e-6, quantize=True)
    for name, t in dict(y=y.float(), scale=scales, sum=total).items():
        ref.assert_within(t, val[name], bound[name], name)
    assert (y.float().abs().amax(-1)[[0, 1, 2, 4]] == 448).all()


def test_strides_and_places(cuda_device):
    """Rows of a wider tensor, a broadcast row, rows on no 16-byte word; the sum and its gradient in place."""
    gen = torch.Generator().manual_seed(2)
    wide = torch.randn(50, 3, 200, generator=gen).to(BF16).cuda()
    s = dict(x=wide[:, 0, :96], residual=wide[:, 1, 1:97].clone(), weight=torch.ones(96, device="cuda", dtype=BF16))
    check(s, wide[:, 2, 3:99], wide[:, 2, 100:196])
    s["x"] = wide[:1, 0, :96].expand(50, 96)
    want = check(s, wide[:1, 2, :96].expand(50, 96), None)
    place = s["residual"].contiguous()
    y, total, _ = based_rms_fwd(s["x"], s["weight"], residual=place, sum_out=place)
    assert total.data_ptr() == place.data_ptr() and torch.equal(total, want["sum"]) and torch.equal(y, want["y"])
    with pytest.raises(BasedError):
        based_rms_fwd(place, s["weight"], residual=s["residual"].contiguous(), sum_out=place)


def test_infinities_stay_in_their_rows(cuda_device):
    s, dy, dsum = inputs((6, 520), F32, F32)
    y = based_rms_fwd(s["x"], s["weight"], residual=s["residual"])[0]
    s["x"][2, 5] = math.inf
    s["x"][4, 7] = math.nan
    z, total, _ = based_rms_fwd(s["x"], s["weight"], residual=s["residual"])
    assert torch.equal(z[[0, 1, 3, 5]], y[[0, 1, 3, 5]]) and z[4].isnan().all() and not z[2].isfinite().all()
    z8, _, scales = based_rms_fwd(s["x"], s["weight"], residual=s["residual"], quantize=True)
    assert scales[[0, 1, 3, 5]].isfinite().all() and z8[[0, 1, 3, 5]].float().isfinite().all() and z8[4].float().isnan().all()


def test_small_and_large_magnitudes(cuda_device):
    for c in (1e-15, 1e15):
        s, dy, dsum = inputs((4, 200), F32, F32)
        s["x"], s["residual"] = s["x"] * c, s["residual"] * c
        check(s, dy, None, eps=0.0)
    s, _, _ = inputs((4, 64), F32, F32, weight="none")
    y, _, scales = based_rms_fwd(s["x"] * 1e-30, torch.full((64,), 1e-20, device="cuda"), eps=1.0, quantize=True)
    assert y.float().isfinite().all() and scales.isfinite().all() and (scales > 0).all()


def test_results_repeat(cuda_device):
    s, dy, dsum = inputs((3000, 1000), BF16, F32)
    a = based_rms_bwd(dy, s["residual"], s["weight"], dsum=dsum)
    ws = torch.full((ops.rms_bwd_workspace_size(3000, 1000),), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = based_rms_bwd(dy, s["residual"], s["weight"], dsum=dsum, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(BasedError):
        based_rms_bwd(dy, s["residual"], s["weight"], dsum=dsum, workspace=ws[:-4])


@pytest.mark.parametrize("dtype,stream", [(F32, F32), (BF16, F32)])
def test_autograd(cuda_device, dtype, stream):
    s, dy, dsum = inputs((7, 120), dtype, stream)
    val, bound = ref.rms(s["x"], s["weight"], s["residual"], 1e-6, dy, dsum)
    t = {n: x.clone().requires_grad_() for n, x in s.items()}
    y, total = rms_norm(t["x"], t["weight"], t["residual"])
    torch.autograd.backward([y, total], [dy, dsum])
    ref.assert_within(t["residual"].grad, val["ds"], bound["ds"], "ds")
    name = "dx" if stream != dtype else "ds"
    ref.assert_within(t["x"].grad, val[name], bound[name], "dx")
    ref.assert_within(t["weight"].grad, val["dweight"], bound["dweight"], "dweight")
    # the stream alone, and no residual, with gradients that are broadcast
    t = {n: x.clone().requires_grad_() for n, x in s.items()}
    rms_norm(t["x"], t["weight"], t["residual"])[1].sum().backward()
    assert (t["x"].grad == 1).all() and (t["residual"].grad == 1).all() and t["x"].grad.dtype == dtype
    t = {n: x.clone().requires_grad_() for n, x in s.items()}
    y, same = rms_norm(t["x"].transpose(0, 1).contiguous().transpose(0, 1), t["weight"])
    (y.sum() + same.sum()).backward()
    assert t["x"].grad.isfinite().all()


def test_empty(cuda_device):
    x, w = torch.empty(0, 16, device="cuda"), torch.ones(16, device="cuda")
    y, total, _ = based_rms_fwd(x, w, residual=x)
    ds, dx, dw = based_rms_bwd(x, x, w)
    assert y.shape == total.shape == ds.shape == x.shape and (dw == 0).all()
    y, _, scales = based_rms_fwd(x, w, quantize=True)
    assert y.shape == x.shape and scales.shape == (0,)
