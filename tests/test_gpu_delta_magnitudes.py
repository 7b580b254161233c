"""The gated delta rule where magnitudes differ widely within a call: what is large and does not reach a result must not cost it bits.

Bounds are those of more_ops_reference.py: roundings of float16 pairs relative to the terms that make up a result."""
import math

import pytest
import torch

import more_ops_reference as ref
from linear_attention_gb300 import based_delta_bwd, based_delta_fwd
from test_gpu_delta import inputs

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NAMES = "q k v beta gate".split()
GRADS = "dq dk dv dbeta dgate dstate".split()


def run(s, more, do, dfinal):
    """The kernels' results, the 64-bit ones and their bounds."""
    o, final, saved = based_delta_fwd(**s, **more, save=True)
    grads = based_delta_bwd(*(s[n] for n in NAMES), do, saved, dfinal=dfinal, lengths=more["lengths"])
    args = *(s[n] for n in NAMES), None, more["state"], more["lengths"], do, dfinal
    val = ref.delta_rows(*args)
    return dict(o=o, final=final, **dict(zip(GRADS, grads))), val, ref.delta_bounds(val, *args)


def near(got, val, dtype, names, rows=slice(None), channels=slice(None)):
    """assert_near on a part: rows of all results, channels of those that have the values' ones."""
    for n in names:
        cut = (slice(None), rows, slice(None), channels) if n in ("o", "dv") else (slice(None), rows)
        ref.assert_near(got[n][cut], val[n][cut], dtype, n)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [1e3, 1e4, 1e6])
def test_a_masked_row_of_large_values(cuda_device, dtype, c):
    """beta 0: whatever lies in the row's v is not written, and no other row sees it."""
    s, more, do, dfinal = inputs(2, 200, 2, 2, 64, 48, dtype, seed=11)
    s["beta"][:, 20] = 0.0
    s["v"][:, 20] *= c
    got, val, bound = run(s, more, do, dfinal)
    for n in val:
        ref.assert_within(got[n], val[n], bound[n], n)
    near(got, val, dtype, ("o", "dq", "dk", "dv", "dgate"))
    # the rows behind: dbeta of row 20 is as large as its v
    near(got, val, dtype, ("dbeta",), rows=slice(21, None))
    # the masked row's values reach dbeta alone
    plain = dict(s, v=s["v"].clone())
    plain["v"][:, 20] = 0.0
    clean, exact, _ = run(plain, more, do, dfinal)
    assert all(torch.equal(exact[n], val[n]) for n in ("o", "final", "dq", "dk", "dv", "dgate", "dstate"))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [1e3, 1e5])
def test_large_values_in_front_of_a_cleared_state(cuda_device, dtype, c):
    s, more, do, dfinal = inputs(2, 260, 2, 1, 64, 48, dtype, seed=12)
    s["v"][:, :70] *= c
    s["gate"][:, 70] = -math.inf
    more["state"] = more["state"] * c
    got, val, bound = run(s, more, do, dfinal)
    # Rows 64 to 79 are scaled together, for rows 64 to 69: the pairs of row j's correction E_j are off by half of float16's least step, 2^-25, where
    # the scale brings the largest |step E| to 2^14 at least: by 2^-39 of that, over j's step. o_i takes beta_j scale |q_i k_j| <= 2 step_j / 8
    # of it from each of the rows 70 .. i: at most 10 x 2 / 8 x 2^-39 max |E|.
    E = []
    for t in range(64, 70):
        front = {n: x[:, :t] for n, x in s.items()}
        S = ref.delta_rows(*(front[n] for n in NAMES), None, more["state"], None)["final"]
        a, k = s["gate"][:, t].double().exp().cpu(), s["k"][:, t].cpu().double().expand(-1, 2, -1)
        E.append(s["v"][:, t].cpu().double() - a[..., None] * torch.einsum("bhkv,bhk->bhv", S, k))
    bound["o"][:, 70:80] += 2.5 * 2.0 ** -39 * torch.stack(E).abs().max()
    for n in val:  # (the gradients' rows that are scaled with them are held to nothing)
        rows = [slice(None)] if n in ("o", "final", "dstate") else [slice(0, 64), slice(80, None)]
        for r in rows:
            ref.assert_within(got[n][:, r], val[n][:, r], bound[n][:, r], n)
    # behind the sixteen rows in which the state is cleared
    near(got, val, dtype, ("o", "dq", "dk", "dv", "dbeta", "dgate"), rows=slice(80, None))
    final = val["final"]
    err = (got["final"].cpu().double() - final).square().mean().sqrt() / final.square().mean().sqrt()
    assert err <= 2.0 ** -16, float(err)  # as assert_near's float32


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [1e-5, 1e4])
def test_a_slice_of_channels_of_another_size(cuda_device, dtype, c):
    """16 channels of the values c times as large, and their gradients 1 / c times: their share of dq and dk is that of the others."""
    s, more, do, dfinal = inputs(2, 150, 4, 2, 64, 64, dtype, seed=13)
    part = slice(16, 32)
    s["v"][..., part] *= c
    more["state"][..., part] *= c
    do[..., part] /= c
    dfinal[..., part] /= c
    got, val, bound = run(s, more, do, dfinal)
    for n in val:
        ref.assert_within(got[n], val[n], bound[n], n)
    near(got, val, dtype, ("dq", "dk", "dbeta", "dgate"))
    for channels in (slice(0, 16), part, slice(32, 64)):
        near(got, val, dtype, ("o", "dv"), channels=channels)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_zero_key_with_large_values(cuda_device, dtype):
    """A row that writes nothing because its key is 0."""
    s, more, do, dfinal = inputs(2, 200, 2, 2, 64, 32, dtype, seed=14)
    s["k"][:, 37] = 0.0
    s["v"][:, 37] *= 1e4
    got, val, bound = run(s, more, do, dfinal)
    for n in val:
        ref.assert_within(got[n], val[n], bound[n], n)
    near(got, val, dtype, ("o", "dq", "dv", "dbeta", "dgate"))
    near(got, val, dtype, ("dk",), rows=slice(38, None))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_values_of_heavy_tails(cuda_device, dtype):
    """Values of Student's t with two degrees of freedom: every chunk has a few that stand out."""
    s, more, do, dfinal = inputs(1, 1024, 2, 2, 64, 32, dtype, seed=15)
    gen = torch.Generator().manual_seed(15)
    t = torch.randn(1, 1024, 2, 32, generator=gen) / (torch.randn(1, 1024, 2, 2, generator=gen).square().mean(-1, keepdim=True).sqrt() + 1e-4)
    s["v"] = t.clamp(-1e4, 1e4).to(dtype).cuda()
    got, val, bound = run(s, more, do, dfinal)
    for n in val:
        ref.assert_within(got[n], val[n], bound[n], n)
    near(got, val, dtype, ("o", "dq", "dk", "dv", "dgate"))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_steps_of_many_magnitudes(cuda_device, dtype):
    """beta from 2^-20 to 2 and of either sign, on values that make what each row writes about as large; and 0."""
    s, more, do, dfinal = inputs(2, 150, 4, 2, 64, 32, dtype, seed=16)
    gen = torch.Generator().manual_seed(16)
    e = -14.0 * torch.rand(2, 150, 4, generator=gen)
    e = torch.where(torch.rand(2, 150, 4, generator=gen) < 0.3, e, -torch.rand(2, 150, 4, generator=gen))
    sign = torch.where(torch.rand(2, 150, 4, generator=gen) < 0.1, -1.0, 1.0)
    s["beta"] = (torch.exp2(e) * sign).to(dtype).cuda()
    s["beta"][:, 10::40] = 0.0
    s["beta"][:, 11::40] = 2.0
    s["v"] = (s["v"].float() / torch.exp2(e)[..., None].cuda()).to(dtype)
    got, val, bound = run(s, more, do, dfinal)
    for n in val:
        ref.assert_within(got[n], val[n], bound[n], n)
    near(got, val, dtype, ("o", "dq", "dv", "dgate"))
    if dtype == F32:
        t = dict(s, beta=torch.where(torch.rand(2, 150, 4, generator=gen).cuda() < 0.2, 2.0 ** -20, s["beta"]))
        got, val, bound = run(t, more, do, dfinal)
        for n in val:
            ref.assert_within(got[n], val[n], bound[n], n)
