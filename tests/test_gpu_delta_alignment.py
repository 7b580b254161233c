"""What depends on the alignment of rows and outputs: of the delta rule's passes only their time, of its step and of the residual
stream's norm the order of sums."""
import pytest
import torch

import more_ops_reference as ref
from linear_attention_gb300 import based_delta_bwd, based_delta_fwd, based_delta_step, based_rms_bwd, based_rms_fwd
from test_gpu_delta import inputs

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NAMES = "q k v beta gate".split()


def shifted(t, by=1):
    """The same values, `by` elements behind a 16-byte word."""
    room = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    out = room[by:].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("dtype,K,V", [(F32, 64, 32), (BF16, 128, 48), (F16, 40, 72)])
def test_the_passes_give_the_same_bits(cuda_device, dtype, K, V):
    s, more, do, dfinal = inputs(2, 100, 4, 2, K, V, dtype, seed=21, lengths=[100, 70])
    odd = {n: shifted(t) for n, t in s.items()}
    o, final, saved = based_delta_fwd(**s, **more, save=True)
    p, last, kept = based_delta_fwd(**odd, state=shifted(more["state"]), lengths=more["lengths"], save=True, out=shifted(o), final_state=shifted(final))
    assert torch.equal(p, o) and torch.equal(last, final)
    a = based_delta_bwd(*(s[n] for n in NAMES), do, saved, dfinal=dfinal, lengths=more["lengths"])
    b = based_delta_bwd(*(odd[n] for n in NAMES), shifted(do), kept, dfinal=shifted(dfinal), lengths=more["lengths"])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("by", [1, 2, 3])
def test_the_step_of_a_pool_anywhere(cuda_device, by):
    s, _, _, _ = inputs(3, 1, 4, 2, 48, 64, BF16, seed=22)
    pool = torch.randn(5, 4, 48, 64, generator=torch.Generator().manual_seed(22)).cuda()
    val = ref.delta_rows(*(s[n] for n in NAMES), None, pool[:3], None)
    bound = ref.delta_bounds(val, *(s[n] for n in NAMES), None, pool[:3], None)
    for place in (pool.clone(), shifted(pool, by)):
        o = based_delta_step(**{n: t[:, 0] for n, t in s.items()}, pool=place)
        ref.assert_within(o[:, None], val["o"], bound["o"], "o")
        ref.assert_within(place[:3], val["final"], bound["final"], "pool")
        assert torch.equal(place[3:], pool[3:])


@pytest.mark.parametrize("C", [64, 1000, 4096])
def test_the_norm_of_rows_anywhere(cuda_device, C):
    gen = torch.Generator().manual_seed(23)
    x, r, dy, ds = ((torch.randn(7, C, generator=gen) * f).to(t).cuda() for f, t in ((1, BF16), (2, F32), (1, BF16), (1, F32)))
    w = (1 + 0.3 * torch.randn(C, generator=gen)).to(BF16).cuda()
    val, bound = ref.rms(x, w, r, 1e-6, dy, ds)
    for move in (lambda t: t, shifted):
        y, total, _ = based_rms_fwd(move(x), move(w), residual=move(r))
        back = based_rms_bwd(move(dy), move(total), move(w), dsum=move(ds))
        for n, t in dict(y=y, sum=total, ds=back[0], dx=back[1], dweight=back[2]).items():
            ref.assert_within(t, val[n], bound[n], n)
