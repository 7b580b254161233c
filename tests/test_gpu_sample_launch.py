"""A row's token does not depend on how a call is launched: alone or in a batch, on 16-byte words or not."""
import pytest
import torch

import more_ops_reference as ref
from linear_attention_gb300 import based_sample
from test_gpu_sample import row

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def border_numbers(x, limits, steps=6):
    """float32 numbers at and around the borders between kept tokens, where one rounding of a sum decides."""
    _, prob = ref.sample_order(x, limits.get("temperature", 1.0), limits.get("top_k"), limits.get("top_p"), limits.get("min_p"))
    up = down = prob.cumsum(0)[:-1].float()
    u = [up]
    for _ in range(steps):
        up, down = torch.nextafter(up, torch.tensor(1.0)), torch.nextafter(down, torch.tensor(0.0))
        u += [up, down]
    u = torch.cat(u)
    return u[u < 1]


def check(x, limits, most=2400):
    u = border_numbers(x, limits)[:most].cuda()
    x = x.cuda()
    tokens, probs = based_sample(x.expand(u.numel(), -1), u, **limits)
    few = [based_sample(x.expand(min(3, u.numel() - i), -1), u[i:i + 3], **limits) for i in range(0, u.numel(), 3)]
    assert torch.equal(torch.cat([t for t, _ in few]), tokens) and torch.equal(torch.cat([p for _, p in few]), probs)
    # the same row on no 16-byte word: other threads see other tokens first
    odd = torch.cat([x.new_zeros(1), x])[1:]
    t, p = based_sample(odd.expand(u.numel(), -1), u, **limits)
    assert torch.equal(t, tokens) and torch.equal(p, probs)


@pytest.mark.parametrize("V,dtype,limits", [(30000, BF16, dict(top_k=250)), (30000, BF16, dict(top_k=255, top_p=0.95, min_p=0.001)),
                                          (20000, F16, dict(top_k=256, temperature=1.5)), (50000, F32, dict(top_k=200)),
                                          (2000, F32, dict(top_k=230)), (16000, F32, dict(top_p=0.5))])
def test_rows_of_any_order(cuda_device, V, dtype, limits):
    check(row(V, dtype, V), limits)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("limits", [dict(top_k=160), dict(top_k=160, min_p=0.02)])
def test_kept_tokens_side_by_side(cuda_device, seed, limits):
    """Pairs of large tokens, in the words of few threads where one CTA has the row and of many where sixteen have: one launch sums what it
    has listed, the other goes through the row."""
    x = row(30000, F32, seed, 0.3)
    gen = torch.Generator().manual_seed(seed)
    words = (torch.arange(12)[:, None] * 40 + 512 * torch.arange(7)).flatten()[:80]
    for i in (0, 1):
        x[8 * words + i] = 4 + torch.rand(80, generator=gen)
    check(x.to(BF16), limits)
