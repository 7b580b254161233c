"""Sampling from rows most of whose tokens lie far below the largest: a type's lowest value as a mask, long tails, small temperatures."""
import math

import pytest
import torch

from linear_attention_gb300 import based_sample
from test_gpu_sample import check, row

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def masked(V, live, dtype, seed=0, tail=0, low=None):
    """`live` ordinary logits and `tail` ones 60 below them at random places; the lowest value elsewhere."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.full((V,), torch.finfo(dtype).min if low is None else low).to(dtype)
    at = torch.randperm(V, generator=gen)
    x[at[:live]] = row(live, dtype, seed)
    x[at[live:live + tail]] = row(tail, dtype, seed + 1) - 60
    return x


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V,live", [(300, 10), (2000, 10), (2000, 1999), (5000, 300), (20000, 40), (50001, 3000)])
def test_the_lowest_value_as_a_mask(cuda_device, dtype, V, live):
    """top_k below, at and above the number of unmasked tokens, with and without the other limits."""
    x = masked(V, live, dtype, V)
    for k in {1, live - 1, live, live + 1, min(V, live + 200), min(V, 1500), V - 1, V}:
        for temperature in (1.0, 0.2):
            check(x, top_k=k, temperature=temperature)
            check(x, top_k=k, temperature=temperature, top_p=0.8)
    check(x, top_p=0.9, min_p=0.01)
    check(x)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tokens_beyond_the_last_bin_s_edge(cuda_device, dtype):
    """Unmasked tokens more than 46 temperatures below the largest share their bin with masked ones."""
    for V, live, tail, ks in ((2000, 10, 300, (200, 310, 311, 1500)), (5000, 3500, 500, (3400, 3600, 4000, 4001, 4200, 4999)),
                              (5000, 100, 500, (90, 400, 600, 601, 3000)), (60000, 40000, 500, (39000, 40100, 40500, 40501, 50000)),
                              (130001, 500, 400, (300, 700, 900, 901, 2000, 40000, 130000))):
        x = masked(V, live, dtype, V, tail)
        for k in ks:
            check(x, top_k=k)
            check(x, top_k=k, top_p=0.7, min_p=0.001)


def test_differences_beyond_float32(cuda_device):
    """Differences that times the inverse temperature, or already by themselves, are infinite."""
    x = row(3000, F32, 3)
    for t in (1e-36, 1e-37, 3e-38, 1e-39):
        for k in (1, 50, 500, 2999):
            check(x, top_k=k, temperature=t)
        check(x, top_k=300, top_p=0.9, temperature=t)
    y = masked(3000, 20, F32, 4)
    y[7] = torch.finfo(F32).max
    for limits in (dict(top_k=5), dict(top_k=300), dict(top_k=300, top_p=0.9), dict(top_p=0.9), {}):
        check(y, **limits)


def test_masked_rows_beside_others(cuda_device):
    """A batch whose rows differ in what is masked; each row's own limits."""
    gen = torch.Generator().manual_seed(6)
    N, V = 24, 4001
    x = torch.stack([masked(V, n, F32, n, tail) for n, tail in zip((1, 2, 40, 300, 1000, 4000) * 4, (0, 30, 300, 0, 2500, 1) * 4)])
    k = torch.randint(1, V, (N,), generator=gen).to(torch.int32)
    p, u = torch.rand(N, generator=gen) * 0.5 + 0.5, torch.rand(N, generator=gen)
    got, probs = based_sample(x.cuda(), u.cuda(), top_k=k.cuda(), top_p=p.cuda())
    for i in range(N):
        t, q = based_sample(x[i:i + 1].cuda(), u[i:i + 1].cuda(), top_k=int(k[i]), top_p=float(p[i]))
        assert t.item() == got[i].item() and abs(q.item() - probs[i].item()) <= 2.0 ** -20 * q.item()
        assert x[i, t.item()] > -math.inf and x[i, t.item()] > x[i].max() - 50 and 0 < q.item() <= 1
