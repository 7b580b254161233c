"""The scaled embedding and its gradient on the GPU."""
import pytest
import torch

import ops_reference as ref
from linear_attention_gb300.based import BasedError
from linear_attention_gb300.ops import based_embed_bwd, based_embed_fwd, embed_bwd_workspace_size

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def draw(N, V, D, dtype, seed, idt=torch.int32, padding=0.0):
    gen = torch.Generator().manual_seed(seed)
    rank = torch.exp(torch.rand(N, generator=gen, dtype=torch.float64) * torch.log(torch.tensor(V + 1.0))).long() - 1
    ids = torch.randperm(V, generator=gen)[rank.clamp(0, V - 1)]
    ids[torch.rand(N, generator=gen) < padding] = -1
    table, dy = torch.randn(V, D, generator=gen).to(dtype).cuda(), torch.randn(N, D, generator=gen).to(dtype).cuda()
    return ids.to(idt).cuda(), table, dy


def check_fwd(ids, table, scale):
    y = based_embed_fwd(ids, table, scale)
    V = table.shape[0]
    live = ((ids >= 0) & (ids < V))[..., None]
    # one product in float32, rounded once: nothing to tolerate
    want = torch.where(live, (table[ids.clamp(0, V - 1).long()].float() * scale), 0.0).to(table.dtype)
    assert torch.equal(y, want)


def check_bwd(ids, dy, V, scale, dtype):
    got = based_embed_bwd(ids, dy, V, scale, dtype=dtype)
    val, bound = ref.embed_grad(ids, dy, V, scale, dtype)
    ref.assert_within(got, val, bound, "dtable")


SIZES = [(1, 1, 1), (1, 5, 8), (2, 2, 3), (31, 7, 64), (32, 7, 64), (33, 1000, 65), (64, 2, 128), (65, 1, 8), (512, 8192, 512),
         (1000, 1023, 100), (1024, 1024, 32), (1025, 1025, 33), (5000, 50, 256), (5000, 70000, 72), (3000, 300, 4104)]


@pytest.mark.parametrize("N,V,D", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_sizes(N, V, D, dtype, cuda_device):
    ids, table, dy = draw(N, V, D, dtype, N + D, padding=0.1 if N % 2 else 0.0)
    check_fwd(ids, table, 1.7)
    check_bwd(ids, dy, V, 1.7, F32)
    check_bwd(ids, dy, V, 0.3, dtype)


def test_id_types_padding_and_axes(cuda_device):
    for idt in (torch.int32, torch.int64):
        ids, table, dy = draw(600, 90, 48, BF16, 1, idt)
        ids[5], ids[6], ids[7] = -1, 90, 2 ** 31 - 1
        if idt == torch.int64:
            ids[8], ids[9] = 2 ** 32 + 3, -2 ** 40
        check_fwd(ids, table, 2.0)
        check_bwd(ids, dy, 90, 2.0, F32)
        y = based_embed_fwd(ids.view(4, 150), table, 2.0)
        assert y.shape == (4, 150, 48) and torch.equal(y.view(600, 48), based_embed_fwd(ids, table, 2.0))
        assert torch.equal(based_embed_bwd(ids.view(4, 150), dy.view(4, 150, 48), 90), based_embed_bwd(ids, dy, 90))
    none = torch.full((70,), -1, dtype=torch.int32, device="cuda")
    dy[:70] = float("nan")  # the rows of padding tokens are not summed anywhere
    assert (based_embed_fwd(none, table) == 0).all() and (based_embed_bwd(none, dy[:70], 90) == 0).all()


@pytest.mark.parametrize("N", [1, 31, 32, 33, 64, 95, 1000, 40000])
def test_one_token_everywhere(N, cuda_device):
    # every position holds the same id: its run crosses every tile
    ids = torch.full((N,), 3, dtype=torch.int32, device="cuda")
    dy = torch.randn(N, 40, generator=torch.Generator().manual_seed(N)).to(BF16).cuda()
    check_bwd(ids, dy, 5, 1.0, F32)


def test_runs_at_every_place_of_a_tile(cuda_device):
    gen = torch.Generator().manual_seed(2)
    for first in range(0, 70, 3):
        counts = [first, 1, 2, 40, 31, 32, 33, 64, 1, 97]
        ids = torch.repeat_interleave(torch.arange(10), torch.tensor(counts))
        ids = ids[torch.randperm(len(ids), generator=gen)].to(torch.int32).cuda()
        dy = torch.randn(len(ids), 16, generator=gen).cuda()
        check_bwd(ids, dy, 11, 1.0, F32)


@pytest.mark.parametrize("V", [3, 1022, 1023, 1024, 2 ** 20 - 1, 2 ** 20, 5_000_000])
def test_vocabularies_around_the_digits_of_the_sort(V, cuda_device):
    gen = torch.Generator().manual_seed(V)
    ids = torch.randint(0, V, (3000,), generator=gen)
    ids[:3] = torch.tensor([0, V - 1, V // 2])
    dy = torch.randn(3000, 4, generator=gen)
    got = based_embed_bwd(ids.to(torch.int32).cuda(), dy.cuda(), V)
    val, bound = ref.embed_grad(ids, dy, V, 1.0, F32)
    ref.assert_within(got, val, bound, V)


def test_many_tokens(cuda_device):
    # more than the 128 sorting CTAs hold in one chunk each
    ids, _, dy = draw(300_000, 20_000, 16, BF16, 3, padding=0.05)
    check_bwd(ids, dy, 20_000, 1.0, F32)


def test_strides_and_alignment(cuda_device):
    ids, table, dy = draw(500, 60, 160, BF16, 4)
    for a, b in ((0, 64), (96, 160), (1, 65), (3, 100)):
        check_fwd(ids, table[:, a:b], 1.5)
        check_bwd(ids, dy[:, a:b], 60, 1.5, F32)
    check_bwd(ids, dy[:1].expand(500, 160), 60, 1.0, F32)
    buf = torch.full((60 * 64 + 9,), 7.0, device="cuda")  # a table that starts off a 16-byte boundary
    out = buf[1:60 * 64 + 1].view(60, 64)
    based_embed_bwd(ids, dy[:, :64], 60, out=out)
    assert torch.equal(out, based_embed_bwd(ids, dy[:, :64], 60)) and buf[0] == 7 and (buf[60 * 64 + 1:] == 7).all()
    half = torch.full((60 * 33 + 9,), 7.0, dtype=BF16, device="cuda")
    based_embed_bwd(ids, dy[:, :33], 60, dtype=BF16, out=half[3:60 * 33 + 3].view(60, 33))
    assert (half[:3] == 7).all() and (half[60 * 33 + 3:] == 7).all()


def test_determinism_streams_graphs_and_workspace(cuda_device):
    ids, table, dy = draw(20000, 3000, 136, BF16, 5, padding=0.1)
    want = (based_embed_fwd(ids, table, 3.0), based_embed_bwd(ids, dy, 3000, 3.0))
    for _ in range(3):
        assert torch.equal(based_embed_bwd(ids, dy, 3000, 3.0), want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (based_embed_fwd(ids, table, 3.0, stream=side), based_embed_bwd(ids, dy, 3000, 3.0, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    n = embed_bwd_workspace_size(20000, 3000, 136)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(based_embed_bwd(ids, dy, 3000, 3.0, workspace=ws[:n]), want[1]) and (ws[n:] == 255).all()
    with pytest.raises(BasedError):
        based_embed_bwd(ids, dy, 3000, 3.0, workspace=ws[:n - 4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = (based_embed_fwd(ids, table, 3.0), based_embed_bwd(ids, dy, 3000, 3.0))
    ids.copy_(ids.flip(0))
    want = (based_embed_fwd(ids, table, 3.0), based_embed_bwd(ids, dy, 3000, 3.0))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, cap))


def test_gradient_against_differences(cuda_device):
    # the lookup is linear in the table: a step of 1 leaves rounding alone
    ids, table, dy = draw(200, 12, 8, F32, 6, padding=0.1)
    grad = based_embed_bwd(ids, dy, 12, 0.5)
    for i in range(0, 96, 7):
        moved = table.clone()
        moved.view(-1)[i] += 1
        diff = ((based_embed_fwd(ids, moved, 0.5).double() - based_embed_fwd(ids, table, 0.5).double()) * dy.double()).sum()
        assert abs(float(diff) - float(grad.view(-1)[i])) <= 200 * 2.0 ** -20 * float(dy.abs().max())


def test_offsets_past_32_bits(cuda_device):
    V, D = (1 << 21) + 2, 1024  # a table and a gradient of more than 2^31 elements
    ids = torch.tensor([V - 1, 0, V - 1, 1 << 20, V], dtype=torch.int32, device="cuda")
    table = torch.zeros(V, D, dtype=BF16, device="cuda")
    table[V - 1], table[1 << 20] = 3, 5
    y = based_embed_fwd(ids, table, 2.0)
    assert y[:, 0].tolist() == [6, 0, 6, 10, 0] and torch.equal(y, y[:, :1].expand(5, D))
    del table
    dy = torch.tensor([[1.0], [2.0], [4.0], [8.0], [16.0]], device="cuda").expand(5, D).to(BF16).contiguous()
    grad = based_embed_bwd(ids, dy, V, dtype=BF16)
    assert (grad[V - 1] == 5).all() and (grad[0] == 2).all() and (grad[1 << 20] == 8).all()
    assert int((grad != 0).sum()) == 3 * D


@pytest.mark.parametrize("filler", [1200, 6000])
def test_runs_at_every_place_of_a_tile_among_many_tokens(filler, cuda_device):
    # enough tokens for the counting sort, with short and with long tiles
    gen = torch.Generator().manual_seed(3)
    for first in (0, 1, 5, 8, 13, 31, 32, 40, 63, 64, 69):
        counts = [first, 1, 2, 40, 31, 32, 33, 64, 1, 97, 0, filler, 3, 400]
        ids = torch.repeat_interleave(torch.arange(14), torch.tensor(counts))
        ids[torch.rand(len(ids), generator=gen) < 0.02] = -1
        ids = ids[torch.randperm(len(ids), generator=gen)].to(torch.int32).cuda()
        dy = torch.randn(len(ids), 16, generator=gen).cuda()
        check_bwd(ids, dy, 15, 1.0, F32)


@pytest.mark.parametrize("N", [1, 7, 8, 127, 128, 129, 250, 512, 513, 1000, 1023, 1024, 1025, 1030])
def test_token_counts_around_the_direct_ranking(N, cuda_device):
    for V in (5, 900, 2 ** 22 - 1, 2 ** 22, 2 ** 22 + 5):
        gen = torch.Generator().manual_seed(N + V)
        ids = torch.randint(0, V, (N,), generator=gen)
        ids[: N // 3] = V - 1
        ids[N // 2: N // 2 + 2] = -1
        dy = torch.randn(N, 2, generator=gen)
        got = based_embed_bwd(ids.to(torch.int32).cuda(), dy.cuda(), V)
        val, bound = ref.embed_grad(ids, dy, V, 1.0, F32)
        ref.assert_within(got, val, bound, (N, V))


def check_exactly(ids, V, D, seed):
    """Gradients of small whole numbers: every float32 sum below 2^24 is exact, and one missing row shows."""
    dy = torch.randint(-8, 9, (ids.numel(), D), generator=torch.Generator().manual_seed(seed))
    live = (ids >= 0) & (ids < V)
    want = torch.zeros(V, D, dtype=torch.int64).index_add(0, ids[live].long(), dy[live])
    for dtype in (F32, BF16, F16):
        got = based_embed_bwd(ids.cuda(), dy.to(dtype).cuda(), V)
        assert torch.equal(got.cpu().long(), want) and torch.equal(got.cpu(), want.float())


@pytest.mark.parametrize("N", [8192, 8193, 40000, 300_000])
def test_one_token_everywhere_exactly(N, cuda_device):
    # tiles of 32 rows: from one run over all of them to runs that begin and end around them
    check_exactly(torch.full((N,), 3, dtype=torch.int32), 5, 40, N)
    ids = torch.full((N,), 3, dtype=torch.int32)
    ids[::5], ids[7], ids[N // 2] = 1, -1, 4
    check_exactly(ids, 5, 9, N + 1)


def test_runs_at_every_place_of_a_long_tile(cuda_device):
    # 8192 tokens and more: tiles of 32 rows, more tokens than one chunk of eight CTAs
    gen = torch.Generator().manual_seed(4)
    for first in (0, 1, 5, 13, 30, 31, 32, 33, 40, 63, 64, 69):
        counts = [first, 1, 2, 40, 31, 32, 33, 64, 1, 97, 0, 9000, 3, 400, 290]
        ids = torch.repeat_interleave(torch.arange(15), torch.tensor(counts))
        ids[torch.rand(len(ids), generator=gen) < 0.02] = -1
        check_exactly(ids[torch.randperm(len(ids), generator=gen)].to(torch.int32), 16, 16, first)


@pytest.mark.parametrize("N,V,D", [(8193, 45_000, 256), (9000, 45_000, 256), (20_000, 90_001, 256), (32_768, 150_000, 256),
                                   (32_769, 150_000, 256), (70_000, 3_000, 24)])
def test_sorts_of_eight_and_sixteen_ctas(N, V, D, cuda_device):
    # eight sort up to 32768 tokens where the gradient has at least 4480 bytes a token
    gen = torch.Generator().manual_seed(N)
    ids = torch.randint(0, V, (N,), generator=gen)
    ids[: N // 3] = torch.randint(0, 50, (N // 3,), generator=gen)
    ids[torch.rand(N, generator=gen) < 0.05] = -1
    check_exactly(ids[torch.randperm(N, generator=gen)].to(torch.int32), V, D, N)


def test_bits_do_not_depend_on_strides_and_alignment(cuda_device):
    for N, V in ((700, 90), (3000, 90), (9000, 300)):
        ids, _, dy = draw(N, V, 72, BF16, N)
        wide = torch.zeros(N, 81, dtype=BF16, device="cuda")
        for off in (1, 8):
            wide[:, off:off + 72] = dy
            assert torch.equal(based_embed_bwd(ids, wide[:, off:off + 72], V), based_embed_bwd(ids, dy, V))
