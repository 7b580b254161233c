"""The gated linear recurrence on the GPU against its 64-bit form (tests/ops_reference.py)."""
import pytest
import torch

import ops_reference as ref
from linear_attention_gb300.ops import SAVE_ROWS, based_scan_bwd, based_scan_fwd, based_scan_step

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def draw(B, T, D, mode, dtype, seed, packed=False):
    gen = torch.Generator().manual_seed(seed)
    f = torch.randn(B, T, D, generator=gen) * 2 + 1.5
    g = f if mode == "sigmoid" else torch.nn.functional.logsigmoid(f)
    x, dy = torch.randn(B, T, D, generator=gen), torch.randn(B, T, D, generator=gen)
    state, dfinal = torch.randn(B, D, generator=gen), torch.randn(B, D, generator=gen)
    g, x, dy = g.to(dtype).cuda(), x.to(dtype).cuda(), dy.to(dtype).cuda()
    if packed:  # parts of one wider tensor
        both = torch.zeros(B, T, 3 * D, dtype=dtype, device="cuda")
        both[..., :D], both[..., D:2 * D], both[..., 2 * D:] = g, x, dy
        g, x, dy = both[..., :D], both[..., D:2 * D], both[..., 2 * D:]
    return g, x, dy, state.cuda(), dfinal.cuda()


def check(g, x, dy, state, dfinal, mode, lengths=None, what=""):
    y, final, saved = based_scan_fwd(g, x, mode=mode, state=state, lengths=lengths, save=True)
    dgate, dx, dstate = based_scan_bwd(g, x, dy, saved, mode=mode, dfinal=dfinal, lengths=lengths)
    torch.cuda.synchronize()
    val, bound = ref.scan(g, x, mode, state, lengths, dy, dfinal)
    for name, got in dict(y=y, final=final, dgate=dgate, dx=dx, dstate=dstate).items():
        ref.assert_within(got, val[name], bound[name], (what, name))


LENGTHS = [1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000, 2049]


@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("mode", ["log", "sigmoid"])
def test_lengths(T, mode, cuda_device):
    for dtype, D in ((BF16, 66), (F32, 35), (F16, 33)):
        check(*draw(2, T, D, mode, dtype, T), mode, what=(T, dtype))


@pytest.mark.parametrize("D", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 130, 200, 1024])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_widths(D, dtype, cuda_device):
    check(*draw(3, 150, D, "sigmoid", dtype, D), "sigmoid", what=(D, dtype))


@pytest.mark.parametrize("B,T,D", [(1, 5000, 64), (40, 70, 256), (1, 700, 2048), (9, 260, 1536), (300, 3, 64)])
def test_shapes_of_the_grid(B, T, D, cuda_device):
    # few and many (batch, channel) blocks for the same work
    for mode in ("log", "sigmoid"):
        check(*draw(B, T, D, mode, BF16, B + T), mode, what=(B, T, D, mode))


@pytest.mark.parametrize("mode", ["log", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_padding_is_not_read_and_keeps_the_state(mode, dtype, cuda_device):
    B, T, D = 8, 333, 70
    g, x, dy, state, dfinal = draw(B, T, D, mode, dtype, 5)
    lengths = torch.tensor([333, 0, 1, 64, 65, 200, -7, 900], dtype=torch.int32, device="cuda")
    for b, n in enumerate(lengths.clamp(0, T).tolist()):
        g[b, n:], x[b, n:], dy[b, n:] = float("nan"), float("inf"), float("-inf")
    check(g, x, dy, state, dfinal, mode, lengths)
    y, final, _ = based_scan_fwd(g, x, mode=mode, state=state, lengths=lengths)
    assert torch.equal(final[1], state[1]) and torch.equal(final[6], state[6])
    assert (y[1] == 0).all() and (y[3, 64:] == 0).all()


@pytest.mark.parametrize("D", [64, 77])
def test_strides_and_broadcasts(D, cuda_device):
    check(*draw(2, 140, D, "sigmoid", BF16, 1, packed=True), "sigmoid", what="packed")
    check(*draw(2, 140, D, "log", F32, 2, packed=True), "log", what="packed")
    # time-major storage, one gate for all batch entries, one for all rows
    g, x, dy, state, dfinal = draw(2, 140, D, "log", BF16, 3)
    tm = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    check(tm(g), tm(x), tm(dy), state, dfinal, "log", what="time-major")
    check(g[:1].expand(2, 140, D), x, dy[:, :1].expand(2, 140, D), state, dfinal, "log", what="broadcast")
    # a start that no wide load can take
    big = torch.zeros(2 * 140 * D + 1, dtype=BF16, device="cuda")
    big[1:] = g.reshape(-1)
    check(big[1:].view(2, 140, D), x, dy, state, dfinal, "log", what="odd start")


def test_extreme_gates(cuda_device):
    inf = float("inf")
    for dtype in (F32, BF16):
        g, x, dy, state, dfinal = draw(1, 200, 64, "sigmoid", dtype, 4)
        g[0, 50], g[0, 60:70], g[0, 199], g[0, 120, 3] = -inf, inf, -1000.0 if dtype == F32 else -300.0, 80.0
        y, final, saved = based_scan_fwd(g, x, state=state, save=True)
        dgate, dx, dstate = based_scan_bwd(g, x, dy, saved, dfinal=dfinal)
        # gates wide open: the state stays and nothing of the input enters
        assert (dx[0, 60:70] == 0).all() and (dgate[0, 60:70] == 0).all()
        val, bound = ref.scan(g, x, "sigmoid", state, None, dy, dfinal)
        for name, got in dict(y=y, final=final, dgate=dgate, dx=dx, dstate=dstate).items():
            ref.assert_within(got, val[name], bound[name], name)
        lg, x, dy, state, dfinal = draw(1, 200, 64, "log", dtype, 4)
        lg[0, 70], lg[0, 80:90] = -inf, 0.0              # clear the state; sum without decay
        check(lg, x, dy, state, dfinal, "log", what="log")
        y, _, _ = based_scan_fwd(lg, x, mode="log", state=state)
        assert torch.equal(y[0, 70], x[0, 70])


def test_nan_stays_in_its_sequence_and_channel(cuda_device):
    g, x, _, state, _ = draw(2, 150, 64, "sigmoid", BF16, 6)
    want, _, _ = based_scan_fwd(g, x, state=state)
    g2, x2 = g.clone(), x.clone()
    g2[0, 20, 5], x2[1, 30, 7] = float("nan"), float("nan")
    got, _, _ = based_scan_fwd(g2, x2, state=state)
    bad = torch.zeros(2, 150, 64, dtype=torch.bool, device="cuda")
    bad[0, 20:, 5], bad[1, 30:, 7] = True, True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


def test_long_sequence_and_determinism(cuda_device):
    g, x, dy, state, dfinal = draw(1, 20011, 34, "sigmoid", BF16, 7)
    check(g, x, dy, state, dfinal, "sigmoid")
    runs = []
    for _ in range(3):
        y, final, saved = based_scan_fwd(g, x, state=state, save=True)
        runs.append((y, final, saved, *based_scan_bwd(g, x, dy, saved, dfinal=dfinal)))
    for other in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(runs[0], other))


def test_split_calls_equal_one_call(cuda_device):
    # a prompt in two parts, the second from the first's last state, in place
    g, x, _, state, _ = draw(2, 500, 96, "sigmoid", F32, 8)
    y, final, _ = based_scan_fwd(g, x, state=state)
    carry = state.clone()
    parts = [based_scan_fwd(g[:, a:b], x[:, a:b], state=carry, final_state=carry)[0] for a, b in ((0, 201), (201, 500))]
    val, bound = ref.scan(g, x, "sigmoid", state)
    ref.assert_within(torch.cat(parts, 1), val["y"], bound["y"], "parts")
    ref.assert_within(carry, val["final"], bound["final"], "carry")


def test_gradient_against_differences(cuda_device):
    # d loss / d inputs by central differences of the kernel's own forward pass, in float32: the
    # step 2^-6 leaves (2^-6)^2 / 6 |f'''| <= 1e-4 of curvature and 2^-18 / 2^-6 of rounding
    B, T, D = 1, 20, 4
    for mode in ("log", "sigmoid"):
        g, x, dy, state, dfinal = draw(B, T, D, mode, F32, 9)

        def loss(g, x, s):
            y, final, _ = based_scan_fwd(g, x, mode=mode, state=s)
            return float((y.double() * dy.double()).sum() + (final.double() * dfinal.double()).sum())

        _, _, saved = based_scan_fwd(g, x, mode=mode, state=state, save=True)
        grads = based_scan_bwd(g, x, dy, saved, mode=mode, dfinal=dfinal)
        for which, t in enumerate((g, x, state)):
            for i in range(0, t.numel(), 7):
                args = [g, x, state]
                vals = []
                for sign in (1, -1):
                    moved = t.clone()
                    moved.view(-1)[i] += sign * 2.0 ** -6
                    args[which] = moved
                    vals.append(loss(*args))
                diff = (vals[0] - vals[1]) / 2.0 ** -5
                got = float(grads[which].reshape(-1)[i])
                scale = float(grads[which].abs().max())
                assert abs(diff - got) <= 2e-3 * max(1.0, scale), (mode, which, i, diff, got)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("mode", ["log", "sigmoid"])
def test_step(dtype, mode, cuda_device):
    for N, D, S in ((1, 1, 1), (1, 1024, 1), (5, 33, 9), (7, 64, 7), (300, 130, 311), (2, 4096, 4)):
        gen = torch.Generator().manual_seed(N * D)
        g, x, _, _, _ = draw(N, 1, D, mode, dtype, N + D)
        g, x = g[:, 0], x[:, 0]
        pool = torch.randn(S, D, generator=gen).cuda()
        slots = torch.randperm(S, generator=gen)[:N].to(torch.int32).cuda()
        val, bound = ref.scan(g[:, None], x[:, None], mode, pool[slots.long()])
        kept = pool.clone()
        y = based_scan_step(g, x, pool, mode=mode, slots=slots)
        ref.assert_within(y[:, None], val["y"], bound["y"], (N, D, "y"))
        ref.assert_within(pool[slots.long()], val["final"], bound["final"], (N, D, "pool"))
        rest = torch.ones(S, dtype=torch.bool)
        rest[slots.long().cpu()] = False
        assert torch.equal(pool[rest.cuda()], kept[rest.cuda()])
        if N == S:  # without slots
            again = kept.clone()
            y2 = based_scan_step(g, x, again, mode=mode)
            val, bound = ref.scan(g[:, None], x[:, None], mode, kept)
            ref.assert_within(y2[:, None], val["y"], bound["y"], (N, D, "no slots"))
            ref.assert_within(again, val["final"], bound["final"], (N, D, "no slots"))


def test_step_idle_slots_and_strides(cuda_device):
    both = torch.randn(4, 200, device="cuda").to(BF16)
    pool = torch.randn(3, 100, device="cuda")
    kept = pool.clone()
    slots = torch.tensor([2, -1, 3, 0], dtype=torch.int32, device="cuda")
    y = based_scan_step(both[:, :100], both[:, 100:], pool, slots=slots)
    assert (y[1] == 0).all() and (y[2] == 0).all() and torch.equal(pool[1], kept[1])
    val, bound = ref.scan(both[[0, 3], None, :100], both[[0, 3], None, 100:], "sigmoid", kept[[2, 0]])
    ref.assert_within(y[[0, 3]][:, None], val["y"], bound["y"], "y")
    ref.assert_within(pool[[2, 0]], val["final"], bound["final"], "pool")


def test_steps_follow_the_scan(cuda_device):
    g, x, _, state, _ = draw(3, 40, 128, "sigmoid", BF16, 12)
    y, final, _ = based_scan_fwd(g, x, state=state)
    pool = state.clone()
    ys = torch.stack([based_scan_step(g[:, t], x[:, t], pool) for t in range(40)], 1)
    val, bound = ref.scan(g, x, "sigmoid", state)
    ref.assert_within(ys, val["y"], bound["y"], "y")
    ref.assert_within(pool, val["final"], bound["final"], "pool")


def test_nothing_is_written_past_the_outputs(cuda_device):
    for B, T, D, dtype in ((2, 77, 33, BF16), (1, 130, 66, BF16), (3, 65, 31, F32)):
        g, x, _, state, _ = draw(B, T, D, "log", dtype, 13)
        n, m = B * T * D, B * D
        buf, fin = torch.full((n + 512,), 7.0, dtype=dtype, device="cuda"), torch.full((m + 256,), 7.0, device="cuda")
        based_scan_fwd(g, x, mode="log", state=state, out=buf[:n].view(B, T, D), final_state=fin[:m].view(B, D))
        assert (buf[n:] == 7).all() and (fin[m:] == 7).all()


def test_side_stream_and_graph(cuda_device):
    g, x, dy, state, dfinal = draw(2, 300, 128, "sigmoid", BF16, 14)
    want = based_scan_fwd(g, x, state=state, save=True)
    wgrad = based_scan_bwd(g, x, dy, want[2], dfinal=dfinal)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = based_scan_fwd(g, x, state=state, save=True, stream=side)
    ggrad = based_scan_bwd(g, x, dy, got[2], dfinal=dfinal, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*want, *wgrad), (*got, *ggrad)))
    pool = state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, gfinal, gsaved = based_scan_fwd(g, x, state=state, save=True)
        gr = based_scan_bwd(g, x, dy, gsaved, dfinal=dfinal)
        st = based_scan_step(g[:, 0], x[:, 0], pool)
    g.copy_(g.flip(1))
    want = based_scan_fwd(g, x, state=state, save=True)
    wgrad = based_scan_bwd(g, x, dy, want[2], dfinal=dfinal)
    wpool = state.clone()
    wst = based_scan_step(g[:, 0], x[:, 0], wpool)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*want, *wgrad, wst, wpool), (gy, gfinal, gsaved, *gr, st, pool)))


def test_offsets_past_32_bits(cuda_device):
    # two batch entries 2^31 + 64 elements apart
    D, T = 64, 70
    far = (1 << 31) + 64
    buf = torch.zeros(far + T * D, dtype=BF16, device="cuda")
    g, x, dy, state, dfinal = draw(2, T, D, "log", BF16, 15)
    wide = buf.as_strided((2, T, D), (far, D, 1))
    wide.copy_(x)
    check(g, wide, dy, state, dfinal, "log", what="far input")
    del buf, wide
    # an output of more than 2^31 elements: constant gates and inputs over all rows
    T = (1 << 25) + 5
    g1 = torch.full((1, 1, D), -0.5, dtype=BF16, device="cuda").expand(1, T, D)
    x1 = torch.full((1, 1, D), 0.25, dtype=BF16, device="cuda").expand(1, T, D)
    y, final, _ = based_scan_fwd(g1, x1, mode="log")
    limit = 0.25 / (1 - torch.exp(torch.tensor(-0.5, dtype=torch.float64)))
    # the fixed point: each row's error of DELTA (a h + u) is summed with ratio a
    allowed = 2.0 ** -20 * float(limit) / (1 - 0.607)
    assert (final.double() - limit.to(final.device)).abs().max() <= allowed
    assert (y[0, -1].double() - limit.to(final.device)).abs().max() <= allowed + ref.half_step(BF16) * float(limit)
    assert torch.equal(y[0, -1], y[0, 1 << 20]) and torch.equal(y[0, (1 << 24) + 3], y[0, -1])


@pytest.mark.parametrize("dtype,D", [(BF16, 34), (BF16, 35), (F32, 33), (F16, 31)])
def test_many_rows_that_start_anywhere(dtype, D, cuda_device):
    # as many tiles as fill the GPU, of rows that no 16-byte word starts on; between them, NaN
    B, T = 320, 660
    for mode in ("log", "sigmoid"):
        g, x, dy, state, dfinal = draw(B, T, D, mode, dtype, 18)
        lengths = torch.arange(B, dtype=torch.int32, device="cuda") * T // (B - 1)
        for lens in (None, lengths):
            check(g, x, dy, state, dfinal, mode, lens, what=(dtype, D, mode))
        wide = torch.full((B, T, D + 5), float("nan"), dtype=dtype, device="cuda")
        wide[:, :, 3:3 + D] = x
        check(g, wide[:, :, 3:3 + D], dy, state, dfinal, mode, lengths, what=(dtype, D, mode, "inner"))


def test_rows_far_apart(cuda_device):
    # rows 2^24 elements apart: a tile's rows span more than 2^32 bytes
    D, T, far = 40, 130, 1 << 24
    for dtype in (BF16, F32):
        g, x, dy, state, dfinal = draw(1, T, D, "sigmoid", dtype, 16)
        buf = torch.zeros((T - 1) * far + D, dtype=dtype, device="cuda")
        wide = buf.as_strided((1, T, D), (T * far, far, 1))
        wide.copy_(x)
        check(g, wide, dy, state, dfinal, "sigmoid", what="far rows")
        del buf, wide


def test_many_batch_entries(cuda_device):
    # more than one axis of the grid takes
    B, T, D = 65535 + 70, 2, 3
    g, x, dy, state, dfinal = draw(B, T, D, "log", BF16, 17)
    check(g, x, dy, state, dfinal, "log", what="many")


def in_a_new_thread(work):
    """What work() returns in a thread of its own, which remembers no shapes of earlier calls."""
    import threading
    got = []
    thread = threading.Thread(target=lambda: got.append(work()))
    thread.start()
    thread.join()
    return got[0]


@pytest.mark.parametrize("B,T,D", [(240, 831, 31), (304, 1535, 31)])
@pytest.mark.parametrize("mode", ["log", "sigmoid"])
def test_bits_do_not_depend_on_the_calls_before(B, T, D, mode, cuda_device):
    # shapes for which another number of CTAs is best with padding than without; decays near 1, so that
    # what the tiles in front pass on is not lost in rounding
    gen = torch.Generator(device="cuda").manual_seed(B)
    g, x, dy = (torch.randn(B, T, D, generator=gen, device="cuda") for _ in range(3))
    g = g + 6 if mode == "sigmoid" else -0.01 * g.abs()
    lengths = torch.randint(0, T + 1, (B,), generator=gen, device="cuda").to(torch.int32)

    def grads(lens):
        y, final, saved = based_scan_fwd(g, x, mode=mode, lengths=lens, save=True)
        return y, final, saved, *based_scan_bwd(g, x, dy, saved, mode=mode, lengths=lens)

    for lens, other in ((lengths, None), (None, lengths)):
        want = in_a_new_thread(lambda: grads(lens))
        got = in_a_new_thread(lambda: (grads(other), grads(lens))[1])
        assert all(torch.equal(p, q) for p, q in zip(want, got))
    # as many rows as there are, told by lengths or not: other CTAs, the same bits
    full = torch.full((B,), T, dtype=torch.int32, device="cuda")
    assert all(torch.equal(p, q) for p, q in zip(in_a_new_thread(lambda: grads(full)), in_a_new_thread(lambda: grads(None))))


@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 33), (BF16, 64), (BF16, 35), (F16, 35)])
def test_growing_log_gates(dtype, D, cuda_device):
    # exp of the gates' sum over a tile, or over sixteen rows, passes float32; what the rows make of it does not:
    # the inputs are zero but for the last few rows, the gradients but for the first few
    for gates, rows in (((3.0, 40.0), (10, 2)), ((0.7, 2.0), (100, 30))):
        g, x, dy, state, dfinal = draw(2, 200, D, "log", dtype, 21)
        for b in range(2):
            n = rows[b] if dtype != F16 else min(rows[b], 2)  # float16 ends at 65504
            g[b], x[b, :-n], dy[b, n:] = gates[b] if dtype != F16 else min(gates[b], 9.0), 0, 0
        check(g, x, dy, 0 * state, 0 * dfinal, "log", what=gates)
    # a channel that grows leaves its neighbours' bits alone
    g, x, dy, state, dfinal = draw(2, 200, D, "log", dtype, 22)
    want = based_scan_fwd(g, x, mode="log", state=state, save=True)
    want = *want, *based_scan_bwd(g, x, dy, want[2], mode="log", dfinal=dfinal)
    g2 = g.clone()
    g2[:, :, 4] = 30.0
    got = based_scan_fwd(g2, x, mode="log", state=state, save=True)
    got = *got, *based_scan_bwd(g2, x, dy, got[2], mode="log", dfinal=dfinal)
    rest = torch.arange(D, device="cuda") != 4
    assert all(torch.equal(p[..., rest], q[..., rest]) for p, q in zip(want, got))


@pytest.mark.parametrize("T", [90, 3000])
def test_growth_of_a_small_state(T, cuda_device):
    # from 1e-30 by a factor of e^1.5 a row, for 80 rows wherever they lie: e^120 in all
    g, x, dy, state, dfinal = draw(3, T, 40, "log", F32, 23)
    g[:], x[:], dy[:] = 0, 0, 0
    for b, first in enumerate((0, 7, T - 80)):
        g[b, first:first + 80] = 1.5
    check(g, x, dy, state * 1e-30, dfinal * 1e-30, "log", what=T)
    g[:, :] = -1.5
    g[1, 0], g[2] = 100.0, 1.4  # e^100 is infinite: a state of zero times it is NaN, in any order
    y, final, _ = based_scan_fwd(g, x, mode="log", state=0 * state)
    assert (y[0] == 0).all() and torch.isnan(y[1]).all() and (y[2] == 0).all() and (final[2] == 0).all()


@pytest.mark.parametrize("dtype,D", [(F32, 33), (BF16, 64)])
def test_growth_that_is_cleared(dtype, D, cuda_device):
    # products over a warp's rows that overflow before a decay of exactly 0, of a state of zero; beside them ordinary
    # channels, and NaN gates that stay NaN
    for at in (3, 9, 70, 150):
        g, x, dy, state, dfinal = draw(2, 200, D, "log", dtype, at)
        g[:, at:at + 6, 1::2], x[:, :at + 6, 1::2], dy[:, at:, 1::2] = 30.0, 0, 0
        g[:, at + 6, 1::2] = -float("inf")
        state[:, 1::2], dfinal[:, 1::2] = 0, 0
        check(g, x, dy, state, dfinal, "log", what=at)
        g[:, at + 8, 0] = float("nan")
        y, final, _ = based_scan_fwd(g, x, mode="log", state=state)
        assert torch.isnan(y[:, at + 8:, 0]).all() and torch.isnan(final[:, 0]).all() and torch.isfinite(y[:, :, 1:]).all()


@pytest.mark.parametrize("mode", ["log", "sigmoid"])
def test_an_infinite_state_stays_infinite(mode, cuda_device):
    # the decays' product over some rows underflows, and 0 times infinity is NaN: no row alone does that
    for dtype, D in ((F32, 64), (BF16, 33), (BF16, 64)):
        g, x, _, state, _ = draw(1, 700, D, mode, dtype, 24)
        want, _, _ = based_scan_fwd(g, x, mode=mode, state=state)
        g[0, :, 3] = -3.0
        x[0, 5, 3] = float("inf")
        got, final, _ = based_scan_fwd(g, x, mode=mode, state=state)
        assert (got[0, 5:, 3] == float("inf")).all() and final[0, 3] == float("inf")
        rest = torch.arange(D, device="cuda") != 3
        assert torch.equal(got[..., rest], want[..., rest])


@pytest.mark.parametrize("mode", ["log", "sigmoid"])
def test_float32_decays_over_their_range(mode, cuda_device):
    # one row from a state of 1 and an input of 0 shows the decay itself. expf is off by 2^-22 at most, the addition by
    # 2^-24, the reciprocal by 2^-23, the multiply-add by 2^-24: 2^-21 in all
    g = torch.linspace(-20, 0 if mode == "log" else 20, 8192, device="cuda").view(8, 1, 1024)
    zero, one = torch.zeros_like(g), torch.ones(8, 1024, device="cuda")
    want = torch.exp(g.double()) if mode == "log" else torch.sigmoid(g.double())
    y, final, _ = based_scan_fwd(g, zero, mode=mode, state=one)
    pool = one.clone()
    z = based_scan_step(g[:, 0], zero[:, 0], pool, mode=mode)
    for got in (y[:, 0], final, z, pool):
        assert ((got.double() - want[:, 0]) / want[:, 0]).abs().max() <= 2.0 ** -21


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mode", ["log", "sigmoid"])
def test_bits_do_not_depend_on_strides_and_alignment(dtype, mode, cuda_device):
    for B, T, D in ((2, 700, 64), (40, 130, 136)):
        g, x, dy, state, dfinal = draw(B, T, D, mode, dtype, 25)
        lengths = torch.arange(B, dtype=torch.int32, device="cuda") * T // B

        def run(g, x, dy, lens):
            y, final, saved = based_scan_fwd(g, x, mode=mode, state=state, lengths=lens, save=True)
            return y, final, saved, *based_scan_bwd(g, x, dy, saved, mode=mode, dfinal=dfinal, lengths=lens)

        for lens in (None, lengths):
            want = run(g, x, dy, lens)
            wide = torch.zeros(B, T, 3 * D + 3, dtype=dtype, device="cuda")
            parts = [wide[..., k * (D + 1):][..., 1:D + 1] for k in range(3)]
            for p, t in zip(parts, (g, x, dy)):
                p.copy_(t)
            assert all(torch.equal(p, q) for p, q in zip(want, run(*parts, lens)))
