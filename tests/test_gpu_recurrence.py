"""GPU parity of the gated linear recurrence (scan, backward, single-token step)
against the 64-bit forms in stack_reference.py, element by element with the
error bounds derived there."""
import math

import pytest
import torch

from tests import stack_reference as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def draw(shape, dtype, seed, la=(1e-3, 1.0)):
    g = torch.Generator().manual_seed(seed)
    lo, hi = math.log(la[0]), math.log(la[1])
    log_alpha = -torch.exp(lo + (hi - lo) * torch.rand(shape, generator=g))
    x = torch.randn(shape, generator=g)
    return log_alpha.to(dtype), x.to(dtype), g


def check_fwd(kda, log_alpha, x, h0, cu=None):
    """log_alpha, x: CPU, dense [N,T,D] or packed [T,D]."""
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    h, end = kda.recurrence_fwd(dev(log_alpha), dev(x), dev(h0), cu_seqlens=dev(cu))
    torch.cuda.synchronize()
    spans = [(n, slice(None)) for n in range(x.shape[0])] if cu is None else \
        [(None, slice(int(b), int(e))) for b, e in zip(cu[:-1], cu[1:])]
    for i, (n, s) in enumerate(spans):
        la_i, x_i, h_i = (t[s] if n is None else t[n] for t in (log_alpha, x, h))
        (want, slack), (want_end, slack_end) = R.recurrence_fwd(la_i, x_i, None if h0 is None else h0[i])
        R.close(h_i, want, slack, f"h of sequence {i}")
        R.close(end[i], want_end, slack_end, f"h_T of sequence {i}")
    return h, end


def check_bwd(kda, log_alpha, h, h0, dh, dh_T, cu=None):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    g = kda.recurrence_bwd(dev(log_alpha), dev(h), dev(h0), dev(dh), dev(dh_T), cu_seqlens=dev(cu))
    torch.cuda.synchronize()
    spans = [(n, slice(None)) for n in range(h.shape[0])] if cu is None else \
        [(None, slice(int(b), int(e))) for b, e in zip(cu[:-1], cu[1:])]
    for i, (n, s) in enumerate(spans):
        pick = lambda t: t[s] if n is None else t[n]  # noqa: E731
        want = R.recurrence_bwd(pick(log_alpha), pick(h), None if h0 is None else h0[i], pick(dh),
                                None if dh_T is None else dh_T[i])
        R.close(pick(g["dx"]), *want["dx"], f"dx of sequence {i}")
        R.close(pick(g["dlog_alpha"]), *want["dlog_alpha"], f"dlog_alpha of sequence {i}")
        R.close(g["dh0"][i], *want["dh0"], f"dh0 of sequence {i}")
    return g


SHAPES = [(1, 1, 1), (2, 1, 64), (1, 2, 7), (3, 31, 8), (1, 127, 100), (2, 128, 64), (1, 129, 65), (2, 300, 37),
          (1, 513, 136), (1, 1025, 40), (5, 64, 513), (1, 3000, 4), (2, 700, 1001)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_and_backward(cuda_lib, dtype, shape):
    N, T, D = shape
    log_alpha, x, g = draw(shape, DT[dtype], 11 + T)
    h0 = torch.randn(N, D, generator=g)
    h, _ = check_fwd(cuda_lib, log_alpha, x, h0)
    check_fwd(cuda_lib, log_alpha, x, None)
    dh, dT = torch.randn(shape, generator=g).to(DT[dtype]), torch.randn(N, D, generator=g)
    check_bwd(cuda_lib, log_alpha, h.cpu(), h0, dh, dT)
    check_bwd(cuda_lib, log_alpha, h.cpu(), None, dh, None)


@pytest.mark.parametrize("lens", [[5], [0], [0, 1, 130, 0, 17], [128, 128, 1, 257], [1] * 40, [900, 3, 0], [0, 3000, 1, 700]])
@pytest.mark.parametrize("D", [8, 50, 192])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed(cuda_lib, dtype, D, lens):
    T, N = sum(lens), len(lens)
    log_alpha, x, g = draw((T, D), DT[dtype], 3 + T)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    h0 = torch.randn(N, D, generator=g)
    h, _ = check_fwd(cuda_lib, log_alpha, x, h0, cu)
    dh, dT = torch.randn(T, D, generator=g).to(DT[dtype]), torch.randn(N, D, generator=g)
    check_bwd(cuda_lib, log_alpha, h.cpu(), h0, dh, dT, cu)


@pytest.mark.parametrize("lens", [[700, 0, 1500, 20, 900], [600, 600, 600, 600, 600]])
def test_packed_many_rows(cuda_lib, lens):
    """Rows enough for one large CTA each, the longest sequences first, ties among them."""
    T, N, D = sum(lens), len(lens), 1000
    log_alpha, x, g = draw((T, D), torch.bfloat16, 4 + T)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    h0 = torch.randn(N, D, generator=g)
    h, _ = check_fwd(cuda_lib, log_alpha, x, h0, cu)
    check_bwd(cuda_lib, log_alpha, h.cpu(), h0, x, h0, cu)


def test_packed_more_sequences_than_threads(cuda_lib):
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(0, 12, (700,), generator=g).tolist()
    T = sum(lens)
    log_alpha, x, g = draw((T, 24), torch.float32, 7)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    check_fwd(cuda_lib, log_alpha, x, torch.randn(700, 24, generator=g), cu)


def test_packed_equals_dense_bits(cuda_lib):
    log_alpha, x, g = draw((3, 200, 72), torch.bfloat16, 5)
    h0 = torch.randn(3, 72, generator=g).cuda()
    dense = cuda_lib.recurrence_fwd(log_alpha.cuda(), x.cuda(), h0)
    cu = torch.tensor([0, 200, 400, 600], dtype=torch.int32, device="cuda")
    packed = cuda_lib.recurrence_fwd(log_alpha.cuda().view(600, 72), x.cuda().view(600, 72), h0, cu_seqlens=cu)
    assert torch.equal(dense[0].view(600, 72), packed[0]) and torch.equal(dense[1], packed[1])


def test_packed_bad_offsets_stay_inside(cuda_lib):
    """Offsets outside [0, T] are clamped, a decreasing pair is empty, tokens of no sequence keep what they held."""
    log_alpha, x, g = draw((100, 24), torch.float32, 6)
    h0 = torch.randn(4, 24, generator=g)
    cu = torch.tensor([-5, 20, 10, 60, 900], dtype=torch.int32)  # [0,20), empty, [10,60), [60,100)
    h = torch.full((100, 24), 7.0, device="cuda")
    h, end = cuda_lib.recurrence_fwd(log_alpha.cuda(), x.cuda(), h0.cuda(), cu_seqlens=cu.cuda(), h=h)
    (want, slack), (we, se) = R.recurrence_fwd(log_alpha[60:], x[60:], h0[3])
    R.close(h[60:], want, slack)
    R.close(end[3], we, se)
    assert torch.equal(end[1].cpu(), h0[1])
    cu = torch.tensor([0, 30, 30, 30, 40], dtype=torch.int32)
    h = torch.full((100, 24), 7.0, device="cuda")
    cuda_lib.recurrence_fwd(log_alpha.cuda(), x.cuda(), None, cu_seqlens=cu.cuda(), h=h)
    assert (h[40:] == 7.0).all() and (h[:40] != 7.0).any(1).all()


@pytest.mark.parametrize("T", [0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_sequences_pass_the_state(cuda_lib, dtype, T):
    e = torch.empty(2, T, 40, dtype=DT[dtype], device="cuda")
    h0 = torch.randn(2, 40, device="cuda")
    h, end = cuda_lib.recurrence_fwd(e, e, h0)
    assert h.shape == (2, 0, 40) and torch.equal(end, h0)
    _, end = cuda_lib.recurrence_fwd(e, e)
    assert end.abs().max() == 0
    g = cuda_lib.recurrence_bwd(e, e, h0, e, h0 + 1)
    assert torch.equal(g["dh0"], h0 + 1)
    z = torch.empty(0, 5, 40, dtype=DT[dtype], device="cuda")
    h, end = cuda_lib.recurrence_fwd(z, z)
    assert h.shape == (0, 5, 40) and end.shape == (0, 40)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, -1e-4, -0.5, -30.0, -math.inf])
def test_decay_extremes(cuda_lib, decay, dtype):
    N, T, D = 1, 2100, 16
    g = torch.Generator().manual_seed(9)
    log_alpha = torch.full((N, T, D), decay).to(DT[dtype])
    x, h0 = torch.randn(N, T, D, generator=g).to(DT[dtype]), torch.randn(N, D, generator=g)
    h, _ = check_fwd(cuda_lib, log_alpha, x, h0)
    check_bwd(cuda_lib, log_alpha, h.cpu(), h0, x, h0)


def test_resets_inside_a_sequence(cuda_lib):
    log_alpha, x, g = draw((2, 400, 48), torch.float32, 21)
    log_alpha[:, ::37] = -math.inf
    log_alpha[1, :, 5] = -math.inf
    h0 = torch.randn(2, 48, generator=g)
    h, _ = check_fwd(cuda_lib, log_alpha, x, h0)
    check_bwd(cuda_lib, log_alpha, h.cpu(), h0, x, h0)


def test_nan_stays_in_its_channel(cuda_lib):
    log_alpha, x, _ = draw((1, 300, 64), torch.float32, 22)
    clean, _ = cuda_lib.recurrence_fwd(log_alpha.cuda(), x.cuda())
    x[0, 150, 9] = math.nan
    h, _ = cuda_lib.recurrence_fwd(log_alpha.cuda(), x.cuda())
    bad = torch.isnan(h)
    assert bad[0, 150:, 9].all() and bad.sum() == 150
    keep = ~bad
    assert torch.equal(h[keep], clean[keep])


@pytest.mark.parametrize("N,T,D", [(1, 20000, 64), (1, 9001, 1000), (2, 5000, 30), (1, 6000, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_sequences_on_few_channels(cuda_lib, dtype, N, T, D):
    log_alpha, x, g = draw((N, T, D), DT[dtype], 31)
    h0 = torch.randn(N, D, generator=g)
    h, _ = check_fwd(cuda_lib, log_alpha, x, h0)
    check_bwd(cuda_lib, log_alpha, h.cpu(), h0, x, h0)


def test_states_chain_in_place(cuda_lib):
    log_alpha, x, g = draw((2, 500, 80), torch.float32, 41)
    h0 = torch.randn(2, 80, generator=g)
    state, parts = h0.cuda(), []
    for b, e in ((0, 1), (1, 129), (129, 500)):
        h, out = cuda_lib.recurrence_fwd(log_alpha[:, b:e].contiguous().cuda(), x[:, b:e].contiguous().cuda(), state, h_T=state)
        assert out is state
        parts.append(h)
    for n in range(2):
        (want, slack), (we, se) = R.recurrence_fwd(log_alpha[n], x[n], h0[n])
        R.close(torch.cat(parts, 1)[n], want, 2 * slack)  # each part adds a bound of its own, two at most overlap
        R.close(state[n], we, 2 * se)


def test_outputs_over_inputs(cuda_lib):
    log_alpha, x, g = draw((2, 333, 72), torch.bfloat16, 42)
    la, xd, h0 = log_alpha.cuda(), x.cuda(), torch.randn(2, 72, generator=g).cuda()
    want = cuda_lib.recurrence_fwd(la, xd, h0)
    over = xd.clone()
    h, _ = cuda_lib.recurrence_fwd(la, over, h0, h=over)
    assert h is over and torch.equal(h, want[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 7), (64, 128), (5, 1001), (256, 4096)])
def test_step(cuda_lib, dtype, N, D):
    log_alpha, x, g = draw((N, D), DT[dtype], 51)
    h0 = torch.randn(N, D, generator=g)
    want = log_alpha.double().exp() * h0.double() + x.double()
    slack = 8 * R.U * (want.abs() + h0.double().abs() + x.double().abs())
    state = h0.cuda()
    y, out = cuda_lib.recurrence_step(log_alpha.cuda(), x.cuda(), state)
    assert out is state
    R.close(state, want, slack)
    R.close(y, want, slack)
    keep = h0.cuda()
    y2, out = cuda_lib.recurrence_step(log_alpha.cuda(), x.cuda(), keep, h_out=torch.empty_like(keep))
    assert torch.equal(out, state) and torch.equal(y, y2) and torch.equal(keep.cpu(), h0)


def test_steps_follow_the_scan(cuda_lib):
    log_alpha, x, g = draw((4, 60, 96), torch.float32, 52)
    h0 = torch.randn(4, 96, generator=g)
    state = h0.cuda()
    ys = [cuda_lib.recurrence_step(log_alpha[:, t].contiguous().cuda(), x[:, t].contiguous().cuda(), state)[0] for t in range(60)]
    for n in range(4):
        (want, slack), _ = R.recurrence_fwd(log_alpha[n], x[n], h0[n])
        R.close(torch.stack(ys, 1)[n], want, slack)


def test_equal_bits_and_streams_and_graphs(cuda_lib):
    log_alpha, x, g = draw((2, 1500, 200), torch.bfloat16, 61)
    la, xd, h0 = log_alpha.cuda(), x.cuda(), torch.randn(2, 200, generator=g).cuda()
    want = cuda_lib.recurrence_fwd(la, xd, h0)
    grads = cuda_lib.recurrence_bwd(la, want[0], h0, xd, h0)
    for _ in range(3):
        again = cuda_lib.recurrence_fwd(la, xd, h0)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, end = torch.empty_like(xd), torch.empty_like(h0)
    cuda_lib.recurrence_fwd(la, xd, h0, h=h, h_T=end, stream=side)
    side.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(end, want[1])
    graph = torch.cuda.CUDAGraph()
    la2, x2, s2 = torch.zeros_like(la), torch.zeros_like(xd), torch.zeros_like(h0)
    with torch.cuda.graph(graph):
        got, got_end = cuda_lib.recurrence_fwd(la2, x2, s2)
        g2 = cuda_lib.recurrence_bwd(la2, got, s2, x2, s2)
    la2.copy_(la), x2.copy_(xd), s2.copy_(h0)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want[0]) and torch.equal(got_end, want[1])
        for name in grads:
            assert torch.equal(g2[name], grads[name]), name


def test_a_wait_that_gives_up_is_reported(cuda_lib):
    """The first CTA of each cluster sends nothing: the others' waits run out, the status says so once, and a call after
    it is right."""
    import time
    log_alpha, x, _ = draw((1, 4000, 100), torch.bfloat16, 81)
    la, xd = log_alpha.cuda(), x.cuda()
    assert cuda_lib.recurrence_status() == 0
    torch.cuda.synchronize()
    began = time.perf_counter()
    cuda_lib.recurrence_timeout_test(la, xd, h=torch.empty_like(xd), wait_budget_cycles=1 << 20)
    assert cuda_lib.recurrence_status() == 4
    assert time.perf_counter() - began < 1.0
    assert cuda_lib.recurrence_status() == 0
    check_fwd(cuda_lib, log_alpha, x, None)
    assert cuda_lib.recurrence_status() == 0


@pytest.mark.parametrize("rows", [1, 6, 7, 14, 15, 16, 17, 34, 35, 74, 75, 148, 149])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_cluster_size(cuda_lib, dtype, rows):
    """The numbers of rows (slices of 128 bytes of channels) at which another split is taken."""
    D = rows * (64 if dtype == "bf16" else 32)
    log_alpha, x, g = draw((1, 2600, D), DT[dtype], 90 + rows)
    h0 = torch.randn(1, D, generator=g)
    h, _ = check_fwd(cuda_lib, log_alpha, x, h0)
    check_bwd(cuda_lib, log_alpha, h.cpu(), h0, x, h0)


def test_offsets_past_32_bits(cuda_lib):
    """More than 2^31 elements: the last tokens of the last channels, whose memory is a few tokens."""
    T, D, tail = 530000, 4104, 100
    g = torch.Generator(device="cuda").manual_seed(71)
    la = torch.empty(1, T, D, dtype=torch.bfloat16, device="cuda").uniform_(-3, -1, generator=g)
    x = torch.empty(1, T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    h, end = cuda_lib.recurrence_fwd(la, x)
    (want, slack), (we, se) = R.recurrence_fwd(la[0, -tail:, -50:].cpu(), x[0, -tail:, -50:].cpu())
    R.close(h[0, -40:, -50:], want[-40:], slack[-40:] + 1e-20)  # exp(-60) of what came before
    R.close(end[0, -50:], we, se + 1e-20)
    grads = cuda_lib.recurrence_bwd(la, h, None, x)
    w = R.recurrence_bwd(la[0, -tail:, -50:].cpu(), h[0, -tail:, -50:].cpu(), None, x[0, -tail:, -50:].cpu())
    R.close(grads["dx"][0, -tail + 1:, -50:], w["dx"][0][1:], w["dx"][1][1:])
    R.close(grads["dlog_alpha"][0, -tail + 1:, -50:], w["dlog_alpha"][0][1:], w["dlog_alpha"][1][1:])


def test_refusals(cuda_lib):
    la = torch.zeros(2, 8, 16, device="cuda")
    with pytest.raises(ValueError, match="x: expected"):
        cuda_lib.recurrence_fwd(la, la[:, :4].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        cuda_lib.recurrence_fwd(la, la.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError, match="x: expected"):
        cuda_lib.recurrence_fwd(la, la.bfloat16())
    with pytest.raises(TypeError):
        cuda_lib.recurrence_fwd(la.half(), la.half())
    with pytest.raises(ValueError, match="h0"):
        cuda_lib.recurrence_fwd(la, la, torch.zeros(2, 16, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="packed"):
        cuda_lib.recurrence_fwd(la, la, cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="cu_seqlens"):
        cuda_lib.recurrence_fwd(la[0], la[0], cu_seqlens=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="dense|B,T,D"):
        cuda_lib.recurrence_fwd(la[0], la[0])
    odd = torch.zeros(2 * 8 * 16 + 1, device="cuda")[1:].view(2, 8, 16)
    with pytest.raises(cuda_lib.KDAError, match="misaligned"):
        cuda_lib.recurrence_fwd(odd, la)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays(cuda_lib, dtype):
    """h = exp(log_alpha) from a state of 1 shows the decays of the scan, its backward pass and the step, at all bf16 values
    from -2^-24 to -87. expf is off by 2 U = 2^-23 at most. The scans' 2^(x log2 e) of bf16 inputs: 4 U by the instruction;
    log2 e and the product are rounded by U each, of an exponent y = |x| log2 e, and 2^y is off by ln 2 y of that: 2 |x| U."""
    bits = torch.arange(0xB380, 0xC2AE + 1, dtype=torch.int32).to(torch.int16)
    la = bits.view(torch.bfloat16).to(DT[dtype])[None, None]
    D = la.shape[-1]
    one, zero = torch.ones(1, D, device="cuda"), torch.zeros(1, 1, D, dtype=DT[dtype], device="cuda")
    h, end = cuda_lib.recurrence_fwd(la.cuda(), zero, one)
    grads = cuda_lib.recurrence_bwd(la.cuda(), h, one, zero, one)
    _, step = cuda_lib.recurrence_step(la[0].cuda(), zero[0], one, h_out=torch.empty_like(one))
    x = la[0].double()
    scan = 2 * R.U if dtype == "f32" else (4 + 2 * x.abs()) * R.U
    for got, bound, what in ((end, scan, "scan"), (grads["dh0"], scan, "backward"), (step, 2 * R.U, "step")):
        off = (got.cpu().double() / x.exp() - 1).abs()
        assert bool((off <= bound).all()), (what, float((off / R.U).max()))


@pytest.mark.parametrize("D", [24, 25, 26])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_in_given_memory(cuda_lib, dtype, D):
    """dx over dh; tokens of no sequence keep what dx and dlog_alpha held, before the first sequence and behind the last."""
    log_alpha, x, g = draw((100, D), DT[dtype], 43)
    cu = torch.tensor([7, 30, 30, 71], dtype=torch.int32).cuda()
    h0, dT = (torch.randn(3, D, generator=g).cuda() for _ in range(2))
    la, xd = log_alpha.cuda(), x.cuda()
    h, _ = cuda_lib.recurrence_fwd(la, xd, h0, cu_seqlens=cu, h=torch.zeros_like(xd))
    want = cuda_lib.recurrence_bwd(la, h, h0, xd, dT, cu_seqlens=cu)
    dx, dla = xd.clone(), torch.full_like(la, 7.0)
    got = cuda_lib.recurrence_bwd(la, h, h0, dx, dT, cu_seqlens=cu, dx=dx, dlog_alpha=dla)
    assert got["dx"] is dx and got["dlog_alpha"] is dla and torch.equal(got["dh0"], want["dh0"])
    for name, before in (("dx", xd), ("dlog_alpha", torch.full_like(la, 7.0))):
        assert torch.equal(got[name][7:71], want[name][7:71]), name
        for outside in (slice(0, 7), slice(71, 100)):
            assert torch.equal(got[name][outside], before[outside]), name
    with pytest.raises(ValueError, match="dx: expected"):
        cuda_lib.recurrence_bwd(la, h, h0, xd, dT, cu_seqlens=cu, dx=dx[:50])
    with pytest.raises(ValueError, match="dlog_alpha: expected"):
        cuda_lib.recurrence_bwd(la, h, h0, xd, dT, cu_seqlens=cu, dlog_alpha=dla.double())
