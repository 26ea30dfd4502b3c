"""GPU parity of the paged decode attention against the 64-bit form in
stack_reference.py."""
import math

import pytest
import torch

from tests import stack_reference as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(lens, Hq, Hk, d, page, dtype, seed, spare=2, poison=False, std=1.0):
    """A cache whose pages are dealt out in a random order; with `poison` every row that no sequence holds is NaN."""
    g = torch.Generator().manual_seed(seed)
    dt, N = DT[dtype], len(lens)
    held = [max(0, l) // page + 1 for l in lens]
    pool = sum(held) + spare
    table = torch.full((N, max(held)), -1, dtype=torch.int32)
    ids = torch.randperm(pool, generator=g).to(torch.int32)
    at = 0
    for n, m in enumerate(held):
        table[n, :m] = ids[at:at + m]
        at += m
    kc, vc = (torch.randn(pool, Hk, page, d, generator=g).to(dt) for _ in range(2))
    if poison:
        keep = torch.zeros(pool, page, dtype=torch.bool)
        for n, l in enumerate(lens):
            for p in range(max(0, l)):
                keep[int(table[n, p // page]), p % page] = True
        for c in (kc, vc):
            c.masked_fill_(~keep[:, None, :, None], math.nan)
    q = (std * torch.randn(N, Hq, d, generator=g)).to(dt)
    k, v = (torch.randn(N, Hk, d, generator=g).to(dt) for _ in range(2))
    return {"q": q, "kc": kc, "vc": vc, "table": table, "lens": torch.tensor(lens, dtype=torch.int32), "k": k, "v": v}


def check(kda, s, put=True, window=0, scale=None):
    c = {n: t.cuda() for n, t in s.items()}
    o, lse = kda.attn_decode(c["q"], c["kc"], c["vc"], c["table"], c["lens"], k=c["k"] if put else None,
                             v=c["v"] if put else None, window=window, scale=scale, return_lse=True)
    torch.cuda.synchronize()
    kc, vc = s["kc"].clone(), s["vc"].clone()
    want_o, want_lse = R.attn_decode(s["q"], kc, vc, s["table"], s["lens"], s["k"] if put else None, s["v"] if put else None, scale, window)
    R.close(o, *want_o, "o")
    R.close(lse, *want_lse, "lse")
    for got, want in ((c["kc"], kc), (c["vc"], vc)):  # the new tokens put, every other row as it was
        assert torch.equal(got.cpu().nan_to_num(nan=77.0), want.nan_to_num(nan=77.0))
    return o, lse


@pytest.mark.parametrize("put", [True, False])
@pytest.mark.parametrize("lens", [[0], [1], [15], [16], [17], [63, 64, 65], [127, 128, 129, 0], [300, 2, -1, 0, 33], [1000]])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lengths(cuda_lib, dtype, d, lens, put):
    check(cuda_lib, make(lens, 4, 2, d, 16, dtype, 3 + sum(lens), poison=True), put)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (8, 1), (16, 1), (17, 1), (40, 1), (5, 5), (16, 16), (12, 4), (20, 4), (56, 8), (64, 2)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_groups(cuda_lib, dtype, Hq, Hk):
    check(cuda_lib, make([70, 0, 201], Hq, Hk, 64, 32, dtype, 5 + Hq, poison=True))
    check(cuda_lib, make([70, 129], Hq, Hk, 128, 32, dtype, 6 + Hq))


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 48, 64, 100, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_page_sizes(cuda_lib, dtype, page):
    check(cuda_lib, make([0, 99, 100, 255, 256, 380], 6, 2, 64, page, dtype, 7 + page, poison=True))


@pytest.mark.parametrize("window", [1, 2, 16, 50, 64, 65, 300, 5000])
@pytest.mark.parametrize("put", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_windows(cuda_lib, dtype, put, window):
    check(cuda_lib, make([0, 1, 64, 70, 333, -1], 8, 2, 128, 48, dtype, 8, poison=True), put, window)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,Hq,Hk", [([20000], 4, 1), ([9000, 1, 300], 8, 2), ([5000] * 3, 16, 8)])
def test_long_contexts(cuda_lib, dtype, lens, Hq, Hk):
    """Few rows and long contexts: the work is split over the length."""
    check(cuda_lib, make(lens, Hq, Hk, 64, 64, dtype, 9))
    check(cuda_lib, make(lens, Hq, Hk, 128, 16, dtype, 10), window=4097)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(cuda_lib, dtype):
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(-1, 260, (333,), generator=g).tolist()
    check(cuda_lib, make(lens, 6, 3, 64, 16, dtype, 12))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sharp_scores(cuda_lib, dtype):
    """Scores that differ by hundreds: the running maximum moves and most weights vanish."""
    check(cuda_lib, make([700, 40], 8, 2, 128, 16, dtype, 13, std=30.0))
    check(cuda_lib, make([700, 40], 8, 2, 128, 16, dtype, 14), scale=3.0)
    check(cuda_lib, make([700, 40], 8, 2, 128, 16, dtype, 14), scale=0.0)
    check(cuda_lib, make([700, 40], 8, 2, 128, 16, dtype, 14), scale=-0.2)


def test_bad_pages_are_not_attended(cuda_lib):
    for dtype in ("f32", "bf16"):
        s = make([100, 100, 100, 15], 4, 2, 64, 16, dtype, 15)
        s["table"][0, 2] = -1                 # a hole
        s["table"][1, 3] = 1 << 30            # far outside the cache
        s["table"][2, 6] = s["kc"].shape[0]   # the page of the new token: one past the last
        s["table"][3, 0] = -7                 # the only page: an empty row
        o, lse = check(cuda_lib, s)
        assert o[3].abs().max() == 0 and torch.isinf(lse[3]).all()


def test_lengths_past_the_table(cuda_lib):
    for dtype in ("f32", "bf16"):
        s = make([64, 64, 64], 4, 2, 64, 16, dtype, 16)
        s["lens"] = torch.tensor([79, 80, 2_000_000_000], dtype=torch.int32)  # room for 80 positions
        s["table"] = torch.arange(15, dtype=torch.int32).view(3, 5)
        check(cuda_lib, s)
        check(cuda_lib, s, put=False)
        check(cuda_lib, s, window=30)
        s["lens"] = torch.tensor([-5, -2147483648, 2147483647], dtype=torch.int32)
        check(cuda_lib, s)


def test_shared_prefix_pages(cuda_lib):
    """Two sequences read the same full pages and end in pages of their own."""
    s = make([70, 90], 8, 2, 128, 16, "bf16", 17)
    s["table"][1, :4] = s["table"][0, :4]
    check(cuda_lib, s)


def test_infinite_keys(cuda_lib):
    """A score of -infinity drops its position; a row with no other gives 0."""
    for dtype in ("f32", "bf16"):
        s = make([40, 0], 2, 1, 64, 16, dtype, 18)
        s["q"] = s["q"].abs()
        s["kc"][int(s["table"][0, 0]), 0, 3] = -math.inf
        s["k"][1] = -math.inf
        c = {n: t.cuda() for n, t in s.items()}
        o, lse = cuda_lib.attn_decode(c["q"], c["kc"], c["vc"], c["table"], c["lens"], k=c["k"], v=c["v"], return_lse=True)
        assert o[1].abs().max() == 0 and (lse[1] == -math.inf).all()
        s["kc"][int(s["table"][0, 0]), 0, 3] = -1e4  # as good as dropped
        kc, vc = s["kc"].clone(), s["vc"].clone()
        (want, slack), _ = R.attn_decode(s["q"][:1], kc, vc, s["table"][:1], s["lens"][:1], s["k"][:1], s["v"][:1])
        (_, calm), _ = R.attn_decode(s["q"][:1], kc * (kc.abs() < 1e3), vc, s["table"][:1], s["lens"][:1], s["k"][:1], s["v"][:1])
        R.close(o[:1], want, 4 * calm)  # the finite keys set the scores' error


def test_infinite_values(cuda_lib):
    """An attended infinity comes out as one where its weight is positive, and stays in its channel."""
    for dtype in ("f32", "bf16"):
        s = make([40], 4, 2, 64, 16, dtype, 23)
        s["vc"][int(s["table"][0, 1]), 0, 5, 7] = math.inf
        s["vc"][int(s["table"][0, 1]), 1, 5, 9] = -math.inf
        c = {n: t.cuda() for n, t in s.items()}
        o = cuda_lib.attn_decode(c["q"], c["kc"], c["vc"], c["table"], c["lens"], k=c["k"], v=c["v"])
        assert (o[0, :2, 7] == math.inf).all() and (o[0, 2:, 9] == -math.inf).all()
        o[0, :2, 7] = o[0, 2:, 9] = 0
        assert torch.isfinite(o).all()


def test_decode_loop_fills_the_cache(cuda_lib):
    """From an empty cache, token by token: each step equals attention over what came before."""
    N, Hq, Hk, d, page, steps = 3, 8, 2, 64, 16, 40
    g = torch.Generator().manual_seed(19)
    table = torch.randperm(9, generator=g).to(torch.int32).view(3, 3)
    kc, vc = (torch.full((9, Hk, page, d), math.nan) for _ in range(2))
    kg, vg, lens = kc.bfloat16().cuda(), vc.bfloat16().cuda(), torch.zeros(N, dtype=torch.int32, device="cuda")
    kc, vc = kc.bfloat16(), vc.bfloat16()
    for t in range(steps):
        q, k, v = (torch.randn(N, h, d, generator=g).bfloat16() for h in (Hq, Hk, Hk))
        o = cuda_lib.attn_decode(q.cuda(), kg, vg, table.cuda(), lens, k=k.cuda(), v=v.cuda())
        want, _ = R.attn_decode(q, kc, vc, table, [t] * N, k, v)
        R.close(o, *want, f"step {t}")
        lens += 1


def test_equal_bits_streams_and_graphs(cuda_lib):
    s = {n: t.cuda() for n, t in make([3000, 10, 777, -1], 16, 4, 128, 32, "bf16", 20).items()}

    def call(c, **kw):
        return cuda_lib.attn_decode(c["q"], c["kc"], c["vc"], c["table"], c["lens"], k=c["k"], v=c["v"], return_lse=True, **kw)

    want = call(s)
    for _ in range(3):
        again = call(s)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, ws = torch.empty_like(want[0]), torch.empty(max(16, cuda_lib.attn_decode_workspace_size(4, 16, 4, 128)), dtype=torch.uint8, device="cuda")
    call(s, o=o, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(o, want[0])
    # two graphs with one workspace, replayed in turn on one stream; lengths change between replays
    other = {n: t.cuda() for n, t in make([5, 2000, 64, 500], 16, 4, 128, 32, "bf16", 21).items()}
    want2 = call(other)
    ws.fill_(255)
    graphs = []
    for c in (s, other):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(c, workspace=ws)
        graphs.append((graph, out))
    for _ in range(2):
        for (graph, out), w in zip(graphs, (want, want2)):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])
    other["lens"].copy_(torch.tensor([1, 900, 60, -1]))
    graphs[1][0].replay()
    torch.cuda.synchronize()
    fresh = call(other)
    assert torch.equal(graphs[1][1][0], fresh[0]) and torch.equal(graphs[1][1][1], fresh[1])


def test_two_streams_at_once(cuda_lib):
    sets = [{n: t.cuda() for n, t in make([4000, 100 + i], 8, 2, 128, 16, "bf16", 22 + i).items()} for i in range(2)]
    want = [cuda_lib.attn_decode(c["q"], c["kc"], c["vc"], c["table"], c["lens"], k=c["k"], v=c["v"]) for c in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (c, st) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(st):
                got[i].append(cuda_lib.attn_decode(c["q"], c["kc"], c["vc"], c["table"], c["lens"], k=c["k"], v=c["v"]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_offsets_past_32_bits(cuda_lib):
    """A cache of more than 2^31 elements, pages at its end."""
    pages, page, d = 140000, 128, 128
    kc, vc = (torch.zeros(pages, 1, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(31)
    small = make([300, 129], 4, 1, d, page, "bf16", 32, spare=0)
    n_small = small["kc"].shape[0]
    base = pages - n_small
    kc[base:], vc[base:] = small["kc"].cuda(), small["vc"].cuda()
    table = torch.where(small["table"] >= 0, small["table"] + base, small["table"])
    o = cuda_lib.attn_decode(small["q"].cuda(), kc, vc, table.cuda(), small["lens"].cuda(), k=small["k"].cuda(), v=small["v"].cuda())
    k2, v2 = small["kc"].clone(), small["vc"].clone()
    want, _ = R.attn_decode(small["q"], k2, v2, small["table"], small["lens"], small["k"], small["v"])
    R.close(o, *want)
    assert torch.equal(kc[base:].cpu(), k2) and torch.equal(vc[base:].cpu(), v2)
    assert not kc[:base].any() and not vc[:base].any()
    del g


def test_no_rows_and_no_pages(cuda_lib):
    z = torch.zeros(0, 4, 64, device="cuda")
    cache = torch.zeros(3, 2, 16, 64, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    assert cuda_lib.attn_decode(z, cache, cache.clone(), torch.zeros(0, 2, **i32), torch.zeros(0, **i32)).shape == (0, 4, 64)
    q = torch.randn(2, 4, 64, device="cuda")
    none = torch.zeros(0, 2, 16, 64, device="cuda")
    o, lse = cuda_lib.attn_decode(q, none, none.clone(), torch.zeros(2, 0, **i32), torch.tensor([0, 9], **i32), return_lse=True)
    assert o.abs().max() == 0 and torch.isinf(lse).all()
    o = cuda_lib.attn_decode(q, none, none.clone(), torch.zeros(2, 3, **i32), torch.tensor([0, 9], **i32))
    assert o.abs().max() == 0


def test_refusals(cuda_lib):
    s = {n: t.cuda() for n, t in make([20, 3], 4, 2, 64, 16, "bf16", 40).items()}
    f = lambda **kw: cuda_lib.attn_decode(*[{**s, **kw}[n] for n in ("q", "kc", "vc", "table", "lens")], k=kw.get("k"), v=kw.get("v"))  # noqa: E731
    with pytest.raises(ValueError, match="both or neither"):
        f(k=s["k"])
    with pytest.raises(ValueError, match="v_cache"):
        f(vc=s["vc"][:1])
    with pytest.raises(ValueError, match="k_cache"):
        f(kc=s["kc"].float())
    with pytest.raises(ValueError, match="seq_lens"):
        f(lens=s["lens"].long())
    with pytest.raises(ValueError, match="page_table"):
        f(table=s["table"][:1])
    with pytest.raises(ValueError, match="k: expected"):
        f(k=s["k"][:, :1].contiguous(), v=s["v"])
    with pytest.raises(cuda_lib.KDAError, match="INVALID"):
        f(q=s["q"][:, :3].contiguous())
    with pytest.raises(cuda_lib.KDAError, match="UNSUPPORTED"):
        f(q=s["q"][..., :32].contiguous(), kc=s["kc"][..., :32].contiguous(), vc=s["vc"][..., :32].contiguous())
    with pytest.raises(cuda_lib.KDAError, match="INVALID"):
        cuda_lib.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], window=-1)
    with pytest.raises(cuda_lib.KDAError, match="INVALID"):
        cuda_lib.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], scale=math.nan)
    with pytest.raises(TypeError):
        cuda_lib.attn_decode(s["q"].half(), s["kc"].half(), s["vc"].half(), s["table"], s["lens"])


@pytest.mark.parametrize("d,Hq", [(64, 4), (128, 4), (64, 64), (128, 64)])
def test_long_sums_are_rounded_to_nearest(cuda_lib, d, Hq):
    """All values 1: o is the sum of the weights over itself, so a sum that is rounded towards zero shows as o < 1. A warp
    adds W tiles of 16 positions: W roundings in the numerator and 2 W in the denominator, some twenty where pieces are
    joined. Rounded to nearest they are independent, each 2^-24 at most: 6 2^-24 sqrt(3 W + 20). Within a tile the products
    may be summed as the MMA likes, six steps of 2^-23, and a weight's second tf32 part is cut 2^-22 below it."""
    N, Hk, page, L = 256, 4, 64, 4096
    g = torch.Generator("cuda").manual_seed(41)
    kc = torch.randn(L // page, Hk, page, d, device="cuda", generator=g)
    vc = torch.ones_like(kc)
    table = torch.arange(L // page, dtype=torch.int32, device="cuda").repeat(N, 1)  # every row reads the same pages
    lens = torch.full((N,), L, dtype=torch.int32, device="cuda")
    q = torch.randn(N, Hq, d, device="cuda", generator=g)
    o = cuda_lib.attn_decode(q, kc, vc, table, lens)
    W = N * Hk * (L // 16) / 1036  # 1036: the fewest warps that share the work
    assert float((o.double() - 1).abs().max()) <= 6 * 2 ** -24 * math.sqrt(3 * W + 20) + 8 * 2 ** -23


# Which warps hold a pair: (lengths, Hq, Hk, page). The work is cut into equal ranges for the 1000 to 2000 warps of a call,
# so a few long rows are split (32 warps join the pieces of fewer than 16 pairs, 8 those of fewer than 148, one the others)
# and among many short ones some pairs are whole.
SPLITS = {"32 warps join": ([20000], 2, 1, 256), "8 warps join": ([2000] * 16, 4, 2, 256), "a warp joins": ([300] * 40, 8, 4, 100),
          "whole pairs": ([60] * 256, 16, 8, 16), "17 heads": ([20000], 17, 1, 256)}


@pytest.mark.parametrize("what", ["q", "k", "v"])
@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attended_nan_comes_out(cuda_lib, dtype, split, what):
    """A NaN query, or a page of NaN keys or values, longer than a piece, makes its heads NaN, whichever warps hold them."""
    lens, Hq, Hk, page = SPLITS[split]
    s = make(lens, Hq, Hk, 64, page, dtype, 51)
    if what == "q":
        s["q"][len(lens) // 2, Hq - 1] = math.nan
    else:
        pages = s["table"][len(lens) // 2]
        s[what + "c"][int(pages[min(1, len(pages) - 1)]), Hk - 1, : min(page, lens[0] // 2)] = math.nan
    o, lse = check(cuda_lib, s)
    bad, G = torch.zeros(len(lens), Hq, dtype=torch.bool), Hq // Hk
    bad[len(lens) // 2, Hq - 1 if what == "q" else Hq - G:] = True
    assert torch.equal(o.isnan().any(-1).cpu(), bad) and torch.equal(o.isnan().all(-1).cpu(), bad)
    assert torch.equal(lse.isnan().cpu(), bad if what != "v" else torch.zeros_like(bad))


@pytest.mark.parametrize("Hq,Hk", [(4, 2), (16, 1), (20, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_bf16_caches_keep_the_weights(cuda_lib, d, Hq, Hk):
    """On bf16 caches only the output is rounded to bf16. The bound is that of 32-bit weights, and beside it what two bf16
    parts leave of a weight (2^-8 of 2^-8 of it) and what the MMA cuts from its sums: for each tile two products of four
    steps, 2^-23 of the weighted magnitudes each."""
    s = make([1, 2, 3, 17, 40, 700], Hq, Hk, d, 16, "bf16", 61)
    c = {n: t.cuda() for n, t in s.items()}
    o = cuda_lib.attn_decode(c["q"], c["kc"], c["vc"], c["table"], c["lens"], k=c["k"], v=c["v"])
    f = {n: t.float() if t.is_floating_point() else t for n, t in s.items()}
    (want, slack), _ = R.attn_decode(f["q"], f["kc"], f["vc"], f["table"], f["lens"], f["k"], f["v"])
    (size, _), _ = R.attn_decode(f["q"], f["kc"], f["vc"].abs(), f["table"], f["lens"], f["k"], f["v"].abs())
    tiles = (s["lens"].double()[:, None, None] + 16) // 16
    R.close(o, want, slack + (2.0 ** -16 + 8 * tiles * 2.0 ** -23) * size)
