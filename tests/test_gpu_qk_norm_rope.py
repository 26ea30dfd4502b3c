"""GPU parity of the query/key norm with the position rotation, forward and
backward, against the 64-bit forms in stack_reference.py."""
import math

import pytest
import torch

from tests import stack_reference as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(n, Hq, Hk, d, rot, dtype, seed, weights=True, far=1000, pos_dtype=torch.int64, fused=True, std=2.0):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    qkv = (std * torch.randn(n, (Hq + 2 * Hk) * d, generator=g)).to(dt)
    s = {"q": qkv[:, : Hq * d].unflatten(1, (Hq, d)), "k": qkv[:, Hq * d: (Hq + Hk) * d].unflatten(1, (Hk, d))}
    if not fused:
        s = {name: t.contiguous() for name, t in s.items()}
    s["wq"], s["wk"] = ((1 + 0.3 * torch.randn(d, generator=g)).to(dt) if weights else None for _ in range(2))
    s["cos"] = s["sin"] = s["pos"] = None
    if rot:
        ang = torch.arange(far)[:, None].double() * 10000.0 ** (-torch.arange(0, rot, 2).double() / rot)
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        s["pos"] = torch.randint(0, far, (n,), generator=g).to(pos_dtype)
    s["dq"], s["dk"] = torch.randn(n, Hq, d, generator=g).to(dt), torch.randn(n, Hk, d, generator=g).to(dt)
    return s


def on_gpu(s):
    """The same tensors there, with the strides they have here."""
    out = {}
    for name, t in s.items():
        if t is None or t.is_contiguous():
            out[name] = None if t is None else t.cuda()
        else:
            base = torch.empty(0, dtype=t.dtype).set_(t.untyped_storage()).cuda()
            out[name] = base.as_strided(t.shape, t.stride(), t.storage_offset())
    return out


def check(kda, s, norm="rms", eps=1e-6, scale=1.0, interleaved=False, backward=True):
    c = on_gpu(s)
    kw = dict(norm=norm, eps=eps, q_scale=scale, interleaved=interleaved)
    args = (c["wq"], c["wk"], c["cos"], c["sin"], c["pos"])
    qo, ko = kda.qk_norm_rope(c["q"], c["k"], *args, **kw)
    torch.cuda.synchronize()
    for name, x, w, got, sc in (("q", s["q"], s["wq"], qo, scale), ("k", s["k"], s["wk"], ko, 1.0)):
        R.close(got, *R.qk_norm_rope(x, w, s["cos"], s["sin"], s["pos"], norm, eps, sc, interleaved), name)
    if not backward:
        return
    g = kda.qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], *args, **kw)
    torch.cuda.synchronize()
    for name, x, w, dy, sc in (("q", s["q"], s["wq"], s["dq"], scale), ("k", s["k"], s["wk"], s["dk"], 1.0)):
        dx, dw = R.qk_norm_rope_bwd(dy, x, w, s["cos"], s["sin"], s["pos"], norm, eps, sc, interleaved)
        R.close(g["d" + name], *dx, "d" + name)
        if w is None:
            assert g[f"d{name}_weight"] is None
        else:
            R.close(g[f"d{name}_weight"], *dw, f"d{name}_weight")


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("d,rot", [(8, 0), (16, 16), (24, 16), (40, 32), (64, 64), (64, 32), (80, 48), (96, 96), (128, 128), (128, 64), (160, 0),
                                   (192, 96), (256, 256), (248, 240)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_sizes(cuda_lib, dtype, d, rot, norm):
    check(cuda_lib, make(7, 6, 2, d, rot, dtype, 3 + d + rot), norm)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,Hq,Hk", [(1, 1, 1), (2, 32, 8), (33, 5, 1), (130, 3, 3), (1, 64, 64), (700, 4, 2), (3, 7, 0), (3, 0, 5)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_counts(cuda_lib, dtype, n, Hq, Hk, interleaved):
    check(cuda_lib, make(n, Hq, Hk, 64, 64, dtype, 5 + n), interleaved=interleaved, scale=0.125)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_positions(cuda_lib, dtype, norm, weights):
    check(cuda_lib, make(50, 4, 4, 128, 0, dtype, 7, weights=weights), norm, eps=1e-5)


@pytest.mark.parametrize("interleaved", [False, True])
def test_interleaved_head_sizes(cuda_lib, interleaved):
    for d, rot in ((16, 16), (64, 32), (96, 80), (128, 128), (256, 144)):
        for dtype in ("f32", "bf16"):
            check(cuda_lib, make(9, 3, 2, d, rot, dtype, d), interleaved=interleaved)


def test_many_rows(cuda_lib):
    """More rows than one pass of the grid, for the weights' sums."""
    for dtype in ("f32", "bf16"):
        check(cuda_lib, make(1500, 8, 2, 64, 32, dtype, 13))


def test_far_and_bad_positions(cuda_lib):
    s = make(6, 2, 2, 64, 64, "f32", 15, far=100000)
    s["pos"] = torch.tensor([0, 99999, 65536, 100000, -1, 1 << 40])  # the last three are clamped
    check(cuda_lib, s)
    s["pos"] = torch.tensor([0, 99999, 65536, 100000, -1, 1 << 30], dtype=torch.int32)
    check(cuda_lib, s)


def test_one_side_has_weights(cuda_lib):
    s = make(40, 4, 2, 64, 64, "bf16", 16)
    s["wk"] = None
    check(cuda_lib, s)
    s = make(40, 4, 2, 64, 64, "f32", 16)
    s["wq"] = None
    check(cuda_lib, s)


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_zero_tiny_and_huge_heads(cuda_lib, dtype, norm):
    s = make(8, 2, 2, 64, 64, dtype, 17, fused=False)
    s["q"][0] = 0
    s["q"][1] *= 1e-18
    s["q"][2] *= 1e18   # the squares leave 32 bits
    s["q"][3] *= 1e30
    s["k"][4, 1] = 0
    s["k"][5] *= 1e-3
    check(cuda_lib, s, norm, backward=False)
    s["q"][2:4] = make(8, 2, 2, 64, 64, dtype, 18, fused=False)["q"][2:4]  # gradients of such heads leave 32 bits themselves
    check(cuda_lib, s, norm)


def test_nan_and_infinity_stay_in_their_head(cuda_lib):
    s = make(5, 4, 2, 128, 128, "f32", 19)
    c = on_gpu(s)
    clean = cuda_lib.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], c["pos"])
    c["q"][1, 2, 5], c["q"][3, 0, 0] = math.nan, math.inf
    got = cuda_lib.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], c["pos"])
    bad = torch.isnan(got[0]).any(-1)
    assert bad.nonzero().tolist() == [[1, 2], [3, 0]]
    assert torch.equal(got[0][~bad], clean[0][~bad]) and torch.equal(got[1], clean[1])


def test_in_place_and_leading_dimensions(cuda_lib):
    s = on_gpu(make(24, 4, 2, 64, 64, "bf16", 20, fused=False))
    want = cuda_lib.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"])
    q, k = s["q"].clone(), s["k"].clone()
    got = cuda_lib.qk_norm_rope(q, k, s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    four = cuda_lib.qk_norm_rope(s["q"].view(4, 6, 4, 64), s["k"].view(4, 6, 2, 64), s["wq"], s["wk"], s["cos"], s["sin"], s["pos"].view(4, 6))
    assert four[0].shape == (4, 6, 4, 64) and torch.equal(four[0].view(24, 4, 64), want[0])


def test_head_major_strides(cuda_lib):
    """[H, n, d] memory seen as [n, H, d]."""
    s = on_gpu(make(24, 4, 2, 64, 64, "f32", 21, fused=False))
    args = (s["wq"], s["wk"], s["cos"], s["sin"], s["pos"])
    want = cuda_lib.qk_norm_rope(s["q"], s["k"], *args)
    qt, kt = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (s["q"], s["k"]))
    got = cuda_lib.qk_norm_rope(qt, kt, *args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # one vector for all heads: a stride of zero
    one = s["k"][:, :1].expand(24, 4, 64)
    got = cuda_lib.qk_norm_rope(s["q"], one, *args)
    want = cuda_lib.qk_norm_rope(s["q"], one.contiguous(), *args)
    assert torch.equal(got[1], want[1])


def test_no_tokens(cuda_lib):
    s = on_gpu(make(0, 4, 2, 64, 64, "f32", 22, fused=False))
    args = (s["wq"], s["wk"], s["cos"], s["sin"], s["pos"])
    q, k = cuda_lib.qk_norm_rope(s["q"], s["k"], *args)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    g = cuda_lib.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], *args)
    assert g["dq_weight"].abs().max() == 0 and g["dk_weight"].abs().max() == 0


def test_equal_bits_streams_and_graphs(cuda_lib):
    s = on_gpu(make(900, 8, 2, 128, 64, "bf16", 23))
    args = (s["wq"], s["wk"], s["cos"], s["sin"], s["pos"])
    want = cuda_lib.qk_norm_rope(s["q"], s["k"], *args)
    grads = cuda_lib.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], *args)
    again = cuda_lib.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], *args)
    assert all(torch.equal(grads[x], again[x]) for x in grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, k = torch.empty_like(want[0]), torch.empty_like(want[1])
    cuda_lib.qk_norm_rope(s["q"], s["k"], *args, q_out=q, k_out=k, stream=side)
    side.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    graph = torch.cuda.CUDAGraph()
    s2 = {x: None if t is None else torch.zeros_like(t) for x, t in s.items()}
    args2 = (s2["wq"], s2["wk"], s2["cos"], s2["sin"], s2["pos"])
    with torch.cuda.graph(graph):
        q, k = cuda_lib.qk_norm_rope(s2["q"], s2["k"], *args2)
        g = cuda_lib.qk_norm_rope_bwd(s2["dq"], s2["dk"], s2["q"], s2["k"], *args2)
    for x in s2:
        s2[x].copy_(s[x])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        assert all(torch.equal(g[x], grads[x]) for x in g)


def test_offsets_past_32_bits(cuda_lib):
    n, H, d = 65800, 256, 128  # 2.16e9 elements
    g = torch.Generator(device="cuda").manual_seed(29)
    q = torch.empty(n, H, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    k = torch.empty(n, 1, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    qo, ko = cuda_lib.qk_norm_rope(q, k, norm="l2")
    R.close(qo[-2:], *R.qk_norm_rope(q[-2:].cpu(), None, None, None, None, "l2", 1e-6))
    R.close(ko[-2:], *R.qk_norm_rope(k[-2:].cpu(), None, None, None, None, "l2", 1e-6))
    grads = cuda_lib.qk_norm_rope_bwd(qo, ko, q, k, norm="l2")
    (dq, slack), _ = R.qk_norm_rope_bwd(qo[-2:].cpu(), q[-2:].cpu(), None, None, None, None, "l2", 1e-6)
    R.close(grads["dq"][-2:], dq, slack)


def test_refusals(cuda_lib):
    s = on_gpu(make(6, 4, 2, 64, 64, "bf16", 30))
    q, k, tab = s["q"], s["k"], (s["cos"], s["sin"], s["pos"])
    f = cuda_lib.qk_norm_rope
    with pytest.raises(ValueError, match="norm"):
        f(q, k, norm="layer")
    with pytest.raises(ValueError, match="k: expected"):
        f(q, k.float())
    with pytest.raises(ValueError, match="q_weight"):
        f(q, k, torch.ones(32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="tables"):
        f(q, k, positions=s["pos"])
    with pytest.raises(ValueError, match="one per token"):
        f(q, k, None, None, s["cos"], s["sin"], s["pos"][:3])
    with pytest.raises(TypeError, match="positions"):
        f(q, k, None, None, s["cos"], s["sin"], s["pos"].float())
    with pytest.raises(ValueError, match="contiguous"):
        f(q.transpose(1, 2).contiguous().transpose(1, 2), k)
    with pytest.raises(cuda_lib.KDAError, match="INVALID"):
        f(q, k, *[None] * 2, *tab, eps=0.0)
    with pytest.raises(cuda_lib.KDAError, match="UNSUPPORTED"):
        f(q[..., :60].contiguous(), k[..., :60].contiguous())
    with pytest.raises(cuda_lib.KDAError, match="UNSUPPORTED"):  # 40 of the 64 channels
        f(q, k, None, None, s["cos"][:, :20].contiguous(), s["sin"][:, :20].contiguous(), s["pos"])
    odd = torch.zeros(6 * 4 * 66, dtype=torch.bfloat16, device="cuda").view(6, 4, 66)[..., :64]
    with pytest.raises(cuda_lib.KDAError, match="INVALID"):  # heads 132 bytes apart
        f(odd, k)
    with pytest.raises(ValueError, match="dq_out"):
        cuda_lib.qk_norm_rope_bwd(s["dq"][:3], s["dk"], q, k)
    with pytest.raises(cuda_lib.KDAError, match="workspace"):
        cuda_lib.qk_norm_rope_bwd(s["dq"], s["dk"], q, k, s["wq"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_eps(cuda_lib, dtype, norm):
    """An eps beside which heads whose squares leave 32 bits are small, like, and large."""
    s = make(12, 2, 2, 64, 64, dtype, 32, fused=False)
    for t, f in ((1, 1e15), (2, 1e18), (3, 1e19), (4, 1e20), (5, 1e25)):
        s["q"][t] *= f
        s["k"][t] *= f
    for eps in (1e30, 1e37, 2.5e38):
        check(cuda_lib, s, norm, eps=eps)


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("d,rot", [(8, 0), (64, 64), (128, 64), (256, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_huge_heads(cuda_lib, dtype, d, rot, norm):
    """Heads whose squares leave 32 bits, beside ordinary ones of the same warp; their gradients do not (1e-18 to 1e-36)."""
    s = make(40, 4, 2, d, rot, dtype, 31, fused=False)
    for t, f in ((1, 1e18), (2, 3e19), (7, 1e30), (8, 1e36)):
        s["q"][t, 1] *= f
        s["k"][t + 2] *= f
    check(cuda_lib, s, norm)
    check(cuda_lib, s, norm, interleaved=True, scale=0.125)
