"""CPU pins of the 64-bit forms in stack_reference.py: closed forms, central
differences for the gradients, and mistakes that the comparison must catch."""
import math

import pytest
import torch

from tests import stack_reference as R


def _g(seed):
    return torch.Generator().manual_seed(seed)


def test_recurrence_closed_forms():
    T, D = 9, 3
    x = torch.randn(T, D, generator=_g(1), dtype=torch.float64)
    (h, _), (end, _) = R.recurrence_fwd(torch.zeros(T, D), x)  # no decay: a running sum
    torch.testing.assert_close(h, x.cumsum(0))
    assert torch.equal(end, h[-1])
    (h, _), _ = R.recurrence_fwd(torch.full((T, D), -math.inf), x, torch.ones(D))  # full decay: the input
    assert torch.equal(h, x)
    la = -torch.rand(T, D, generator=_g(2), dtype=torch.float64)  # no input: a running product
    (h, _), _ = R.recurrence_fwd(la, torch.zeros(T, D), torch.ones(D))
    torch.testing.assert_close(h, la.cumsum(0).exp())


@pytest.mark.parametrize("with_state", [False, True])
def test_recurrence_gradients_against_differences(with_state):
    T, D, eps = 6, 2, 1e-6
    g = _g(3)
    la, x = -torch.rand(T, D, generator=g, dtype=torch.float64), torch.randn(T, D, generator=g, dtype=torch.float64)
    h0, dh = torch.randn(D, generator=g, dtype=torch.float64), torch.randn(T, D, generator=g, dtype=torch.float64)
    dT = torch.randn(D, generator=g, dtype=torch.float64) if with_state else None

    def loss(la, x, h0):
        (h, _), (end, _) = R.recurrence_fwd(la, x, h0)
        return (h * dh).sum() + (0 if dT is None else (end * dT).sum())

    (h, _), _ = R.recurrence_fwd(la, x, h0)
    got = R.recurrence_bwd(la, h, h0, dh, dT)
    for name, arg in (("dlog_alpha", 0), ("dx", 1), ("dh0", 2)):
        base = [la, x, h0]
        want = torch.zeros_like(base[arg])
        for i in range(base[arg].numel()):
            ends = []
            for sign in (1, -1):
                moved = [t.clone() for t in base]
                moved[arg].view(-1)[i] += sign * eps
                ends.append(loss(*moved))
            want.view(-1)[i] = (ends[0] - ends[1]) / (2 * eps)
        torch.testing.assert_close(got[name][0], want, rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_qk_gradients_against_differences(norm, interleaved):
    n, H, d, rot, eps = 2, 2, 24, 16, 1e-6
    g = _g(4)
    x, w = torch.randn(n, H, d, generator=g, dtype=torch.float64), torch.randn(d, generator=g, dtype=torch.float64)
    dy = torch.randn(n, H, d, generator=g, dtype=torch.float64)
    ang = torch.randn(5, rot // 2, generator=g, dtype=torch.float64)
    args = (ang.cos(), ang.sin(), torch.tensor([3, 1]), norm, 1e-3, 0.7, interleaved)
    (dx, _), (dw, _) = R.qk_norm_rope_bwd(dy, x, w, *args)
    for name, t, got in (("x", x, dx), ("w", w, dw)):
        want = torch.zeros_like(t)
        for i in range(t.numel()):
            ends = []
            for sign in (1, -1):
                m = t.clone()
                m.view(-1)[i] += sign * eps
                y, _ = R.qk_norm_rope(m if name == "x" else x, m if name == "w" else w, *args)
                ends.append((y * dy).sum())
            want.view(-1)[i] = (ends[0] - ends[1]) / (2 * eps)
        torch.testing.assert_close(got, want, rtol=1e-5, atol=1e-7)


def test_qk_closed_forms():
    x = torch.randn(3, 2, 16, generator=_g(5), dtype=torch.float64)
    y, _ = R.qk_norm_rope(x, None, None, None, None, "l2", 1e-12)
    torch.testing.assert_close(y.norm(dim=-1), torch.ones(3, 2, dtype=torch.float64))
    ang = torch.rand(4, 8, generator=_g(6), dtype=torch.float64)
    for inter in (False, True):  # a rotation keeps norms, and the inner product depends on the distance alone
        z, _ = R.qk_norm_rope(x, None, ang.cos(), ang.sin(), torch.tensor([0, 2, 3]), "l2", 1e-12, interleaved=inter)
        torch.testing.assert_close(z.norm(dim=-1), torch.ones(3, 2, dtype=torch.float64))
    freq = torch.rand(8, generator=_g(7), dtype=torch.float64)
    ang = torch.arange(9)[:, None] * freq
    dots = []
    for a, b in ((1, 4), (5, 8)):
        p = [R.qk_norm_rope(x[i:i + 1], None, ang.cos(), ang.sin(), torch.tensor([at]), "l2", 1e-12)[0] for i, at in ((0, a), (1, b))]
        dots.append((p[0] * p[1]).sum(-1))
    torch.testing.assert_close(dots[0], dots[1])


def test_attention_closed_forms_and_masks():
    g = _g(8)
    N, Hq, Hk, d, page = 3, 4, 2, 8, 4
    kc, vc = torch.randn(5, Hk, page, d, generator=g), torch.randn(5, Hk, page, d, generator=g)
    table = torch.tensor([[4, 0], [2, -1], [1, 3]], dtype=torch.int32)
    q, k, v = (torch.randn(N, h, d, generator=g) for h in (Hq, Hk, Hk))
    k2, v2 = kc.clone(), vc.clone()
    (o, _), (lse, _) = R.attn_decode(q, k2, v2, table, torch.tensor([5, 0, -1]), k, v)
    assert torch.equal(k2[0, :, 1], k[0]) and torch.equal(v2[2, :, 0], v[1])  # put where the table says
    torch.testing.assert_close(o[1], v[1].double().repeat_interleave(2, 0))      # one position: its value
    assert o[2].abs().max() == 0 and torch.isinf(lse[2]).all()                    # a padded row
    K = torch.cat([k2[4, 0], k2[0, 0, :2]]).double()
    V = torch.cat([v2[4, 0], v2[0, 0, :2]]).double()
    s = d ** -0.5 * K @ q[0, 1].double()
    torch.testing.assert_close(o[0, 1], torch.softmax(s, 0) @ V)
    torch.testing.assert_close(lse[0, 1], torch.logsumexp(s, 0))
    (w, _), _ = R.attn_decode(q, k2, v2, table, torch.tensor([5, 0, -1]), k, v, window=1)  # the new token alone
    torch.testing.assert_close(w[0], v[0].double().repeat_interleave(2, 0))


def test_the_comparison_catches_mistakes():
    g = _g(9)
    la, x = -0.1 * torch.rand(50, 4, generator=g), torch.randn(50, 4, generator=g)
    (h, s), _ = R.recurrence_fwd(la, x)
    R.close(h.float(), h, s)
    R.close(h.bfloat16(), h, s)
    with pytest.raises(AssertionError):
        R.close(h.float() * (1 + 1e-3), h, s)
    with pytest.raises(AssertionError):
        R.close((h * (1 + 2 ** -6)).bfloat16(), h, s)
    moved = la.roll(1, 0)  # the decay of the token before
    (wrong, _), _ = R.recurrence_fwd(moved, x)
    with pytest.raises(AssertionError):
        R.close(wrong.bfloat16(), h, s)
    bad = h.float()
    bad[3, 1] = float("nan")
    with pytest.raises(AssertionError):
        R.close(bad, h, s)
