"""Plain 64-bit forms of the operators beside the gated delta rule (test
infrastructure only): the gated linear recurrence, the query/key norm with the
position rotation, and the attention of one new token over a paged cache, each
with the error that a 32-bit evaluation may make of it.

Everything is torch float64 on the CPU, token by token and row by row. A result
comes as (value, slack): slack is the largest error, element by element, of an
evaluation whose sums and products are rounded to 32 bits (U = 2^-24 a
rounding), before the rounding to the output's type, which `close` adds.
"""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def close(got, want, slack, what=""):
    """|got - want| <= slack + one rounding to got's type, element by element (and the same non-finite values)."""
    got_d = got.detach().cpu().double()
    assert got_d.shape == want.shape, (what, got_d.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got_d), fine), f"{what}: other non-finite places"
    assert torch.equal(got_d[~fine].nan_to_num(nan=7.0), want[~fine].nan_to_num(nan=7.0)), f"{what}: other non-finite values"
    # a rounding of a value that is itself off by slack, and the type's smallest step near zero
    bound = slack + half_step(got.dtype) * (want.abs() + slack) + torch.finfo(got.dtype).smallest_normal
    over = ((got_d - want).abs() - bound)[fine]
    if over.numel():
        worst = over.max().item()
        assert worst <= 0, f"{what}: {worst:.3e} beyond the bound (largest error {(got_d - want).abs()[fine].max().item():.3e})"


# ---------------------------------------------------------------- gated linear recurrence


def _scan(a, x, h):
    """h_t = a_t h_{t-1} + x_t over the first dimension, and the final state."""
    out = torch.empty_like(x)
    for t in range(x.shape[0]):
        h = a[t] * h + x[t]
        out[t] = h
    return out, h


def _recurrence_slack(a, x, h0):
    """The decay over a span of m tokens is off by at most m * 8U (an exponential to 3U and a product a token, or the
    exponential of a 32-bit sum), and every addition rounds once: the errors obey the recurrence themselves, fed by 8U of
    the sum of magnitudes. Sums of log_alpha over a span of total decay S are off by log2(span) * U * S <= 16 U S, and
    S e^-S < 1, which adds 16U of the largest state."""
    size, end = _scan(a, x.abs(), h0.abs())
    slack, slack_end = _scan(a, 8 * U * size, 8 * U * h0.abs())
    top = 16 * U * (torch.cat([size, h0.abs()[None]]).amax(0) if x.shape[0] else h0.abs())
    return slack + top, slack_end + top


def recurrence_fwd(log_alpha, x, h0=None):
    """One sequence: log_alpha, x [T, D]; h0 [D]. ((h, slack), (h_T, slack))."""
    a, x = log_alpha.double().exp(), x.double()
    h0 = torch.zeros(x.shape[1], dtype=torch.float64) if h0 is None else h0.double()
    h, end = _scan(a, x, h0)
    s, s_end = _recurrence_slack(a, x, h0)
    return (h, s), (end, s_end if x.shape[0] else torch.zeros_like(s_end))


def recurrence_bwd(log_alpha, h, h0, dh, dh_T=None):
    """One sequence, h the given [T, D] output. dict of (value, slack): dx, dlog_alpha, dh0."""
    a, h, dh = log_alpha.double().exp(), h.double(), dh.double()
    zero = torch.zeros(dh.shape[1], dtype=torch.float64)
    h0 = zero if h0 is None else h0.double()
    c = zero if dh_T is None else dh_T.double()
    T = dh.shape[0]
    # c_{t-1} = a_t c_t + a_t dh_t: the forward recurrence over the reversed tokens
    af, gf = a.flip(0), (a * dh).flip(0)
    cs, end = _scan(af, gf, c)
    s, s_end = _recurrence_slack(af, gf, c)
    after = torch.cat([c[None], cs[:-1]]) if T else cs
    s_after = torch.cat([torch.zeros_like(s_end)[None], s[:-1]]) if T else s
    before = torch.cat([h0[None], h[:-1]]) if T else h
    dx = dh + after.flip(0)
    dla = cs.flip(0) * before
    return {"dx": (dx, s_after.flip(0) + 2 * U * dx.abs()), "dlog_alpha": (dla, s.flip(0) * before.abs() + 2 * U * dla.abs()),
            "dh0": (end, s_end if T else torch.zeros_like(s_end))}


# ---------------------------------------------------------------- query/key norm and rotation


def _pairs(d, rot, interleaved):
    """Channels (first, second) of every rotated pair, in the tables' column order."""
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _rotate(y, cos, sin, interleaved, back=False):
    """y [n, H, d]; cos, sin [n, rot/2]."""
    if cos is None:
        return y
    i, j = _pairs(y.shape[-1], 2 * cos.shape[1], interleaved)
    c, s = cos[:, None], sin[:, None] * (-1 if back else 1)
    out = y.clone()
    out[..., i] = y[..., i] * c - y[..., j] * s
    out[..., j] = y[..., j] * c + y[..., i] * s
    return out


def _sizes(y, cos, sin, interleaved):
    """Sum of the magnitudes that a rotation adds."""
    if cos is None:
        return y.abs()
    return _rotate(y.abs(), cos.abs(), -sin.abs(), interleaved).abs() + _rotate(y.abs(), cos.abs(), sin.abs(), interleaved).abs()


def _tables(cos, sin, positions):
    if positions is None:
        return None, None
    p = positions.reshape(-1).long().clamp(0, cos.shape[0] - 1)
    return cos.double()[p], sin.double()[p]


def _r(x, norm, eps):
    share = 1.0 / x.shape[-1] if norm == "rms" else 1.0
    # the magnitudes squared may leave 64 bits only for values past 1e150: not drawn
    return 1 / ((x * x).sum(-1, keepdim=True) * share + eps).sqrt(), share


def qk_norm_rope(x, w, cos, sin, positions, norm, eps, scale=1.0, interleaved=False):
    """One side: x [n, H, d]. (y, slack)."""
    x = x.double()
    c, s = _tables(cos, sin, positions)
    r, _ = _r(x, norm, eps)
    y = x * r * (1.0 if w is None else w.double())
    out = scale * _rotate(y, c, s, interleaved)
    # a sum of d squares rounds d times at most, halved by the root; root, products, rotation: 12 more
    return out, (x.shape[-1] / 2 + 12) * U * abs(scale) * _sizes(y, c, s, interleaved)


def qk_norm_rope_bwd(dy, x, w, cos, sin, positions, norm, eps, scale=1.0, interleaved=False):
    """One side: (dx, slack), (dw, slack)."""
    x, dy, d = x.double(), dy.double(), x.shape[-1]
    c, s = _tables(cos, sin, positions)
    r, share = _r(x, norm, eps)
    u = scale * _rotate(dy, c, s, interleaved, back=True)
    u_size = abs(scale) * _sizes(dy, c, s, interleaved)
    n = x * r
    wd = 1.0 if w is None else w.double()
    dot = (u * wd * n).sum(-1, keepdim=True)
    dx = r * (u * wd - n * share * dot)
    size = r * (u_size * abs(wd) + n.abs() * share * (u_size * abs(wd) * n.abs()).sum(-1, keepdim=True)) if w is None else \
        r * (u_size * wd.abs() + n.abs() * share * (u_size * wd.abs() * n.abs()).sum(-1, keepdim=True))
    dw = (u * n).sum((0, 1))
    rows = x.shape[0] * x.shape[1]
    return (dx, (2 * d + 24) * U * size), (dw, (rows + d / 2 + 24) * U * (u_size * n.abs()).sum((0, 1)))


# ---------------------------------------------------------------- paged decode attention


def attn_decode(q, kc, vc, table, lens, k=None, v=None, scale=None, window=0):
    """q [N, Hq, d] ...; kc, vc are updated in place as the operator does. ((o, slack), (lse, slack))."""
    N, Hq, d = q.shape
    n_pages, Hk, page, _ = kc.shape
    scale = d ** -0.5 if scale is None else scale
    weights = 0.0 if q.dtype == torch.float32 else half_step(q.dtype)  # the softmax weights' own rounding
    o, lse = torch.zeros(N, Hq, d, dtype=torch.float64), torch.full((N, Hq), -math.inf, dtype=torch.float64)
    so, sl = torch.zeros_like(o), torch.zeros_like(lse)
    cap = table.shape[1] * page
    for n in range(N):
        held = int(lens[n])
        if held < 0:
            continue
        total = held + (k is not None)
        rows_k, rows_v = [], []
        for p in range(max(0, total - window) if window else 0, min(total, cap)):
            at = int(table[n, p // page])
            if not 0 <= at < n_pages:
                continue
            if k is not None and p == held:
                kc[at, :, p % page] = k[n]
                vc[at, :, p % page] = v[n]
            rows_k.append(kc[at, :, p % page])
            rows_v.append(vc[at, :, p % page])
        if not rows_k:
            continue
        kk, vv = torch.stack(rows_k, 1).double(), torch.stack(rows_v, 1).double()  # [Hk, L, d]
        for h in range(Hq):
            K, V, x = kk[h // (Hq // Hk)], vv[h // (Hq // Hk)], q[n, h].double()
            s = scale * (K @ x)
            off = (d + 4) * U * abs(scale) * (K.abs() @ x.abs()).max()  # of a score
            p = torch.softmax(s, 0)
            o[n, h], lse[n, h] = p @ V, torch.logsumexp(s, 0)
            # a weight is off by its score's error and 8U; sums of L terms, rescaled as the maximum grows
            each = 2 * off + (2 * len(s) + 32) * U + 2 * weights
            so[n, h] = each * (p @ V.abs())
            sl[n, h] = off + (2 * len(s) + 32) * U + 4 * U * (abs(lse[n, h]) + s.abs().max())
    return (o, so), (lse, sl)
