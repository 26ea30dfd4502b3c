"""Measured cases of the operators that stand beside the gated delta rule in a hybrid decoder stack.

Three families:
  recurrence  h_t = exp(log_alpha_t) * h_{t-1} + x_t per channel: the scan over long sequences (dense or packed), its
              backward pass and its single-token step
  qk          the norm of every query and key head with the position rotation in the same pass, and its backward pass
  attn        the attention of one new token per sequence over a paged key-value cache

`run` computes a case in plain torch operations where `own` is false, and through the package where it is true.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # One decode step of a recurrent layer for a full serving batch.
        {"name": "step_n256_d4096_bf16", "op": "step", "n": 256, "d": 4096, "dtype": "bf16"},
        # Training forward of the framework's B4 H32 T8192 d128 workload, its 4096 channels as one recurrence.
        {"name": "scan_b4_t8192_d4096_bf16", "op": "scan", "b": 4, "t": 8192, "d": 4096, "packed": False, "dtype": "bf16"},
        # One long document, a width that no vector load divides, a last tile of one token.
        {"name": "scan_b1_t16385_d1001_f32", "op": "scan", "b": 1, "t": 16385, "d": 1001, "packed": False, "dtype": "f32"},
        # Prefill of nine requests of very different lengths, packed.
        {"name": "scan_packed9_t16384_d2048_bf16", "op": "scan", "b": 9, "t": 16384, "d": 2048, "packed": True, "dtype": "bf16"},
        # Training backward of half of the dense workload above.
        {"name": "scan_bwd_b2_t8192_d4096_bf16", "op": "scan_bwd", "b": 2, "t": 8192, "d": 4096, "packed": False, "dtype": "bf16"},
        # Queries and keys of one decode step, 64 sequences, out of a fused projection.
        {"name": "qk_n64_hq32_hk8_d128_rms_bf16", "op": "qk", "n": 64, "hq": 32, "hk": 8, "d": 128, "rot": 128, "norm": "rms", "dtype": "bf16"},
        # The inputs of the framework's B4 H32 T8192 d128 prefill: L2-normalised queries and keys, no positions.
        {"name": "qk_n32768_h32_d128_l2_bf16", "op": "qk", "n": 32768, "hq": 32, "hk": 32, "d": 128, "rot": 0, "norm": "l2", "dtype": "bf16"},
        # Training backward of a softmax layer's queries and keys, half of each head rotated.
        {"name": "qk_bwd_n8192_hq32_hk8_d128_bf16", "op": "qk_bwd", "n": 8192, "hq": 32, "hk": 8, "d": 128, "rot": 64, "norm": "rms", "dtype": "bf16"},
        # One user with a 128K context.
        {"name": "attn_n1_l131072_hq32_hk8_d128_bf16", "op": "attn", "n": 1, "lo": 131072, "hi": 131072, "hq": 32, "hk": 8, "d": 128, "page": 64, "window": 0, "dtype": "bf16"},
        # A serving batch whose contexts differ by a factor of 64.
        {"name": "attn_n64_l256_16384_hq32_hk8_bf16", "op": "attn", "n": 64, "lo": 256, "hi": 16384, "hq": 32, "hk": 8, "d": 128, "page": 32, "window": 0, "dtype": "bf16"},
        # Many short requests, the first of them without any context, one key-value head for each query head.
        {"name": "attn_n256_l0_300_h16_d64_bf16", "op": "attn", "n": 256, "lo": 0, "hi": 300, "hq": 16, "hk": 16, "d": 64, "page": 16, "window": 0, "dtype": "bf16"},
        # 32-bit cache, five query heads to a key-value head, a sliding window that ends inside pages.
        {"name": "attn_n7_l100_9000_hq20_hk4_w1000_f32", "op": "attn", "n": 7, "lo": 100, "hi": 9000, "hq": 20, "hk": 4, "d": 128, "page": 48, "window": 1000, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "scan_bwd", "scan_bwd", "qk", "qk", "qk_bwd", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "step":
        return {"op": op, "n": _log(rng, 1, 512), "d": _log(rng, 64, 8192), "dtype": dtype}
    if op in ("scan", "scan_bwd"):
        # widths of heads times head sizes mostly, any width else
        d = rng.choice([128 * _log(rng, 1, 64), 64 * _log(rng, 1, 64), _log(rng, 30, 4096)])
        t = _log(rng, 1, 65536)
        b = _log(rng, 1, max(1, min(16, (1 << 26) // (t * d) or 1)))
        packed = rng.random() < 0.4
        if packed:
            t = max(t, 2 * b)
        while b * t * d > (1 << 26):
            t = t // 2 + 1
        return {"op": op, "b": b, "t": t, "d": d, "packed": packed, "dtype": dtype}
    if op in ("qk", "qk_bwd"):
        hk = rng.choice([1, 2, 4, 5, 8, 16, 32])
        hq = hk * rng.choice([1, 1, 2, 3, 4, 8])
        d = rng.choice([64, 64, 96, 128, 128, 256])
        n = _log(rng, 1, max(2, min(32768, (1 << 26) // ((hq + hk) * d))))
        rot = rng.choice([0, d, d, d // 2])
        return {"op": op, "n": n, "hq": hq, "hk": hk, "d": d, "rot": rot, "norm": rng.choice(["rms", "l2"]), "dtype": dtype}
    hk = rng.choice([1, 2, 4, 8, 16])
    hq = hk * rng.choice([1, 2, 3, 4, 6, 8, 16])
    d = rng.choice([64, 128])
    n = _log(rng, 1, 256)
    # the longest context is bounded by what the largest listed batch reads
    hi = _log(rng, 1, max(2, min(131072, (1 << 28) // (n * hk * d))))
    lo = rng.choice([0, 1, hi // 10 + 1, hi])
    window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    return {"op": "attn", "n": n, "lo": min(lo, hi), "hi": hi, "hq": hq, "hk": hk, "d": d, "page": rng.choice([16, 32, 48, 64, 128]),
            "window": window, "dtype": dtype}


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly over their logarithm; a length of 0 where lo is 0."""
    if n == 1:
        return [hi]
    a = max(1, lo)
    got = [int(round(a * (hi / a) ** (i / (n - 1)))) for i in range(n)]
    return [lo] + got[1:]


def _packed_lengths(b, t):
    """b lengths that sum to t, each about twice the one before, the first of them empty if there are several."""
    if b == 1:
        return [t]
    share = [0.0] + [2.0 ** min(i, 5) for i in range(1, b)]
    got = [int(t * s / sum(share)) for s in share]
    got[-1] += t - sum(got)
    return got


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _log_alpha(shape, dtype, g):
    # decays that forget within a token up to ones that hold for a thousand
    return (-torch.exp(torch.empty(shape, device="cuda").uniform_(math.log(1e-3), 0.0, generator=g))).to(dtype)


def prepare(case, seed):
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dtype, std=1.0):
        return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g).to(dtype)

    op, s = case["op"], {"op": case["op"], "dtype": dtype}
    if op == "step":
        n, d = case["n"], case["d"]
        s |= {"la": _log_alpha((n, d), dtype, g), "x": normal(n, d), "h": normal(n, d, dtype=torch.float32),
              "h_out": torch.empty(n, d, device="cuda")}
    elif op in ("scan", "scan_bwd"):
        b, t, d = case["b"], case["t"], case["d"]
        shape = (t, d) if case["packed"] else (b, t, d)
        s |= {"la": _log_alpha(shape, dtype, g), "x": normal(*shape), "h0": normal(b, d, dtype=torch.float32), "cu": None}
        if case["packed"]:
            lens = torch.tensor(_packed_lengths(b, t))[torch.randperm(b, generator=torch.Generator().manual_seed(seed))]
            s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to("cuda", torch.int32)
        if op == "scan_bwd":  # a training step has the outputs of its forward pass
            s["h"] = _plain_scan(s)[0]
            s |= {"dh": normal(*shape), "dh_T": normal(b, d, dtype=torch.float32), "x": None}
    elif op in ("qk", "qk_bwd"):
        n, hq, hk, d, rot = (case[k] for k in ("n", "hq", "hk", "d", "rot"))
        qkv = normal(n, (hq + 2 * hk) * d, std=2.0)  # one projection gives queries, keys and values
        s |= {"q": qkv[:, : hq * d].unflatten(1, (hq, d)), "k": qkv[:, hq * d: (hq + hk) * d].unflatten(1, (hk, d)),
              "wq": None, "wk": None, "cos": None, "sin": None, "pos": None, "norm": case["norm"], "eps": 1e-6}
        if case["norm"] == "rms":
            s |= {"wq": (1 + normal(d, dtype=torch.float32, std=0.1)).to(dtype), "wk": (1 + normal(d, dtype=torch.float32, std=0.1)).to(dtype)}
        if rot:
            far = 65536
            angle = torch.arange(far, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
            s |= {"cos": angle.cos().float().cuda(), "sin": angle.sin().float().cuda(),
                  "pos": torch.randint(0, far, (n,), generator=g, device="cuda")}
        if op == "qk_bwd":
            s |= {"dq": normal(n, hq, d), "dk": normal(n, hk, d)}
    else:
        n, hq, hk, d, page = (case[k] for k in ("n", "hq", "hk", "d", "page"))
        lens = torch.tensor(_spread(n, case["lo"], case["hi"]))[torch.randperm(n, generator=torch.Generator().manual_seed(seed))]
        held = (lens + page) // page  # pages with room for the new token
        most = int(held.max())
        pool = int(held.sum()) + 3
        ids = torch.randperm(pool, generator=torch.Generator().manual_seed(seed + 1), dtype=torch.int64)[: int(held.sum())].to(torch.int32)
        table = torch.full((n, most), -1, dtype=torch.int32)
        table[torch.arange(most)[None] < held[:, None]] = ids
        s |= {"q": normal(n, hq, d), "k": normal(n, hk, d), "v": normal(n, hk, d), "kc": normal(pool, hk, page, d), "vc": normal(pool, hk, page, d),
              "table": table.cuda(), "lens": lens.to(torch.int32).cuda(), "window": case["window"], "scale": d ** -0.5}
    return s


def _starts(cu, b, t):
    """For every packed sequence: its first and last token, and whether it has any."""
    cu = cu.long()
    return cu[:-1].clamp(max=t - 1), (cu[1:] - 1).clamp(min=0), cu[1:] > cu[:-1]


def _doubling(a, h):
    """Prefix of h_t = a_t h_{t-1} + h_t along dimension -2: after k rounds a token holds the sum over its last 2^k."""
    s = 1
    while s < h.shape[-2]:
        h = torch.cat([h[..., :s, :], h[..., s:, :] + a[..., s:, :] * h[..., :-s, :]], -2)
        a = torch.cat([a[..., :s, :], a[..., s:, :] * a[..., :-s, :]], -2)
        s *= 2
    return h


def _plain_scan(s):
    a, h, h0 = s["la"].float().exp(), s["x"].float().clone(), s["h0"]
    if s["cu"] is None:
        h[:, 0] += a[:, 0] * h0
        h = _doubling(a, h)
        return h.to(s["dtype"]), h[:, -1].clone()
    first, last, some = _starts(s["cu"], h0.shape[0], h.shape[0])
    h[first[some]] += a[first[some]] * h0[some]
    a[first[some]] = 0
    h = _doubling(a, h)
    return h.to(s["dtype"]), torch.where(some[:, None], h[last], h0)


def _plain_scan_bwd(s):
    a, lam, h, h0 = s["la"].float().exp(), s["dh"].float().clone(), s["h"].float(), s["h0"]
    if s["cu"] is None:
        lam[:, -1] += s["dh_T"]
        nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
        lam = _doubling(nxt.flip(1), lam.flip(1)).flip(1)
        before = torch.cat([h0[:, None], h[:, :-1]], 1)
        return lam.to(s["dtype"]), (lam * a * before).to(s["dtype"]), lam[:, 0] * a[:, 0]
    first, last, some = _starts(s["cu"], h0.shape[0], h.shape[0])
    lam[last[some]] += s["dh_T"][some]
    nxt = torch.cat([a[1:], torch.zeros_like(a[:1])], 0)
    nxt[last[some]] = 0
    lam = _doubling(nxt.flip(0), lam.flip(0)).flip(0)
    before = torch.cat([h[:1], h[:-1]], 0)
    before[first[some]] = h0[some]
    return lam.to(s["dtype"]), (lam * a * before).to(s["dtype"]), torch.where(some[:, None], lam[first] * a[first], s["dh_T"])


def _turn(x, cos, sin):
    """Rotates the first 2 * cos.shape[-1] channels, channel i with channel i + half."""
    half = cos.shape[-1]
    lo, hi, rest = x[..., :half], x[..., half: 2 * half], x[..., 2 * half:]
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin, rest], -1)


def _plain_qk(x, w, s):
    x = x.float()
    total = (x * x).sum(-1, keepdim=True)
    y = x * torch.rsqrt((total / x.shape[-1] if s["norm"] == "rms" else total) + s["eps"])
    if w is not None:
        y = y * w.float()
    if s["pos"] is not None:
        y = _turn(y, s["cos"][s["pos"]][:, None], s["sin"][s["pos"]][:, None])
    return y.to(s["dtype"])


def _plain_qk_bwd(dy, x, w, s):
    x, u = x.float(), dy.float()
    total = (x * x).sum(-1, keepdim=True)
    share = 1 / x.shape[-1] if s["norm"] == "rms" else 1.0
    r = torch.rsqrt(total * share + s["eps"])
    if s["pos"] is not None:
        u = _turn(u, s["cos"][s["pos"]][:, None], -s["sin"][s["pos"]][:, None])
    n = x * r
    dw = None if w is None else (u * n).sum((0, 1))
    u = u if w is None else u * w.float()
    return (r * (u - n * (share * (u * n).sum(-1, keepdim=True)))).to(s["dtype"]), dw


def _plain_attn(s):
    n, hq, d = s["q"].shape
    kc, vc, table, page = s["kc"], s["vc"], s["table"].long(), s["kc"].shape[2]
    hk, at = kc.shape[1], s["lens"].long()
    where = table.gather(1, (at // page)[:, None])[:, 0]
    kc[where, :, at % page] = s["k"]
    vc[where, :, at % page] = s["v"]
    held = table.clamp(min=0)
    k = kc[held].float().transpose(1, 2).reshape(n, hk, -1, d)
    v = vc[held].float().transpose(1, 2).reshape(n, hk, -1, d)
    place = torch.arange(k.shape[2], device="cuda")[None]
    seen = place <= at[:, None]
    if s["window"]:
        seen = seen & (place > at[:, None] - s["window"])
    q = s["q"].float().view(n, hk, hq // hk, d) * s["scale"]
    score = (q @ k.transpose(2, 3)).masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total
    return o.view(n, hq, d).to(s["dtype"]), (top + total.log()).view(n, hq), kc, vc


def run(s):
    op = s["op"]
    if own:
        import gated_delta_rule_134_b200 as kda
        if op == "step":
            return kda.recurrence_step(s["la"], s["x"], s["h"], h_out=s["h_out"])
        if op == "scan":
            return kda.recurrence_fwd(s["la"], s["x"], s["h0"], cu_seqlens=s["cu"])
        if op == "scan_bwd":
            g = kda.recurrence_bwd(s["la"], s["h"], s["h0"], s["dh"], s["dh_T"], cu_seqlens=s["cu"])
            return g["dx"], g["dlog_alpha"], g["dh0"]
        if op == "qk":
            return kda.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], norm=s["norm"], eps=s["eps"])
        if op == "qk_bwd":
            g = kda.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], norm=s["norm"], eps=s["eps"])
            return g["dq"], g["dk"], g["dq_weight"], g["dk_weight"]
        o, lse = kda.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], k=s["k"], v=s["v"], scale=s["scale"], window=s["window"], return_lse=True)
        return o, lse, s["kc"], s["vc"]
    if op == "step":
        h = s["la"].float().exp() * s["h"] + s["x"].float()
        return h.to(s["dtype"]), h
    if op == "scan":
        return _plain_scan(s)
    if op == "scan_bwd":
        return _plain_scan_bwd(s)
    if op == "qk":
        return _plain_qk(s["q"], s["wq"], s), _plain_qk(s["k"], s["wk"], s)
    if op == "qk_bwd":
        dq, dwq = _plain_qk_bwd(s["dq"], s["q"], s["wq"], s)
        dk, dwk = _plain_qk_bwd(s["dk"], s["k"], s["wk"], s)
        return dq, dk, dwq, dwk
    return _plain_attn(s)


def work(case):
    es, op = BYTES[case["dtype"]], case["op"]
    if op == "step":
        cells = case["n"] * case["d"]
        return {"bytes": cells * (3 * es + 8), "flops": 2 * cells}
    if op in ("scan", "scan_bwd"):
        cells, states = (1 if case["packed"] else case["b"]) * case["t"] * case["d"], case["b"] * case["d"]
        if op == "scan":
            return {"bytes": 3 * es * cells + 8 * states, "flops": 2 * cells}
        return {"bytes": 5 * es * cells + 12 * states, "flops": 4 * cells}
    if op in ("qk", "qk_bwd"):
        rows, tables = case["n"] * (case["hq"] + case["hk"]), case["n"] * (case["rot"] * 4 + 8 if case["rot"] else 0)
        cells = rows * case["d"]
        return {"bytes": (2 if op == "qk" else 3) * es * cells + tables, "flops": (8 if op == "qk" else 16) * cells}
    n, hq, hk, d = (case[k] for k in ("n", "hq", "hk", "d"))
    seen = [min(x + 1, case["window"] or x + 1) for x in _spread(n, case["lo"], case["hi"])]
    # the new token's key and value are read from the call's arguments and written once; every other row is read once
    rows = 2 * hk * d * es
    return {"bytes": sum(seen) * rows + n * rows + n * hq * (2 * d * es + 4), "flops": 4 * sum(seen) * hq * d}


def _exact_scan(a, x, h, reset):
    """Token by token in 64 bits; `reset` gives {token: state to begin from}."""
    out = torch.empty_like(x)
    for t in range(x.shape[0]):
        h = reset.get(t, h)
        h = torch.addcmul(x[t], a[t], h)
        out[t] = h
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, z = s["op"], {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if op == "step":
        h = torch.exp(z["la"]) * z["h"] + z["x"]
        return h, h
    if op in ("scan", "scan_bwd"):
        a = torch.exp(z["la"])
        if s["cu"] is None:  # tokens first
            spans, a = [(0, case["t"])], a.transpose(0, 1)
            h0 = z["h0"][None]
        else:
            c = s["cu"].tolist()
            spans, h0 = list(zip(c[:-1], c[1:])), z["h0"]
        first = lambda v: v.transpose(0, 1) if s["cu"] is None else v  # noqa: E731
        batch = (lambda v: v[0]) if s["cu"] is None else (lambda v: v)
        if op == "scan":
            out = _exact_scan(a, first(z["x"]), h0[0], {lo: h0[i] for i, (lo, hi) in enumerate(spans) if hi > lo})
            end = torch.stack([out[hi - 1] if hi > lo else h0[i] for i, (lo, hi) in enumerate(spans)])
            return first(out).contiguous(), batch(end).contiguous()
        g, h = first(z["dh"]), first(z["h"])
        end = z["dh_T"][None] if s["cu"] is None else z["dh_T"]
        dx, dla, dh0 = torch.empty_like(g), torch.empty_like(g), torch.empty_like(h0)
        for i, (lo, hi) in enumerate(spans):
            c = end[i]
            for t in range(hi - 1, lo - 1, -1):
                dx[t] = c = c + g[t]
                c = a[t] * c
                dla[t] = c * (h[t - 1] if t > lo else h0[i])
            dh0[i] = c
        return first(dx).contiguous(), first(dla).contiguous(), batch(dh0).contiguous()
    if op in ("qk", "qk_bwd"):
        def matrix(rot):
            """[n, rot/2, 2, 2] turns of every token."""
            c, n = z["cos"][s["pos"]], z["sin"][s["pos"]]
            return torch.stack([torch.stack([c, -n], -1), torch.stack([n, c], -1)], -2)

        def one(x, w):
            norm = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
            y = x / torch.sqrt((norm ** 2 / x.shape[-1] if s["norm"] == "rms" else norm ** 2) + s["eps"])
            y = y if w is None else w * y
            if case["rot"]:
                pair = torch.stack(y[..., : case["rot"]].chunk(2, -1), -1)
                pair = torch.einsum("nfij,nhfj->nhif", matrix(case["rot"]), pair)
                y = torch.cat([pair.flatten(2), y[..., case["rot"]:]], -1)
            return y

        got = []
        for x, w, dy in (("q", "wq", "dq"), ("k", "wk", "dk")):
            if op == "qk":
                got.append(one(z[x], z[w]))
                continue
            leaf = [z[x].clone().requires_grad_()] + ([] if z[w] is None else [z[w].clone().requires_grad_()])
            grads = torch.autograd.grad(one(leaf[0], leaf[1] if len(leaf) > 1 else None), leaf, z[dy])
            got.append(grads)
        return tuple(got) if op == "qk" else (got[0][0], got[1][0], got[0][1] if len(got[0]) > 1 else None, got[1][1] if len(got[1]) > 1 else None)
    n, hq, d = s["q"].shape
    hk, page = s["kc"].shape[1], s["kc"].shape[2]
    o, lse = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda"), torch.empty(n, hq, dtype=torch.float64, device="cuda")
    kc, vc, table = s["kc"], s["vc"], s["table"].tolist()
    for i, length in enumerate(s["lens"].tolist()):
        kc[table[i][length // page], :, length % page] = s["k"][i]
        vc[table[i][length // page], :, length % page] = s["v"][i]
        begin = max(0, length + 1 - s["window"]) if s["window"] else 0
        ids = torch.tensor(table[i][: length // page + 1], device="cuda")
        k = kc[ids].transpose(0, 1).flatten(1, 2)[:, begin: length + 1].double()
        v = vc[ids].transpose(0, 1).flatten(1, 2)[:, begin: length + 1].double()
        score = s["scale"] * torch.einsum("hgd,htd->hgt", z["q"][i].view(hk, -1, d), k)
        lse[i] = torch.logsumexp(score, -1).flatten()
        o[i] = torch.einsum("hgt,htd->hgd", torch.softmax(score, -1), v).reshape(hq, d)
    return o, lse, kc.double(), vc.double()
