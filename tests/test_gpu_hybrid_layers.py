"""The operators together, as the layers of a hybrid decoder stack run them: a
prompt and then single tokens through a delta-rule layer (L2-normalised queries
and keys), a softmax layer (RMS norm, rotation, paged cache) and a gated linear
recurrence. Every layer's outputs are checked against 64-bit forms on the inputs
that the layer saw, and the single tokens must continue what the prompt left."""
import numpy as np
import pytest
import torch

import oracle
from tests import stack_reference as R

pytestmark = pytest.mark.gpu

DELTA_BAR = 2e-2  # the bf16 bar of the delta rule's own parity tests: max|x - ref| / max|ref|


def rel_err(x, ref):
    x, ref = np.asarray(x, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    return float(np.abs(x - ref).max() / np.abs(ref).max())


def test_prompt_and_decode(cuda_lib):
    kda = cuda_lib
    B, T, steps, H, Hq, Hk, d, page = 2, 150, 5, 2, 8, 2, 128, 32
    far, rot = 400, 64
    g = torch.Generator().manual_seed(77)
    total = T + steps
    bf = lambda *shape, std=1.0: (std * torch.randn(*shape, generator=g)).bfloat16()  # noqa: E731
    ang = torch.arange(far)[:, None].double() * 10000.0 ** (-torch.arange(0, rot, 2).double() / rot)
    cos, sin = ang.cos().float(), ang.sin().float()
    wq, wk = (1 + bf(d, std=0.1)).bfloat16(), (1 + bf(d, std=0.1)).bfloat16()
    # projections of all tokens, as the layers would get them
    lin = {"qk": bf(B, total, 2 * H, d), "v": bf(B, total, H, d), "la": -torch.rand(B, total, H, d, generator=g).bfloat16() * 0.1,
           "beta": torch.sigmoid(torch.randn(B, total, H, generator=g)).bfloat16()}
    att = {"qkv": bf(B, total, Hq + 2 * Hk, d)}
    rec = {"la": -torch.rand(B, total, H * d, generator=g).bfloat16(), "x": bf(B, total, H * d)}
    dev = lambda t: t.cuda()  # noqa: E731
    cosd, sind, wqd, wkd = map(dev, (cos, sin, wq, wk))

    # ---- the prompt
    qk = dev(lin["qk"][:, :T].contiguous())
    q, k = kda.qk_norm_rope(qk[:, :, :H], qk[:, :, H:], norm="l2", eps=1e-6)
    R.close(q.view(-1, H, d), *R.qk_norm_rope(lin["qk"][:, :T, :H].reshape(-1, H, d), None, None, None, None, "l2", 1e-6))
    sl = lambda t, a, b: dev(t[:, a:b].contiguous())  # noqa: E731
    o, S = kda.chunk_fwd(q, k, sl(lin["v"], 0, T), sl(lin["la"], 0, T), sl(lin["beta"], 0, T))
    qh, kh = [q.cpu()], [k.cpu()]
    ro, rS = oracle.recurrent(q.cpu(), k.cpu(), lin["v"][:, :T], lin["la"][:, :T], lin["beta"][:, :T])
    assert rel_err(o.float().cpu(), ro) <= DELTA_BAR and rel_err(S.cpu(), rS) <= DELTA_BAR

    qkv = dev(att["qkv"][:, :T].contiguous())
    pos = torch.arange(T, device="cuda").repeat(B)
    aq, ak = kda.qk_norm_rope(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], wqd, wkd, cosd, sind, pos)
    # the prompt's keys and values into the pages
    held = -(-(total) // page)
    table = torch.randperm(B * held, generator=g).to(torch.int32).view(B, held)
    kc = torch.full((B * held, Hk, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    at = torch.arange(T)
    for b in range(B):
        where, row = table[b][at // page].long(), at % page
        kc[where.cuda(), :, row.cuda()] = ak[b]
        vc[where.cuda(), :, row.cuda()] = qkv[b, :, Hq + Hk:]
    h, hT = kda.recurrence_fwd(sl(rec["la"], 0, T), sl(rec["x"], 0, T))

    # ---- single tokens, the states in place
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
    kcr, vcr = kc.cpu(), vc.cpu()
    outs, hs, state = [], [h.cpu()], hT.clone()
    for t in range(T, total):
        one = dev(lin["qk"][:, t].contiguous())
        q1, k1 = kda.qk_norm_rope(one[:, :H], one[:, H:], norm="l2", eps=1e-6)
        o1, S = kda.decode_step(q1, k1, dev(lin["v"][:, t].contiguous()), dev(lin["la"][:, t].contiguous()),
                                dev(lin["beta"][:, t].contiguous()), S)
        qh.append(q1.cpu()[:, None]), kh.append(k1.cpu()[:, None]), outs.append(o1.float().cpu())

        new = dev(att["qkv"][:, t].contiguous())
        p1 = torch.full((B,), t, device="cuda")
        q2, k2 = kda.qk_norm_rope(new[:, :Hq], new[:, Hq:Hq + Hk], wqd, wkd, cosd, sind, p1)
        R.close(q2, *R.qk_norm_rope(att["qkv"][:, t, :Hq], wq, cos, sin, p1.cpu(), "rms", 1e-6))
        v2 = new[:, Hq + Hk:].contiguous()
        a = kda.attn_decode(q2, kc, vc, dev(table), lens, k=k2, v=v2)
        want, _ = R.attn_decode(q2.cpu(), kcr, vcr, table, [t] * B, k2.cpu(), v2.cpu())
        R.close(a, *want, f"attention at {t}")
        lens += 1

        y, state = kda.recurrence_step(dev(rec["la"][:, t].contiguous()), dev(rec["x"][:, t].contiguous()), state)
        hs.append(y.cpu()[:, None])
    torch.cuda.synchronize()
    # the whole run of each recurrent layer, prompt and single tokens as one sequence
    ro, rS = oracle.recurrent(torch.cat(qh, 1), torch.cat(kh, 1), lin["v"], lin["la"], lin["beta"])
    assert rel_err(torch.stack(outs, 1), ro[:, T:]) <= DELTA_BAR and rel_err(S.cpu(), rS) <= DELTA_BAR
    for b in range(B):
        (want, slack), (end, slack_end) = R.recurrence_fwd(rec["la"][b], rec["x"][b])
        R.close(torch.cat(hs, 1)[b], want, 2 * slack)  # the prompt's bound and the steps'
        R.close(state[b], end, 2 * slack_end)


def test_training_step_gradients(cuda_lib):
    """A loss through the query/key norm and the delta rule, and one through the recurrence: the chained backward calls
    against the 64-bit chain rule on the same intermediate tensors."""
    kda = cuda_lib
    B, T, H, d = 1, 70, 2, 64
    g = torch.Generator().manual_seed(78)
    x = 2 * torch.randn(B, T, 2 * H, d, generator=g)
    v, beta = torch.randn(B, T, H, d, generator=g), torch.sigmoid(torch.randn(B, T, H, generator=g))
    la, dO = -torch.rand(B, T, H, d, generator=g) * 0.1, torch.randn(B, T, H, d, generator=g)
    xd = x.cuda()
    q, k = kda.qk_norm_rope(xd[:, :, :H], xd[:, :, H:], norm="l2", eps=1e-6)
    gr = kda.chunk_bwd(q, k, v.cuda(), la.cuda(), beta.cuda(), None, dO.cuda())
    gx = kda.qk_norm_rope_bwd(gr["dq"], gr["dk"], xd[:, :, :H], xd[:, :, H:], norm="l2", eps=1e-6)
    for name, side, part in (("dq", "dq", x[:, :, :H]), ("dk", "dk", x[:, :, H:])):
        want, _ = R.qk_norm_rope_bwd(gr[side].cpu().view(-1, H, d), part.reshape(-1, H, d), None, None, None, None, "l2", 1e-6)
        R.close(gx[name].view(-1, H, d), *want, name)
    # against differences of the whole loss, in the direction of the gradient itself (64-bit oracle)
    def loss(xx):
        n = xx.double() / (xx.double().square().sum(-1, keepdim=True) + 1e-6).sqrt()
        o, _ = oracle.recurrent(n[:, :, :H], n[:, :, H:], v, la, beta)
        return float((np.asarray(o, dtype=np.float64) * dO.double().numpy()).sum())

    full = torch.cat([gx["dq"], gx["dk"]], 2).cpu().double()
    way = full / full.norm()
    eps = 1e-3
    slope = (loss(x.double() + eps * way) - loss(x.double() - eps * way)) / (2 * eps)
    # central differences leave eps^2 of a third derivative, 1e-6 of the slope's scale; the gradient is 32-bit: 1e-4
    assert abs(slope - float(full.norm())) <= 1e-3 * abs(slope)
