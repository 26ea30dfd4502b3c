"""Calls on a stream that is not the current one: what they allocate belongs to
that stream, so neither earlier nor later work of the current stream touches it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

CYCLES = 100_000_000  # about 50 ms: the other stream is surely behind


def calls(kda):
    g = torch.Generator("cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    la, x, dh = -torch.rand(2, 300, 264, device="cuda", generator=g), rand(2, 300, 264), rand(2, 300, 264)
    h, _ = kda.recurrence_fwd(la, x)
    q, k, wq, wk = rand(500, 6, 64), rand(500, 2, 64), rand(64), rand(64)
    dq, dk = rand(500, 6, 64), rand(500, 2, 64)
    aq, kc, vc = rand(5, 6, 64), rand(40, 2, 16, 64), rand(40, 2, 16, 64)
    table = torch.randperm(40, device="cuda", generator=g).to(torch.int32).view(5, 8)
    lens = torch.tensor([0, 3, 70, 128, 17], dtype=torch.int32, device="cuda")

    def bwd(s):
        r = kda.recurrence_bwd(la, h, None, dh, stream=s)
        return r["dx"], r["dlog_alpha"], r["dh0"]

    def qk_bwd(s):
        r = kda.qk_norm_rope_bwd(dq, dk, q, k, wq, wk, stream=s)
        return r["dq"], r["dk"], r["dq_weight"], r["dk_weight"]

    return {
        "recurrence_fwd": lambda s: kda.recurrence_fwd(la, x, stream=s),
        "recurrence_bwd": bwd,
        "recurrence_step": lambda s: kda.recurrence_step(la[0], x[0], dh[0], h_out=torch.empty_like(dh[0]), stream=s)[:1],
        "qk_norm_rope": lambda s: kda.qk_norm_rope(q, k, wq, wk, stream=s),
        "qk_norm_rope_bwd": qk_bwd,
        "attn_decode": lambda s: kda.attn_decode(aq, kc, vc, table, lens, return_lse=True, stream=s),
    }


def poison(sizes):
    """Zeros all over memory of the sizes that a call takes, by work that the current stream has yet to do."""
    for _ in range(3):
        for t in [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]:
            t.zero_()


@pytest.mark.parametrize("name", ["recurrence_fwd", "recurrence_bwd", "recurrence_step", "qk_norm_rope", "qk_norm_rope_bwd",
                                  "attn_decode"])
@pytest.mark.parametrize("behind", ["current", "given"])
def test_memory_of_a_given_stream(cuda_lib, name, behind):
    call = calls(cuda_lib)[name]
    want = [t.clone() for t in call(None)]
    sizes = [t.numel() * t.element_size() for t in want]
    sizes += [cuda_lib.attn_decode_workspace_size(5, 6, 2, 64), cuda_lib.load().kda_qk_norm_rope_bwd_workspace_size(500, 6, 2, 64)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if behind == "current":  # its pending writes to memory that it has given back
        torch.cuda._sleep(CYCLES)
        poison(sizes)
        got = call(side)
    else:  # its later writes to memory that the call has given back
        with torch.cuda.stream(side):
            torch.cuda._sleep(CYCLES)
        got = call(side)
        poison(sizes)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_more_tokens_than_the_calls_count(cuda_lib):
    q = torch.randn(1, 1, 8, device="cuda").expand(2 ** 32 + 5, 1, 8)
    with pytest.raises(ValueError, match="tokens"):
        cuda_lib.qk_norm_rope(q, q)
