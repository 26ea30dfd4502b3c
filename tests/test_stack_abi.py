"""CPU tests of the C-ABI boundary of the recurrence, the query/key norm and the
decode attention: bad arguments are refused with a status before anything is
launched, and the Python binding refuses CPU tensors. Every combination below
fails validation, so nothing reaches a device."""
import ctypes
import math

import pytest
import torch

import gated_delta_rule_134_b200 as kda

P = [ctypes.c_void_p(0x1000 * (i + 1)) for i in range(20)]
ODD = ctypes.c_void_p(0x9008)
HALF = ctypes.c_void_p(0x9002)


def rec_fwd(la=P[0], x=P[1], h0=None, h=P[2], h_T=None, cu=None, N=1, T=4, D=8, dtype=1):
    return kda.load().kda_recurrence_fwd(la, x, h0, h, h_T, cu, N, T, D, dtype, None)


def rec_bwd(la=P[0], h=P[1], h0=None, dh=P[2], dT=None, dx=P[3], dla=P[4], d0=None, cu=None, N=1, T=4, D=8, dtype=1):
    return kda.load().kda_recurrence_bwd(la, h, h0, dh, dT, dx, dla, d0, cu, N, T, D, dtype, None)


@pytest.mark.parametrize("bad", [dict(la=None), dict(x=None), dict(h=None), dict(la=ODD), dict(x=ODD), dict(h=ODD), dict(h0=ODD),
                                 dict(h_T=ODD), dict(cu=HALF), dict(N=-1), dict(T=-1), dict(D=0), dict(dtype=2), dict(N=1 << 30, D=4096), dict(D=(1 << 30) + 1)])
def test_recurrence_fwd_refuses(bad):
    assert rec_fwd(**bad) == 1


@pytest.mark.parametrize("bad", [dict(la=None), dict(h=None), dict(dh=None), dict(dx=None), dict(dla=None), dict(dla=ODD), dict(h=ODD),
                                 dict(h0=ODD), dict(dT=ODD), dict(d0=ODD), dict(cu=HALF), dict(N=-1), dict(T=-1), dict(D=-3), dict(dtype=-1)])
def test_recurrence_bwd_refuses(bad):
    assert rec_bwd(**bad) == 1


def test_recurrence_timeout_hook_refuses():
    f = kda.load().kda_recurrence_timeout_test
    good = dict(la=P[0], x=P[1], h=P[2], N=1, T=600, D=64, dtype=1, budget=1 << 20)
    for bad in (dict(budget=0), dict(budget=-1), dict(budget=(1 << 31) + 1), dict(T=100), dict(D=4096), dict(N=0), dict(N=40, D=128),
                dict(x=None), dict(h=ODD), dict(dtype=5)):
        a = {**good, **bad}
        assert f(a["la"], a["x"], a["h"], a["N"], a["T"], a["D"], a["dtype"], a["budget"], None) == 1, bad


def test_recurrence_step_refuses():
    f = kda.load().kda_recurrence_step
    good = P[:5]
    for i in range(5):
        for worse in (None, ODD):
            p = list(good)
            p[i] = worse
            assert f(*p, 2, 8, 1, None) == 1
    assert f(*good, -1, 8, 1, None) == 1
    assert f(*good, 2, 0, 1, None) == 1
    assert f(*good, 2, 8, 3, None) == 1
    assert f(*[None] * 5, 0, 8, 1, None) == 0  # nothing to do


def qk(q=P[0], k=P[1], wq=None, wk=None, cos=P[2], sin=P[3], pos=P[4], pos_bytes=8, qo=P[5], ko=P[6], n=2, Hq=4, Hk=2, d=64, rot=64,
       far=10, qt=256, qh=64, kt=128, kh=64, norm=1, eps=1e-6, inter=0, dtype=1, bwd=False, dq=P[7], dk=P[8], dwq=None, dwk=None, ws=None, ws_len=0):
    lib = kda.load()
    tail = (n, Hq, Hk, d, rot, far, qt, qh, kt, kh, norm, eps, 1.0, inter, dtype)
    if bwd:
        return lib.kda_qk_norm_rope_bwd(dq, dk, q, k, wq, wk, cos, sin, pos, pos_bytes, qo, ko, dwq, dwk, *tail, ws, ws_len, None)
    return lib.kda_qk_norm_rope(q, k, wq, wk, cos, sin, pos, pos_bytes, qo, ko, *tail, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("bad,status", [
    (dict(q=None), 1), (dict(k=ODD), 1), (dict(wq=ODD), 1), (dict(wk=ODD), 1), (dict(cos=None), 1), (dict(sin=ODD), 1), (dict(pos=ctypes.c_void_p(0x5004)), 1),
    (dict(pos=HALF, pos_bytes=4), 1), (dict(pos_bytes=2), 1), (dict(qo=None), 1), (dict(ko=ODD), 1), (dict(n=-1), 1), (dict(Hq=-1), 1),
    (dict(Hk=-2), 1), (dict(Hq=70000), 1), (dict(d=60), 2), (dict(d=264), 2), (dict(d=0), 2), (dict(rot=8), 2), (dict(rot=24), 2), (dict(rot=80), 2), (dict(far=0), 1),
    (dict(qt=260), 1), (dict(qh=68), 1), (dict(kt=1), 1), (dict(kh=-4), 1), (dict(norm=2), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1),
    (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(inter=2), 1), (dict(dtype=9), 1)])
def test_qk_refuses(bad, status, bwd):
    assert qk(**bad, bwd=bwd) == status


@pytest.mark.parametrize("bad", [dict(dq=None), dict(dk=ODD), dict(dwq=P[9]), dict(dwq=P[9], ws=P[10], ws_len=8), dict(dwk=P[9], ws=ODD, ws_len=1 << 30), dict(dwk=ODD)])
def test_qk_bwd_refuses(bad):
    assert qk(**bad, bwd=True) == 1


def test_qk_workspace_size():
    lib = kda.load()
    assert lib.kda_qk_norm_rope_bwd_workspace_size(100, 8, 2, 128) > 0
    assert lib.kda_qk_norm_rope_bwd_workspace_size(-1, 8, 2, 128) == 0
    assert lib.kda_qk_norm_rope_bwd_workspace_size(100, 8, 2, 100) == 0


def attn(q=P[0], k=P[1], v=P[2], kc=P[3], vc=P[4], table=P[5], lens=P[6], o=P[7], lse=None, N=2, Hq=4, Hk=2, d=64, pages=8, page=16,
         most=4, window=0, scale=0.1, dtype=1, ws=ctypes.c_void_p(0x100000), ws_len=1 << 40):
    return kda.load().kda_attn_decode(q, k, v, kc, vc, table, lens, o, lse, N, Hq, Hk, d, pages, page, most, window, scale, dtype, ws, ws_len, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), 1), (dict(q=ODD), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(k=ODD), 1), (dict(v=ODD), 1), (dict(kc=None), 1), (dict(vc=ODD), 1),
    (dict(table=None), 1), (dict(table=HALF), 1), (dict(lens=None), 1), (dict(lens=HALF), 1), (dict(o=None), 1), (dict(o=ODD), 1), (dict(lse=HALF), 1),
    (dict(N=-1), 1), (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(Hk=0), 1), (dict(Hk=-2), 1), (dict(d=96), 2), (dict(d=256), 2), (dict(pages=-1), 1), (dict(page=0), 1),
    (dict(most=-1), 1), (dict(most=1 << 28, page=16), 1), (dict(N=1 << 28), 1), (dict(N=1 << 21, most=1 << 25, page=16), 1), (dict(pages=1 << 30, page=2), 1), (dict(pages=1 << 26, page=16), 1), (dict(window=-1), 1), (dict(scale=math.nan), 1), (dict(dtype=2), 1)])
def test_attn_refuses(bad, status):
    assert attn(**bad) == status


def test_attn_workspace():
    lib = kda.load()
    assert lib.kda_attn_decode_workspace_size(4, 5, 2, 64) == 0   # not a multiple
    assert lib.kda_attn_decode_workspace_size(4, 8, 2, 96) == 0
    need = lib.kda_attn_decode_workspace_size(4, 8, 2, 128)
    if need:
        assert attn(N=4, Hq=8, d=128, ws=None, ws_len=0) == 1
        assert attn(N=4, Hq=8, d=128, ws_len=need - 1) == 1
        assert attn(N=4, Hq=8, d=128, ws=ODD, ws_len=need) == 1


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.recurrence_fwd(x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.recurrence_bwd(x, x, None, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.recurrence_step(x[0], x[0], x[0])
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.qk_norm_rope(x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.qk_norm_rope_bwd(x, x, x, x)
    q, cache = torch.zeros(2, 4, 64), torch.zeros(3, 2, 16, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.attn_decode(q, cache, cache, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


def test_binding_refuses_sizes_past_int32():
    far = torch.empty(2 ** 32 + 5, 1, device="meta")
    cu = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: kda.recurrence_fwd(far, far, cu_seqlens=cu), lambda: kda.recurrence_fwd(far[None], far[None]),
                 lambda: kda.recurrence_step(far, far, far)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    q, cache = torch.zeros(1, 1, 64), torch.zeros(1, 1, 16, 64)
    for window in (2 ** 32 + 5, -2 ** 32):
        with pytest.raises(ValueError, match="window"):
            kda.attn_decode(q, cache, cache, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), window=window)


@pytest.mark.parametrize("bad", ["other device", "expanded", "strided"])
def test_binding_refuses_workspaces_that_are_not_its_memory(bad):
    """Tensors that stand for CUDA tensors without memory: a call that went on would fail in another way."""
    from torch._subclasses import FakeTensorMode
    with FakeTensorMode():
        cuda = dict(device="cuda", dtype=torch.bfloat16)
        i32 = dict(device="cuda", dtype=torch.int32)
        size = 1 << 24
        ws = {"other device": lambda: torch.empty(size, dtype=torch.uint8),
              "expanded": lambda: torch.empty(1, device="cuda", dtype=torch.uint8).expand(size),
              "strided": lambda: torch.empty(size, 2, device="cuda", dtype=torch.uint8)[:, 0]}[bad]()
        q, cache = torch.empty(2, 4, 64, **cuda), torch.empty(3, 2, 16, 64, **cuda)
        with pytest.raises(ValueError, match="workspace"):
            kda.attn_decode(q, cache, cache, torch.empty(2, 2, **i32), torch.empty(2, **i32), workspace=ws)
        w = torch.empty(64, **cuda)
        with pytest.raises(ValueError, match="workspace"):
            kda.qk_norm_rope_bwd(q, q, q, q, w, w, workspace=ws)


def test_tokens_of_the_longest_packed_batches(tmp_path):
    """What the recurrence's plan goes by, compiled for the host: sequences of 2^30 tokens must not count as negative."""
    import shutil
    import subprocess

    from gated_delta_rule_134_b200 import build
    src, exe = tmp_path / "tokens.cpp", tmp_path / "tokens"
    src.write_text("""#include <cstdio>
#include "kda_internal.h"
int main() {
    const int cu = 0, sizes[][2] = {{1, 5}, {2, 5}, {2, 0x7fffffff}, {1 << 26, 0x7fffffff}};
    for (auto& s : sizes) {
        kda::RecurrenceArgs a{};
        a.N = s[0]; a.T = s[1];
        const long long dense = kda::tokens_of(a);
        a.cu_seqlens = &cu;
        std::printf("%lld %lld\\n", dense, kda::tokens_of(a));
    }
}
""")
    cuda = str(build.NVCC).rsplit("/bin/", 1)[0]
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-I", cuda + "/include", str(src), "-o", str(exe)], check=True)
    got = [tuple(map(int, line.split())) for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    assert got == [(5, 5), (5, 3), (0x7fffffff, 1 << 30), (0x7fffffff, 32)]
