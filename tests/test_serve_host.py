"""Host-side checks of the serving operators' C ABI that need no GPU: bad
arguments are refused before the device is touched, workspaces are sized."""
import ctypes as C

import pytest

import verify_markov_head_gb300 as vm


@pytest.fixture(scope="module")
def host():
    return C.cast((C.c_float * 64)(), C.c_void_p)


def test_workspace_sizes():
    assert vm.dspark_cache_workspace_bytes(64, 32, 8, 128, 8) > 0
    assert vm.dspark_cache_workspace_bytes(64, 33, 8, 128, 8) == 0      # heads that do not divide
    assert vm.dspark_cache_workspace_bytes(64, 32, 8, 100, 8) == 0      # head size not a multiple of 8
    assert vm.dspark_cache_workspace_bytes(64, 32, 8, 264, 8) == 0
    assert vm.dspark_cache_workspace_bytes(4097, 32, 8, 128, 8) == 0
    assert vm.dspark_cache_workspace_bytes(64, 32, 8, 128, 18) == 0     # a block longer than gamma allows
    assert vm.dspark_logits_workspace_bytes(64, 8) >= 64 * 9 * 4
    assert vm.dspark_logits_workspace_bytes(64, 18) == 0
    assert vm.dspark_logits_workspace_bytes(0, 8) == 0


def test_plan_refuses_bad_sizes_and_host_memory(host):
    ok = dict(B=4, pages=100, width=8, page=16, T=32)

    def call(p=None, **kw):
        a = {**ok, **kw}
        return vm._lib.dspark_cache_plan(p, p, p, a["B"], p, p, a["pages"], p, a["width"], a["page"], p, p, p, p, p, p, p,
                                         a["T"], None, None)

    assert call(None) == -1 and call(host) == -1
    for kw in (dict(B=0), dict(B=4097), dict(pages=0), dict(page=0), dict(page=5000), dict(pages=1 << 28),
               dict(width=0), dict(width=1 << 28), dict(T=-1)):
        assert call(host, **kw) == -1, kw


def test_append_refuses_bad_arguments(host):
    def call(p, t=1, ks=256, vs=256, T=4, ps=4096, pages=10, page=16, heads=2, D=128):
        return vm._lib.dspark_cache_append(p, p, t, ks, vs, p, T, p, p, ps, pages, page, heads, D, None, None)

    assert call(None) == -1 and call(host) == -1
    assert call(host, t=2) == -4                                        # unknown type
    for kw in (dict(ks=255), dict(vs=260), dict(ks=128), dict(ps=4000), dict(D=12), dict(heads=0), dict(T=-1)):
        assert call(host, **kw) == -1, kw
    assert call(None, T=0) == 0                                         # nothing to write


def test_attention_refuses_bad_arguments(host):
    def call(p, qs=1024, t=1, ps=16384, page=16, width=4, B=2, N=4, Hq=8, Hkv=2, D=128, new=2, scale=1.0, ws=None, nb=0):
        return vm._lib.dspark_cache_attention(p, qs, p, p, t, ps, 10, page, p, width, p, p, p, B, N, Hq, Hkv, D, new,
                                              scale, p, None, ws, nb, None)

    assert call(None) == -1 and call(host) == -1
    assert call(host, t=5) == -4
    for kw in (dict(Hkv=3), dict(D=4), dict(new=0), dict(new=18), dict(scale=-1.0), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(qs=1023), dict(qs=512), dict(ps=100), dict(B=0), dict(N=-1), dict(width=0)):
        assert call(host, **kw) == -1, kw
    assert call(None, N=0) == 0


def test_logits_refuse_bad_arguments(host):
    def call(p, t=0, rs=64, B=2, R=3, V=64, hist=None, hist_len=None, draft=None, ds=0, nb=1 << 20,
             fill=float("-inf")):
        return vm._lib.dspark_logits_process(p, t, rs, p, B, R, V, hist, 4, hist_len, None, draft, ds, None, None, None,
                                             None, None, None, 0, None, fill, None, p, nb, None)

    assert call(None) == -1 and call(host) == -1
    assert call(host, t=3) == -4
    for kw in (dict(V=60), dict(V=0), dict(rs=63), dict(R=18), dict(R=0), dict(B=0), dict(B=70000), dict(nb=0),
               dict(fill=float("nan"))):
        assert call(host, **kw) == -1, kw
