"""Host-side checks of the cache in 4 bits, the rotary positions and the sampling
that need no GPU: bad arguments are refused before the device is touched,
workspaces are sized, frequencies and turns are formed."""
import ctypes as C
import math
from fractions import Fraction

import pytest
import torch

import verify_markov_head_gb300 as vm


@pytest.fixture(scope="module")
def host():
    return C.cast((C.c_float * 64)(), C.c_void_p)


def _rows(call, t=1, ks=256, vs=256, T=4, ps=2048, ss=256, pages=10, page=16, heads=2, D=128, ke=0, ve=0, p=None):
    if call == "append":
        return vm._lib.dspark_cache_append4(p, p, t, ks, vs, p, T, p, p, p, p, ps, ss, pages, page, heads, D, ke, ve, None, None)
    return vm._lib.dspark_cache_read4(p, p, p, p, ps, ss, pages, page, heads, D, ke, ve, p, T, p, p, t, ks, vs, None, None)


@pytest.mark.parametrize("call", ["append", "read"])
def test_rows_refuse_bad_arguments(call, host):
    assert _rows(call) == -1 and _rows(call, p=host) == -1              # null, and host memory
    assert _rows(call, t=2, T=0) == -4                                  # unknown type
    assert _rows(call, T=0) == 0                                        # nothing to do
    for kw in (dict(ks=255), dict(vs=260), dict(ks=128), dict(ps=2047), dict(ps=2052), dict(ss=255), dict(D=120), dict(D=272), dict(D=0),
               dict(heads=0), dict(heads=5000), dict(T=-1), dict(pages=0), dict(page=0), dict(page=5000), dict(pages=1 << 28), dict(ke=65), dict(ke=-65), dict(ve=65)):
        assert _rows(call, **{**dict(T=0), **kw}) == -1, kw
    assert _rows(call, T=0, ps=2056, ss=257, ke=-64, ve=64) == 0


def test_attention_refuses_bad_arguments(host):
    def call(p=None, qs=1024, t=1, ps=2048, ss=256, page=16, width=4, B=2, N=0, Hq=8, Hkv=2, D=128, new=2, scale=1.0, ke=0, ve=0, nb=0):
        return vm._lib.dspark_cache_attention4(p, qs, t, p, p, p, p, ps, ss, 10, page, ke, ve, p, width, p, p, p, B, N, Hq, Hkv, D, new,
                                               scale, p, None, p, nb, None)

    assert call() == 0
    assert call(N=4) == -1 and call(host, N=4) == -1
    assert call(t=5) == -4
    for kw in (dict(Hkv=3), dict(D=120), dict(D=8), dict(D=272), dict(new=0), dict(new=18), dict(scale=-1.0), dict(scale=0.0), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(scale=1e-30, ke=-64), dict(scale=1e30, ke=64), dict(qs=1023), dict(qs=512), dict(ps=2047), dict(ps=2056),
               dict(ss=255), dict(ss=257), dict(ke=65), dict(ve=-65), dict(B=0), dict(B=4097), dict(N=-1), dict(width=0), dict(width=(1 << 27) - 15)):
        assert call(**kw) == -1, kw
    # rows of 40 bytes of codes and 5 of scales: addresses of 8 and of 1
    assert call(D=80, qs=640, ps=1288, ss=161) == 0 and call(D=80, qs=640, ps=1284, ss=161) == -1


@pytest.mark.parametrize("heads,new", [(1, 1), (8, 1), (3, 3), (2, 8), (16, 1), (4, 8), (8, 8), (16, 8)])
def test_the_workspace_holds_two_tiles_of_rows_a_worker(heads, new):
    """Sums, maximum and weight of each row on 152 SMs: a warp to a tile of up to 32
    rows (12 warps an SM for 8 rows up to head size 128, else 8), or an SM to one of 64."""
    rows = heads * new
    for D in (16, 64, 128, 256):
        tile = 8 if rows <= 8 else 16 if rows <= 16 or D > 128 else 32
        warps = 12 if tile == 8 and D <= 128 else 8
        most = max(warps * tile, 64 if rows > 32 and D == 128 else 0)
        n = vm.dspark_cache4_workspace_bytes(3, 2 * heads, 2, D, new)
        assert n >= 256 + 152 * warps * 32 + 2 * 152 * most * (D + 2) * 4 and n >= vm.dspark_cache_workspace_bytes(3, 2 * heads, 2, D, new)
    assert vm.dspark_cache4_workspace_bytes(3, 2 * heads, 2, 120, new) == 0 and vm.dspark_cache4_workspace_bytes(0, 2 * heads, 2, 128, new) == 0


def test_rope_refuses_bad_arguments(host):
    def call(p=None, T=0, qs=1024, ks=256, t=1, rotary=128, mult=1.0, qos=1024, kos=256, Hq=8, Hkv=2, D=128):
        return vm._lib.dspark_rope(p, qs, p, ks, t, p, p, rotary, 0, mult, p, qos, p, kos, T, Hq, Hkv, D, None)

    assert call() == 0 and call(ks=0, kos=0, Hkv=0) == 0
    assert call(T=2) == -1 and call(host, T=2) == -1
    assert call(t=2) == -4
    for kw in (dict(T=-1), dict(Hq=0), dict(Hkv=-1), dict(Hq=8191, Hkv=2, qs=1 << 21, qos=1 << 21), dict(D=12), dict(D=264), dict(rotary=0), dict(rotary=3), dict(rotary=130),
               dict(mult=float("inf")), dict(mult=float("nan")), dict(qs=1020), dict(qs=1023), dict(qos=1020), dict(ks=128), dict(kos=260), dict(kos=128)):
        assert call(**kw) == -1, kw


def test_sampling_refuses_bad_arguments(host):
    assert vm.dspark_sample_workspace_bytes(0) > 0 and vm.dspark_sample_workspace_bytes(1 << 20) > 0
    assert vm.dspark_sample_workspace_bytes(-1) == 0 and vm.dspark_sample_workspace_bytes((1 << 20) + 1) == 0

    def call(p=None, t=0, rs=64, N=0, V=64, nb=1 << 20):
        return vm._lib.dspark_sample(p, t, rs, N, V, p, None, None, None, None, p, None, p, nb, None)

    assert call() == 0 and call(V=1 << 19) == 0
    assert call(N=2) == -1 and call(host, N=2) == -1
    assert call(t=3) == -4
    for kw in (dict(N=-1), dict(N=(1 << 20) + 1), dict(V=0), dict(V=(1 << 19) + 1), dict(N=2, rs=63), dict(N=2, V=65), dict(N=2, rs=66), dict(N=2, t=1, rs=68)):
        assert call(**kw) == -1, kw


# ------------------------------------------------------------------- binding
def _i(*s):
    return torch.zeros(s, dtype=torch.int32)


def _ws():
    buf = torch.zeros(1 << 24, dtype=torch.uint8)
    return type("W", (), {"buf": buf, "buf4": buf})


@pytest.mark.parametrize("call", ["append", "read", "attention"])
def test_the_binding_refuses_caches_that_do_not_fit(call):
    c = vm.Cache4(6, 2, 16, 64, device="cpu")
    k, ks = c.k, c.k_scale
    x = torch.zeros((3, 4 if call == "attention" else 2, 64), dtype=torch.bfloat16)

    def run(k=k, v=k, ks=ks, vs=ks, x=x, y=None, **kw):
        y = torch.empty(x.shape, dtype=x.dtype) if y is None else y
        if call == "append":
            vm.dspark_cache_append4(x, y, _i(x.shape[0]), k, v, ks, vs, stream=0, **kw)
        elif call == "read":
            vm.dspark_cache_read4(k, v, ks, vs, _i(x.shape[0]), x, y, stream=0, **kw)
        else:
            vm.dspark_cache_attention4(x, k, v, ks, vs, _i(1, 4), _i(1), _i(2), _i(2), y, _ws(), max_new=3, stream=0, **kw)

    with pytest.raises(vm.DsparkError):                          # all in order, but not on the device
        run()
    both = torch.zeros((6, 2, 2, 16, 32), dtype=torch.uint8)     # keys and values of a page side by side: fits
    with pytest.raises(vm.DsparkError):
        run(k=both[:, 0], v=both[:, 1])
    with pytest.raises(vm.DsparkError):
        run(k_exp=65)
    for kw in (dict(v=k[:5]), dict(v=both[:, 0]), dict(ks=ks[:5]), dict(vs=ks[..., :2]), dict(ks=ks[:, :1], vs=ks[:, :1]), dict(k=k.transpose(1, 2), v=k.transpose(1, 2)),
               dict(k=k[..., :16], v=k[..., :16]), dict(k=k[0]), dict(x=x[..., :32]), dict(x=x[:, :, None]),
               dict(x=torch.zeros((3, 64, x.shape[1]), dtype=torch.bfloat16).transpose(1, 2)), dict(y=x[:2]), dict(y=x.float())):
        with pytest.raises(ValueError):
            run(**kw)
    for kw in (dict(k=k.view(torch.int8), v=k.view(torch.int8)), dict(ks=ks.float()), dict(x=x.half(), y=x.half()), dict(k=None), dict(k_exp="1"), dict(v_exp=0.5)):
        with pytest.raises(TypeError):
            run(**kw)


def test_the_binding_refuses_heads_that_do_not_fit_rope():
    q, k, pos, table = torch.zeros((3, 4, 64)), torch.zeros((3, 2, 64)), _i(3), vm.RopeTable(32, device="cpu")
    with pytest.raises(vm.DsparkError):                          # all in order, but not on the device
        vm.dspark_rope(q, k, pos, table, stream=0)
    with pytest.raises(vm.DsparkError):
        vm.dspark_rope(q, None, pos, table, stream=0)
    with pytest.raises(vm.DsparkError):
        vm.dspark_rope(torch.zeros((3, 4, 16)), None, pos, table, stream=0)  # more turned than there is
    for a in ((q, k[:2], pos), (q, k[..., :32], pos), (q, k.bfloat16(), pos), (q, k, pos[:2]), (q[0], k, pos), (q.transpose(1, 2), None, pos),
              (q, k, pos, table, q[:2]), (q, k, pos, table, q.bfloat16()), (q, k, pos, table, q, k.bfloat16()), (q, None, pos, table, q, k)):
        with pytest.raises(ValueError):
            vm.dspark_rope(*a, **({} if len(a) > 3 else dict(table=table)), stream=0)
    for a in ((q.half(), None, pos), (q, k, pos.long())):
        with pytest.raises(TypeError):
            vm.dspark_rope(*a, table, stream=0)


def test_the_binding_refuses_rows_that_do_not_fit_sampling():
    x, f, tok = torch.zeros((3, 64)), torch.zeros(3), _i(3)
    good = dict(temperature=f, top_k=_i(3), top_p=f, min_p=f, logprob=f)
    run = lambda x=x, u=f, tok=tok, **kw: vm.dspark_sample(x, u, tok, _ws(), stream=0, **kw)  # noqa: E731
    with pytest.raises(vm.DsparkError):                          # all in order, but not on the device
        run(**good)
    for kw in (dict(u=f[:2]), dict(tok=_i(4)), dict(x=x[0]), dict(x=torch.zeros((64, 3)).T), dict(temperature=f[:2]), dict(top_k=_i(2)),
               dict(top_p=f[None]), dict(min_p=f[:0]), dict(logprob=torch.zeros(4))):
        with pytest.raises(ValueError):
            run(**{**good, **kw})
    for kw in (dict(x=x.half()), dict(u=f.double()), dict(tok=tok.long()), dict(top_k=f), dict(top_p=_i(3)), dict(logprob=f.bfloat16()), dict(u=None)):
        with pytest.raises(TypeError):
            run(**{**good, **kw})


# --------------------------------------------------------------- frequencies
def test_frequencies_follow_their_formulas():
    """Each to some roundings of 64 bits (powers and logarithms, 2^-50)."""
    r, base, f, n = 64, 10000.0, 4.0, 2048
    plain = [base ** (-2 * i / r) for i in range(r // 2)]

    def near(a, b):
        assert len(a) == len(b) and all(abs(x - y) <= 2.0 ** -50 * abs(y) for x, y in zip(a, b))

    got, mult = vm.rope_frequencies(r, base)
    near(got, plain)
    assert mult == 1.0
    got, mult = vm.rope_frequencies(r, base, dict(kind="linear", factor=f))
    near(got, [x / f for x in plain])
    got, mult = vm.rope_frequencies(r, base, dict(kind="ntk", factor=f))
    assert got[0] == 1.0 and abs(got[-1] * f / plain[-1] - 1) < 2.0 ** -48
    got, mult = vm.rope_frequencies(r, base, dict(kind="yarn", factor=f, trained=n))
    assert mult == 0.1 * math.log(f) + 1.0
    turns = [n * x / (2 * math.pi) for x in plain]
    for i in range(r // 2):
        # (the ramp's ends lie up to a pair further out)
        wider = turns[min(i + 1, r // 2 - 1)]
        if wider > 32:
            assert got[i] == plain[i]
        if turns[max(i - 1, 0)] < 1:
            assert got[i] == plain[i] / f
        assert plain[i] / f <= got[i] <= plain[i]
    assert vm.rope_frequencies(r, base, dict(kind="yarn", factor=f, trained=n, mult=2.0))[1] == 2.0
    got, _ = vm.rope_frequencies(r, base, dict(kind="wavelength", factor=f, trained=n, low=1, high=4))
    for x, y, t in zip(got, plain, turns):
        want = y if t > 4 else y / f if t < 1 else y * (t - 1) / 3 + y / f * (1 - (t - 1) / 3)
        assert abs(x - want) <= 2.0 ** -48 * y
    for bad in (dict(kind="other"), dict(kind="yarn"), dict(kind="wavelength", trained=n, low=4, high=4), dict(kind="linear", factor=0.0),
                dict(kind="linear", trained=4), dict(factor=float("nan")), dict(kind="yarn", trained=n, slow=0), dict(kind="wavelength", trained=-1)):
        with pytest.raises(ValueError):
            vm.rope_frequencies(r, base, bad)
    for a in ((0,), (3,), (64, 0.0), (64, float("inf")), (2, 10000.0, dict(kind="ntk", factor=2.0)), (64, 0.5, dict(kind="yarn", trained=n))):
        with pytest.raises(ValueError):
            vm.rope_frequencies(*a)


def test_turns_are_the_frequencies_in_64_bits():
    """To half a unit of 2^-64 turns; a full turn a position is none."""
    # 2 pi to 60 digits (Machin's formula in fractions)
    def arctan(n):
        x, total, k = Fraction(1, n), Fraction(0), 0
        while k < 130:
            total += x / (2 * k + 1) * (-1) ** k
            x /= n * n
            k += 1
        return total

    turn = 8 * (4 * arctan(5) - arctan(239))
    for freq in ([1.0, 0.25], [1e-9, -1e-9], [6.25, 100.0]):
        t = vm.RopeTable(4, frequencies=freq, device="cpu")
        for got, f in zip(t.turns.tolist(), freq):
            off = (Fraction(f) / turn * 2 ** 64 - got) % 2 ** 64
            assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 2 ** 20)
    assert abs(vm.RopeTable(2, frequencies=[2 * math.pi], device="cpu").turns.item()) < 2 ** 14
    for a, kw in (((4,), dict(frequencies=[1.0])), ((4,), dict(frequencies=[1.0, float("nan")]))):
        with pytest.raises(ValueError):
            vm.RopeTable(*a, device="cpu", **kw)


def test_a_cache_of_4_bits_has_whole_groups():
    c = vm.Cache4(5, 2, 16, 96, k_exp=-1, v_exp=2, device="cpu")
    assert [tuple(t.shape) for t in c.tensors] == [(5, 2, 16, 48)] * 2 + [(5, 2, 16, 6)] * 2
    assert (c.k_exp, c.v_exp) == (-1, 2) and not any(t.any() for t in c.tensors)
    with pytest.raises(ValueError):
        vm.Cache4(5, 2, 16, 100, device="cpu")
