"""GPU tests of the cache in 4 bits and the sampling at the edges of their types:
queries that are no numbers, light tokens, cuts that change nothing, flat rows."""
import numpy as np
import pytest
import torch

from tests import _serve4_ref as ref
from tests import test_gpu_serve4 as s4
from tests.test_gpu_serve4 import BF16, F32, _attend, _cache, _case, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vm():
    import verify_markov_head_gb300 as vm
    return vm


def _check(q, arrays, table, lens, q_off, scale, got, lse, k_exp=0, v_exp=0):
    """test_gpu_serve4's check, and the logarithms are NaN where the definition's are and nowhere else."""
    s4._check(q, arrays, table, lens, q_off, scale, got, lse, k_exp, v_exp)
    K, V = ref.values(arrays[0], arrays[2], k_exp), ref.values(arrays[1], arrays[3], v_exp)
    _, want, _, _ = ref.attention(_np(q), K, V, table, lens, q_off, scale, q.dtype == BF16)
    a, b = q_off[0], q_off[-1]
    np.testing.assert_array_equal(np.isnan(_np(lse)[a:b]), np.isnan(want[a:b]))


# ----------------------------------------------------------------- attention
# (rows of a key head, tokens of the block): registers, few requests and many rows on the tensor cores
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,n", [(3, 3), (16, 4), (24, 2), (32, 8), (40, 5), (64, 4), (136, 8)])
def test_a_query_that_is_no_number_reaches_its_own_row_alone(vm, rows, n, dtype):
    """NaN and infinities in four rows of a block: every other row keeps its own bound."""
    rng = np.random.default_rng(rows)
    P, lens, D = 16, [500, 90], 128
    G, q_off = rows // n, np.array([0, n, 2 * n])
    pages, table = _case(rng, 2, P, lens, D, 2)
    arrays = _cache(rng, pages, 2, P, D)
    q = torch.from_numpy(rng.standard_normal((2 * n, 2 * G, D))).to(dtype).cuda()
    clean, clean_lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, n)
    assert status == 0
    bad = [(0, 0, float("nan")), (n - 1, G - 1, float("inf")), (n, G, float("-inf")), (2 * n - 1, 2 * G - 1, float("nan"))]
    for t, h, x in bad:
        q[t, h, 77] = x
    got, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, n)
    assert status == 0
    _check(q, arrays, table, lens, q_off, np.float32(D ** -0.5), got, lse)
    for t, h, _ in bad:
        assert bool(torch.isnan(got[t, h]).all()) and bool(torch.isnan(lse[t, h]))


@pytest.mark.parametrize("lo,hi", [(-60, 0), (0, 60), (-110, -20)])
@pytest.mark.parametrize("rows,n", [(24, 2), (64, 4), (136, 8)])
def test_rows_of_a_tile_keep_their_own_precision(vm, rows, n, lo, hi):
    """Queries of sizes 2^lo .. 2^hi in one block: a row is as exact as by itself."""
    rng = np.random.default_rng(rows + hi)
    P, lens, D, G = 16, [300], 128, rows // n
    pages, table = _case(rng, 1, P, lens, D, 1)
    arrays = _cache(rng, pages, 1, P, D)
    size = 2.0 ** rng.permutation(np.linspace(lo, hi, n * G).round())
    q = torch.from_numpy(np.clip(rng.standard_normal((n, G, D)), -1, 1) * size.reshape(n, G, 1)).to(BF16).cuda()
    for at in (lo, (lo + hi) // 2, hi):                     # scores of ordinary size from the smallest rows, the middle ones, the largest
        scale = float(2.0 ** -at)
        got, lse, status = _attend(vm, rng, q, arrays, table, lens, np.array([0, n]), n, scale=scale)
        assert status == 0
        _check(q, arrays, table, lens, np.array([0, n]), scale, got, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,Hq,Hkv,D,P,new,lens", [
    (1, 8, 1, 128, 16, 1, [9000]), (1, 32, 4, 128, 64, 8, [2000]), (1, 24, 1, 128, 16, 1, [3000]), (3, 4, 1, 256, 32, 3, [4000, 0, 33]), (2, 6, 2, 96, 24, 2, [700, 1])])
def test_a_value_that_is_no_number_leaves_the_logarithm(vm, B, Hq, Hkv, D, P, new, lens, dtype):
    """NaN groups among the values, over segments that several CTAs share: lse stays a number, out is NaN in that group alone."""
    rng = np.random.default_rng(D + Hq)
    q_off = np.concatenate([[0], np.cumsum(np.minimum(new, lens))])
    pages, table = _case(rng, B, P, lens, D, Hkv)
    arrays = _cache(rng, pages, Hkv, P, D, spread=0.1)       # (weights of one size: none underflows)
    for pos in (0, lens[0] // 2, lens[0] - 1):
        arrays[3][table[0, pos // P], Hkv - 1, pos % P, 1] = 0x7F
    q = torch.from_numpy(rng.standard_normal((int(q_off[-1]), Hq, D))).to(dtype).cuda()
    got, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, new)
    assert status == 0 and not bool(torch.isnan(lse).any())
    _check(q, arrays, table, lens, q_off, np.float32(D ** -0.5), got, lse)
    # and a key that is no number: the whole rows that see it
    arrays[2][table[0, 5 // P], 0, 5 % P, 2] = 0x7F
    got, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, new)
    assert status == 0 and bool(torch.isnan(lse[0, :Hq // Hkv]).all())
    _check(q, arrays, table, lens, q_off, np.float32(D ** -0.5), got, lse)


# ------------------------------------------------------------------ sampling
def _model_rows(rng, N, V, dtype):
    """Rows of a model's kind: some candidates stand out, their lead falls with the rank."""
    x = rng.standard_normal((N, -(-V // 8) * 8)) * 1.5
    for r in x:
        r[rng.choice(V, 400, replace=False)] += 9 - rng.uniform(1.2, 1.8) * np.log(np.arange(1, 401))
    return torch.from_numpy(x).to(dtype).cuda()[:, :V]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1000, 32003, 151936])
def test_top_k_beyond_the_entries_that_weigh_something(vm, V, dtype):
    """Low temperatures: fewer entries than top_k weigh anything, and the cut changes nothing."""
    rng = np.random.default_rng(V)
    N = 12
    x = _model_rows(rng, N, V, dtype)
    x[0, :] = float("-inf")
    x[0, V // 2], x[0, V - 1] = 1.0, 1.0                    # fewer entries than top_k at all
    x[1, 7:] -= 1e4
    u = rng.random(N).astype(np.float32)
    for T in (0.02, 0.05, 0.1):
        for k in (20, 50, 200, 600, 5000):
            for p, m in ((None, None), (0.9, None), (0.5, 1e-3)):
                args = (np.full(N, T), np.full(N, k), None if p is None else np.full(N, p), None if m is None else np.full(N, m))
                tok, lp, status = s4._sample(vm, x, u, *args)
                assert status == 0
                s4._check_rows(x, u, *args, tok, lp)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [129280, 151936, 1 << 19])
def test_many_light_entries_count_with_their_whole_weight(vm, V, dtype):
    """One entry far above all others, which are equal or nearly so: the share that
    is not its own is the sum of weights of 2^-24 to 2^-47."""
    rng = np.random.default_rng(V)
    gaps = np.array([24.3, 30.3, 33.3, 36.5, 38.7, 40.4, 44.6, 47.1])
    N = len(gaps)
    x = torch.zeros((N, V + 8 - V % 8), dtype=dtype)[:, :V]
    x[:, 1::2] = -0.01                                      # (bf16 holds it well enough)
    x[:, 70001] = torch.from_numpy(gaps * np.log(2)).to(dtype)
    x, u = x.cuda(), rng.uniform(0.2, 0.8, N).astype(np.float32)
    one, k = np.ones(N), np.full(N, V - 3)
    for args in ((None,) * 4, (None, None, one * (1 - 2.0 ** -24), None), (None, k, None, None), (None, None, None, one * 1e-30), (one * 0.9, k, one * (1 - 2.0 ** -23), None)):
        tok, lp, status = s4._sample(vm, x, u, *args)
        assert status == 0 and (tok == 70001).all()
        s4._check_rows(x, u, *args, tok, lp)
    # rows of few light entries among heavy ones, whose unit is coarser
    x[:, :1000] = 30.0
    for args in ((None,) * 4, (None, None, one * 0.999, None), (one * 5, None, one * 0.9, None)):
        tok, lp, status = s4._sample(vm, x, u, *args)
        assert status == 0
        s4._check_rows(x, u, *args, tok, lp)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [600, 5000, 151936])
@pytest.mark.parametrize("T", [1.0, 0.3])
def test_the_logarithm_of_a_light_token(vm, V, dtype, T):
    """u = 0 draws the first id that weighs something, however little."""
    rng = np.random.default_rng(V)
    far = np.array([5.0, 12.0, 18.0, 22.0, 25.0, 27.0, 29.0])
    N = len(far)
    x = torch.from_numpy(rng.standard_normal((N, -(-V // 8) * 8))).to(dtype)[:, :V]
    x[:, V // 2] = 8.0
    x[:, 0] = torch.from_numpy(8.0 - far * T).to(dtype)
    x, one = x.cuda(), np.ones(N)
    for k in (None, 500, V - 1):
        tok, lp, status = s4._sample(vm, x, np.zeros(N), T=one * T, k=None if k is None else np.full(N, k))
        assert status == 0
        for i, row in enumerate(_np(x)):
            w = np.exp((row - row.max()) / float(np.float32(T)))
            if k is not None:
                w[np.argsort(-row, kind="stable")[k:]] = 0
            assert tok[i] == np.flatnonzero(w)[0]
            want = np.log(w[tok[i]] / w.sum())
            # a difference, a quotient and a sum rounded to binary32, the logarithm's own, and 2^-29
            assert abs(lp[i] - want) <= 2.0 ** -29 + 4 * ref.EPS32 * abs(want), (i, tok[i], lp[i], want)


# ------------------------------------------------------------------ refusals
def test_rows_and_caches_that_overlap_are_refused(vm):
    T, H, D, P, pages = 5, 2, 64, 4, 5
    slots = s4._cu(np.arange(T))
    c = vm.Cache4(pages, H, P, D)
    wide = torch.randn((T, 4, H, D), device="cuda")
    k, v = wide[:, 0], wide[:, 1]

    def append(k=k, v=v, slots=slots, kc=c.k, vc=c.v, ks=c.k_scale, vs=c.v_scale):
        vm.dspark_cache_append4(k, v, slots, kc, vc, ks, vs)

    def read(k=wide[:, 2], v=wide[:, 3], slots=slots, kc=c.k, vc=c.v, ks=c.k_scale, vs=c.v_scale):
        vm.dspark_cache_read4(kc, vc, ks, vs, slots, k, v)

    append()
    read()
    assert bool(wide[:, 2].any(2).any(1).all())
    rows = H * P * D // 2
    blob = torch.zeros(pages * 4 * rows, dtype=torch.uint8, device="cuda")
    part = lambda at, w: blob[at:at + pages * H * P * w].view(pages, H, P, w)  # noqa: E731
    both = torch.zeros((pages, 2, H, P, D // 2), dtype=torch.uint8, device="cuda")
    append(kc=both[:, 0], vc=both[:, 1])                    # pages in each other's gaps
    append(kc=part(0, D // 2), vc=part(pages * rows, D // 2))
    for kw in (dict(kc=c.v), dict(vs=c.k_scale),
               dict(kc=part(0, D // 2), vc=part(pages * rows - 16, D // 2)), dict(ks=part(0, D // 16), vc=part(0, D // 2)),
               dict(kc=part(0, D // 2), k=blob[:T * H * D * 4].view(F32).view(T, H, D)), dict(kc=part(0, D // 2), slots=blob[:4 * T].view(torch.int32))):
        with pytest.raises(vm.DsparkError):
            append(**kw)
    out = torch.zeros((T + 1, H, D), device="cuda")
    for kw in (dict(k=out[1:], v=out[1:]), dict(k=out[1:], v=out[:-1]), dict(k=wide[:, 2], v=wide[:, 2]), dict(kc=part(0, D // 2), v=blob[:T * H * D * 4].view(F32).view(T, H, D)),
               dict(k=blob[:T * H * D * 4].view(F32).view(T, H, D), slots=blob[64:64 + 4 * T].view(torch.int32))):
        with pytest.raises(vm.DsparkError):
            read(**kw)
    read(v=wide[:, 1])                                      # (what was written may be read over)


def test_attention_refuses_results_that_overlap(vm):
    rng = np.random.default_rng(1)
    P, lens, D, N = 16, [40, 3], 64, 4
    pages, table = _case(rng, 2, P, lens, D, 2)
    ts = [torch.from_numpy(a).cuda() for a in _cache(rng, pages, 2, P, D)]
    lists = [s4._cu(table), s4._cu(lens), s4._cu([0, 2, 4]), s4._cu([0, 1, 2])]
    ws = vm.CacheWorkspace(2, 4, 2, D, 2)
    wide = torch.randn((N + 1, 4, D), device="cuda")
    q, out, lse = wide[:N], torch.empty((N, 4, D), device="cuda"), torch.empty((N, 4), device="cuda")

    def call(q=q, out=out, lse=lse, ts=ts, lists=lists, ws=ws):
        vm.dspark_cache_attention4(q, *ts, *lists, out, ws, max_new=2, lse=lse)

    call()
    big = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    f = lambda at, *s: big[at:at + 4 * int(np.prod(s))].view(F32).view(*s)  # noqa: E731
    for kw in (dict(out=q), dict(out=wide[1:]), dict(lse=out[0].view(-1)[:16].view(4, 4)), dict(lse=q[1].reshape(-1)[:16].view(4, 4)),
               dict(out=ws.buf4[256:256 + 4 * N * 4 * D].view(F32).view(N, 4, D)),
               dict(out=f(0, N, 4, D), ts=[big[:ts[0].numel()].view_as(ts[0])] + ts[1:]), dict(lse=f(0, N, 4), ts=ts[:3] + [big[:ts[3].numel()].view_as(ts[3])]),
               dict(lse=f(0, N, 4), lists=lists[:2] + [big[16:28].view(torch.int32)] + lists[3:])):
        with pytest.raises(vm.DsparkError):
            call(**kw)
    assert s4._status(vm, ws) == 0


def test_a_workspace_without_room_for_four_bits_is_the_smaller_one(vm):
    sizes = (3, 8, 2, 128, 8)
    ws, both = vm.CacheWorkspace(*sizes, four_bits=False), vm.CacheWorkspace(*sizes)
    n, n4 = vm.dspark_cache_workspace_bytes(*sizes), vm.dspark_cache4_workspace_bytes(*sizes)
    assert len(ws.buf) == len(both.buf) == n < n4 == len(both.buf4) and ws.buf4 is None and len(ws.tensor) < n + 512
    B, P, lens = 3, 16, np.array([100, 40, 8])
    rng = np.random.default_rng(2)
    pages, table = _case(rng, B, P, lens, 128, 2)
    k, v = (torch.from_numpy(rng.standard_normal((pages, 2, P, 128))).to(BF16).cuda() for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((24, 8, 128))).to(BF16).cuda()
    lists = [s4._cu(table), s4._cu(lens), s4._cu([0, 8, 16, 24]), s4._cu([0, 2, 3, 4])]
    outs = [torch.empty_like(q) for _ in range(2)]
    for w, out in zip((ws, both), outs):
        vm.dspark_cache_attention(q, k, v, *lists, out, w, max_new=8)
        assert s4._status(vm, w) == 0
    assert torch.equal(*outs)
    with pytest.raises(ValueError):
        vm.dspark_cache_attention4(q, *vm.Cache4(pages, 2, P, 128).tensors, *lists, outs[0], ws, max_new=8)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_flat_rows_of_many_different_entries(vm, dtype):
    """A step of weights holds more entries than a list, few of them equal (bf16: some)."""
    rng = np.random.default_rng(17)
    N, V = 5, 151936
    x = torch.from_numpy(rng.standard_normal((N, V)) * np.array([0.3, 0.3, 1.5, 1.5, 0.01])[:, None]).to(dtype).cuda()
    u = rng.random(N).astype(np.float32)
    T = np.array([1.0, 2.0, 5.0, 10.0, 1.0])
    for k, p in ((None, 0.5), (None, 0.03), (50000, None), (70000, 0.6), (V - 2, 0.999)):
        args = (T, None if k is None else np.full(N, k), None if p is None else np.full(N, p), None)
        tok, lp, status = s4._sample(vm, x, u, *args)
        assert status == 0
        s4._check_rows(x, u, *args, tok, lp)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [20001, 70003, 151936])
def test_a_long_row_is_the_same_however_many_ctas_take_it(vm, V, dtype):
    """One row is taken by up to 16 CTAs, many by two or one each: tokens and logarithms, bit by bit."""
    rng = np.random.default_rng(V)
    N = 160
    x = torch.empty((N, -(-V // 8) * 8), dtype=dtype, device="cuda")[:, :V]
    x.copy_(torch.randn((N, V), generator=torch.Generator(device="cuda").manual_seed(V), device="cuda") * 2)
    x[::3] *= 0.1                                           # flat rows, whose unit is coarser
    x[1::3, V // 3] = 40.0                                  # and rows of one entry far above the others
    u, T = rng.random(N).astype(np.float32), rng.choice([0.05, 0.7, 1.0, 4.0], N)
    k, p, m = rng.choice([0, 3, 300, 2000, V - 5], N), rng.choice([0.5, 0.95, 1.0], N), rng.choice([0.0, 0.01], N)
    for args in ((None,) * 4, (T, None, None, None), (T, k, None, m), (T, None, p, None), (T, k, p, m)):
        tok, lp, status = s4._sample(vm, x, u, *args)
        assert status == 0
        for a, b in ((0, 1), (1, 2), (2, 3), (5, 12), (10, 60)):
            part = [None if v is None else v[a:b] for v in args]
            t, l, _ = s4._sample(vm, x[a:b], u[a:b], *part)
            assert (t == tok[a:b]).all() and (l == lp[a:b]).all()
