"""GPU tests of the cache in 4 bits, the rotary positions and the sampling
against the 64-bit references of tests/_serve4_ref.py."""
import numpy as np
import pytest
import torch

from tests import _serve4_ref as ref

pytestmark = pytest.mark.gpu
BAD_LENGTH, BAD_INPUT, DEAD_ROW, BAD_PAGE = 2, 8, 16, 32
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def vm():
    import verify_markov_head_gb300 as vm
    return vm


def _cu(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _status(vm, ws):
    return vm.dspark_sync_status(ws.buf)[1]


# ------------------------------------------------------- writing and reading
def _rows(rng, T, H, D, dtype):
    """Entries of many sizes, among them borders between codes and between scales."""
    x = rng.standard_normal((T, H, D)) * 2.0 ** rng.integers(-9, 9, (T, H, D // 16)).repeat(16, 2)
    x[rng.random(x.shape) < 0.02] = 0
    groups = x.reshape(-1, 16)
    for i in range(0, len(groups), 3):                      # multiples of a quarter of a scale, the largest 6 scales
        s = ref.SCALES[rng.integers(8, 100)]
        groups[i] = s * rng.integers(-24, 25, 16) / 4
        groups[i, rng.integers(0, 16)] = 6 * s
    for i in range(1, len(groups), 7):                      # the largest at a border between two scales
        a = rng.integers(1, 125)
        groups[i, rng.integers(0, 16)] = 3 * (ref.SCALES[a] + ref.SCALES[a + 1])
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("T,H,D,P,dtype,k_exp,v_exp", [
    (1, 1, 16, 1, BF16, 0, 0), (37, 2, 64, 8, BF16, 0, -3), (200, 8, 128, 16, BF16, 2, 1), (61, 3, 96, 5, F32, -4, 0),
    (33, 1, 256, 64, F32, 0, 7), (90, 2, 80, 24, BF16, 0, 0), (19, 5, 48, 3, F32, 64, -64),
])
def test_rows_are_quantised_and_read_back_exactly(vm, T, H, D, P, dtype, k_exp, v_exp):
    rng = np.random.default_rng(T * D)
    pages = -(-T // P) + 3
    wide = torch.empty((T, 3 * H, D), dtype=dtype)          # slices of a wider projection
    wide[:, :H], wide[:, 2 * H:] = _rows(rng, T, H, D, dtype), _rows(rng, T, H, D, dtype)
    k, v = wide.cuda()[:, :H], wide.cuda()[:, 2 * H:]
    if k_exp == 64:
        k, v = (k.double() * 2.0 ** 60).to(dtype), (v.double() * 2.0 ** -60).to(dtype)
    slots = rng.permutation(pages * P)[:T].astype(np.int32)
    slots[rng.random(T) < 0.1] = -1
    # pages of codes with a gap between them, everything set to a pattern that has to stay
    big = torch.full((pages, 2, H, P, D // 2), 0xA5, dtype=torch.uint8, device="cuda")
    kc, vc = big[:, 0], big[:, 1]
    ks, vs = (torch.full((pages, H, P, D // 16), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(2))
    ws = vm.LogitsWorkspace(1, 1)
    vm.dspark_cache_append4(k, v, _cu(slots), kc, vc, ks, vs, k_exp=k_exp, v_exp=v_exp, ws=ws)
    for x, c, s, e in ((k, kc, ks, k_exp), (v, vc, vs, v_exp)):
        want_c, want_s = np.full(tuple(c.shape), 0xA5, np.uint8), np.full(tuple(s.shape), 0x5A, np.uint8)
        codes, scales = ref.quantise(_np(x), e)
        at = slots >= 0
        want_c[slots[at] // P, :, slots[at] % P], want_s[slots[at] // P, :, slots[at] % P] = codes[at], scales[at]
        np.testing.assert_array_equal(s.cpu().numpy(), want_s)
        np.testing.assert_array_equal(c.cpu().numpy(), want_c)
    back = torch.full((T, 3, H, D), 7.0, dtype=dtype, device="cuda")
    vm.dspark_cache_read4(kc, vc, ks, vs, _cu(slots), back[:, 0], back[:, 2], k_exp=k_exp, v_exp=v_exp, ws=ws)
    for i, x, e in ((0, k, k_exp), (2, v, v_exp)):
        want = ref.values(*ref.quantise(_np(x), e), e)
        want[slots < 0] = 7
        np.testing.assert_array_equal(_np(back[:, i]), want)
    assert bool((back[:, 1] == 7).all())
    assert _status(vm, ws) == 0


def test_infinities_saturate_and_a_nan_marks_its_group(vm):
    x = torch.zeros((4, 1, 32))
    x[0, 0, :16] = torch.arange(16) - 8.0
    x[0, 0, 3] = float("inf")
    x[1, 0, 5], x[1, 0, 20] = float("nan"), 3.0
    x[2, 0, 1], x[2, 0, 17] = -1e38, 5000.0
    x[3, 0, 0] = 1e-40
    for dtype in (F32, BF16):
        k = x.to(dtype).cuda()
        c = vm.Cache4(2, 1, 4, 32)
        back = torch.empty_like(k), torch.empty_like(k)
        slots = _cu([0, 1, 2, 3])
        vm.dspark_cache_append4(k, -k, slots, *c.tensors)
        vm.dspark_cache_read4(*c.tensors, slots, *back)
        for got, sign in zip(back, (1, -1)):
            got = _np(got) * sign
            want = ref.values(*ref.quantise(_np(k), 0), 0)
            assert np.isnan(got[1, 0, :16]).all() and not np.isnan(got[1, 0, 16:]).any()
            want[1, 0, :16] = got[1, 0, :16] = 0
            np.testing.assert_array_equal(got, want)
            assert got[0, 0, 3] == 2688 and got[2, 0, 1] == -2688 and got[2, 0, 17] == 2688


def test_slots_beyond_the_cache_are_skipped_and_reported(vm):
    c = vm.Cache4(3, 1, 4, 16)
    k = torch.ones((4, 1, 16), dtype=BF16, device="cuda")
    ws = vm.LogitsWorkspace(1, 1)
    slots = _cu([11, 12, -5, 2 ** 31 - 1])
    vm.dspark_cache_append4(k, k, slots, *c.tensors, ws=ws)
    assert _status(vm, ws) == BAD_PAGE
    assert int((c.k != 0).any(3).sum()) == 1 and bool((c.k[2, 0, 3] != 0).all())
    out = torch.full_like(k, 9.0)
    vm.dspark_cache_read4(*c.tensors, slots, out, out.clone(), ws=ws)
    assert _status(vm, ws) == BAD_PAGE
    # (1 is 6 scales of 1/6, whose nearest scale is 11/64: 11/64 - 1/6 = 1/192, 1/6 - 10/64 = 2/192)
    assert out[:, 0, 0].tolist() == [6 * 11 / 64, 9, 9, 9]


# ----------------------------------------------------------------- attention
def _cache(rng, pages, H, P, D, dtype=BF16, spread=1.0):
    """Codes and scales of random values, and the garbage bytes of every kind between them."""
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    out = []
    for size in (spread, 0.7):
        x = (torch.randn((pages, H, P, D), generator=g) * size).to(dtype)
        out.append(ref.quantise(_np(x), 0))
    return [out[0][0], out[1][0], out[0][1], out[1][1]]


def _attend(vm, rng, q, arrays, table, kv_len, q_off, max_new, k_exp=0, v_exp=0, scale=None, stride=None, B=None, stream=None, ws=None):
    N, Hq, D = q.shape
    B, Hkv = len(kv_len), arrays[0].shape[1]
    tile_off = np.concatenate([[0], np.cumsum(-(-np.asarray(kv_len) // 64))])
    pad = 3
    wide = torch.full((N, Hq + pad, D), 3.0, dtype=q.dtype, device="cuda")
    wide[:, :Hq] = q
    out = torch.full((N, Hq, D), 77.0, dtype=q.dtype, device="cuda")
    lse = torch.full((N, Hq), 77.0, device="cuda")
    ws = ws or vm.CacheWorkspace(B, Hq, Hkv, D, max_new)
    ts = [torch.from_numpy(a).cuda() for a in arrays]
    vm.dspark_cache_attention4(wide[:, :Hq], *ts, _cu(table), _cu(kv_len), _cu(q_off), _cu(tile_off), out, ws, max_new=max_new,
                               k_exp=k_exp, v_exp=v_exp, scale=scale, lse=lse, stream=stream)
    torch.cuda.synchronize()
    return out, lse, _status(vm, ws)


def _case(rng, B, P, lens, D, Hkv, spare=3):
    lens = np.asarray(lens)
    owned = -(-lens // P)
    pages = int(owned.sum()) + spare
    width = int(owned.max()) + 2 if B else 1
    table = np.full((B, width), -1, np.int32)
    perm, o = rng.permutation(pages), 0
    for b in range(B):
        table[b, :owned[b]] = perm[o:o + owned[b]]
        o += owned[b]
    return pages, table


def _poison(arrays, table, lens, P):
    """Bytes of ones wherever no request's positions lie: NaN scales."""
    free = np.ones((arrays[0].shape[0], P), bool)
    for b, n in enumerate(lens):
        pos = np.arange(n)
        free[table[b, pos // P], pos % P] = False
    for a in arrays:
        a.transpose(0, 2, 1, 3)[free] = 0xFF


def _check(q, arrays, table, lens, q_off, scale, got, lse, k_exp=0, v_exp=0):
    bf16 = q.dtype == BF16
    K, V = ref.values(arrays[0], arrays[2], k_exp), ref.values(arrays[1], arrays[3], v_exp)
    want, want_lse, tol, lse_tol = ref.attention(_np(q), K, V, table, lens, q_off, scale, bf16)
    a, b = q_off[0], q_off[-1]
    x, y = _np(got)[a:b], _np(lse)[a:b]
    err = np.abs(x - want[a:b])
    assert np.array_equal(np.isnan(x), np.isnan(want[a:b]))
    assert (err <= tol[a:b])[~np.isnan(x)].all(), (np.nanmax(err - tol[a:b]), np.nanmax(err / tol[a:b]))
    none = want_lse[a:b] == -np.inf
    assert (y[none] == -np.inf).all()
    some = ~none & ~np.isnan(y)
    assert (np.abs(y[some] - want_lse[a:b][some]) <= lse_tol[a:b][some]).all()
    # rows outside the requests are left as they were
    rest = np.ones(len(_np(got)), bool)
    rest[a:b] = False
    assert (_np(got)[rest] == 77).all() and (_np(lse)[rest] == 77).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,D,P,new,lens", [
    (4, 1, 128, 16, 1, [1000]), (32, 8, 128, 16, 1, [1, 15, 16, 17, 63, 64, 65, 200]), (8, 2, 64, 8, 8, [8, 300, 77, 1, 2]),
    (8, 8, 128, 1, 3, [40, 0, 3, 129]), (16, 2, 96, 24, 4, [100, 4, 513]), (7, 1, 80, 5, 2, [90, 33]), (64, 4, 128, 64, 8, [700, 64, 8]),
    (17, 1, 48, 16, 8, [200, 9]), (4, 2, 256, 16, 8, [150, 300]), (3, 1, 160, 3, 2, [77]), (2, 1, 192, 32, 17, [400, 17, 16]),
    (1, 1, 16, 2, 1, [33, 1]), (5, 5, 32, 16, 5, [64, 65, 5]), (12, 1, 112, 7, 1, [250, 19]), (16, 1, 256, 64, 4, [130]),
    (48, 3, 224, 16, 1, [99, 16]), (9, 1, 64, 128, 1, [5000, 129]), (64, 8, 128, 16, 17, [333]),
])
def test_attention_over_four_bits(vm, Hq, Hkv, D, P, new, lens, dtype):
    rng = np.random.default_rng(Hq * 1000 + D + new)
    B = len(lens)
    n_new = rng.integers(1, new + 1, B)
    n_new[0] = new                                           # (a request may hold fewer positions than it has new tokens)
    q_off = np.concatenate([[0], np.cumsum(n_new)])
    pages, table = _case(rng, B, P, lens, D, Hkv)
    arrays = _cache(rng, pages, Hkv, P, D)
    _poison(arrays, table, lens, P)
    q = (torch.from_numpy(rng.standard_normal((int(q_off[-1]) + 3, Hq, D))) * 2).to(dtype).cuda()
    got, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, new, k_exp=1, v_exp=-2)
    assert status == 0
    _check(q, arrays, table, lens, q_off, np.float32(D ** -0.5), got, lse, 1, -2)


@pytest.mark.parametrize("B,Hq,Hkv,D,P,new,lo,hi", [
    (1, 8, 1, 128, 16, 1, 20000, 20000), (2, 64, 8, 128, 64, 8, 3000, 9000), (300, 8, 2, 64, 16, 1, 0, 90), (40, 32, 8, 128, 16, 2, 1, 400),
    (3, 4, 1, 256, 32, 3, 5000, 6000), (70, 4, 4, 96, 16, 2, 1, 300),
])
def test_attention_split_over_ctas_and_segments(vm, B, Hq, Hkv, D, P, new, lo, hi):
    """Against the same formula in 64 bits on the GPU's values, whole batches at a time."""
    rng = np.random.default_rng(B + D)
    lens = rng.integers(lo, hi + 1, B)
    n_new = np.minimum(rng.integers(0, new + 1, B), lens)
    q_off = np.concatenate([[0], np.cumsum(n_new)])
    pages, table = _case(rng, B, P, lens, D, Hkv)
    arrays = _cache(rng, pages, Hkv, P, D)
    q = torch.from_numpy(rng.standard_normal((int(q_off[-1]), Hq, D))).to(BF16).cuda()
    got, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, new)
    assert status == 0
    _check(q, arrays, table, lens, q_off, np.float32(D ** -0.5), got, lse)
    again = _attend(vm, rng, q, arrays, table, lens, q_off, new)
    assert torch.equal(again[0], got) and torch.equal(again[1], lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_attention_keeps_a_nan_to_the_rows_that_see_it(vm, D, dtype):
    """A group that is NaN in the block's last positions, in a key and in a value."""
    rng = np.random.default_rng(D)
    P, lens, n = 16, [50, 37], 8
    q_off = np.array([0, n, 2 * n])
    pages, table = _case(rng, 2, P, lens, D, 1)
    arrays = _cache(rng, pages, 1, P, D)
    for which, b, pos, group in ((3, 0, 46, 0), (3, 0, 48, D // 16 - 1), (2, 1, 33, 1), (3, 1, 35, 2)):
        arrays[which][table[b, pos // P], 0, pos % P, group] = 0x7F
    q = torch.from_numpy(rng.standard_normal((2 * n, 4, D))).to(dtype).cuda()
    got, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, n)
    assert status == 0
    nan = torch.isnan(got)
    # request 0: group 0 from its fifth token on (position 46), the last group from the seventh
    for i in range(n):
        assert bool(nan[i, :, :16].all()) == (42 + i >= 46) and bool(nan[i, :, D - 16:].all()) == (42 + i >= 48)
        assert not bool(nan[i, :, 16:D - 16].any())
        assert bool(nan[n + i].all()) == (29 + i >= 33) and (29 + i >= 33 or not bool(nan[n + i].any()))
    _check(q[:n], arrays, table[:1], lens[:1], q_off[:2], np.float32(D ** -0.5), got[:n], lse[:n])


def test_attention_leaves_out_bad_pages(vm):
    rng = np.random.default_rng(3)
    P, lens, D = 16, [100, 70], 128
    q_off = np.array([0, 2, 3])
    pages, table = _case(rng, 2, P, lens, D, 2)
    table[0, 2], table[1, 4] = pages, -7
    arrays = _cache(rng, pages, 2, P, D)
    for dtype in (BF16, F32):
        q = torch.from_numpy(rng.standard_normal((3, 8, D))).to(dtype).cuda()
        got, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, 2)
        assert status == BAD_PAGE
        _check(q, arrays, table, lens, q_off, np.float32(D ** -0.5), got, lse)


def test_attention_reports_lengths_and_offsets_that_do_not_fit(vm):
    rng = np.random.default_rng(4)
    P, D = 16, 128
    pages, table = _case(rng, 2, P, [64, 64], D, 1)
    arrays = _cache(rng, pages, 1, P, D)
    for dtype in (BF16, F32):
        q = torch.from_numpy(rng.standard_normal((4, 4, D))).to(dtype).cuda()
        for lens, q_off in (([64, 10 ** 6], [0, 2, 4]), ([64, -3], [0, 2, 4]), ([64, 64], [0, 2, 9]), ([64, 64], [0, 4, 2]),
                            ([64, 64], [0, 2, 2 ** 31 - 1])):
            out = torch.zeros((4, 4, D), dtype=dtype, device="cuda")
            ws = vm.CacheWorkspace(2, 4, 1, D, 2)
            vm.dspark_cache_attention4(q, *(torch.from_numpy(a).cuda() for a in arrays), _cu(table), _cu(lens), _cu(q_off), _cu([0, 1, 2]),
                                       out, ws, max_new=2)
            assert _status(vm, ws) & BAD_LENGTH, (lens, q_off)


@pytest.mark.parametrize("size", [1e-30, 1e-3, 300.0, 1e30])
def test_attention_with_queries_of_any_size(vm, size):
    """Rows of q are scaled by powers of two: scores of a fixed size from queries of any."""
    rng = np.random.default_rng(9)
    P, lens, D = 16, [300], 128
    pages, table = _case(rng, 1, P, lens, D, 1)
    arrays = _cache(rng, pages, 1, P, D)
    q = torch.from_numpy(rng.standard_normal((2, 4, D)) * size).to(BF16).cuda()
    q[0, 1] = 0
    scale = float(np.float32(0.2 / size))
    got, lse, _ = _attend(vm, rng, q, arrays, table, lens, [0, 2], 2, scale=scale)
    _check(q, arrays, table, lens, np.array([0, 2]), scale, got, lse)


@pytest.mark.parametrize("rising", [True, False])
def test_attention_with_scores_that_rise_or_fall_along_the_context(vm, rising):
    """Every unit of positions moves the references, or none but the first; weights of
    many sizes, most of them far below the largest."""
    rng = np.random.default_rng(10)
    P, n, D = 16, 1200, 128
    pages, table = _case(rng, 1, P, [n], D, 1)
    x = torch.from_numpy(rng.standard_normal((n, D)) * 0.02)
    x[:, 16:] += torch.linspace(-2, 2, n)[:, None].double() * (1 if rising else -1)
    arrays = _cache(rng, pages, 1, P, D)
    c, s = ref.quantise(_np(x.to(BF16)), 0)
    pos = np.arange(n)
    arrays[0][table[0, pos // P], 0, pos % P], arrays[2][table[0, pos // P], 0, pos % P] = c, s
    q = torch.ones((2, 8, D), dtype=BF16, device="cuda") * torch.arange(1, 9, device="cuda")[None, :, None] / 4
    got, lse, _ = _attend(vm, rng, q, arrays, table, [n], [0, 2], 2, scale=0.25)
    _check(q, arrays, table, [n], np.array([0, 2]), 0.25, got, lse)


# --------------------------------------------------------------------- rope
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rotary,far", [
    (1, 1, 0, 8, 2, 10), (5, 4, 2, 64, 64, 10000), (33, 3, 1, 128, 128, 2 ** 31 - 1), (7, 2, 2, 96, 48, 1 << 20), (64, 8, 1, 80, 80, 4096),
    (9, 1, 1, 256, 64, 1 << 22), (12, 2, 1, 40, 26, 5000), (2500, 2, 1, 64, 32, 131072), (3, 2, 1, 128, 6, 99),
])
def test_rope_matches_the_formula(vm, T, Hq, Hkv, D, rotary, far, inter, dtype):
    rng = np.random.default_rng(T + D + rotary)
    x = torch.from_numpy(rng.standard_normal((T, Hq + Hkv + 1, D)) * 3).to(dtype).cuda()
    pos = rng.integers(0, far + 1, T).astype(np.int32)
    pos[0] = far
    pos[rng.random(T) < 0.1] = -1 - rng.integers(0, 5)
    table = vm.RopeTable(rotary, base=10000.0, mult=1.25)
    freq = np.array(vm.rope_frequencies(rotary)[0])
    want, tol = ref.rope(_np(x), pos, freq, np.float64(np.float32(1.25)), rotary, inter, ref.EPS16 if dtype == BF16 else ref.EPS32)
    hidden = pos < 0
    out = torch.full((T, Hq + Hkv + 2, D), 5.0, dtype=dtype, device="cuda")
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv] if Hkv else None
    qo, ko = out[:, 1:1 + Hq], out[:, 1 + Hq:1 + Hq + Hkv] if Hkv else None
    vm.dspark_rope(q, k, _cu(pos), table, qo, ko, interleaved=inter)
    got = _np(out)
    assert (got[:, 0] == 5).all() and (got[:, 1 + Hq + Hkv:] == 5).all()
    w, t = want[:, :Hq + Hkv], tol[:, :Hq + Hkv]
    w[hidden] = 5
    assert (np.abs(got[:, 1:1 + Hq + Hkv] - w) <= t).all(), np.max(np.abs(got[:, 1:1 + Hq + Hkv] - w) - t)
    # in place: the same bits, the rest as it was
    before = _np(x)
    vm.dspark_rope(q, k, _cu(pos), table, interleaved=inter)
    same = _np(x)
    np.testing.assert_array_equal(same[~hidden, :Hq + Hkv], got[~hidden, 1:1 + Hq + Hkv])
    np.testing.assert_array_equal(same[hidden], before[hidden])
    np.testing.assert_array_equal(same[:, -1], before[:, -1])


def test_rope_turns_back(vm):
    """Frequencies of the other sign undo it; a whole number of turns does nothing."""
    x = torch.randn((50, 4, 64), device="cuda")
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 1000003
    f = vm.rope_frequencies(64, 500000.0)[0]
    y, z = torch.empty_like(x), torch.empty_like(x)
    vm.dspark_rope(x, None, pos, vm.RopeTable(64, frequencies=f), y)
    vm.dspark_rope(y, None, pos, vm.RopeTable(64, frequencies=[-a for a in f]), z)
    assert float((z - x).abs().max()) < 1e-5 * float(x.abs().max())
    vm.dspark_rope(x, None, pos, vm.RopeTable(64, frequencies=[2 * np.pi] * 32), y)
    assert float((y - x).abs().max()) < 1e-5 * float(x.abs().max())


# ------------------------------------------------------------------- sample
def _sample(vm, x, u, T=None, k=None, p=None, m=None, ws=None):
    N = x.shape[0]
    ws = ws or vm.SampleWorkspace(N)
    tok, lp = torch.full((N,), -9, dtype=torch.int32, device="cuda"), torch.empty(N, device="cuda")
    f = lambda a, t=F32: None if a is None else _cu(a, t)  # noqa: E731
    vm.dspark_sample(x, f(u), tok, ws, temperature=f(T), top_k=f(k, torch.int32), top_p=f(p), min_p=f(m), logprob=lp)
    return tok.cpu().numpy(), _np(lp), _status(vm, ws)


def _check_rows(x, u, T, k, p, m, tok, lp):
    xs = _np(x)
    f32 = lambda a, i, d: d if a is None else float(np.float32(a[i]))  # noqa: E731
    for i in range(len(xs)):
        want, wlp, near, near_p = ref.sample(xs[i], f32(u, i, 0), f32(T, i, 1.0), 0 if k is None else int(k[i]), f32(p, i, 1.0), f32(m, i, 0.0))
        # weights are off by 2^-30 of themselves: sums of shares by 2^-30, a draw at a border may go either way
        if near > 2.0 ** -30 and near_p > 2.0 ** -30:
            assert tok[i] == want, (i, tok[i], want, near, near_p)
            # and its logarithm: 2^-29, then two roundings of binary32 and the logarithm's two
            assert abs(lp[i] - wlp) <= 2.0 ** -29 + 4 * ref.EPS32 * abs(wlp) if np.isfinite(wlp) else lp[i] == wlp


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,V", [(1, 1), (3, 2), (5, 7), (40, 100), (64, 1000), (17, 4097), (300, 257), (9, 32003), (3, 151936), (1, 151936), (2, 1 << 19)])
def test_sampling_matches_the_definition(vm, N, V, dtype):
    rng = np.random.default_rng(N * 7 + V)
    pad = -(-V // 8) * 8 + 8
    x = torch.from_numpy(rng.standard_normal((N, pad)) * 3).to(dtype).cuda()[:, :V]
    x[:, ::7] = float("-inf")
    if V > 1:
        x[:, 1] = 4.0
    if V <= 7:
        x[:, 0] = 1.0
    u = rng.random(N).astype(np.float32)
    T, k = rng.choice([0.0, 0.3, 0.7, 1.0, 2.5], N), rng.choice([0, 1, 2, 5, 40, 1000, 10 ** 9, -3], N)
    p, m = rng.choice([0.0, 0.1, 0.5, 0.9, 0.999, 1.0], N), rng.choice([0.0, 0.0, 0.001, 0.2, 1.0], N)
    for args in ((None,) * 4, (T, None, None, None), (T, k, None, None), (T, None, p, None), (T, None, None, m), (T, k, p, m)):
        tok, lp, status = _sample(vm, x, u, *args)
        assert status == 0
        _check_rows(x, u, *args, tok, lp)


def test_sampling_takes_ties_by_the_lowest_id(vm):
    """Rows of few different values: the cut of top-k and top-p lies among equal entries."""
    rng = np.random.default_rng(2)
    N, V = 200, 3001
    pad = 3008
    x = torch.from_numpy(rng.integers(0, 4, (N, pad)).astype(np.float64)).to(BF16).cuda()[:, :V]
    x[::5] = 1.0                                            # all equal
    x[1::5, 1000:] = -0.0
    x[1::5, :1000] = 0.0
    u = rng.random(N).astype(np.float32)
    k, p = rng.integers(1, 2000, N), rng.uniform(0.01, 0.99, N)
    for args in ((None, k, None, None), (None, None, p, None), (None, k, p, None)):
        tok, lp, _ = _sample(vm, x, u, *args)
        _check_rows(x, u, *args, tok, lp)
    top, _, _ = _sample(vm, x, u, T=np.zeros(N))
    assert (top == [int(np.argmax(r)) for r in _np(x)]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sampling_leaves_out_what_is_no_number(vm, dtype):
    x = torch.full((6, 64), float("-inf"), dtype=dtype, device="cuda")
    x[0, 5], x[0, 9] = 1.0, float("nan")
    x[1, 7], x[1, 3] = -2.0, float("inf")
    x[2, :] = float("nan")
    x[4, 63] = -3e38
    x[5, 0], x[5, 1] = 3e38, -3e38
    tok, lp, status = _sample(vm, x, np.full(6, 0.999))
    assert tok.tolist() == [5, 7, -1, -1, 63, 0] and status == BAD_INPUT | DEAD_ROW
    assert lp[[0, 1, 4, 5]].tolist() == [0, 0, 0, 0] and (lp[2:4] == -np.inf).all()
    ok = x[4:]
    _, _, status = _sample(vm, ok, [0.1, 0.2])
    assert status == 0
    tok, _, status = _sample(vm, ok, [0.1, 0.2], T=[-1.0, float("nan")])
    assert tok.tolist() == [63, 0] and status == BAD_INPUT
    tok, _, status = _sample(vm, ok, [0.1, 0.2], p=[float("nan"), 0.5], m=[0.1, float("nan")])
    assert tok.tolist() == [63, 0] and status == BAD_INPUT


@pytest.mark.parametrize("T", [1e-38, 1e-6, 1e-3, 50.0, 1e30])
def test_sampling_at_extreme_temperatures(vm, T):
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((20, 5000)) * 20 + 300).float().cuda()
    x[:, 10] = x.amax(1) + 1e-3
    u = rng.random(20)
    Ts = np.full(20, T)
    for p in (None, np.full(20, 0.8)):
        tok, lp, status = _sample(vm, x, u, T=Ts, p=p)
        assert status == 0
        _check_rows(x, u, Ts, None, p, None, tok, lp)


def test_sampling_at_the_ends_of_the_random_numbers(vm):
    x = torch.zeros((6, 1000), device="cuda")
    x[:, 500:] = float("-inf")
    u = [0.0, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, float("nan")]
    tok, _, _ = _sample(vm, x, u)
    assert tok.tolist() == [0, 499, 499, 499, 0, 0]


def test_sampling_draws_by_the_shares(vm):
    """A grid of u hits every token as often as its share says, to one draw at each border."""
    rng = np.random.default_rng(6)
    row = rng.standard_normal(300) * 2
    n = 4096
    x = torch.from_numpy(row).float().cuda()[None].expand(n, 300).contiguous()
    x = torch.nn.functional.pad(x, (0, 4))[:, :300]
    tok, _, _ = _sample(vm, x, (np.arange(n) + 0.5) / n)
    share = np.exp(_np(x[0]) - _np(x[0]).max())
    got = np.bincount(tok, minlength=300)
    assert np.abs(got - n * share / share.sum()).max() <= 1.0001


# ----------------------------------------------------------------- together
def test_a_step_in_a_graph_on_another_stream(vm):
    """Rotated, written, attended, processed and drawn in one captured graph: replays
    with new inputs give what eager calls on the current stream give, bit by bit."""
    g = torch.Generator(device="cuda").manual_seed(1)
    B, n, Hq, Hkv, D, P, V, width = 5, 3, 8, 2, 64, 16, 1000, 20
    pages = B * width
    i32 = dict(dtype=torch.int32, device="cuda")

    def fresh():
        c = vm.Cache4(pages, Hkv, P, D, k_exp=-1)
        return dict(cache=c, seq=torch.zeros(B, **i32), new=torch.full((B,), n, **i32), owned=torch.zeros(B, **i32), ring=torch.arange(pages, **i32),
                    state=torch.tensor([0, pages], **i32), table=torch.full((B, width), -1, **i32), owned_out=torch.zeros(B, **i32),
                    state_out=torch.zeros(2, **i32), kv_len=torch.zeros(B, **i32), q_off=torch.zeros(B + 1, **i32), tile_off=torch.zeros(B + 1, **i32),
                    slot=torch.zeros(B * n, **i32), pos=torch.zeros(B * n, **i32), qkv=torch.zeros((B * n, Hq + 2 * Hkv, D), dtype=BF16, device="cuda"),
                    out=torch.zeros((B * n, Hq, D), dtype=BF16, device="cuda"), logits=torch.zeros((B, 1, V), device="cuda"),
                    rep=torch.full((B,), 1.2, device="cuda"), u=torch.zeros(B, device="cuda"), tok=torch.zeros(B, **i32),
                    hist=torch.zeros((B, 4), **i32), hist_len=torch.full((B,), 4, **i32), k=torch.full((B,), 50, **i32),
                    ws=vm.CacheWorkspace(B, Hq, Hkv, D, n), lws=vm.LogitsWorkspace(B, 1), sws=vm.SampleWorkspace(B))

    table = vm.RopeTable(D, 10000.0, dict(kind="yarn", factor=4.0, trained=64))

    def step(s):
        q, k, v = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:]
        c = s["cache"]
        vm.dspark_cache_plan(s["seq"], s["new"], s["owned"], s["ring"], s["state"], s["table"], P, owned_out=s["owned_out"],
                             ring_state_out=s["state_out"], kv_len=s["kv_len"], q_off=s["q_off"], tile_off=s["tile_off"], slot_map=s["slot"],
                             positions=s["pos"], ws=s["ws"])
        vm.dspark_rope(q, k, s["pos"], table)
        vm.dspark_cache_append4(k, v, s["slot"], *c.tensors, k_exp=-1, ws=s["ws"])
        vm.dspark_cache_attention4(q, *c.tensors, s["table"], s["kv_len"], s["q_off"], s["tile_off"], s["out"], s["ws"], max_new=n, k_exp=-1)
        s["logits"].copy_((s["out"].float().view(B, n, -1)[:, -1] @ weight)[:, None])
        vm.dspark_logits_process(s["logits"], s["logits"], s["lws"], hist=s["hist"], hist_len=s["hist_len"], rep=s["rep"])
        vm.dspark_sample(s["logits"][:, 0], s["u"], s["tok"], s["sws"], top_k=s["k"])
        s["owned"].copy_(s["owned_out"])
        s["state"].copy_(s["state_out"])
        s["seq"].copy_(s["kv_len"])

    weight = torch.randn((Hq * D, V), generator=g, device="cuda") / 4
    inputs = [(torch.randn((B * n, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF16), torch.rand(B, generator=g, device="cuda")) for _ in range(8)]
    eager, replayed = fresh(), fresh()
    step(fresh())                                           # (loads the kernels)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(replayed)
    for x, u in inputs:
        eager["qkv"].copy_(x)
        eager["u"].copy_(u)
        step(eager)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            replayed["qkv"].copy_(x)
            replayed["u"].copy_(u)
            graph.replay()
        torch.cuda.synchronize()
        for name in ("out", "tok", "table", "seq", "qkv"):
            assert torch.equal(eager[name], replayed[name]), name
        assert torch.equal(eager["cache"].k, replayed["cache"].k)
    # against the formula: the last step's rows over everything that was written
    lens = eager["kv_len"].tolist()
    assert lens == [8 * n] * B
    arrays = [t.cpu().numpy() for t in eager["cache"].tensors]
    lse = torch.zeros(eager["out"].shape[:2], device="cuda")
    K, V_ = ref.values(arrays[0], arrays[2], -1), ref.values(arrays[1], arrays[3], 0)
    want, _, tol, _ = ref.attention(_np(eager["qkv"][:, :Hq]), K, V_, eager["table"].cpu().numpy(), lens, eager["q_off"].tolist(), np.float32(D ** -0.5), True)
    assert (np.abs(_np(eager["out"]) - want) <= tol).all()
    for ws in (eager["ws"], eager["lws"], eager["sws"]):
        assert _status(vm, ws) == 0
    del lse


# ------------------------------------------------- attention on the tensor cores
def test_many_rows_of_128_with_pages_of_any_kind(vm):
    """More than 32 rows a key head: pages that whole copies take (multiples of 8
    positions), others, and pages with room between them."""
    rng = np.random.default_rng(21)
    D, new, lens = 128, 5, [700, 130, 64, 9, 5]
    n_new = np.array([5, 2, 4, 1, 3])
    q_off = np.concatenate([[0], np.cumsum(n_new)])
    q = torch.from_numpy(rng.standard_normal((int(q_off[-1]) + 2, 22, D))).to(BF16).cuda()
    for P in (8, 24, 40, 128, 256, 1, 12, 20):
        pages, table = _case(rng, len(lens), P, lens, D, 2)
        arrays = _cache(rng, pages, 2, P, D)
        _poison(arrays, table, lens, P)
        got, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, new)
        assert status == 0
        _check(q, arrays, table, lens, q_off, np.float32(D ** -0.5), got, lse)
        # keys' and values' pages in turn, and pages a little further apart than they are long
        tile_off = np.concatenate([[0], np.cumsum(-(-np.asarray(lens) // 64))])
        args = (_cu(table), _cu(lens), _cu(q_off), _cu(tile_off))
        for gap in (0, 64):
            kv = torch.full((pages, 2 * 2 * P * 64 + gap), 0xFF, dtype=torch.uint8, device="cuda")
            sc = torch.full((pages, 2 * 2 * P * 8 + gap), 0xFF, dtype=torch.uint8, device="cuda")
            views = []
            for i, (store, w) in enumerate(((kv, 64), (kv, 64), (sc, 8), (sc, 8))):
                at = (i % 2) * 2 * P * w
                view = store[:, at:at + 2 * P * w].unflatten(1, (2, P, w))
                view.copy_(torch.from_numpy(arrays[i]))
                views.append(view)
            out, l2 = torch.full_like(got, 77.0), torch.full_like(lse, 77.0)
            ws = vm.CacheWorkspace(len(lens), 22, 2, D, new)
            vm.dspark_cache_attention4(q, *views, *args, out, ws, max_new=new, lse=l2)
            assert _status(vm, ws) == 0
            _check(q, arrays, table, lens, q_off, np.float32(D ** -0.5), out, l2)


@pytest.mark.parametrize("rows", [33, 64, 65, 97, 136])
def test_many_rows_leave_out_bad_pages_and_keep_a_nan_to_the_rows_that_see_it(vm, rows):
    rng = np.random.default_rng(rows)
    D, P, n = 128, 16, 8 if rows % 8 == 0 else 1
    Hq = rows // n
    lens, q_off = [400, 150, 90], np.array([0, n, 2 * n, 3 * n])
    pages, table = _case(rng, 3, P, lens, D, 1)
    arrays = _cache(rng, pages, 1, P, D)
    # among the last positions of the first request, a value group; in the middle of the second, a key's
    for which, b, pos, group in ((3, 0, 400 - n // 2 - 1, 3), (2, 1, 149, 1), (3, 0, 399, 7)):
        arrays[which][table[b, pos // P], 0, pos % P, group] = 0x7F
    q = torch.from_numpy(rng.standard_normal((3 * n, Hq, D))).to(BF16).cuda()
    q[0, 0] = 0
    got, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, n)
    assert status == 0
    _check(q, arrays, table, lens, q_off, np.float32(D ** -0.5), got, lse)
    assert torch.isnan(got[:n, :, 48:64]).any() and not torch.isnan(got[:n, :, :48]).any()
    table[0, 3], table[0, 20], table[2, 5] = pages, -1, 2 ** 31 - 1
    got, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, n)
    assert status == BAD_PAGE
    _check(q, arrays, table, lens, q_off, np.float32(D ** -0.5), got, lse)
    table[2] = -5                                            # a request whose pages are all bad
    got, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, n)
    assert status == BAD_PAGE and not got[2 * n:].any() and bool((lse[2 * n:] == float("-inf")).all())


@pytest.mark.parametrize("lo,hi", [(-8, 0), (0, 28), (-40, 40), (90, 126), (-126, -100)])
def test_rows_of_very_different_sizes_share_a_tile(vm, lo, hi):
    """The queries of 64 rows, their sizes 2^lo .. 2^hi: each row against its own bound."""
    rng = np.random.default_rng(31)
    P, lens, D, n = 16, [500], 128, 4
    pages, table = _case(rng, 1, P, lens, D, 1)
    arrays = _cache(rng, pages, 1, P, D)
    size = 2.0 ** np.linspace(lo, hi, n * 16).round()
    q = torch.from_numpy(np.clip(rng.standard_normal((n, 16, D)), -1, 1) * size.reshape(n, 16, 1)).to(BF16).cuda()
    scale = 2.0 ** min(max(-(lo + hi) // 2, -100), 100)
    got, lse, status = _attend(vm, rng, q, arrays, table, lens, [0, n], n, scale=float(scale))
    assert status == 0
    # a tile's queries are exact to 2^-40 of its largest entry (the bound of a row of its own is 2^-25 of the row's)
    K, V = ref.values(arrays[0], arrays[2], 0), ref.values(arrays[1], arrays[3], 0)
    want, want_lse, tol, lse_tol = ref.attention(_np(q), K, V, table, lens, [0, n], scale, True)
    more = scale * 2.0 ** -40 * np.abs(_np(q)).max() * np.abs(K).sum(-1).max()
    x, ok = _np(got), np.isfinite(want_lse)
    bound = tol + 2 * more * np.abs(V).max()
    assert (np.abs(x - want) <= bound)[ok].all(), (np.abs(x - want) / bound)[ok].max()


@pytest.mark.parametrize("rows", [8, 64])
def test_scores_below_any_reference(vm, rows):
    """Scores of -10^37 everywhere: the weights are those of the differences."""
    rng = np.random.default_rng(5)
    P, D, n = 16, 128, 90
    pages, table = _case(rng, 1, P, [n], D, 1)
    arrays = _cache(rng, pages, 1, P, D)
    for a in (arrays[0], arrays[2]):
        a[:] = 0x22 if a.shape[-1] == 64 else 0x38          # every key entry 1, its scale 1
    q = torch.full((1, rows, D), -(2.0 ** 122), dtype=BF16, device="cuda")
    got, lse, status = _attend(vm, rng, q, arrays, table, [n], [0, 1], 1, scale=2.0 ** -7)
    assert status == 0
    _check(q, arrays, table, [n], np.array([0, 1]), 2.0 ** -7, got, lse)
    # every weight is the same: the mean, to a weight's and the result's rounding and 90 sums'
    V = ref.values(arrays[1], arrays[3], 0)[table[0, np.arange(n) // P], 0, np.arange(n) % P]
    bound = (ref.EPS16 + ref.EPSH + 100 * 2 * ref.EPS32) * np.abs(V).mean(0)
    assert (np.abs(_np(got)[0] - V.mean(0)) <= 1.01 * bound).all()


def test_expired_waits_are_reported_and_the_workspace_recovers(vm):
    """With a wait bound of 300 cycles the attention on the tensor cores gives up,
    reports a timeout and returns; after dspark_workspace_init the same call
    gives the results of a fresh workspace.  Every wait on the path is bounded."""
    rng = np.random.default_rng(15)
    P, lens, D, n = 16, [3000, 700], 128, 8
    q_off = np.array([0, n, 2 * n])
    pages, table = _case(rng, 2, P, lens, D, 8)
    arrays = _cache(rng, pages, 8, P, D)
    q = torch.from_numpy(rng.standard_normal((2 * n, 64, D))).to(BF16).cuda()
    ws = vm.CacheWorkspace(2, 64, 8, D, n)
    out, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, n, ws=ws)
    assert status == 0
    vm.dspark_workspace_set_wait_limit(ws.buf, 300)
    tile_off = np.concatenate([[0], np.cumsum(-(-np.asarray(lens) // 64))])
    vm.dspark_cache_attention4(q, *(torch.from_numpy(a).cuda() for a in arrays), _cu(table), _cu(lens), _cu(q_off), _cu(tile_off),
                               torch.empty_like(q), ws, max_new=n)
    st, bits = vm.dspark_sync_status(ws.buf)
    assert st == -3 and bits & 4
    vm.dspark_workspace_init(ws.buf)
    again, lse2, status = _attend(vm, rng, q, arrays, table, lens, q_off, n, ws=ws)
    assert status == 0 and torch.equal(again, out) and torch.equal(lse, lse2)


# ------------------------------------------------------------ sampling, the rest
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sampling_where_the_cut_lies_among_more_entries_than_a_list_holds(vm, dtype):
    """Long rows of few different values, and top-k beyond what is gathered: the
    last entry kept is found in the slices themselves."""
    rng = np.random.default_rng(8)
    V, pad = 60001, 60008
    x = torch.from_numpy(rng.integers(0, 3, (8, pad)).astype(np.float64)).to(dtype).cuda()[:, :V]
    x[0] = 2.5
    x[1] = -0.0
    u = np.array([0.0, 0.3, 0.5, 0.9, 0.99, 0.25, 0.75, 0.123])
    k, p = np.array([700, 59999, 20000, 1000, 513, 40000, 60000, 30000]), np.array([0.3, 0.9, 0.5, 0.999, 0.01, 0.7, 0.2, 0.66])
    for args in ((None, k, None, None), (None, None, p, None), (None, k, p, None), (np.full(8, 0.5), k, p, np.full(8, 0.2))):
        tok, lp, status = _sample(vm, x, u, *args)
        assert status == 0
        _check_rows(x, u, *args, tok, lp)


def test_sampling_is_the_same_in_any_batch(vm):
    """A row's token does not depend on the rows beside it or on how many CTAs take it."""
    g = torch.Generator(device="cuda").manual_seed(3)
    N, V = 400, 8200
    x = torch.randn((N, V), generator=g, device="cuda") * 4
    rng = np.random.default_rng(4)
    u, k, p = rng.random(N).astype(np.float32), rng.choice([0, 3, 100, 800], N), rng.choice([0.5, 0.95, 1.0], N)
    tok, lp, _ = _sample(vm, x, u, k=k, p=p)
    for n in (1, 7, 100):
        t, l, _ = _sample(vm, x[:n], u[:n], k=k[:n], p=p[:n])
        assert (t == tok[:n]).all() and (l == lp[:n]).all()


def test_sampling_refuses_results_that_overlap(vm):
    x, f = torch.zeros((4, 64), device="cuda"), torch.zeros(8, device="cuda")
    tok, ws = torch.zeros(8, dtype=torch.int32, device="cuda"), vm.SampleWorkspace(4)
    vm.dspark_sample(x, f[:4], tok[:4], ws, logprob=f[4:])
    for kw in (dict(logprob=f[3:7]), dict(logprob=x[0, :4]), dict(logprob=tok[2:6].view(F32)), dict(top_k=tok[3:7]), dict(temperature=f[4:], logprob=f[4:])):
        with pytest.raises(vm.DsparkError):
            vm.dspark_sample(x, f[:4], tok[:4], ws, **kw)
    assert _status(vm, ws) == 0


def test_rope_refuses_outputs_that_overlap(vm):
    x = torch.randn((6, 8, 64), device="cuda")
    pos, table = torch.arange(6, dtype=torch.int32, device="cuda"), vm.RopeTable(64)
    want = torch.empty_like(x)
    vm.dspark_rope(x, None, pos, table, want)
    q, k = x[:, :5], x[:, 5:]
    for qo, ko in ((x[:, 1:6], None), (x[:, :5], x[:, 4:7]), (x[:, 3:], x[:, :3])):
        with pytest.raises(vm.DsparkError):
            vm.dspark_rope(q, k if ko is not None else None, pos, table, qo, ko)
    vm.dspark_rope(q, k, pos, table)                         # slices of the same rows, in place
    assert torch.equal(x, want)


def test_two_streams_at_once(vm):
    """Two steps' calls on two streams, each with workspaces of its own, give what they give alone."""
    rng = np.random.default_rng(12)
    P, D, n, lens = 16, 128, 4, [2000, 300, 40]
    q_off = n * np.arange(4)
    pages, table = _case(rng, 3, P, lens, D, 2)
    ts = [torch.from_numpy(a).cuda() for a in _cache(rng, pages, 2, P, D)]
    tile_off = np.concatenate([[0], np.cumsum(-(-np.asarray(lens) // 64))])
    args = (_cu(table), _cu(lens), _cu(q_off), _cu(tile_off))
    runs = []
    for i, heads in enumerate((8, 32)):
        g = torch.Generator(device="cuda").manual_seed(i)
        q = torch.randn((3 * n, heads, D), generator=g, device="cuda").to(BF16)
        x = torch.randn((50, 30000), generator=g, device="cuda") * 3
        runs.append(dict(q=q, x=x, u=torch.rand(50, generator=g, device="cuda"), p=torch.full((50,), 0.9, device="cuda"), ws=vm.CacheWorkspace(3, heads, 2, D, n),
                         sws=vm.SampleWorkspace(50), s=torch.cuda.Stream()))

    def call(r, stream):
        out, tok = torch.empty_like(r["q"]), torch.empty(50, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        return out, tok, lambda: (vm.dspark_cache_attention4(r["q"], *ts, *args, out, r["ws"], max_new=n, stream=stream),
                                  vm.dspark_sample(r["x"], r["u"], tok, r["sws"], top_p=r["p"], stream=stream))

    alone = []
    for r in runs:
        out, tok, go = call(r, r["s"])
        go()
        torch.cuda.synchronize()
        alone.append((out, tok))
    both = [call(r, r["s"]) for r in runs]
    for _ in range(5):
        for _, _, go in both:
            go()
    torch.cuda.synchronize()
    for (out, tok, _), (o, t) in zip(both, alone):
        assert torch.equal(out, o) and torch.equal(tok, t)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group,new", [(1, 1), (8, 1), (3, 3), (2, 8), (4, 8), (8, 8), (16, 8)])
def test_attention_stays_within_its_workspace(vm, group, new, D, dtype):
    """Segments split over all workers: what lies behind the workspace is untouched, and a smaller one is refused."""
    rng = np.random.default_rng(group + new)
    P, lens, q_off = 16, [5000, 3000], np.array([0, new, new + 1])
    pages, table = _case(rng, 2, P, lens, D, 2)
    arrays = _cache(rng, pages, 2, P, D)
    q = torch.from_numpy(rng.standard_normal((new + 1, 2 * group, D))).to(dtype).cuda()
    n = vm.dspark_cache4_workspace_bytes(2, 2 * group, 2, D, new)
    big = torch.full((n + (1 << 20),), 0x5a, dtype=torch.uint8, device="cuda")
    ws = vm.CacheWorkspace(2, 2 * group, 2, D, new)
    assert len(ws.buf4) >= n
    ws.buf = ws.buf4 = big[:n]
    vm.dspark_workspace_init(ws.buf)
    got, lse, status = _attend(vm, rng, q, arrays, table, lens, q_off, new, ws=ws)
    assert status == 0 and bool((big[n:] == 0x5a).all())
    fresh, lse2, _ = _attend(vm, rng, q, arrays, table, lens, q_off, new)
    assert torch.equal(got, fresh) and torch.equal(lse, lse2)
    ws.buf4 = big[:n - 256]
    with pytest.raises(vm.DsparkError):
        _attend(vm, rng, q, arrays, table, lens, q_off, new, ws=ws)
