"""GPU tests of the serving operators (paged cache plan, append and attention,
logit controls) against the 64-bit references of tests/_serve_ref.py."""
import numpy as np
import pytest
import torch

from tests import _serve_ref as ref

pytestmark = pytest.mark.gpu
BAD_TOKEN, BAD_LENGTH, BAD_INPUT, DEAD_ROW, BAD_PAGE = 1, 2, 8, 16, 32


@pytest.fixture(scope="module")
def vm():
    import verify_markov_head_gb300 as vm
    return vm


def _cu(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


def _status(vm, ws):
    return vm.dspark_sync_status(ws.buf)[1]


# -------------------------------------------------------------------- plan
def _plan_inputs(rng, B, P, hi, new_hi, width, spare, ended=0.1):
    seq = rng.integers(0, hi + 1, B)
    new = rng.integers(0, new_hi + 1, B)
    owned = -(-seq // P)
    owned = np.minimum(owned + (rng.random(B) < 0.3), width)
    gone = rng.random(B) < ended
    seq[gone] = 0
    new[gone] = 0
    pages = int(owned.sum()) + spare
    perm = rng.permutation(pages)
    table = np.full((B, width), -1)
    o = 0
    for b in range(B):
        table[b, :owned[b]] = perm[o:o + owned[b]]
        o += owned[b]
    head = int(rng.integers(0, pages))
    ring = np.roll(np.concatenate([perm[o:], np.full(o, -7)]), head)
    return [a.astype(np.int32) for a in (seq, new, owned, ring)] + [np.array([head, spare], np.int32), table.astype(np.int32)]


def _run_plan(vm, seq, new, owned, ring, state, table, P, T, ws=None, stream=None):
    B = len(seq)
    e = lambda n: torch.full((n,), -99, dtype=torch.int32, device="cuda")  # noqa: E731
    o = dict(owned_out=e(B), ring_state_out=e(2), kv_len=e(B), q_off=e(B + 1), tile_off=e(B + 1), slot_map=e(T),
             positions=e(T))
    tab, rng_ = _cu(table), _cu(ring)
    args = (_cu(seq), _cu(new), _cu(owned), rng_, _cu(state), tab, P)
    for _ in range(2):                       # the same inputs give the same outputs
        vm.dspark_cache_plan(*args, **o, ws=ws, stream=stream)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in dict(o, block_table=tab, ring=rng_).items()}


@pytest.mark.parametrize("B,P,hi,new_hi,spare", [
    (1, 16, 40, 8, 9), (3, 1, 30, 8, 40), (64, 64, 5000, 8, 128), (513, 16, 300, 8, 700), (33, 24, 100, 90, 400),
    (4096, 8, 50, 3, 4096), (40, 16, 200, 60, 37),     # the last: the ring runs out
])
def test_plan_matches_a_host_allocator(vm, B, P, hi, new_hi, spare):
    rng = np.random.default_rng(B * 1000 + P)
    width = -(-(hi + new_hi) // P) + 1
    seq, new, owned, ring, state, table = _plan_inputs(rng, B, P, hi, new_hi, width, spare)
    T = int(new.sum()) + 5
    want = ref.plan(seq, new, owned, ring, state, table, P, T)
    ws = vm.LogitsWorkspace(1, 1)
    got = _run_plan(vm, seq, new, owned, ring, state, table, P, T, ws)
    bad = want.pop("bad")
    for k, v in want.items():
        np.testing.assert_array_equal(got[k], v, err_msg=k)
    assert _status(vm, ws) == (BAD_PAGE if bad else 0)


def test_plan_reports_short_tables_negative_lengths_and_too_many_tokens(vm):
    rng = np.random.default_rng(5)
    seq, new, owned, ring, state, table = _plan_inputs(rng, 6, 16, 60, 8, 4, 20, ended=0.0)
    seq[1], new[1] = 60, 8                   # 68 positions, a row holds 64
    seq[3] = -5
    new[4] = -1
    ws = vm.LogitsWorkspace(1, 1)
    T = 3
    want = ref.plan(seq, new, owned, ring, state, table, 16, T)
    got = _run_plan(vm, seq, new, owned, ring, state, table, 16, T, ws)
    assert want.pop("bad")
    for k in want:
        if k != "positions":                 # the positions of a negative length are not defined
            np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    assert _status(vm, ws) == BAD_PAGE | BAD_LENGTH


def test_plan_chained_over_steps_never_shares_a_page(vm):
    """Steps with random admitted and accepted counts: at every step the owned
    pages and the free ones are a partition of all pages."""
    rng = np.random.default_rng(8)
    B, P, width, pages = 17, 8, 40, 420
    table, ring = np.full((B, width), -1, np.int32), np.arange(pages, dtype=np.int32)
    seq, owned, state = np.zeros(B, np.int32), np.zeros(B, np.int32), np.array([0, pages], np.int32)
    for step in range(30):
        new = rng.integers(1, 9, B).astype(np.int32)
        ended = rng.random(B) < 0.05
        ended |= seq + 8 > width * P
        seq[ended], new[ended] = 0, 0
        got = _run_plan(vm, seq, new, owned, ring, state, table, P, 8 * B)
        table, ring, owned, state = got["block_table"], got["ring"], got["owned_out"], got["ring_state_out"]
        held = np.concatenate([table[b, :owned[b]] for b in range(B)] + [ring[(state[0] + np.arange(state[1])) % pages]])
        np.testing.assert_array_equal(np.sort(held), np.arange(pages))
        slots = got["slot_map"][got["slot_map"] >= 0]
        assert len(set(slots.tolist())) == int(new.sum())
        seq = seq + np.minimum(new, rng.integers(1, 9, B)).astype(np.int32)     # accepted + 1


M = 2 ** 31 - 1


@pytest.mark.parametrize("news", [[8, 8, M, 8], [8, 2 ** 30, 8, 2 ** 30, 8], [M, M, 0, 0, 8, 0, M, M], [8, M, M], [-2 ** 31, 8, M],
                                  [8] * 31 + [M, 8, M] + [8] * 40])
def test_plan_keeps_numbers_of_tokens_out_of_range_from_the_other_requests(vm, news):
    """A number of new tokens beyond the table's rows counts none, as a negative
    one does; the other requests are planned as if it were not there."""
    rng = np.random.default_rng(len(news))
    B = len(news)
    seq, new, owned, ring, state, table = _plan_inputs(rng, B, 16, 300, 8, 24, 10 + 2 * B, ended=0.0)
    new[:] = news
    wild = (new < 0) | (new > 24 * 16)
    T = 8 * B + 3
    want = ref.plan(seq, np.where(wild, -1, new), owned, ring, state, table, 16, T)
    ws = vm.LogitsWorkspace(1, 1)
    got = _run_plan(vm, seq, new, owned, ring, state, table, 16, T, ws)
    assert want.pop("bad")
    for k in want:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    assert _status(vm, ws) == BAD_PAGE


def test_plan_stops_its_sums_and_reports_too_many_tokens(vm):
    """Numbers of tokens that a row of the table holds, but no ring: their sum
    passes 2^31.  Lengths near 2^31 have no pages."""
    P, n, width = 4096, 1 << 30, (1 << 18) + 1
    seq = np.array([5, 7, 0, 2 ** 31 - 1, 9, 0, 2 ** 31 - 64], np.int32)
    new = np.array([8, n, 8, 8, n, n, 0], np.int32)
    B, T = len(new), 40
    owned = np.array([1, 1, 0, 0, 1, 0, 0], np.int32)
    table = np.full((B, width), -1, np.int32)
    table[0, 0], table[1, 0], table[4, 0] = 3, 1, 4
    ring = np.array([0, 2, 5, -7, -7, -7], np.int32)
    ws = vm.LogitsWorkspace(1, 1)
    got = _run_plan(vm, seq, new, owned, ring, np.array([0, 3], np.int32), table, P, T, ws)
    assert _status(vm, ws) == BAD_PAGE | BAD_LENGTH
    off = np.minimum(np.concatenate([[0], np.cumsum(new.astype(np.int64))]), M)
    np.testing.assert_array_equal(got["q_off"], off)
    # requests are served in order while the ring has pages: the second asks for more than there are
    np.testing.assert_array_equal(got["kv_len"], [13, 0, 0, 0, 0, 0, 0])
    np.testing.assert_array_equal(got["tile_off"], [0, 1, 1, 1, 1, 1, 1, 1])
    np.testing.assert_array_equal(got["owned_out"], owned)
    np.testing.assert_array_equal(got["ring_state_out"], [0, 3])
    np.testing.assert_array_equal(got["slot_map"], list(range(3 * P + 5, 3 * P + 13)) + [-1] * (T - 8))
    np.testing.assert_array_equal(got["positions"][:8], range(5, 13))
    np.testing.assert_array_equal(got["block_table"], table)
    np.testing.assert_array_equal(got["ring"], ring)


def test_plan_refuses_outputs_that_overlap_its_inputs_or_each_other(vm):
    """kv_len in place of seq_len and the like: CTAs read the lengths again while the first one writes."""
    rng = np.random.default_rng(6)
    B, P, T = 40, 16, 300
    seq, new, owned, ring, state, table = _plan_inputs(rng, B, P, 200, 8, 16, 90, ended=0.0)
    i = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    ins = dict(seq_len=_cu(seq), n_new=_cu(new), owned=_cu(owned), ring=_cu(ring), ring_state=_cu(state), block_table=_cu(table))
    outs = dict(owned_out=i(B), ring_state_out=i(2), kv_len=i(B), q_off=i(B + 1), tile_off=i(B + 1), slot_map=i(T), positions=i(T))
    vm.dspark_cache_plan(**ins, page_size=P, **outs)
    torch.cuda.synchronize()
    pair = i(2 * B)
    pair[:B] = ins["seq_len"]
    for kw in (dict(kv_len=ins["seq_len"]), dict(kv_len=ins["n_new"]), dict(owned_out=ins["owned"]), dict(ring_state_out=ins["ring_state"]),
               dict(seq_len=pair[:B], kv_len=pair[B - 1:2 * B - 1]), dict(positions=outs["slot_map"]), dict(tile_off=outs["q_off"]),
               dict(ring_state_out=ins["seq_len"][3:5]), dict(kv_len=ins["block_table"].view(-1)[:B]), dict(slot_map=i(T)[:T], positions=ins["ring"][:T])):
        if kw.get("positions") is not None and kw["positions"].numel() != T:
            kw["slot_map"] = kw["slot_map"][:kw["positions"].numel()].contiguous()
        with pytest.raises(vm.DsparkError):
            vm.dspark_cache_plan(**{**ins, **outs, **kw}, page_size=P)
    vm.dspark_cache_plan(**{**ins, **outs, "seq_len": pair[:B], "kv_len": pair[B:]}, page_size=P)     # side by side
    same = dict(ins, n_new=ins["seq_len"])                                                            # inputs may be one
    vm.dspark_cache_plan(**same, page_size=P, **outs)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D,P", [(1, 1, 8, 1), (5, 3, 64, 24), (700, 8, 128, 16), (333, 2, 80, 64), (0, 2, 64, 8)])
def test_append_writes_exactly_the_slots(vm, T, H, D, P, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    pages = T // P + 4
    qkv = torch.randn((T, 3 * H, D), generator=g, device="cuda").to(dtype)        # tokens at a stride
    kv = torch.randn((pages, 2, H, P, D), generator=g, device="cuda").to(dtype)   # keys and values by turns
    k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    slots = torch.randperm(pages * P, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 3:
        slots[1], slots[3] = -1, pages * P + 7        # skipped; skipped and reported
    want = kv.clone()
    for t in range(T):
        s = int(slots[t])
        if 0 <= s < pages * P:
            want[s // P, 0, :, s % P] = k[t]
            want[s // P, 1, :, s % P] = v[t]
    ws = vm.LogitsWorkspace(1, 1)
    vm.dspark_cache_append(k, v, slots, kv[:, 0], kv[:, 1], ws=ws)
    assert _status(vm, ws) == (BAD_PAGE if T > 3 else 0)
    assert torch.equal(kv.view(torch.int16), want.view(torch.int16))


# --------------------------------------------------------------- attention
def _attention_inputs(rng, lens, news, Hq, Hkv, D, P, dtype, junk=True, q_pad=0, extra_pages=3, wide=0):
    """Caches whose unused places (other pages, rows beyond the length) hold
    NaN, block tables with -1 beyond the owned pages."""
    B, lens, news = len(lens), np.asarray(lens), np.asarray(news)
    per = -(-lens // P)
    width, pages = int(per.max()) + 1 + wide, int(per.sum()) + extra_pages
    perm = rng.permutation(pages)
    table = np.full((B, width), -1)
    k, v = (np.full((pages, Hkv, P, D), np.nan if junk else 0.0, np.float32) for _ in range(2))
    o = 0
    for b in range(B):
        table[b, :per[b]] = perm[o:o + per[b]]
        o += per[b]
        pos = np.arange(lens[b])
        k[table[b, pos // P], :, pos % P] = rng.standard_normal((lens[b], Hkv, D))
        v[table[b, pos // P], :, pos % P] = rng.standard_normal((lens[b], Hkv, D))
    q_off = np.concatenate([[0], np.cumsum(news)])
    N = int(q_off[-1])
    q = torch.as_tensor(rng.standard_normal((N, Hq + q_pad, D)) * 2, dtype=torch.float32).to(dtype).cuda()[:, :Hq]
    tile_off = np.concatenate([[0], np.cumsum(-(-lens // 64))])
    return dict(q=q, k=torch.as_tensor(k).to(dtype).cuda(), v=torch.as_tensor(v).to(dtype).cuda(), table=_cu(table),
                kv_len=_cu(lens), q_off=_cu(q_off), tile_off=_cu(tile_off))


def _attend(vm, a, max_new, scale=None, ws=None, stream=None):
    q = a["q"]
    ws = ws or vm.CacheWorkspace(a["table"].shape[0], q.shape[1], a["k"].shape[1], q.shape[2], max_new)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    vm.dspark_cache_attention(q, a["k"], a["v"], a["table"], a["kv_len"], a["q_off"], a["tile_off"], out, ws,
                              max_new=max_new, scale=scale, lse=lse, stream=stream)
    torch.cuda.synchronize()
    return out, lse, ws


def _check_attention(a, out, lse, scale):
    d = lambda t: t.cpu().double().numpy()  # noqa: E731
    i = lambda t: t.cpu().numpy()  # noqa: E731
    bf = a["q"].dtype == torch.bfloat16
    want, wlse, tol, ltol = ref.attention(d(a["q"]), d(a["k"]), d(a["v"]), i(a["table"]), i(a["kv_len"]), i(a["q_off"]),
                                          scale, ref.EPS16 if bf else 0.0, ref.EPS16 if bf else 4 * ref.EPS32)
    got, glse = d(out), d(lse)
    assert np.isfinite(got).all()
    over = np.abs(got - want) / np.maximum(tol, 1e-30)
    assert (np.abs(got - want) <= tol).all(), over.max()
    empty = np.isinf(wlse)
    np.testing.assert_array_equal(glse[empty], wlse[empty])
    assert (np.abs(glse[~empty] - wlse[~empty]) <= ltol[~empty]).all()


ATTENTION = [
    # lens, news, Hq, Hkv, D, page size
    ([1], [1], 4, 1, 64, 16),
    ([64, 65, 63, 1, 128], [1, 1, 1, 1, 1], 8, 2, 128, 16),
    ([0, 5, 0, 200], [2, 1, 0, 8], 4, 4, 64, 8),               # rows that see nothing, requests without a token
    ([8, 130, 67, 9], [8, 3, 5, 8], 32, 8, 128, 64),           # blocks that fill the cache, ragged
    ([300, 77], [8, 7], 14, 2, 64, 24),                        # 7 heads to a key head, an odd page size
    ([500, 2, 129], [4, 2, 8], 16, 1, 128, 32),                # one key head: several tiles of rows
    ([70], [17], 16, 2, 128, 1),                               # the longest block, pages of one position
    ([1000, 1], [1, 1], 8, 8, 128, 128),                       # no shared heads
    ([90, 33], [8, 2], 6, 2, 80, 16),                          # other head sizes
    ([90, 130], [3, 8], 4, 2, 256, 64),
    ([45, 100], [8, 1], 8, 1, 8, 16),
    ([4100], [8], 8, 2, 64, 64),                               # split over many CTAs
    ([130, 20], [8, 3], 96, 1, 64, 16),                        # 96 heads to a key head
    ([2000, 70, 900], [0, 1, 0], 8, 4, 128, 32),               # requests that wait
    ([9000], [8], 8, 1, 128, 16),                              # one key head, few CTAs with long shares
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention_matches_the_definition(vm, case, dtype):
    lens, news, Hq, Hkv, D, P = ATTENTION[case]
    rng = np.random.default_rng(case)
    a = _attention_inputs(rng, lens, news, Hq, Hkv, D, P, dtype, q_pad=case % 3)
    out, lse, ws = _attend(vm, a, max(max(news), 1))
    _check_attention(a, out, lse, D ** -0.5)
    assert _status(vm, ws) == 0
    again, lse2, _ = _attend(vm, a, max(max(news), 1), ws=ws)      # the same bits on a used workspace
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lens,news,Hq,Hkv,D,P", [
    ([500, 2, 129], [4, 2, 8], 16, 1, 128, 32), ([70, 1], [17, 1], 16, 2, 128, 8), ([130, 20], [8, 3], 96, 1, 64, 16),
    ([3000], [8], 16, 1, 128, 64),
])
def test_attention_with_128_rows_at_once(vm, lens, news, Hq, Hkv, D, P):
    """Block tables for long contexts (most of them empty here): more than 64 rows
    of a key head are taken together."""
    rng = np.random.default_rng(len(lens) + Hq)
    a = _attention_inputs(rng, lens, news, Hq, Hkv, D, P, torch.bfloat16, wide=400000 // P)
    out, lse, ws = _attend(vm, a, max(news))
    _check_attention(a, out, lse, D ** -0.5)
    assert _status(vm, ws) == 0
    again, lse2, _ = _attend(vm, a, max(news), ws=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("P,group,new,wide", [(8, 1, 8, 0), (16, 4, 4, 0), (64, 4, 8, 0), (128, 8, 1, 0), (32, 12, 8, 400000), (5, 3, 8, 0), (1, 2, 4, 0), (12, 8, 8, 0)])
@pytest.mark.parametrize("D", [16, 40, 80, 96, 112, 120, 192, 256, 136])
def test_attention_of_other_head_sizes(vm, D, P, group, new, wide):
    """Heads that do not fill a tile's row, or fill two; pages that are no
    multiple of 8 positions; 8 to 96 rows of a key head (wide: 96 at once); lengths about the tiles' ends; q and cache with
    gaps between tokens and pages; positions beyond the lengths hold NaN."""
    rng = np.random.default_rng(D + P)
    lens = [300, 1, 0, 128, 129, 64, 700]
    news = np.minimum([new, 1, 2, new, max(new - 1, 1), new, new], new)
    a = _attention_inputs(rng, lens, news, 2 * group, 2, D, P, torch.bfloat16, q_pad=1, wide=wide // P)
    kv = torch.stack([a["k"], a["v"]], 1)
    a = dict(a, k=kv[:, 0], v=kv[:, 1])
    out, lse, ws = _attend(vm, a, new)
    _check_attention(a, out, lse, D ** -0.5)
    assert _status(vm, ws) == 0
    again, lse2, _ = _attend(vm, a, new, ws=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group,new", [(1, 1), (8, 1), (3, 3), (2, 8), (4, 8), (8, 8), (16, 8)])
def test_attention_stays_within_its_workspace(vm, group, new, dtype):
    """Segments split over all SMs, both kinds of tables; what lies behind the workspace is untouched."""
    D, P = 64, 16
    for wide in (0, 300000 // P):
        a = _attention_inputs(np.random.default_rng(group + new), [5000, 3000], [new, 1], 2 * group, 2, D, P, dtype, wide=wide)
        n = vm.dspark_cache_workspace_bytes(2, 2 * group, 2, D, new)
        ws = vm.CacheWorkspace(2, 2 * group, 2, D, new)
        big = torch.full((16 << 20,), 0x5a, dtype=torch.uint8, device="cuda")       # 256-byte aligned, far larger
        ws.buf = big[:n]
        vm.dspark_workspace_init(ws.buf)
        out, lse, _ = _attend(vm, a, new, ws=ws)
        _check_attention(a, out, lse, D ** -0.5)
        assert bool((big[n:] == 0x5a).all())


def test_attention_of_a_large_ragged_batch(vm):
    rng = np.random.default_rng(77)
    lens = rng.integers(1, 400, 150)
    news = np.minimum(lens, rng.integers(1, 9, 150))
    a = _attention_inputs(rng, lens, news, 8, 2, 64, 16, torch.bfloat16)
    out, lse, ws = _attend(vm, a, 8)
    _check_attention(a, out, lse, 64 ** -0.5)


@pytest.mark.parametrize("dtype,Hq", [(torch.bfloat16, 2), (torch.bfloat16, 8), (torch.float32, 2)])
def test_attention_of_a_long_context(vm, dtype, Hq):
    """131071 positions of one key head beside a short request: split over all SMs."""
    rng = np.random.default_rng(78)
    a = _attention_inputs(rng, [131071, 9], [2, 8], Hq, 1, 64, 64, dtype)
    out, lse, ws = _attend(vm, a, 8)
    _check_attention(a, out, lse, 64 ** -0.5)
    assert _status(vm, ws) == 0


def test_attention_scale_and_large_scores(vm):
    """A large scale makes the softmax a maximum: no overflow, the running
    maximum carries over the tiles."""
    rng = np.random.default_rng(3)
    a = _attention_inputs(rng, [700, 40], [8, 8], 8, 2, 128, 16, torch.bfloat16)
    out, lse, _ = _attend(vm, a, 8, scale=3.0)
    _check_attention(a, out, lse, 3.0)


def _vary_block_values(a, b, P, bad):
    """The value of the last position of request b set to `bad` in every head."""
    pos = int(a["kv_len"][b]) - 1
    a["v"][int(a["table"][b, pos // P]), :, pos % P, ::3] = bad


@pytest.mark.parametrize("dtype,Hq,wide", [(torch.bfloat16, 8, 0), (torch.float32, 8, 0), (torch.bfloat16, 32, 30000)])
@pytest.mark.parametrize("D,P", [(128, 16), (96, 16), (256, 16), (128, 1), (256, 12)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_later_drafts_value_never_reaches_an_earlier_row(vm, bad, D, P, dtype, Hq, wide):
    """A draft whose value is not finite: the rows before it, which do not see
    it, are as they were; its own row is not finite where the value is not."""
    rng = np.random.default_rng(4)
    a = _attention_inputs(rng, [70, 64, 8], [8, 5, 8], Hq, 2, D, P, dtype, wide=wide)
    clean, _, _ = _attend(vm, a, 8)
    for b in range(3):
        _vary_block_values(a, b, P, bad)
    got, _, _ = _attend(vm, a, 8)
    last = (a["q_off"][1:] - 1).tolist()
    for t in range(got.shape[0]):
        if t in last:
            assert not torch.isfinite(got[t, :, ::3].float()).any()
            assert torch.isfinite(got[t, :, 1::3].float()).all()
        else:
            assert torch.equal(got[t], clean[t])


@pytest.mark.parametrize("P", [64, 20])
def test_attention_reads_pages_beyond_32_bit_offsets(vm, P):
    """Pages whose element offset passes 2^31, in caches of 2 x 4.4 GB."""
    H, D = 8, 128
    pages = (1 << 31) // (H * P * D) + 600
    k = torch.zeros((pages, H, P, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    rng = np.random.default_rng(9)
    a = _attention_inputs(rng, [200, 64], [8, 1], 16, H, D, P, torch.bfloat16, extra_pages=0)
    n = a["k"].shape[0]
    k[pages - n:], v[pages - n:] = a["k"], a["v"]
    big = dict(a, k=k, v=v, table=torch.where(a["table"] >= 0, a["table"] + pages - n, -1))
    out, lse, _ = _attend(vm, a, 8)
    out2, lse2, ws = _attend(vm, big, 8)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and _status(vm, ws) == 0
    new_k = torch.randn((1, H, D), device="cuda").to(torch.bfloat16)
    vm.dspark_cache_append(new_k, new_k, _cu([pages * P - 1]), k, v)
    assert torch.equal(k[pages - 1, :, P - 1], new_k[0])


def test_attention_on_another_stream_and_interleaved_caches(vm):
    rng = np.random.default_rng(12)
    a = _attention_inputs(rng, [300, 20], [8, 2], 8, 2, 128, 16, torch.bfloat16)
    out, lse, _ = _attend(vm, a, 8)
    kv = torch.stack([a["k"], a["v"]], 1)                   # [pages, 2, heads, page, dim]
    b = dict(a, k=kv[:, 0], v=kv[:, 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out2, lse2, _ = _attend(vm, b, 8, stream=s)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("P", [16, 4])
def test_attention_reports_bad_pages_and_lengths(vm, P):
    rng = np.random.default_rng(13)
    a = _attention_inputs(rng, [100, 50], [2, 2], 4, 2, 64, P, torch.bfloat16)
    out, _, ws = _attend(vm, a, 2)
    hurt = dict(a, table=a["table"].clone())
    hurt["table"][1, 1] = a["k"].shape[0]                   # a page that does not exist
    got, _, _ = _attend(vm, hurt, 2, ws=ws)
    assert _status(vm, ws) == BAD_PAGE
    assert torch.equal(got[:2], out[:2]) and torch.isfinite(got.float()).all()
    got, _, _ = _attend(vm, a, 1, ws=vm.CacheWorkspace(2, 4, 2, 64, 2))
    ws2 = vm.CacheWorkspace(2, 4, 2, 64, 2)
    _attend(vm, a, 1, ws=ws2)                               # two tokens a request, one announced
    assert _status(vm, ws2) == BAD_LENGTH
    far = dict(a, kv_len=a["kv_len"] + 100000)
    _attend(vm, far, 2, ws=ws2)
    assert _status(vm, ws2) & BAD_LENGTH


def _rows_as_defined(a, out, lse, requests):
    """The rows of these requests against the definition."""
    q_off, n = a["q_off"].cpu(), a["kv_len"].shape[0]
    take = torch.cat([torch.arange(int(q_off[b]), int(q_off[b + 1])) for b in range(n) if b in requests]).cuda()
    news = [int(q_off[b + 1] - q_off[b]) for b in range(n) if b in requests]
    keep = torch.tensor([b for b in range(n) if b in requests], device="cuda")
    part = dict(a, q=a["q"][take], table=a["table"][keep], kv_len=a["kv_len"][keep], q_off=_cu(np.concatenate([[0], np.cumsum(news)])))
    _check_attention(part, out[take], lse[take], a["q"].shape[2] ** -0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,P", [(3, 16), (3, 4), (70, 64)])
def test_attention_reports_tile_offsets_of_an_earlier_step(vm, B, P, dtype):
    """The lengths grew and tile_off did not: status bit 1 where a request has a
    tile more; the requests with as many tiles as before are as they should be."""
    rng = np.random.default_rng(B + P)
    lens = rng.integers(9, 700, B)
    lens[0], lens[1] = 128, 127                    # one position more: a new tile; none
    news = rng.integers(1, 9, B)
    a = _attention_inputs(rng, lens + 1, news, 8, 2, 64, P, dtype)
    old = np.concatenate([[0], np.cumsum(-(-lens // 64))])
    grown = -(-(lens + 1) // 64) > -(-lens // 64)
    assert grown[0] and not grown[1]
    out, lse, ws = _attend(vm, dict(a, tile_off=_cu(old)), 8)
    assert _status(vm, ws) == BAD_LENGTH
    _rows_as_defined(a, out, lse, np.flatnonzero(~grown).tolist())
    out, lse, ws = _attend(vm, a, 8, ws=ws)
    _rows_as_defined(a, out, lse, list(range(B)))
    assert _status(vm, ws) == 0


@pytest.mark.parametrize("dtype,D,wide", [(torch.bfloat16, 64, 0), (torch.float32, 64, 0), (torch.bfloat16, 256, 0), (torch.bfloat16, 64, 40000)])
@pytest.mark.parametrize("B", [2, 5, 70])
def test_attention_reports_tile_offsets_out_of_range(vm, B, D, dtype, wide):
    """Entries that do not ascend, negative and large ones between good ones: the
    status bit, nothing written beside the rows, and the workspace as good as before."""
    rng = np.random.default_rng(B + D)
    lens, P = rng.integers(1, 700, B), 16
    a = _attention_inputs(rng, lens, np.minimum(lens, 8), 8, 2, D, P, dtype, wide=wide)
    want, wlse, ws = _attend(vm, a, 8)
    off = a["tile_off"].cpu().numpy()
    total, width = int(off[-1]), a["table"].shape[1]
    room = B * -(-width * P // 64)                 # tiles that the tables could hold
    N = want.shape[0]
    big = torch.full((N + 8, *want.shape[1:]), 7.0, dtype=dtype, device="cuda")
    cases = []
    for i in range(1, B, max(1, B // 3)):
        for x in (-2 ** 31, -(1 << 25), -1, 1 << 25, 2 ** 31 - 1, total + 3, int(off[i + 1]) + 1, int(off[i - 1]) - 1):
            cases.append(np.concatenate([off[:i], [x], off[i + 1:]]))
    cases += [np.concatenate([[0], np.sort(off[1:B])[::-1], [total]]), np.concatenate([off[:B], [total - 1]]),
              np.concatenate([off[:B], [min(room, total + 100)]]), np.concatenate([off[:B], [room + 1]]), np.full(B + 1, -1),
              off + 1, np.where(np.arange(B + 1) < B, 0, total)]
    for o in cases:
        if (o == off).all():
            continue
        vm.dspark_cache_attention(a["q"], a["k"], a["v"], a["table"], a["kv_len"], a["q_off"], _cu(o), big[4:N + 4], ws, max_new=8)
        assert _status(vm, ws) == BAD_LENGTH, o
        assert bool((big[:4] == 7).all()) and bool((big[N + 4:] == 7).all())
    out, lse, _ = _attend(vm, a, 8, ws=ws)
    assert torch.equal(out, want) and torch.equal(lse, wlse) and _status(vm, ws) == 0


@pytest.mark.parametrize("Hq,Hkv,new,D,P", [(4, 4, 1, 128, 16), (8, 2, 3, 64, 16), (16, 2, 4, 128, 64), (8, 2, 8, 96, 16), (8, 2, 8, 64, 4),
                                            (16, 2, 8, 128, 16), (16, 2, 8, 64, 8), (16, 2, 8, 256, 16), (8, 2, 8, 256, 12), (16, 2, 8, 80, 1)])
def test_attention_of_up_to_64_rows_holds_its_weights_to_2_to_the_minus_15(vm, Hq, Hkv, new, D, P):
    """4 to 64 rows a key head: a weight w enters the second product as its leading 8
    bits, cut off, and the rest of (1 + 2^-20) w rounded to 8 bits: off by at most
    2^-8 (2^-7 + 2^-20) w + 2^-20 w.  The product's 2 len / 16 additions in binary32
    may each cut off 2^-23 of the sum of magnitudes."""
    rng = np.random.default_rng(Hq + D + P)
    lens = [700, 64, 129]
    a = _attention_inputs(rng, lens, [new] * 3, Hq, Hkv, D, P, torch.bfloat16)
    out, _, ws = _attend(vm, a, new)
    d = lambda t: t.cpu().double().numpy()  # noqa: E731
    i = lambda t: t.cpu().numpy()  # noqa: E731
    weight = 2.0 ** -8 * (2.0 ** -7 + 2.0 ** -20) + 2.0 ** -20 + max(lens) / 8 * 2.0 ** -23
    want, _, tol, _ = ref.attention(d(a["q"]), d(a["k"]), d(a["v"]), i(a["table"]), i(a["kv_len"]), i(a["q_off"]), D ** -0.5, weight, ref.EPS16)
    assert _status(vm, ws) == 0
    assert (np.abs(d(out) - want) <= tol).all(), (np.abs(d(out) - want) / tol).max()


@pytest.mark.parametrize("dtype,Hq,wide", [(torch.bfloat16, 2, 0), (torch.bfloat16, 8, 0), (torch.bfloat16, 16, 0), (torch.bfloat16, 32, 30000),
                                           (torch.float32, 8, 0)])
def test_an_infinite_value_in_the_history_gives_the_infinity_of_the_definition(vm, dtype, Hq, wide):
    """Values that every row sees, with weights that are powers of two and others."""
    rng = np.random.default_rng(44)
    a = _attention_inputs(rng, [300, 20], [8, 8], Hq, 2, 64, 16, dtype, wide=wide)
    clean, _, _ = _attend(vm, a, 8)
    for b, pos, dim, bad in ((0, 0, 0, float("inf")), (0, 130, 1, -float("inf")), (0, 250, 2, float("nan")), (0, 5, 3, float("inf")),
                             (0, 200, 3, float("inf")), (0, 7, 4, float("inf")), (0, 8, 4, -float("inf")), (1, 3, 5, -float("inf"))):
        a["v"][int(a["table"][b, pos // 16]), :, pos % 16, dim] = bad
    a["q"][9] = 0                                   # all weights of this row are 1
    got, _, _ = _attend(vm, a, 8)
    inf = float("inf")
    for b, dim, value in ((0, 0, inf), (0, 1, -inf), (0, 3, inf), (1, 5, -inf)):
        assert bool((got[8 * b:8 * b + 8, :, dim] == value).all()), (b, dim)
    assert bool(torch.isnan(got[:8, :, [2, 4]]).all())
    assert torch.equal(got[:8, :, 5:], clean[:8, :, 5:]) and torch.equal(got[10:, :, 6:], clean[10:, :, 6:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_reports_query_offsets_out_of_range(vm, dtype):
    """q_off beyond N, descending, negative, and so large that the tokens behind
    them pass 2^31: status bit 1, the other requests' rows as they should be."""
    rng = np.random.default_rng(40)
    lens, news, B, N = [70, 5, 130, 40], [2, 3, 1, 2], 4, 8
    a = _attention_inputs(rng, lens, news, 4, 2, 64, 16, dtype)
    off = a["q_off"].tolist()
    M = 2 ** 31 - 1
    for bad, good in (([0, 2, 5, 9, 11], [0, 1]), ([0, 2, M, -2 ** 31, -2 ** 31 + 1], [0]), ([0, 2, 5, M, -2 ** 31], [0, 1]),
                      ([-3, 2, 5, 6, 8], [1, 2, 3]), ([0, 2, 5, 4, 4], [0, 1]), ([M - 2, M, M, M, M], []), ([0, 2, 5, 6, M], [0, 1, 2]),
                      ([-2 ** 31, M, -2 ** 31, M, -2 ** 31], [])):
        big = torch.full((N + 40, 4, 64), 7.0, dtype=dtype, device="cuda")
        ws = vm.CacheWorkspace(B, 4, 2, 64, 3)
        lse = torch.full((N, 4), 7.0, device="cuda")
        vm.dspark_cache_attention(a["q"], a["k"], a["v"], a["table"], a["kv_len"], _cu(bad), a["tile_off"], big[20:20 + N], ws,
                                  max_new=3, lse=lse)
        assert _status(vm, ws) == BAD_LENGTH, bad
        assert bool((big[:20] == 7).all()) and bool((big[20 + N:] == 7).all())
        for b in good:
            assert bad[b:b + 2] == off[b:b + 2]
        if good:
            _rows_as_defined(a, big[20:20 + N], lse, good)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_reports_query_offsets_of_requests_without_positions(vm, dtype):
    """More tokens than max_new, or rows beyond N, of a request with an empty cache."""
    rng = np.random.default_rng(41)
    a = _attention_inputs(rng, [70, 0, 20], [2, 2, 2], 4, 2, 64, 16, dtype)
    out, lse, ws = _attend(vm, a, 2)
    assert _status(vm, ws) == 0
    _rows_as_defined(a, out, lse, [0, 1, 2])
    for lens, bad, good in (([70, 0, 20], [0, 2, 6, 6], [0]), ([70, 20, 0], [0, 2, 4, 2 ** 31 - 1], [0, 1]), ([0, 20, 70], [-1, 2, 4, 6], [1, 2]),
                            ([70, 20, 0], [0, 2, 4, 3], [0, 1])):
        a = _attention_inputs(rng, lens, [2, 2, 2], 4, 2, 64, 16, dtype)
        big = torch.full((46, 4, 64), 7.0, dtype=dtype, device="cuda")
        lse = torch.full((6, 4), 7.0, device="cuda")
        vm.dspark_cache_attention(a["q"], a["k"], a["v"], a["table"], a["kv_len"], _cu(bad), a["tile_off"], big[20:26], ws,
                                  max_new=2, lse=lse)
        assert _status(vm, ws) == BAD_LENGTH, bad
        assert bool((big[:20] == 7).all()) and bool((big[26:] == 7).all())
        _rows_as_defined(a, big[20:26], lse, good)


def test_attention_in_a_cuda_graph(vm):
    rng = np.random.default_rng(14)
    a = _attention_inputs(rng, [300, 20], [8, 2], 8, 2, 128, 16, torch.bfloat16)
    out, lse, ws = _attend(vm, a, 8)
    got = torch.empty_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        vm.dspark_cache_attention(a["q"], a["k"], a["v"], a["table"], a["kv_len"], a["q_off"], a["tile_off"], got, ws,
                                  max_new=8)
    for _ in range(3):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, out)


# ------------------------------------------------------------------ logits
def _logit_inputs(rng, B, R, V, dtype, L, masked=0.5, allowed=0.3):
    x = torch.as_tensor(rng.standard_normal((B, R, V)) * 3, dtype=torch.float32).to(dtype)
    hist = (V * rng.random((B, L)) ** 4).astype(np.int32)
    hist_len = rng.integers(0, L + 1, B).astype(np.int32)
    hist[np.arange(L)[None] >= hist_len[:, None]] = -12345      # beyond the length: never read
    draft = (V * rng.random((B, R)) ** 4).astype(np.int32)      # one more than is used
    mask = rng.random((B, R, V)) < allowed
    mask[rng.random(B) >= masked] = True
    mask[:, :, 3] = True
    bias = []
    for _ in range(B):
        ids = np.sort(rng.choice(V, size=rng.integers(0, min(V, 40)), replace=False))
        bias.append({int(i): float(np.float32(rng.standard_normal() * 4)) for i in ids})
    f = lambda lo, hi: rng.uniform(lo, hi, B).astype(np.float32)  # noqa: E731
    return dict(x=x, hist=hist, hist_len=hist_len, prompt_len=(hist_len // 2).astype(np.int32), draft=draft, mask=mask,
                bias=bias, rep=f(0.7, 1.5), freq=f(-0.5, 0.7), pres=f(-0.3, 0.8))


def _words(mask):
    B, R, V = mask.shape
    W = -(-V // 32)
    bits = np.zeros((B, R, W * 32), np.uint64)
    bits[:, :, :V] = mask
    w = (bits.reshape(B, R, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return torch.as_tensor(w.astype(np.uint32).view(np.int32)).cuda()


def _process(vm, a, ws=None, x=None, out=None, **drop):
    x = a["x"].cuda() if x is None else x
    B, R, V = x.shape
    ws = ws or vm.LogitsWorkspace(B, R)
    out = torch.empty((B, R, V), dtype=x.dtype, device="cuda") if out is None else out
    live = torch.full((B, R), -9, dtype=torch.int32, device="cuda")
    tok = [i for b in a["bias"] for i in b]
    val = [w for b in a["bias"] for w in b.values()]
    off = np.concatenate([[0], np.cumsum([len(b) for b in a["bias"]])])
    kw = dict(hist=_cu(a["hist"]), hist_len=_cu(a["hist_len"]), prompt_len=_cu(a["prompt_len"]), draft_tok=_cu(a["draft"]),
              rep=_cu(a["rep"], torch.float32), freq=_cu(a["freq"], torch.float32), pres=_cu(a["pres"], torch.float32),
              bias_tok=_cu(tok), bias_val=_cu(val, torch.float32), bias_off=_cu(off), mask=_words(a["mask"]), live=live)
    kw.update(drop)
    vm.dspark_logits_process(x, out, ws, **kw)
    torch.cuda.synchronize()
    return out, live, ws


def _check_logits(a, out, live, x=None, **drop):
    x = (a["x"] if x is None else x).double().numpy()
    B, R, V = x.shape
    z, none = np.zeros(B), [dict() for _ in range(B)]
    bf = out.dtype == torch.bfloat16
    want, tol = ref.logits(x, a["hist"], z.astype(int) if "hist" in drop else a["hist_len"], a["prompt_len"], a["draft"],
                           z + 1 if "rep" in drop else a["rep"].astype(float), z if "freq" in drop else a["freq"].astype(float),
                           z if "pres" in drop else a["pres"].astype(float), none if "bias_off" in drop else a["bias"],
                           None if "mask" in drop else a["mask"], ref.EPS16 if bf else 0.0)
    got = out.cpu().double().numpy()
    fin = np.isfinite(want)
    np.testing.assert_array_equal(np.isfinite(got), fin)
    np.testing.assert_array_equal(np.isneginf(got), np.isneginf(want))
    err = np.abs(got[fin] - want[fin])
    assert (err <= tol[fin]).all(), err.max()
    np.testing.assert_array_equal(live.cpu().numpy(), (want > -np.inf).sum(2))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,R,V,L", [(1, 1, 8, 1), (3, 8, 1024, 50), (2, 17, 4104, 300), (5, 7, 32008, 3000), (40, 2, 264, 17)])
def test_logits_match_the_definition(vm, B, R, V, L, dtype):
    rng = np.random.default_rng(B * R + V)
    a = _logit_inputs(rng, B, R, V, dtype, L)
    out, live, ws = _process(vm, a)
    _check_logits(a, out, live)
    assert _status(vm, ws) == 0
    again, live2, _ = _process(vm, a, ws=ws)                     # the counters are clear again
    assert torch.equal(out, again) and torch.equal(live, live2)


@pytest.mark.parametrize("drop", [("mask",), ("bias_off",), ("rep", "freq", "pres"), ("hist", "hist_len", "prompt_len"),
                                  ("freq", "pres", "mask", "bias_off")])
def test_logits_without_some_controls(vm, drop):
    rng = np.random.default_rng(len(drop))
    a = _logit_inputs(rng, 3, 8, 4104, torch.float32, 200)
    out, live, _ = _process(vm, a, **{k: None for k in drop})
    _check_logits(a, out, live, **{k: None for k in drop})


def test_logits_with_an_empty_history(vm):
    rng = np.random.default_rng(20)
    a = _logit_inputs(rng, 2, 3, 1024, torch.float32, 10)
    want, live, _ = _process(vm, a, hist=None, hist_len=None, prompt_len=None)
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    for hist in (torch.empty((2, 0), dtype=torch.int32, device="cuda"), _cu(a["hist"])):
        got, live2, _ = _process(vm, a, hist=hist, hist_len=z, prompt_len=z)
        assert torch.equal(got, want) and torch.equal(live, live2)


@pytest.mark.parametrize("B,V", [(1, 1024), (3, 8200)])
def test_logits_without_a_history_but_with_its_stride(vm, B, V):
    """The C call with hist = NULL beside the row widths a caller always passes: nothing is read there."""
    rng = np.random.default_rng(B)
    a = _logit_inputs(rng, B, 4, V, torch.float32, 10)
    want, live, _ = _process(vm, a, hist=None, hist_len=None, prompt_len=None, draft_tok=None, bias_off=None)
    x, words = a["x"].cuda(), _words(a["mask"])
    f = [_cu(a[k], torch.float32) for k in ("rep", "freq", "pres")]
    ws = vm.LogitsWorkspace(B, 4)
    out, got = torch.empty_like(x), torch.zeros_like(live)
    st = vm._lib.dspark_logits_process(x.data_ptr(), 0, V, out.data_ptr(), B, 4, V, None, 8192, None, None, None, 17,
                                       *[t.data_ptr() for t in f], None, None, None, 0, words.data_ptr(), float("-inf"),
                                       got.data_ptr(), ws.buf.data_ptr(), ws.buf.numel(), None)
    torch.cuda.synchronize()
    assert st == 0 and _status(vm, ws) == 0
    assert torch.equal(out, want) and torch.equal(got, live)


def test_logits_in_place_and_strided_rows(vm):
    rng = np.random.default_rng(21)
    a = _logit_inputs(rng, 4, 5, 1032, torch.bfloat16, 60)
    want, live, _ = _process(vm, a)
    x = a["x"].cuda()
    got, live2, _ = _process(vm, a, x=x, out=x)
    assert torch.equal(got, want) and torch.equal(live, live2)
    wide = torch.full((4, 5, 1032 + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :, :1032] = a["x"].cuda()
    got, live2, _ = _process(vm, a, x=wide[:, :, :1032])
    assert torch.equal(got, want) and torch.equal(live, live2)


def test_logits_with_infinities_nan_and_the_lowest_value(vm):
    """NaN or infinity under the mask disappear; -inf and the type's lowest
    value in allowed places stay what the formula makes of them."""
    rng = np.random.default_rng(22)
    for dtype in (torch.float32, torch.bfloat16):
        a = _logit_inputs(rng, 2, 4, 520, dtype, 40, masked=1.0)
        hidden = torch.as_tensor(~a["mask"])
        x = a["x"].clone()
        low = torch.finfo(dtype).min
        x[:, :, 10:60] = -float("inf")
        x[:, :, 60:110] = low
        x[hidden] = float("nan")
        x[:, 1][hidden[:, 1]] = float("inf")
        out, live, _ = _process(vm, a, x=x.cuda())
        y = out.float().cpu()
        assert torch.isneginf(y[hidden]).all()
        assert not torch.isnan(y).any() and not (y == float("inf")).any()
        seen = ~hidden
        assert torch.isneginf(y[:, :, 10:60]).all()
        np.testing.assert_array_equal(live.cpu().numpy(), (y > -float("inf")).sum(2).numpy())
        assert (y[:, :, 60:110][seen[:, :, 60:110]] < -1e38).all()


def test_logits_report_rows_with_nothing_left_and_bad_inputs(vm):
    rng = np.random.default_rng(23)
    a = _logit_inputs(rng, 3, 4, 1024, torch.float32, 50)
    a["mask"][1, 2] = False
    out, live, ws = _process(vm, a)
    _check_logits(a, out, live)
    assert int(live[1, 2]) == 0 and _status(vm, ws) == DEAD_ROW
    a["mask"][1, 2] = True
    ok, _, _ = _process(vm, a, ws=ws)
    assert _status(vm, ws) == 0
    hist = a["hist"].copy()
    hist_len = a["hist_len"].copy()
    hist_len[0] = 50
    hist[0, 7] = 1024
    _process(vm, dict(a, hist=np.where(hist < 0, 0, hist), hist_len=hist_len), ws=ws)
    assert _status(vm, ws) == BAD_TOKEN
    long = a["hist_len"].copy()
    long[2] = 51
    _process(vm, dict(a, hist=np.where(a["hist"] < 0, 0, a["hist"]), hist_len=long), ws=ws)
    assert _status(vm, ws) == BAD_LENGTH
    rep = a["rep"].copy()
    rep[0] = 0.0
    _process(vm, dict(a, rep=rep), ws=ws)
    assert _status(vm, ws) == BAD_INPUT
    tok = _cu([5, 5])
    _process(vm, a, ws=ws, bias_tok=tok, bias_val=tok.float(), bias_off=_cu([0, 2, 2, 2]))
    assert _status(vm, ws) == BAD_TOKEN
    _process(vm, a, ws=ws, bias_tok=tok, bias_val=tok.float(), bias_off=_cu([0, 9, 9, 9]))
    assert _status(vm, ws) == BAD_LENGTH


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_skip_invalid_biases_and_keep_the_valid_ones(vm, dtype):
    """Ids out of range, out of order or twice: an entry counts where its id is
    above every valid one before it, whatever stands beside it."""
    rng = np.random.default_rng(26)
    V = 4104
    rows = [[10, -1], [100, 3, 200], [5, 5], [2 ** 31 - 1, 7, 4103], [4104, 4103], [9, 9, 9, 11, -2 ** 31, 12, 11, 13],
            [100, 3, 50, 100, 4000], [0, 1, 2], [-1], [], [4103, 0, 4102], rng.integers(-50, V + 50, 300).tolist()]
    a = _logit_inputs(rng, len(rows), 3, V, dtype, 40)
    vals = [rng.standard_normal(len(r)).astype(np.float32) * 8 for r in rows]
    kept = []
    for r, w in zip(rows, vals):
        top, d = -1, {}
        for v, y in zip(r, w):
            if top < v < V:
                top, d[v] = v, float(y)
        kept.append(d)
    assert sum(map(len, kept)) < sum(map(len, rows))
    off = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
    out, live, ws = _process(vm, dict(a, bias=kept), bias_tok=_cu(sum(rows, [])), bias_val=_cu(np.concatenate(vals), torch.float32), bias_off=_cu(off))
    assert _status(vm, ws) == BAD_TOKEN
    _check_logits(dict(a, bias=kept), out, live)
    want, live2, _ = _process(vm, dict(a, bias=kept), ws=ws)
    assert _status(vm, ws) == 0 and torch.equal(out, want) and torch.equal(live, live2)


def test_logits_with_a_finite_fill(vm):
    """The rows of a draft take a finite value under the mask; the entries left
    and the rows with nothing left are counted as with -inf."""
    rng = np.random.default_rng(24)
    for dtype in (torch.float32, torch.bfloat16):
        a = _logit_inputs(rng, 3, 4, 1024, dtype, 50)
        a["mask"][2, 1] = False
        low, live, ws = _process(vm, a)
        assert _status(vm, ws) == DEAD_ROW
        got, live2, _ = _process(vm, a, ws=ws, fill=-1e4)
        assert _status(vm, ws) == DEAD_ROW
        assert torch.equal(live, live2)
        fill = torch.tensor(-1e4, dtype=dtype, device="cuda")
        assert torch.equal(got, torch.where(torch.as_tensor(a["mask"]).cuda(), low, fill))


# ------------------------------------------- the operators around the step
@pytest.mark.parametrize("B,V,r,wdt,mode", [(4, 1024, 32, torch.float32, 0), (5, 4104, 64, torch.bfloat16, 0),
                                            (1, 4104, 64, torch.bfloat16, 0), (70, 8200, 128, torch.bfloat16, 1)])
def test_a_constrained_step_matches_the_oracle(vm, B, V, r, wdt, mode):
    """A grammar that leaves 0.2 % of the vocabulary, on the draft's rows and the
    target's: the whole step draws what the oracle draws from the same rows, and
    every emitted token is allowed where it stands."""
    import oracle
    import workload

    w = workload.custom("tiny", B=B, V=V, r=r, w_dtype=wdt, seed=3, mode=mode)
    inp = workload.inputs(w, device="cuda")
    G = w.gamma
    rng = np.random.default_rng(7)
    allowed = rng.random((B, 1, V)) < 0.002          # the same law in every row of a request
    allowed[:, :, 7] = True
    words = _words(np.repeat(allowed, G + 1, 1))
    ws = vm.LogitsWorkspace(B, G + 1)
    vm.dspark_logits_process(inp["target"], inp["target"], ws, mask=words)
    vm.dspark_logits_process(inp["U"], inp["U"], vm.LogitsWorkspace(B, G), mask=words[:, :G].contiguous(), fill=-1e4)
    buf = vm.StepBuffers(B, G, V, r)
    vm.run_step(inp, buf, mode=mode, seed=5)
    assert vm.dspark_sync_status(buf.ws.buf) == (0, 0) and _status(vm, ws) == 0
    want = oracle.step({k: (v.cpu() if torch.is_tensor(v) else v) for k, v in inp.items()}, mode=mode, seed=5)
    np.testing.assert_array_equal(buf.draft_tok.cpu().numpy(), want["draft"]["tok"])
    n = int(buf.out_off[-1])
    tok, req = buf.out_tok[:n].cpu().numpy(), buf.out_req[:n].cpu().numpy()
    np.testing.assert_array_equal(tok, want["out"]["out_tok"])
    assert allowed[req, 0, tok].all()


# ------------------------------------------------------------ expired waits
def test_expired_waits_are_reported_and_the_workspace_recovers(vm):
    """With a wait bound of 300 cycles the attention and the logit controls give
    up, report a timeout and return; after dspark_workspace_init the same calls
    give the results of a fresh workspace.  Every wait on the path is bounded."""
    rng = np.random.default_rng(15)
    a = _attention_inputs(rng, [3000, 700], [8, 8], 32, 8, 128, 16, torch.bfloat16)
    out, lse, ws = _attend(vm, a, 8)
    vm.dspark_workspace_set_wait_limit(ws.buf, 300)
    _attend(vm, a, 8, ws=ws)
    st, bits = vm.dspark_sync_status(ws.buf)
    assert st == -3 and bits & 4
    vm.dspark_workspace_init(ws.buf)
    again, lse2, _ = _attend(vm, a, 8, ws=ws)
    assert _status(vm, ws) == 0 and torch.equal(again, out) and torch.equal(lse, lse2)
    # 17 rows: more than the ring holds, so the producer waits for the warps that
    # are still reading the history
    b = _logit_inputs(rng, 4, 17, 32008, torch.float32, 5000)
    want, live, lw = _process(vm, b)
    vm.dspark_workspace_set_wait_limit(lw.buf, 300)
    _process(vm, b, ws=lw)
    st, bits = vm.dspark_sync_status(lw.buf)
    assert st == -3 and bits & 4
    vm.dspark_workspace_init(lw.buf)
    got, live2, _ = _process(vm, b, ws=lw)
    assert _status(vm, lw) == 0 and torch.equal(got, want) and torch.equal(live, live2)


# ---------------------------------------------------------------- refusals
def test_the_binding_refuses_wrong_shapes_types_and_strides(vm):
    rng = np.random.default_rng(31)
    a = _attention_inputs(rng, [20], [2], 4, 2, 64, 16, torch.bfloat16)
    ws = vm.CacheWorkspace(1, 4, 2, 64, 2)
    out = torch.empty_like(a["q"])
    call = lambda **kw: vm.dspark_cache_attention(*[{**a, "out": out, **kw}[n] for n in (  # noqa: E731
        "q", "k", "v", "table", "kv_len", "q_off", "tile_off", "out")], kw.get("ws", ws), max_new=kw.get("max_new", 2),
        scale=kw.get("scale"))
    call()
    for kw, err in ((dict(q=a["q"].float()), ValueError), (dict(v=a["v"][:, :, ::2]), ValueError),
                    (dict(kv_len=a["kv_len"].long()), TypeError), (dict(tile_off=a["tile_off"][:1]), ValueError),
                    (dict(k=a["k"].transpose(1, 2), v=a["v"].transpose(1, 2)), ValueError),
                    (dict(max_new=18), vm.DsparkError), (dict(max_new=0), vm.DsparkError),
                    (dict(scale=0.0), vm.DsparkError), (dict(scale=float("nan")), vm.DsparkError),
                    (dict(k=a["k"][:, :, :, :60].contiguous(), v=a["v"][:, :, :, :60].contiguous()), ValueError)):
        with pytest.raises(err):
            call(**kw)
    with pytest.raises(vm.DsparkError):                       # a workspace for fewer rows
        big = _attention_inputs(rng, [20], [2], 64, 2, 64, 16, torch.bfloat16)
        vm.dspark_cache_attention(big["q"], big["k"], big["v"], big["table"], big["kv_len"], big["q_off"],
                                  big["tile_off"], torch.empty_like(big["q"]), ws, max_new=2)
    with pytest.raises(ValueError):
        vm.CacheWorkspace(1, 5, 2, 64, 2)
    x = torch.zeros((2, 3, 64), device="cuda")
    lw = vm.LogitsWorkspace(2, 3)
    for kw, err in ((dict(hist=_cu(np.zeros((2, 4)))), ValueError), (dict(draft_tok=_cu(np.zeros((2, 1)))), ValueError),
                    (dict(rep=torch.ones(2, dtype=torch.float64, device="cuda")), TypeError),
                    (dict(mask=_cu(np.zeros((2, 3, 3)))), ValueError)):
        with pytest.raises(err):
            vm.dspark_logits_process(x, torch.empty_like(x), lw, **kw)
    odd = torch.zeros((2, 3, 60), device="cuda")
    with pytest.raises(vm.DsparkError):
        vm.dspark_logits_process(odd, torch.empty_like(odd), lw)
    with pytest.raises(vm.DsparkError):
        many = torch.zeros((70, 3, 64), device="cuda")         # a workspace for fewer requests
        vm.dspark_logits_process(many, torch.empty_like(many), lw)
