"""The serving operators around the draft + verify step, as they are measured.

Four operators stand between one verification and the next: the plan of a paged
key-value cache (block tables, slot map and offsets from request lengths), the
append of new keys and values, the attention of a block's new tokens over the
cache, and the controls on logits (penalties, biases, grammar masks) before the
draws.  Each case is one call as a decode loop makes it.  `own` selects the
library's kernels; otherwise `run` computes the same from elementary torch
operations in 32 bits.

Shapes: 32 query heads over 8 key-value heads of 128 (and 64 over 8), blocks of
gamma + 1 = 8 tokens, vocabularies 151936 and 129280, batches of 1 to 512.
"""
import math

import torch

own = False

TILE = 64          # cache positions per attention tile (tile_off counts these)
VOCABS = (151936, 129280)


def listed():
    att = dict(op="attention", q_heads=32, kv_heads=8, head_dim=128, dtype="bf16")
    plan = dict(op="plan", chunk=2048)
    app = dict(op="append", kv_heads=8, head_dim=128, dtype="bf16")
    log = dict(op="logits", rows=8)
    return [
        # the smallest call: one request, one new token, a short context (latency)
        dict(att, name="attention b1 one token", B=1, page=16, new=1, ragged=False, lo=1000, hi=1000),
        # a batch verifying whole blocks: gamma + 1 tokens of every request, ragged contexts
        dict(att, name="attention b64 block", B=64, page=64, new=8, ragged=False, lo=1024, hi=8192),
        # one request with a long context and 8 query heads per key head: split over the length
        dict(att, name="attention b1 block 131k", q_heads=64, B=1, page=64, new=8, ragged=False, lo=131072, hi=131072),
        # plain decoding of a large batch, small pages, short to middling contexts
        dict(att, name="attention b256 one token", q_heads=64, B=256, page=16, new=1, ragged=False, lo=128, hi=4096),
        # a small fp32 model, odd lengths, a different number of tokens in each block
        dict(att, name="attention b4 fp32", q_heads=8, kv_heads=2, head_dim=64, dtype="fp32", B=4, page=16, new=8,
             ragged=True, lo=1, hi=301),
        # the plan of an ordinary step: 64 requests, a block each
        dict(plan, name="plan b64", B=64, page=64, lo=1024, hi=8192, prefill=0),
        # 512 requests in small pages, an eighth of them taking in a prompt chunk
        dict(plan, name="plan b512 prompts", B=512, page=16, lo=128, hi=32768, prefill=64),
        # the keys and values of 64 blocks of 8 tokens
        dict(app, name="append b64 block", tokens=512, page=64),
        # a prompt chunk: 32768 tokens, cut from a fused projection's output
        dict(app, name="append 32k", tokens=32768, page=64),
        # one request's block: latency, a long history
        dict(log, name="logits b1", B=1, V=151936, dtype="fp32", history=8192, bias=64, masked=0.0, allowed=1.0),
        # the 64-request step: an fp32 target, a quarter of the requests under a tight grammar
        dict(log, name="logits b64", B=64, V=151936, dtype="fp32", history=4096, bias=32, masked=0.25, allowed=0.01),
        # the 256-request step: a bf16 target, half of the requests under a loose grammar
        dict(log, name="logits b256 bf16", B=256, V=129280, dtype="bf16", history=2048, bias=16, masked=0.5,
             allowed=0.9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "plan", "append", "logits", "logits"])
    if op == "attention":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        group = rng.choice([1, 2, 4, 7, 8, 16])
        kv = rng.choice([1, 2, 4, 8])
        hi = _log(rng, 1, 65536)
        B = max(1, min(256, _log(rng, 1, 256), 400000 // (kv * max(hi, 64)) * 4))
        if dtype == "fp32":
            hi, B = min(hi, 8192), min(B, 16)
        return dict(op=op, q_heads=kv * group, kv_heads=kv, head_dim=rng.choice([64, 128]), dtype=dtype, B=B,
                    page=rng.choice([8, 16, 32, 64, 128, 24]), new=rng.randint(1, 8), ragged=rng.random() < 0.5,
                    lo=max(1, int(hi * rng.choice([0.02, 0.3, 1.0]))), hi=hi)
    if op == "plan":
        B = _log(rng, 1, 512)
        hi = _log(rng, 16, 32768)
        return dict(op=op, B=B, page=rng.choice([8, 16, 24, 32, 64, 128]), chunk=_log(rng, 16, 2048),
                    prefill=rng.randint(0, B // 8), lo=max(1, hi // rng.choice([1, 8, 64])), hi=hi)
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 32768), kv_heads=rng.choice([1, 2, 4, 8]),
                    head_dim=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    page=rng.choice([8, 16, 24, 32, 64, 128]))
    B = _log(rng, 1, 128)
    return dict(op=op, B=B, rows=rng.randint(1, 8), V=rng.choice([1024, 4104, 32008, *VOCABS]),
                dtype=rng.choice(["bf16", "fp32"]), history=_log(rng, 1, 16384), bias=_log(rng, 1, 300),
                masked=rng.choice([0.0, 0.3, 1.0]), allowed=rng.choice([0.001, 0.1, 0.99]))


# ------------------------------------------------------------------ inputs
def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _scan(x):
    """[n] -> [n+1]: the exclusive sums and the total."""
    return torch.nn.functional.pad(torch.cumsum(x, 0), (1, 0)).to(torch.int32)


def _tables(owned, width, pages, g):
    """Block tables whose rows hold owned[b] distinct pages; the other pages in a ring that starts anywhere."""
    B = owned.numel()
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    used = int(owned.sum())
    held = torch.arange(width, device="cuda")[None] < owned[:, None]
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[held] = perm[:used]
    head = int(torch.randint(0, pages, (1,), generator=g, device="cuda"))
    ring = torch.roll(torch.cat([perm[used:], perm[:used]]), head).contiguous()
    return table, ring, torch.tensor([head, pages - used], dtype=torch.int32, device="cuda")


def _prepare_attention(case, g):
    B, P, dt = case["B"], case["page"], _type(case)
    n_new = torch.full((B,), case["new"], dtype=torch.int32, device="cuda")
    if case["ragged"]:                                      # the admitted prefixes of a scheduled step
        n_new = 1 + (5 * torch.arange(B, device="cuda", dtype=torch.int32) + 2) % case["new"]
    kv_len = torch.maximum(_ints(g, case["lo"], case["hi"], B), n_new)
    owned = (kv_len + P - 1) // P
    pages = int(owned.sum()) + 7
    width = -(-max(case["hi"], case["new"]) // P) + 1
    table, _, _ = _tables(owned, width, pages, g)
    shape = (pages, case["kv_heads"], P, case["head_dim"])
    q_off = _scan(n_new)
    N = int(q_off[-1])
    q = torch.randn((N, case["q_heads"], case["head_dim"]), generator=g, device="cuda") * 2
    return dict(q=q.to(dt), k=torch.randn(shape, generator=g, device="cuda").to(dt),
                v=torch.randn(shape, generator=g, device="cuda").to(dt), table=table, kv_len=kv_len, q_off=q_off,
                tile_off=_scan((kv_len + TILE - 1) // TILE), scale=case["head_dim"] ** -0.5,
                out=torch.empty_like(q, dtype=dt), lse=torch.empty(q.shape[:2], device="cuda"))


def _prepare_plan(case, g):
    B, P = case["B"], case["page"]
    seq = _ints(g, case["lo"], case["hi"], B)
    n_new = _ints(g, 1, 8, B)                               # the admitted drafts and the token before them
    order = torch.randperm(B, generator=g, device="cuda")
    n_new[order[:case["prefill"]]] = case["chunk"]
    owned = (seq + P - 1) // P
    owned += (_ints(g, 0, 3, B) == 0).to(torch.int32)       # a page kept from rejected drafts
    gone = order[B - B // 32:]                              # requests that have ended give their pages back
    seq[gone] = 0
    n_new[gone] = 0
    width = -(-(case["hi"] + max(8, case["chunk"])) // P) + 1
    pages = B * (-(-case["hi"] // P) + 3) + case["prefill"] * (-(-case["chunk"] // P) + 1)
    table, ring, ring_state = _tables(owned, width, pages, g)
    T = 8 * B + case["prefill"] * case["chunk"]
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(seq_len=seq, n_new=n_new, owned=owned.contiguous(), ring=ring, ring_state=ring_state, table=table, page=P,
                owned_out=torch.empty(B, **i32), ring_state_out=torch.empty(2, **i32), kv_len=torch.empty(B, **i32),
                q_off=torch.empty(B + 1, **i32), tile_off=torch.empty(B + 1, **i32),
                slot_map=torch.empty(T, **i32), positions=torch.empty(T, **i32))


def _prepare_append(case, g):
    T, H, D, P, dt = case["tokens"], case["kv_heads"], case["head_dim"], case["page"], _type(case)
    pages = -(-T * 5 // (4 * P)) + 3
    # rows of a fused projection: the queries (four heads to a key head), the keys, the values
    qkv = torch.randn((T, 6 * H, D), generator=g, device="cuda").to(dt)
    runs = -(-T // P)                                       # runs of a page's slots, as a plan leaves them
    first = torch.randperm(pages, generator=g, device="cuda")[:runs] * P
    slots = (first[:, None] + torch.arange(P, device="cuda")[None]).reshape(-1)[:T].to(torch.int32).contiguous()
    slots[_ints(g, 0, 63, T) == 0] = -1                     # padding tokens
    return dict(key=qkv[:, 4 * H:5 * H], value=qkv[:, 5 * H:], slot_map=slots,
                k=torch.zeros((pages, H, P, D), dtype=dt, device="cuda"),
                v=torch.zeros((pages, H, P, D), dtype=dt, device="cuda"))


def _prepare_logits(case, g):
    B, R, V, L, dt = case["B"], case["rows"], case["V"], case["history"], _type(case)
    W = -(-V // 32)
    logits = torch.randn((B, R, V), generator=g, device="cuda").mul_(2).to(dt)
    hist_len = _ints(g, max(1, L // 2), L, B)
    # text repeats itself: tokens from a skewed law over the vocabulary
    u = torch.rand((B, L), generator=g, device="cuda")
    hist = (V * u ** 3).to(torch.int32).clamp_(0, V - 1)
    draft = (V * torch.rand((B, max(1, R - 1)), generator=g, device="cuda") ** 3).to(torch.int32).clamp_(0, V - 1)
    n_bias = _ints(g, 0, case["bias"], B)
    ids = (torch.arange(case["bias"], device="cuda")[None] * (V // case["bias"])
           + _ints(g, 0, V // case["bias"] - 1, B * case["bias"]).view(B, -1))
    kept = torch.arange(ids.shape[1], device="cuda")[None] < n_bias[:, None]
    ids = torch.sort(torch.where(kept, ids, V), 1).values   # ascending in each request
    tok = ids[ids < V].to(torch.int32).contiguous()
    mask = None
    if case["masked"] > 0:
        constrained = torch.rand(B, generator=g, device="cuda") < case["masked"]
        constrained[0] = True
        bits = torch.rand((B, R, W * 32), generator=g, device="cuda") < case["allowed"]
        bits |= ~constrained[:, None, None]
        bits[:, :, 5 % V] = True                            # the grammar always leaves a token
        weights = torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
        mask = torch.empty((B, R, W), dtype=torch.int32, device="cuda")
        for b in range(B):
            word = (bits[b].view(R, W, 32).to(torch.int64) * weights).sum(-1)
            mask[b] = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)
    f = lambda lo, hi: lo + (hi - lo) * torch.rand(B, generator=g, device="cuda")  # noqa: E731
    return dict(logits=logits, hist=hist, hist_len=hist_len, prompt_len=(hist_len * 0.6).to(torch.int32), draft_tok=draft if R > 1 else None,
                rep=f(1.0, 1.3), freq=f(-0.2, 0.6), pres=f(0.0, 0.5), bias_tok=tok,
                bias_val=torch.randn(tok.numel(), generator=g, device="cuda") * 3, bias_off=_scan(n_bias), mask=mask,
                out=torch.empty_like(logits), live=torch.empty((B, R), dtype=torch.int32, device="cuda"))


_PREPARE = dict(attention=_prepare_attention, plan=_prepare_plan, append=_prepare_append, logits=_prepare_logits)


def prepare(case, seed):
    s = _PREPARE[case["op"]](case, _gen(seed))
    s["op"] = case["op"]
    s["case"] = case
    return s


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import verify_markov_head_gb300 as vm

    op, case = s["op"], s["case"]
    if op == "attention":
        if "ws" not in s:
            s["ws"] = vm.CacheWorkspace(case["B"], case["q_heads"], case["kv_heads"], case["head_dim"], case["new"])
        vm.dspark_cache_attention(s["q"], s["k"], s["v"], s["table"], s["kv_len"], s["q_off"], s["tile_off"], s["out"],
                                  s["ws"], max_new=case["new"], scale=s["scale"], lse=s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    if op == "plan":
        vm.dspark_cache_plan(s["seq_len"], s["n_new"], s["owned"], s["ring"], s["ring_state"], s["table"], s["page"],
                             owned_out=s["owned_out"], ring_state_out=s["ring_state_out"], kv_len=s["kv_len"],
                             q_off=s["q_off"], tile_off=s["tile_off"], slot_map=s["slot_map"],
                             positions=s["positions"])
        return {k: s[k] for k in _PLAN_OUT}
    if op == "append":
        vm.dspark_cache_append(s["key"], s["value"], s["slot_map"], s["k"], s["v"])
        return dict(k=s["k"], v=s["v"])
    if "ws" not in s:
        s["ws"] = vm.LogitsWorkspace(case["B"], case["rows"])
    vm.dspark_logits_process(s["logits"], s["out"], s["ws"], hist=s["hist"], hist_len=s["hist_len"],
                             prompt_len=s["prompt_len"], draft_tok=s["draft_tok"], rep=s["rep"], freq=s["freq"],
                             pres=s["pres"], bias_tok=s["bias_tok"], bias_val=s["bias_val"], bias_off=s["bias_off"],
                             mask=s["mask"], live=s["live"])
    return dict(out=s["out"], live=s["live"])


# ------------------------------------------------------------------ plain forms
_PLAN_OUT = ("table", "ring", "owned_out", "ring_state_out", "kv_len", "q_off", "tile_off", "slot_map", "positions")


def _plain_attention(s):
    q, table, kv_len, q_off = s["q"], s["table"], s["kv_len"].long(), s["q_off"].long()
    B, Hkv, D = table.shape[0], s["k"].shape[1], q.shape[2]
    G, nq = q.shape[1] // Hkv, s["case"]["new"]
    n = q_off[1:] - q_off[:-1]
    i = torch.arange(nq, device=q.device)
    have = i[None] < n[:, None]                                             # [B, nq]
    row = torch.where(have, q_off[:-1, None] + i[None], 0)
    Q = q.float()[row].view(B, nq, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, nq * G, D)
    pages = table.clamp(min=0).long()
    K = s["k"][pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D).float()  # [B, Hkv, W*P, D]
    S = torch.matmul(Q, K.transpose(2, 3)) * s["scale"]
    del K
    pos = torch.arange(S.shape[3], device=q.device)
    last = kv_len[:, None] - n[:, None] + i[None]                            # the position of token i
    seen = (pos[None, None] <= last[:, :, None]) & (pos[None, None] < kv_len[:, None, None])
    S.masked_fill_(~seen.repeat_interleave(G, 1)[:, None], -math.inf)
    top = S.amax(3, keepdim=True).clamp(min=-3e38)
    S.sub_(top).exp_()
    total = S.sum(3, keepdim=True)
    V = s["v"][pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    V = torch.where((pos[None] < kv_len[:, None])[:, None, :, None], V, 0).float()
    O = torch.matmul(S, V) / total.clamp(min=1e-37)
    lse = (top + total.log()).view(B, Hkv, nq, G).permute(0, 2, 1, 3).reshape(B, nq, -1)
    O = O.view(B, Hkv, nq, G, D).permute(0, 2, 1, 3, 4).reshape(B, nq, Hkv * G, D)
    return dict(out=O[have].to(q.dtype), lse=lse[have])


def _plain_plan(s):
    P, table, ring = s["page"], s["table"], s["ring"].long()
    seq, new, owned = s["seq_len"].long(), s["n_new"].long(), s["owned"].long()
    n, width = ring.numel(), table.shape[1]
    head, free = s["ring_state"].long()[0], s["ring_state"].long()[1]
    want = seq + new
    goal = (want + P - 1) // P
    over = goal > width
    need = torch.where(over, 0, (goal - owned).clamp(min=0))
    off = torch.cumsum(need, 0) - need
    ok = ~over & ((need == 0) | (off + need <= free))
    give = torch.where(ok, (owned - goal).clamp(min=0), 0)
    back = torch.cumsum(give, 0) - give
    popped = torch.where(ok, need, 0).sum()
    j = torch.arange(width, device=table.device)[None]
    taken = ok[:, None] & (j >= owned[:, None]) & (j < goal[:, None])
    table[taken] = ring[(head + off[:, None] + j - owned[:, None])[taken] % n].to(torch.int32)
    freed = ok[:, None] & (j >= goal[:, None]) & (j < owned[:, None])
    s["ring"][(head + free + back[:, None] + j - goal[:, None])[freed] % n] = table[freed]
    kv_len = torch.where(ok, want, 0)
    q_off = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    tile_off = torch.nn.functional.pad(torch.cumsum((kv_len + TILE - 1) // TILE, 0), (1, 0))
    t = torch.arange(s["slot_map"].numel(), device=table.device)
    b = (torch.searchsorted(q_off, t, right=True) - 1).clamp(max=seq.numel() - 1)
    pos = seq[b] + t - q_off[b]
    inside = (t < q_off[-1]) & ok[b]
    page = table[b, torch.where(inside, pos // P, 0)].long()
    slot = torch.where(inside, page * P + pos % P, -1)
    return dict(table=table, ring=s["ring"], owned_out=torch.where(ok, goal, owned).to(torch.int32),
                ring_state_out=torch.stack([(head + popped) % n, free - popped + give.sum()]).to(torch.int32),
                kv_len=kv_len.to(torch.int32), q_off=q_off.to(torch.int32), tile_off=tile_off.to(torch.int32),
                slot_map=slot.to(torch.int32), positions=torch.where(t < q_off[-1], pos, -1).to(torch.int32))


def _plain_append(s):
    slots, P = s["slot_map"].long(), s["k"].shape[2]
    at = slots >= 0
    page, row = slots[at] // P, slots[at] % P
    s["k"][page, :, row] = s["key"][at]
    s["v"][page, :, row] = s["value"][at]
    return dict(k=s["k"], v=s["v"])


def _plain_logits(s):
    x, hist = s["logits"], s["hist"].long()
    B, R, V = x.shape
    i = torch.arange(hist.shape[1], device=x.device)[None]
    known = i < s["hist_len"][:, None]
    output = known & (i >= s["prompt_len"][:, None])
    count = torch.zeros((B, V), device=x.device).scatter_add_(1, hist, output.float())
    prompt = torch.zeros((B, V), device=x.device).scatter_add_(1, hist, (known & ~output).float())
    step = torch.zeros((B, R, V), device=x.device)
    step[:, 0] = count
    if s["draft_tok"] is not None:
        step[:, 1:].scatter_(2, s["draft_tok"][:, :R - 1, None].long(), 1.0)
    count = step.cumsum_(1)
    out = x.float()
    rep = s["rep"][:, None, None]
    out = torch.where((count > 0) | (prompt > 0)[:, None], torch.where(out > 0, out / rep, out * rep), out)
    out = out - s["freq"][:, None, None] * count - s["pres"][:, None, None] * (count > 0)
    bias = torch.zeros((B, V), device=x.device)
    owner = torch.searchsorted(s["bias_off"][1:].long(), torch.arange(s["bias_tok"].numel(), device=x.device), right=True)
    bias[owner, s["bias_tok"].long()] = s["bias_val"]
    out += bias[:, None]
    if s["mask"] is not None:
        v = torch.arange(V, device=x.device)
        out.masked_fill_(((s["mask"][:, :, v // 32] >> (v % 32)) & 1) == 0, -math.inf)
    out = out.to(x.dtype)
    return dict(out=out, live=(out > -math.inf).sum(2).to(torch.int32))


_PLAIN = dict(attention=_plain_attention, plan=_plain_plan, append=_plain_append, logits=_plain_logits)


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    es = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "attention":
        new = case["new"]
        if case["ragged"]:
            new = sum(1 + (5 * b + 2) % case["new"] for b in range(case["B"])) / case["B"]
        keys = case["B"] * max(new, (case["lo"] + case["hi"]) / 2)
        rows = case["B"] * new * case["q_heads"]
        D = case["head_dim"]
        return dict(bytes=keys * case["kv_heads"] * D * 2 * es + keys / case["page"] * 4 + rows * (D * 2 * es + 4),
                    flops=4.0 * (keys / case["B"]) * rows * D)
    if case["op"] == "plan":
        B, P = case["B"], case["page"]
        T = 8 * B + case["prefill"] * case["chunk"]
        fresh = 4.5 * B + case["prefill"] * case["chunk"]
        # lengths in and out, the slot map and positions, the pages that change hands (read, and written)
        return dict(bytes=4.0 * (3 * B + 4 * B + 2 * T + 2 * fresh / P), flops=0.0)
    if case["op"] == "append":
        return dict(bytes=case["tokens"] * (case["kv_heads"] * case["head_dim"] * 2 * 2.0 * es + 4), flops=0.0)
    B, R, V = case["B"], case["rows"], case["V"]
    n, m = B * R * V, case["masked"]
    read = (1 - m) + m * case["allowed"]                    # a masked entry need not be read
    return dict(bytes=n * es * (1 + read) + (n / 8 if m else 0) + B * (case["history"] * 0.75 + case["bias"]) * 4,
                flops=float(n * 4))


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return dict(attention=_exact_attention, plan=lambda s: None, append=_exact_append, logits=_exact_logits)[case["op"]](s)


def _exact_attention(s):
    case = s["case"]
    P, G = case["page"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    lens, offs = s["kv_len"].tolist(), s["q_off"].tolist()
    if sum(lens) * case["q_heads"] * case["new"] * case["head_dim"] * 4 > 2e12:
        return None
    for b, L in enumerate(lens):
        n = offs[b + 1] - offs[b]
        pages = s["table"][b, :-(-L // P)].long()
        for h in range(case["kv_heads"]):
            K = s["k"][pages, h].reshape(-1, case["head_dim"])[:L].double()
            V = s["v"][pages, h].reshape(-1, case["head_dim"])[:L].double()
            q = s["q"][offs[b]:offs[b + 1], h * G:(h + 1) * G].double()
            z = torch.einsum("igd,td->igt", q, K) * s["scale"]
            hidden = torch.arange(L, device="cuda")[None] > (L - n + torch.arange(n, device="cuda"))[:, None]
            z = z.masked_fill(hidden[:, None], -math.inf)
            out[offs[b]:offs[b + 1], h * G:(h + 1) * G] = torch.einsum("igt,td->igd", torch.softmax(z, 2), V)
            lse[offs[b]:offs[b + 1], h * G:(h + 1) * G] = torch.logsumexp(z, 2)
    return dict(out=out, lse=lse)


def _exact_append(s):
    H, P = s["k"].shape[1], s["k"].shape[2]
    got = {}
    for name, new in (("k", s["key"]), ("v", s["value"])):
        flat = s[name].double().transpose(1, 2).reshape(-1, H, new.shape[2])   # one row for each slot
        kept = s["slot_map"] >= 0
        flat.index_copy_(0, s["slot_map"][kept].long(), new[kept].double())
        got[name] = flat.view(-1, P, H, new.shape[2]).transpose(1, 2)
    return got


def _exact_logits(s):
    x = s["logits"]
    B, R, V = x.shape
    out = torch.empty((B, R, V), dtype=torch.float64, device="cuda")
    lens, prompts, offs = s["hist_len"].tolist(), s["prompt_len"].tolist(), s["bias_off"].tolist()
    for b in range(B):
        prompt = torch.bincount(s["hist"][b, :prompts[b]].long(), minlength=V)
        count = torch.bincount(s["hist"][b, prompts[b]:lens[b]].long(), minlength=V)
        bias = torch.zeros(V, dtype=torch.float64, device="cuda")
        bias[s["bias_tok"][offs[b]:offs[b + 1]].long()] = s["bias_val"][offs[b]:offs[b + 1]].double()
        rep, freq, pres = (float(s[k][b]) for k in ("rep", "freq", "pres"))
        for i in range(R):
            if i:
                count[int(s["draft_tok"][b, i - 1])] += 1
            z = x[b, i].double()
            z = torch.where((prompt + count) > 0, torch.where(z > 0, z / rep, z * rep), z)
            z = z - freq * count - pres * (count > 0) + bias
            if s["mask"] is not None:
                words = s["mask"][b, i].long() & 0xFFFFFFFF
                bits = (words[:, None] >> torch.arange(32, device="cuda")) & 1
                z = torch.where(bits.view(-1)[:V] > 0, z, -math.inf)
            out[b, i] = z
    return dict(out=out, live=None)
