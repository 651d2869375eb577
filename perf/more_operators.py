"""More operators of the decode loop, as they are measured.

Around the paged cache: rotary positions of a step's queries and keys, the cache
held in 4 bits (values quantised as they are written, and read back), and the
attention over it.  Behind the logit controls: a token of each row, drawn with
temperature, top-k, top-p and min-p from a given random number.  Each case is
one call as a decode loop makes it (the 4-bit cache is written and read back in
one).  `own` selects the library's kernels; otherwise `run` computes the same
from elementary torch operations.

A cache in 4 bits: 16 neighbouring entries of a head share a scale s (8 bits:
sign, 4 of exponent, 3 of mantissa), an entry is one of 0, 1/2, 1, 3/2, 2, 3, 4,
6 with a sign, and stands for entry * s * 2^e with one exponent e for the keys
and one for the values.

Shapes: 32 query heads over 8 key-value heads of 128 (and 64 over 8), blocks of
gamma + 1 = 8 tokens, vocabularies 151936 and 129280, batches of 1 to 512.
"""
import math

import torch

own = False

TILE = 64          # cache positions per attention tile (tile_off counts these)
GROUP = 16         # entries that share a scale
VOCABS = (151936, 129280)


def listed():
    att = dict(op="attention4", q_heads=32, kv_heads=8, head_dim=128, dtype="bf16")
    app = dict(op="append4", kv_heads=8, head_dim=128, dtype="bf16")
    rope = dict(op="rope", q_heads=32, kv_heads=8, head_dim=128, dtype="bf16")
    smp = dict(op="sample", dtype="fp32")
    return [
        # the smallest call: one request, one new token, a short context (latency)
        dict(att, name="attention4 b1 one token", B=1, page=16, new=1, ragged=False, lo=1000, hi=1000),
        # a batch verifying whole blocks: gamma + 1 tokens of every request, ragged contexts
        dict(att, name="attention4 b64 block", B=64, page=64, new=8, ragged=False, lo=1024, hi=8192),
        # one request with a long context and 8 query heads per key head: split over the length
        dict(att, name="attention4 b1 block 131k", q_heads=64, B=1, page=64, new=8, ragged=False, lo=131072, hi=131072),
        # plain decoding of a large batch, small pages, short to middling contexts
        dict(att, name="attention4 b256 one token", q_heads=64, B=256, page=16, new=1, ragged=False, lo=128, hi=4096),
        # a small fp32 model, odd lengths, a different number of tokens in each block
        dict(att, name="attention4 b4 fp32", q_heads=8, kv_heads=2, head_dim=64, dtype="fp32", B=4, page=16, new=8,
             ragged=True, lo=1, hi=301),
        # the keys and values of 64 blocks of 8 tokens
        dict(app, name="append4 b64 block", tokens=512, page=64),
        # a prompt chunk: 32768 tokens, cut from a fused projection's output
        dict(app, name="append4 32k", tokens=32768, page=64),
        # the queries and keys of 64 blocks, a context stretched eightfold by parts
        dict(rope, name="rope b64 block", tokens=512, rotary=128, interleaved=False, scaling="yarn", far=65536),
        # a prompt chunk far into a long context, neighbouring pairs in half of the head
        dict(rope, name="rope 32k half of the head", tokens=32768, rotary=64, interleaved=True, scaling="none", far=1048576),
        # one request without drafts: latency
        dict(smp, name="sample b1", rows=1, V=151936, mix=True),
        # 64 requests' rows of a block, each with its request's settings
        dict(smp, name="sample b64 block", rows=512, V=151936, mix=True),
        # a large batch, bf16 logits of the other vocabulary, nothing cut off
        dict(smp, name="sample b256 bf16 whole", rows=256, V=129280, dtype="bf16", mix=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention4", "attention4", "attention4", "append4", "rope", "sample", "sample"])
    if op == "attention4":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        group = rng.choice([1, 2, 4, 7, 8, 16])
        kv = rng.choice([1, 2, 4, 8])
        hi = _log(rng, 1, 65536)
        B = max(1, min(256, _log(rng, 1, 256), 400000 // (kv * max(hi, 64)) * 4))
        if dtype == "fp32":
            hi, B = min(hi, 8192), min(B, 16)
        return dict(op=op, q_heads=kv * group, kv_heads=kv, head_dim=rng.choice([64, 96, 128]), dtype=dtype, B=B,
                    page=rng.choice([8, 16, 32, 64, 128, 24]), new=rng.randint(1, 8), ragged=rng.random() < 0.5,
                    lo=max(1, int(hi * rng.choice([0.02, 0.3, 1.0]))), hi=hi)
    if op == "append4":
        return dict(op=op, tokens=_log(rng, 1, 32768), kv_heads=rng.choice([1, 2, 4, 8]),
                    head_dim=rng.choice([64, 96, 128]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    page=rng.choice([8, 16, 24, 32, 64, 128]))
    if op == "rope":
        kv, head = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128])
        return dict(op=op, tokens=_log(rng, 1, 16384), q_heads=kv * rng.choice([1, 4, 7]), kv_heads=kv, head_dim=head,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), rotary=rng.choice([head, head // 2, head - 16]),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "yarn", "wavelength"]),
                    far=_log(rng, 64, 1 << 22))
    return dict(op=op, rows=_log(rng, 1, 256), V=rng.choice([1000, 4097, 32003, *VOCABS]),
                dtype=rng.choice(["bf16", "fp32"]), mix=rng.random() < 0.7)


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


def _quantise(x, e):
    """Codes [.., D / 2] (even entries in the low half of a byte) and scales [.., D / 16] of x [.., D]."""
    y = x.float().view(*x.shape[:-1], -1, GROUP) * 2.0 ** -e
    s = (y.abs().amax(-1) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float()[..., None]
    # next to a border between two codes: the quotient in 64 bits
    r = torch.where(f > 0, y.double() / f.double().clamp(min=1e-9), 0.0)
    a = r.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8)
            + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) + (a > 5).to(torch.uint8))
    code += torch.signbit(y).to(torch.uint8) * 8
    code = code.view(*x.shape[:-1], -1, 2)
    return code[..., 0] + code[..., 1] * 16, s.view(torch.uint8)


def _values(codes, scales, e):
    """What codes and scales stand for, in fp32 (exactly)."""
    level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    level = torch.cat([level, -level])
    x = level[torch.stack([codes & 15, codes >> 4], -1).long()].view(*codes.shape[:-1], -1, GROUP)
    return (x * (scales.view(torch.float8_e4m3fn).float() * 2.0 ** e)[..., None]).view(*codes.shape[:-1], -1)


def _prepare_attention(case, g):
    B, P, dt = case["B"], case["page"], _type(case)
    H, D = case["kv_heads"], case["head_dim"]
    n_new = torch.full((B,), case["new"], dtype=torch.int32, device="cuda")
    if case["ragged"]:                                      # the admitted prefixes of a scheduled step
        n_new = 1 + (5 * torch.arange(B, device="cuda", dtype=torch.int32) + 2) % case["new"]
    kv_len = torch.maximum(_ints(g, case["lo"], case["hi"], B), n_new)
    owned = (kv_len + P - 1) // P
    pages = int(owned.sum()) + 7
    width = -(-max(case["hi"], case["new"]) // P) + 1
    held = torch.arange(width, device="cuda")[None] < owned[:, None]
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[held] = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[:pages - 7]
    q_off = _scan(n_new)
    q = torch.randn((int(q_off[-1]), case["q_heads"], D), generator=g, device="cuda") * 2
    s = dict(q=q.to(dt), table=table, kv_len=kv_len, q_off=q_off, tile_off=_scan((kv_len + TILE - 1) // TILE),
             scale=D ** -0.5, k_exp=-1, v_exp=-5, out=torch.empty_like(q, dtype=dt), lse=torch.empty(q.shape[:2], device="cuda"))
    # a few entries of every head's keys are larger than the others
    wide = 1 + 2 * (torch.rand((H, 1, D), generator=g, device="cuda") < 0.05)
    for name, e, size in (("k", -1, wide), ("v", -5, 0.2)):
        s[name] = torch.empty((pages, H, P, D // 2), dtype=torch.uint8, device="cuda")
        s[name + "s"] = torch.empty((pages, H, P, D // GROUP), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (H * P * D))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            x = (torch.randn((n, H, P, D), generator=g, device="cuda") * size).to(dt)
            s[name][p:p + n], s[name + "s"][p:p + n] = _quantise(x, e)
    return s


def _prepare_append(case, g):
    T, H, D, P, dt = case["tokens"], case["kv_heads"], case["head_dim"], case["page"], _type(case)
    pages = -(-T * 5 // (4 * P)) + 3
    # rows of a fused projection: the queries (four heads to a key head), the keys, the values
    qkv = torch.randn((T, 6 * H, D), generator=g, device="cuda").to(dt)
    runs = -(-T // P)                                       # runs of a page's slots, as a plan leaves them
    first = torch.randperm(pages, generator=g, device="cuda")[:runs] * P
    slots = (first[:, None] + torch.arange(P, device="cuda")[None]).reshape(-1)[:T].to(torch.int32).contiguous()
    slots[_ints(g, 0, 63, T) == 0] = -1                     # padding tokens
    u8 = dict(dtype=torch.uint8, device="cuda")
    return dict(key=qkv[:, 4 * H:5 * H], value=qkv[:, 5 * H:], slot_map=slots, k_exp=-1, v_exp=-2,
                k=torch.zeros((pages, H, P, D // 2), **u8), v=torch.zeros((pages, H, P, D // 2), **u8),
                ks=torch.zeros((pages, H, P, D // GROUP), **u8), vs=torch.zeros((pages, H, P, D // GROUP), **u8),
                k_out=torch.zeros((T, H, D), dtype=dt, device="cuda"), v_out=torch.zeros((T, H, D), dtype=dt, device="cuda"))


_BASE, _FACTOR, _TRAINED = 500000.0, 8.0, 8192    # of every rotary case


def _frequencies(rotary, scaling):
    """Radians per position of each pair (64 bits), and what the rotated part is multiplied by."""
    i = torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda")
    base = _BASE * _FACTOR ** (rotary / (rotary - 2)) if scaling == "ntk" else _BASE
    f = base ** (-i / rotary)
    if scaling == "linear":
        return f / _FACTOR, 1.0
    if scaling == "yarn":
        # pairs that turn more than 32 times within the trained length stay, less than once are stretched
        pair = [rotary * math.log(_TRAINED / (t * 2 * math.pi)) / (2 * math.log(_BASE)) for t in (32, 1)]
        low, high = max(0, math.floor(pair[0])), min(rotary - 1, math.ceil(pair[1]))
        ramp = ((i / 2 - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / _FACTOR * ramp, 0.1 * math.log(_FACTOR) + 1.0
    if scaling == "wavelength":
        # wavelengths above the trained length are stretched, below a quarter of it stay
        smooth = ((_TRAINED * f / (2 * math.pi) - 1) / 3).clamp(0, 1)
        return f * smooth + f / _FACTOR * (1 - smooth), 1.0
    return f, 1.0


def _prepare_rope(case, g):
    T, H, Hq, D, dt = case["tokens"], case["kv_heads"], case["q_heads"], case["head_dim"], _type(case)
    qkv = torch.randn((T, Hq + 2 * H, D), generator=g, device="cuda").to(dt)
    at = torch.arange(T, device="cuda", dtype=torch.int32) % 8 + _ints(g, 0, max(0, case["far"] - 8), -(-T // 8)).repeat_interleave(8)[:T]
    at[_ints(g, 0, 63, T) == 0] = -1                        # padding tokens
    f, m = _frequencies(case["rotary"], case["scaling"])
    return dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + H], positions=at.contiguous(), freq=f, mult=m,
                q_out=torch.zeros((T, Hq, D), dtype=dt, device="cuda"), k_out=torch.zeros((T, H, D), dtype=dt, device="cuda"))


def _prepare_sample(case, g):
    N, V, dt = case["rows"], case["V"], _type(case)
    pad = -(-V // 8) * 8
    logits = torch.randn((N, pad), generator=g, device="cuda") * 1.5
    # a model's row: some candidates stand out, their lead falls with the rank
    some = min(V, 400)
    ids = torch.randint(0, V, (N, some), generator=g, device="cuda")
    lead = 9 - (1.2 + 0.6 * torch.rand((N, 1), generator=g, device="cuda")) * torch.log(torch.arange(1, some + 1, device="cuda"))[None]
    logits.scatter_add_(1, ids, lead.expand(N, some).contiguous())
    logits[:, _ints(g, 0, V - 1, max(1, V // 50)).long()] = -math.inf      # a mask's entries
    f = lambda lo, hi: lo + (hi - lo) * torch.rand(N, generator=g, device="cuda")  # noqa: E731
    some = lambda p, x, off: torch.where(torch.rand(N, generator=g, device="cuda") < p, x, off)  # noqa: E731
    s = dict(logits=logits.to(dt)[:, :V], u=torch.rand(N, generator=g, device="cuda"), temperature=f(0.5, 1.2), top_k=None,
             top_p=None, min_p=None, tok=torch.empty(N, dtype=torch.int32, device="cuda"), logprob=torch.empty(N, device="cuda"))
    if case["mix"]:                                         # each request's own settings, some of them off
        s["temperature"] = some(0.1, torch.zeros(N, device="cuda"), s["temperature"])
        s["top_k"] = some(0.5, _ints(g, 1, 200, N), torch.zeros(N, dtype=torch.int32, device="cuda"))
        s["top_p"] = some(0.6, f(0.5, 0.99), torch.ones(N, device="cuda"))
        s["min_p"] = some(0.3, f(0.001, 0.1), torch.zeros(N, device="cuda"))
    return s


_PREPARE = dict(attention4=_prepare_attention, append4=_prepare_append, rope=_prepare_rope, sample=_prepare_sample)


def prepare(case, seed):
    s = _PREPARE[case["op"]](case, _gen(seed))
    s["op"] = case["op"]
    s["case"] = case
    return s


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import verify_markov_head_gb300 as vm

    op, case = s["op"], s["case"]
    if op == "attention4":
        if "ws" not in s:
            s["ws"] = vm.CacheWorkspace(case["B"], case["q_heads"], case["kv_heads"], case["head_dim"], case["new"])
        vm.dspark_cache_attention4(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["kv_len"], s["q_off"],
                                   s["tile_off"], s["out"], s["ws"], max_new=case["new"], k_exp=s["k_exp"],
                                   v_exp=s["v_exp"], scale=s["scale"], lse=s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    if op == "append4":
        vm.dspark_cache_append4(s["key"], s["value"], s["slot_map"], s["k"], s["v"], s["ks"], s["vs"], k_exp=s["k_exp"],
                                v_exp=s["v_exp"])
        vm.dspark_cache_read4(s["k"], s["v"], s["ks"], s["vs"], s["slot_map"], s["k_out"], s["v_out"], k_exp=s["k_exp"],
                              v_exp=s["v_exp"])
        return dict(k_out=s["k_out"], v_out=s["v_out"])
    if op == "rope":
        if "table" not in s:
            kind = case["scaling"]
            more = dict(linear={}, ntk={}, yarn=dict(trained=_TRAINED), wavelength=dict(trained=_TRAINED))
            scaling = None if kind == "none" else dict(kind=kind, factor=_FACTOR, **more[kind])
            s["table"] = vm.RopeTable(case["rotary"], base=_BASE, scaling=scaling)
        vm.dspark_rope(s["q"], s["k"], s["positions"], s["table"], s["q_out"], s["k_out"], interleaved=case["interleaved"])
        return dict(q_out=s["q_out"], k_out=s["k_out"])
    if "ws" not in s:
        s["ws"] = vm.SampleWorkspace(case["rows"])
    vm.dspark_sample(s["logits"], s["u"], s["tok"], s["ws"], temperature=s["temperature"], top_k=s["top_k"],
                     top_p=s["top_p"], min_p=s["min_p"], logprob=s["logprob"])
    return dict(tok=s["tok"], logprob=s["logprob"])


# ------------------------------------------------------------------ plain forms
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
    flat = lambda x: x[pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, x.shape[3])  # noqa: E731
    K = _values(flat(s["k"]), flat(s["ks"]), s["k_exp"])                     # [B, Hkv, W*P, D]
    S = torch.matmul(Q, K.transpose(2, 3)) * s["scale"]
    del K
    pos = torch.arange(S.shape[3], device=q.device)
    last = kv_len[:, None] - n[:, None] + i[None]                            # the position of token i
    seen = (pos[None, None] <= last[:, :, None]) & (pos[None, None] < kv_len[:, None, None])
    S.masked_fill_(~seen.repeat_interleave(G, 1)[:, None], -math.inf)
    top = S.amax(3, keepdim=True).clamp(min=-3e38)
    S.sub_(top).exp_()
    total = S.sum(3, keepdim=True)
    V = _values(flat(s["v"]), flat(s["vs"]), s["v_exp"])
    V.masked_fill_((pos[None] >= kv_len[:, None])[:, None, :, None], 0.0)
    O = torch.matmul(S, V) / total.clamp(min=1e-37)
    lse = (top + total.log()).view(B, Hkv, nq, G).permute(0, 2, 1, 3).reshape(B, nq, -1)
    O = O.view(B, Hkv, nq, G, D).permute(0, 2, 1, 3, 4).reshape(B, nq, Hkv * G, D)
    return dict(out=O[have].to(q.dtype), lse=lse[have])


def _plain_append(s):
    slots, P = s["slot_map"].long(), s["k"].shape[2]
    at = slots >= 0
    page, row = slots[at] // P, slots[at] % P
    s["k"][page, :, row], s["ks"][page, :, row] = _quantise(s["key"][at], s["k_exp"])
    s["v"][page, :, row], s["vs"][page, :, row] = _quantise(s["value"][at], s["v_exp"])
    s["k_out"][at] = _values(s["k"][page, :, row], s["ks"][page, :, row], s["k_exp"]).to(s["k_out"].dtype)
    s["v_out"][at] = _values(s["v"][page, :, row], s["vs"][page, :, row], s["v_exp"]).to(s["v_out"].dtype)
    return dict(k_out=s["k_out"], v_out=s["v_out"])


def _rotated(x, cos, sin, rotary, interleaved):
    y = x.clone()
    a, b = (x[..., :rotary:2], x[..., 1:rotary:2]) if interleaved else (x[..., :rotary // 2], x[..., rotary // 2:rotary])
    c, d = (y[..., :rotary:2], y[..., 1:rotary:2]) if interleaved else (y[..., :rotary // 2], y[..., rotary // 2:rotary])
    c.copy_(a * cos - b * sin)
    d.copy_(b * cos + a * sin)
    return y


def _plain_rope(s):
    at = s["positions"] >= 0
    angle = (s["positions"].double()[:, None] * s["freq"][None])[:, None]    # angles of far positions: 64 bits
    cos, sin = (angle.cos() * s["mult"]).float(), (angle.sin() * s["mult"]).float()
    rotary, inter = s["case"]["rotary"], s["case"]["interleaved"]
    s["q_out"].copy_(torch.where(at[:, None, None], _rotated(s["q"].float(), cos, sin, rotary, inter), s["q_out"].float()))
    s["k_out"].copy_(torch.where(at[:, None, None], _rotated(s["k"].float(), cos, sin, rotary, inter), s["k_out"].float()))
    return dict(q_out=s["q_out"], k_out=s["k_out"])


def _plain_sample(s):
    x = s["logits"].float()
    N, V = x.shape
    greedy = s["temperature"] <= 0
    T = torch.where(greedy, 1.0, s["temperature"]).double()[:, None]
    top, best = x.max(1)
    best = torch.where(x == top[:, None], torch.arange(V, device=x.device)[None], V).amin(1)      # the lowest index
    val, idx = torch.sort(x, dim=1, descending=True, stable=True)
    # sums over a vocabulary, next to borders: 64 bits
    w = torch.exp((val.double() - top.double()[:, None]) / T)
    if s["top_k"] is not None:
        rank = torch.arange(V, device=x.device)[None]
        w.masked_fill_((s["top_k"][:, None] > 0) & (rank >= s["top_k"][:, None]), 0.0)
    if s["top_p"] is not None:
        c = w.cumsum(1)
        out = (c - w >= s["top_p"].double()[:, None] * c[:, -1:]) & (s["top_p"][:, None] < 1)
        out[:, 0] = False
        w.masked_fill_(out, 0.0)
        del c, out
    if s["min_p"] is not None:
        p = s["min_p"].double()[:, None]
        w.masked_fill_((val.double() < top.double()[:, None] + T * p.clamp(min=1e-300).log()) & (p > 0), 0.0)
    w = torch.zeros_like(w).scatter_(1, idx, w)
    c = w.cumsum(1)
    tok = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(1).clamp(max=V - 1)
    logprob = (w.gather(1, tok[:, None])[:, 0] / c[:, -1]).log()
    return dict(tok=torch.where(greedy, best, tok).to(torch.int32), logprob=torch.where(greedy, 0.0, logprob).float())


_PLAIN = dict(attention4=_plain_attention, append4=_plain_append, rope=_plain_rope, sample=_plain_sample)


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "attention4":
        new = case["new"]
        if case["ragged"]:
            new = sum(1 + (5 * b + 2) % case["new"] for b in range(case["B"])) / case["B"]
        keys = case["B"] * max(new, (case["lo"] + case["hi"]) / 2)
        rows = case["B"] * new * case["q_heads"]
        D = case["head_dim"]
        return dict(bytes=keys * case["kv_heads"] * 2 * (D / 2 + D / GROUP) + keys / case["page"] * 4 + rows * (D * 2 * es + 4),
                    flops=4.0 * (keys / case["B"]) * rows * D)
    if case["op"] == "append4":
        n = case["tokens"] * case["kv_heads"] * case["head_dim"] * 2.0
        # the rows in, codes and scales out, the rows out again; the slots
        return dict(bytes=n * (es + 1 / 2 + 1 / GROUP + es) + case["tokens"] * 4, flops=n * 4)
    if case["op"] == "rope":
        heads = case["q_heads"] + case["kv_heads"]
        return dict(bytes=case["tokens"] * (heads * case["head_dim"] * 2.0 * es + 4), flops=case["tokens"] * heads * case["rotary"] * 3.0)
    n = case["rows"] * case["V"]
    return dict(bytes=n * es + case["rows"] * (6 if case["mix"] else 4) * 4.0, flops=n * 4.0)


# ------------------------------------------------------------------ the definitions in 64 bits
_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def exact(case, seed):
    s = prepare(case, seed)
    return dict(attention4=_exact_attention, append4=_exact_append, rope=_exact_rope, sample=_exact_sample)[case["op"]](s)


def _exact_cache(codes, scales, e):
    x = torch.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=torch.float64, device="cuda")
    level = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), dtype=torch.float64, device="cuda")
    x[..., 0::2], x[..., 1::2] = level[codes.int() % 16], level[codes.int() // 16]
    b = scales.int()
    expo, frac = (b // 8) % 16, (b % 8).double()
    size = torch.where(expo > 0, (1 + frac / 8) * torch.exp2(expo.double() - 7), frac / 8 * 2.0 ** -6)
    return x * size.repeat_interleave(GROUP, -1) * 2.0 ** e


def _exact_attention(s):
    case = s["case"]
    G, D = case["q_heads"] // case["kv_heads"], case["head_dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    lens, offs = s["kv_len"].tolist(), s["q_off"].tolist()
    if sum(lens) * case["q_heads"] * case["new"] * D * 4 > 2e12:
        return None
    for b, L in enumerate(lens):
        n = offs[b + 1] - offs[b]
        pages = s["table"][b, :-(-L // case["page"])].long()
        for h in range(case["kv_heads"]):
            K = _exact_cache(s["k"][pages, h], s["ks"][pages, h], s["k_exp"]).reshape(-1, D)[:L]
            V = _exact_cache(s["v"][pages, h], s["vs"][pages, h], s["v_exp"]).reshape(-1, D)[:L]
            q = s["q"][offs[b]:offs[b + 1], h * G:(h + 1) * G].double()
            z = torch.einsum("igd,td->igt", q, K) * s["scale"]
            hidden = torch.arange(L, device="cuda")[None] > (L - n + torch.arange(n, device="cuda"))[:, None]
            z = z.masked_fill(hidden[:, None], -math.inf)
            out[offs[b]:offs[b + 1], h * G:(h + 1) * G] = torch.einsum("igt,td->igd", torch.softmax(z, 2), V)
            lse[offs[b]:offs[b + 1], h * G:(h + 1) * G] = torch.logsumexp(z, 2)
    return dict(out=out, lse=lse)


def _exact_append(s):
    got = {}
    for name, x, e in (("k_out", s["key"], s["k_exp"]), ("v_out", s["value"], s["v_exp"])):
        y = x.double().reshape(-1, GROUP) * 2.0 ** -e
        # the scale: 8 steps to a power of two, down to 2^-6, ties to the even step
        want = y.abs().amax(1) / 6
        unit = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3)
        scale = (torch.round(want / unit) * unit).clamp(max=448)
        # the nearest level, a tie to the one of even number
        a = (y / torch.where(scale > 0, scale, math.inf)[:, None]).abs()
        level = torch.zeros_like(a)
        for i in range(7):
            border = (_LEVELS[i] + _LEVELS[i + 1]) / 2
            level = torch.where((a > border) | ((a == border) & (i % 2 == 1)), _LEVELS[i + 1], level)
        val = (torch.sign(y) * level * scale[:, None] * 2.0 ** e).view(x.shape)
        got[name] = torch.where((s["slot_map"] >= 0)[:, None, None], val, 0.0)
    return got


def _exact_rope(s):
    case, r = s["case"], s["case"]["rotary"]
    got = {}
    turn = torch.polar(torch.full_like(s["freq"], s["mult"])[None].expand(case["tokens"], -1),
                       s["positions"].double()[:, None] * s["freq"][None])[:, None]
    for name, x in (("q_out", s["q"]), ("k_out", s["k"])):
        y = x.double()
        p = y[..., :r].unflatten(-1, (r // 2, 2)) if case["interleaved"] else y[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(p.contiguous()) * turn)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        y = torch.cat([z.flatten(-2), y[..., r:]], -1)
        got[name] = torch.where((s["positions"] >= 0)[:, None, None], y, 0.0)
    return got


def _exact_sample(s):
    N, V = s["logits"].shape
    lp = torch.zeros(N, dtype=torch.float64, device="cuda")
    for i in range(N):
        x, T = s["logits"][i].double(), float(s["temperature"][i])
        if T <= 0:
            continue
        order = torch.argsort(-x, stable=True)
        p = torch.softmax(x[order] / T, 0)
        k = int(s["top_k"][i]) if s["top_k"] is not None else 0
        if k > 0:
            p[k:] = 0
            p = p / p.sum()
        if s["top_p"] is not None and float(s["top_p"][i]) < 1:
            before = p.cumsum(0) - p
            p[1:] = torch.where(before[1:] < float(s["top_p"][i]), p[1:], 0.0)
        if s["min_p"] is not None and float(s["min_p"][i]) > 0:
            p = torch.where(p >= float(s["min_p"][i]) * p[0] * (1 - 1e-14), p, 0.0)
        q = torch.zeros_like(p)
        q[order] = p / p.sum()
        t = int(torch.searchsorted(q.cumsum(0), torch.tensor(float(s["u"][i]), dtype=torch.float64, device="cuda"), right=True))
        lp[i] = q[min(t, V - 1)].log()
    return dict(tok=None, logprob=lp)
