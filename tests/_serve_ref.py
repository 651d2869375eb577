"""Plain 64-bit references of the serving operators (dspark_cache_plan,
dspark_cache_attention, dspark_logits_process), written from the definitions in
include/dspark.h with loops and numpy, and the error bounds the tests allow."""
import numpy as np
import torch

EPS32 = torch.finfo(torch.float32).eps / 2     # unit roundoff of binary32, 2^-24
EPS16 = torch.finfo(torch.bfloat16).eps / 2    # unit roundoff of bfloat16, 2^-8


def plan(seq_len, n_new, owned, ring, ring_state, table, page_size, T, tile=64):
    """One request after another, as a host-side allocator would."""
    pages, (head, free) = len(ring), ring_state
    table, ring, owned_out = table.copy(), ring.copy(), owned.copy()
    kv_len, q_off, tile_off = [], [0], [0]
    slot_map, positions = np.full(T, -1, np.int32), np.full(T, -1, np.int32)
    popped, asked, pushed, bad = 0, 0, 0, False
    for b, (n, new, own) in enumerate(zip(seq_len.tolist(), n_new.tolist(), owned.tolist())):
        ok = n >= 0 and new >= 0 and 0 <= own <= table.shape[1]
        new = max(0, new)
        goal = -(-(n + new) // page_size)
        ok = ok and goal <= table.shape[1]
        if ok:
            need = max(0, goal - own)
            asked += need
            ok = need == 0 or asked <= free
        if ok:
            for j in range(own, goal):
                table[b, j] = ring[(head + popped) % pages]
                popped += 1
            for j in range(goal, own):
                ring[(head + free + pushed) % pages] = table[b, j]
                pushed += 1
            owned_out[b] = goal
        bad |= not ok
        for i in range(new):
            t = q_off[-1] + i
            if t < T:
                positions[t] = n + i
                if ok:
                    slot_map[t] = table[b, (n + i) // page_size] * page_size + (n + i) % page_size
        kv_len.append(n + new if ok else 0)
        q_off.append(q_off[-1] + new)
        tile_off.append(tile_off[-1] + -(-kv_len[-1] // tile))
    i32 = np.int32
    return dict(block_table=table, ring=ring, owned_out=owned_out.astype(i32),
                ring_state_out=np.array([(head + popped) % pages, free - popped + pushed], i32),
                kv_len=np.array(kv_len, i32), q_off=np.array(q_off, i32), tile_off=np.array(tile_off, i32),
                slot_map=slot_map, positions=positions, bad=bad)


def attention(q, k_cache, v_cache, table, kv_len, q_off, scale, weight_eps, out_eps):
    """out, lse and the error allowed for each.  Arrays are float64; a cache
    position beyond kv_len is never read.

    A score computed in binary32 from D products is off by at most
    d = (D + 4) EPS32 scale sum |q_d k_d|; a weight then by 2 d + 2^-20
    relatively (exponential, running maximum, sum), plus weight_eps where it is
    rounded for the tensor cores; an output by that times sum p |v|, plus its
    own rounding."""
    N, Hq, D = q.shape
    Hkv, P = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    out, lse = np.zeros((N, Hq, D)), np.full((N, Hq), -np.inf)
    out_tol, lse_tol = np.zeros((N, Hq, D)), np.zeros((N, Hq))
    for b in range(len(kv_len)):
        n = q_off[b + 1] - q_off[b]
        for i in range(n):
            last = kv_len[b] - n + i
            if last < 0:
                continue
            pos = np.arange(last + 1)
            page, row = table[b, pos // P], pos % P
            for h in range(Hq):
                K, V = k_cache[page, h // G, row], v_cache[page, h // G, row]
                x = q[q_off[b] + i, h]
                s = (K * x).sum(1) * scale
                d = (D + 4) * EPS32 * scale * np.abs(K * x).sum(1).max()
                top = s.max()
                w = np.exp(s - top)
                p = w / w.sum()
                t = q_off[b] + i
                out[t, h] = p @ V
                lse[t, h] = top + np.log(w.sum())
                rel = 2 * d + 2.0 ** -20 + weight_eps
                out_tol[t, h] = 1.01 * (rel * (p @ np.abs(V)) + out_eps * np.abs(out[t, h])) + 1e-30
                lse_tol[t, h] = 2 * d + 2.0 ** -20 + 4 * EPS32 * abs(lse[t, h])
    return out, lse, out_tol, lse_tol


def logits(x, hist, hist_len, prompt_len, draft_tok, rep, freq, pres, bias, mask, out_eps):
    """The processed rows of x [B, R, V] (float64), the error allowed, and the
    entries left.  bias: a list of {token: value}; mask [B, R, V] bool or None.

    Each of the four additions and the scaling rounds once: 4 EPS32 of the sum
    of the terms' magnitudes, plus the rounding of the result."""
    B, R, V = x.shape
    out, tol = np.empty((B, R, V)), np.empty((B, R, V))
    for b in range(B):
        seen, count = np.zeros(V, bool), np.zeros(V)
        for i, v in enumerate(hist[b, :hist_len[b]]):
            seen[v] = True
            count[v] += i >= prompt_len[b]
        for i in range(R):
            if i:
                count[draft_tok[b, i - 1]] += 1
            y = x[b, i].copy()
            hit = seen | (count > 0)
            with np.errstate(invalid="ignore"):
                y[hit] = np.where(y[hit] > 0, y[hit] / rep[b], y[hit] * rep[b])
                size = np.abs(y) + np.abs(freq[b]) * count + np.abs(pres[b])
                y = y - freq[b] * count - pres[b] * (count > 0)
                for v, w in bias[b].items():
                    y[v] += w
                    size[v] += abs(w)
                if mask is not None:
                    y = np.where(mask[b, i], y, -np.inf)
                out[b, i] = y
                tol[b, i] = 4 * EPS32 * size + out_eps * np.abs(y)
    return out, tol
