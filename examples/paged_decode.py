"""Speculative decoding with a paged cache and constrained logits, end to end.

A toy target model (one attention layer over the paged key-value cache, random
weights) decodes a batch of requests with Markov-head drafts.  Each step, all
on the device and without a host synchronisation:

  dspark_logits_process   the draft's base logits under each request's grammar
  dspark_draft_markov     gamma drafts per request
  dspark_cache_plan       pages, slots and offsets for the block's tokens
  dspark_cache_append     their keys and values
  dspark_cache_attention  their attention over everything before them
  dspark_logits_process   penalties, biases and the grammar on the target rows,
                          row i counting the drafts before it
  dspark_verify           accepted drafts and the next token
  (torch indexing)        histories and lengths advance by accepted + 1

    python examples/paged_decode.py [--requests 8] [--steps 16]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import verify_markov_head_gb300 as vm  # noqa: E402


class ToyTarget:
    """Embedding, one attention layer with a residual, output projection."""

    def __init__(self, V, q_heads, kv_heads, head_dim, max_len, seed=0, dtype=torch.bfloat16, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        d = q_heads * head_dim
        rand = lambda *s, std=1.0: (torch.randn(s, generator=g, device=device) * std).to(dtype)  # noqa: E731
        self.V, self.q_heads, self.kv_heads, self.head_dim = V, q_heads, kv_heads, head_dim
        self.emb, self.pos = rand(V, d), rand(max_len, d, std=0.5)
        self.qkv = rand(d, (q_heads + 2 * kv_heads) * head_dim, std=d ** -0.5)
        self.proj, self.head = rand(d, d, std=d ** -0.5), rand(d, V, std=4 * d ** -0.5)

    def inputs(self, tokens, positions):
        return self.emb[tokens] + self.pos[positions]

    def split(self, x):
        """q [N, q_heads, D], k and v [N, kv_heads, D]: slices of one projection."""
        h = (x @ self.qkv).view(x.shape[0], -1, self.head_dim)
        return h[:, :self.q_heads], h[:, self.q_heads:self.q_heads + self.kv_heads], h[:, self.q_heads + self.kv_heads:]

    def logits(self, x, attended):
        return (x + attended.reshape(x.shape) @ self.proj) @ self.head


class Decoder:
    """The state of B requests: cache pages, histories, grammars, penalties."""

    def __init__(self, model: ToyTarget, B, gamma=7, r=64, page_size=16, max_len=512, pages=None, seed=0, device="cuda"):
        m, D = model, model.head_dim
        i32 = dict(dtype=torch.int32, device=device)
        g = torch.Generator(device=device).manual_seed(seed + 1)
        self.m, self.B, self.gamma, self.P = m, B, gamma, page_size
        width = -(-max_len // page_size)
        pages = pages or B * width
        self.k = torch.zeros((pages, m.kv_heads, page_size, D), dtype=m.emb.dtype, device=device)
        self.v = torch.zeros_like(self.k)
        self.table = torch.full((B, width), -1, **i32)
        self.ring = torch.arange(pages, **i32)
        # inputs and outputs of a plan, exchanged at every step
        self.owned, self.owned_out = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.ring_state, self.ring_state_out = torch.tensor([0, pages], **i32), torch.zeros(2, **i32)
        T = B * (gamma + 1)
        self.kv_len, self.q_off, self.tile_off = torch.zeros(B, **i32), torch.zeros(B + 1, **i32), torch.zeros(B + 1, **i32)
        self.slot_map, self.positions = torch.zeros(T, **i32), torch.zeros(T, **i32)
        self.seq_len = torch.zeros(B, **i32)                 # positions in the cache
        self.hist, self.hist_len = torch.zeros((B, max_len + gamma + 1), **i32), torch.ones(B, **i32)
        self.anchor = torch.randint(0, m.V, (B,), generator=g, device=device, dtype=torch.int32)
        self.hist[:, 0] = self.anchor
        self.prompt_len = torch.ones(B, **i32)
        # a Markov head and base logits that know the target's taste a little
        self.W1 = (torch.randn((m.V, r), generator=g, device=device) * 0.05).to(torch.bfloat16)
        self.W2 = (torch.randn((r, m.V), generator=g, device=device) * 0.05).to(torch.bfloat16)
        self.rep = 1.0 + 0.3 * torch.rand(B, generator=g, device=device)
        self.freq, self.pres = 0.4 * torch.rand(B, generator=g, device=device), 0.2 * torch.rand(B, generator=g, device=device)
        # half of the requests may only use a tenth of the vocabulary
        self.allowed = (torch.rand((B, m.V), generator=g, device=device) < 0.1) | (torch.arange(B, device=device) % 2 == 1)[:, None]
        self.allowed[:, 0] = True
        W = -(-m.V // 32)
        bits = torch.zeros((B, W * 32), dtype=torch.int64, device=device)
        bits[:, :m.V] = self.allowed
        word = (bits.view(B, W, 32) << torch.arange(32, device=device)).sum(2)
        word = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)
        self.mask = word[:, None].expand(B, gamma + 1, W).contiguous()
        self.mask_draft = word[:, None].expand(B, gamma, W).contiguous()
        self.buf = vm.StepBuffers(B, gamma, m.V, r, device)
        self.cache_ws = vm.CacheWorkspace(B, m.q_heads, m.kv_heads, D, gamma + 1, device, four_bits=False)
        self.target_ws, self.draft_ws = vm.LogitsWorkspace(B, gamma + 1, device), vm.LogitsWorkspace(B, gamma, device)
        self.target = torch.empty((B, gamma + 1, m.V), device=device)
        self.U = torch.empty((B, gamma, m.V), device=device)
        self.n_new = torch.full((B,), gamma + 1, **i32)
        self.K = torch.full((B,), gamma, **i32)
        self.emitted = torch.arange(gamma + 1, device=device)[None]

    def step(self, seed, step):
        m, B, G, buf = self.m, self.B, self.gamma, self.buf
        # the draft's base logits: the target's head on the anchor alone
        x = m.inputs(self.anchor.long(), self.seq_len.long())
        self.U.copy_(m.logits(x, m.split(x)[2].repeat_interleave(m.q_heads // m.kv_heads, 1))[:, None].expand(B, G, m.V))
        vm.dspark_logits_process(self.U, self.U, self.draft_ws, mask=self.mask_draft, fill=-1e4)
        vm.dspark_draft_markov(self.U, self.W1, self.W2, self.anchor, buf.draft_tok, buf.lse_q, buf.z_tok, buf.ws,
                               seed=seed, step=step)
        # the block: the anchor and its drafts
        vm.dspark_cache_plan(self.seq_len, self.n_new, self.owned, self.ring, self.ring_state, self.table, self.P,
                             owned_out=self.owned_out, ring_state_out=self.ring_state_out, kv_len=self.kv_len,
                             q_off=self.q_off, tile_off=self.tile_off, slot_map=self.slot_map,
                             positions=self.positions, ws=self.cache_ws)
        block = torch.cat([self.anchor[:, None], buf.draft_tok], 1).view(-1).long()
        x = m.inputs(block, self.positions.long())
        q, k, v = m.split(x)
        vm.dspark_cache_append(k, v, self.slot_map, self.k, self.v, ws=self.cache_ws)
        attended = torch.empty((B * (G + 1), m.q_heads, m.head_dim), dtype=q.dtype, device=q.device)
        vm.dspark_cache_attention(q, self.k, self.v, self.table, self.kv_len, self.q_off, self.tile_off, attended,
                                  self.cache_ws, max_new=G + 1)
        self.target.copy_(m.logits(x, attended).view(B, G + 1, m.V))
        self.raw = self.target.clone()
        vm.dspark_logits_process(self.target, self.target, self.target_ws, hist=self.hist, hist_len=self.hist_len,
                                 prompt_len=self.prompt_len, draft_tok=buf.draft_tok, rep=self.rep, freq=self.freq,
                                 pres=self.pres, mask=self.mask)
        vm.dspark_verify(self.target, self.U, self.W1, self.W2, self.anchor, buf.draft_tok, buf.lse_q, buf.z_tok, self.K,
                         buf.accepted, buf.out_tok, buf.out_req, buf.out_pos, buf.out_off, buf.next_anchor, buf.ws,
                         seed=seed, step=step)
        # advance: accepted drafts, then the new anchor (not yet in the cache)
        keep = self.emitted <= buf.accepted[:, None]
        new = torch.where(self.emitted == buf.accepted[:, None], buf.next_anchor[:, None],
                          torch.cat([buf.draft_tok, buf.next_anchor[:, None]], 1))
        at = self.hist_len[:, None].long() + self.emitted
        self.hist.scatter_(1, at, torch.where(keep, new, self.hist.gather(1, at)))
        self.hist_len += buf.accepted + 1
        self.seq_len += buf.accepted + 1
        self.anchor = buf.next_anchor.clone()
        self.owned, self.owned_out = self.owned_out, self.owned
        self.ring_state, self.ring_state_out = self.ring_state_out, self.ring_state

    def dense_logits(self, tokens):
        """The target's logits after tokens[0], ..: attention over the whole
        sequence at once, without the cache (fp32)."""
        m = self.m
        x = m.inputs(tokens, torch.arange(tokens.numel(), device=tokens.device))
        q, k, v = (t.float() for t in m.split(x))
        G = m.q_heads // m.kv_heads
        s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(G, 1)) * m.head_dim ** -0.5
        n = tokens.numel()
        s = s.masked_fill(torch.ones((n, n), dtype=torch.bool, device=s.device).triu(1), float("-inf"))
        o = torch.einsum("hij,jhd->ihd", s.softmax(2), v.repeat_interleave(G, 1))
        return m.logits(x, o.to(x.dtype)).float()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--vocab", type=int, default=4096)
    a = ap.parse_args(argv)
    max_len = 8 * (a.steps + 1) + 8
    model = ToyTarget(a.vocab, q_heads=8, kv_heads=2, head_dim=64, max_len=max_len)
    d = Decoder(model, a.requests, max_len=max_len)
    worst, accepted = 0.0, 0
    for t in range(a.steps):
        before, block = d.hist_len.clone(), d.anchor.clone()
        d.step(seed=1, step=t)
        accepted += int(d.buf.accepted.sum())
        # the cached path against the whole sequence, on request 0's block
        b, n = 0, int(before[0])
        seq = torch.cat([d.hist[b, :n], d.buf.draft_tok[b]]).long()
        want = d.dense_logits(seq)[n - 1:]
        assert int(seq[n - 1]) == int(block[b])
        worst = max(worst, float((d.raw[b] - want).abs().max() / want.abs().max()))
    for ws in (d.buf.ws, d.cache_ws, d.target_ws, d.draft_ws):
        st, bits = vm.dspark_sync_status(ws.buf)
        assert st == 0, (st, bits)
    ids = torch.arange(d.hist.shape[1], device="cuda")[None]
    mine = (ids >= 1) & (ids < d.hist_len[:, None])
    ok = d.allowed.gather(1, d.hist.long())[mine].all()
    n = int((d.hist_len - 1).sum())
    print(f"{a.requests} requests, {a.steps} steps: {n} tokens, {accepted / (a.steps * a.requests):.2f} drafts accepted a step; "
          f"cached against dense logits: {worst:.2e}; every token allowed: {bool(ok)}; "
          f"pages in use {int(d.owned.sum())}, free {int(d.ring_state[1])}")
    return dict(worst=worst, allowed=bool(ok), tokens=n, accepted=accepted, decoder=d)


if __name__ == "__main__":
    main()
