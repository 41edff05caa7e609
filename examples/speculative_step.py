"""Speculative decoding of a small hybrid model: one KDA layer, one softmax-attention layer.

    python examples/speculative_step.py [steps]

Each step takes every request's last token and K drafted ones through both
layers, decides how many drafts stand, and commits exactly those:

    kda_build_block_tables   pages and slots of the step's new tokens
    kda_cache_append         their keys and values into the paged cache
    kda_paged_attention      the attention layer, over the cache
    kda_decode_multi         the KDA layer; the state is left as it was
    kda_verify_draft         how many drafts stand, and the next token
    kda_decode_multi         the state after the tokens that stand

The model has random weights: a token's q, k, v and gates are rows of tables.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kimi_delta_attention_chunked_gb300 as kda  # noqa: E402
from kimi_delta_attention_chunked_gb300 import inputs  # noqa: E402

VOCAB, HEADS, KV_HEADS, DIM, PAGE = 512, 8, 2, 128, 16


class Model:
    def __init__(self, device, seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
        # KDA layer: per token q, k, v, beta, log_alpha; attention layer: q, k, v
        self.kda = inputs.make_qkv_gates(VOCAB, HEADS, DIM, DIM, torch.bfloat16, gen, device)
        self.q, self.k, self.v = (rnd(VOCAB, h, DIM).bfloat16() for h in (HEADS, KV_HEADS, KV_HEADS))
        self.out = rnd(2 * HEADS * DIM, VOCAB).bfloat16() * 0.05
        self.draft = torch.softmax(rnd(VOCAB, VOCAB), -1)            # the draft model: a table of next-token distributions

    def target(self, o_kda, o_attn):
        """Next-token distributions from both layers' outputs [..., H, DIM]."""
        x = torch.cat([o_kda.flatten(-2), o_attn.flatten(-2)], -1)
        return torch.softmax((x @ self.out).float(), -1)


class Server:
    """The state of N requests: last token, committed tokens, pages, KDA states."""

    def __init__(self, model, n, drafts, blocks=64, seed=1):
        self.model, self.n, self.drafts, self.blocks = model, n, drafts, blocks
        dev = model.q.device
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        self.last = torch.randint(0, VOCAB, (n,), generator=self.gen, device=dev)
        self.text = [[int(t)] for t in self.last]                    # all tokens; the last one is not committed yet
        self.ctx = torch.zeros(n, dtype=torch.int32, device=dev)
        self.pool = n * blocks
        self.table = torch.full((n, blocks), -1, dtype=torch.int32, device=dev)
        self.k_cache = torch.zeros(self.pool, KV_HEADS, PAGE, DIM, dtype=torch.bfloat16, device=dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.S = torch.zeros(n, HEADS, DIM, DIM, device=dev)

    def free_pages(self):
        """Pages that hold no committed token (those of rejected drafts come back)."""
        held = torch.arange(self.blocks, device=self.ctx.device) < ((self.ctx + PAGE - 1) // PAGE)[:, None]
        used = torch.zeros(self.pool, dtype=torch.bool, device=self.ctx.device)
        used[self.table[held].long()] = True
        return torch.nonzero(~used)[:, 0].to(torch.int32)

    def propose(self):
        """K drafted tokens of each request and the distributions they were drawn from."""
        tokens, dists, last = [], [], self.last
        for _ in range(self.drafts):
            p = self.model.draft[last]
            last = torch.multinomial(p, 1, generator=self.gen)[:, 0]
            tokens.append(last)
            dists.append(p)
        return torch.stack(tokens, 1), torch.stack(dists, 1).contiguous()

    def step(self):
        m, n, k = self.model, self.n, self.drafts
        drafted, dists = self.propose()
        run = torch.cat([self.last[:, None], drafted], 1)            # [N, K + 1]
        flat = run.reshape(-1)
        new = torch.full((n,), k + 1, dtype=torch.int32, device=run.device)
        cu, seq, slots, _, _ = kda.kda_build_block_tables(self.ctx, new, self.free_pages(), self.table, PAGE, n * (k + 1))
        kda.kda_cache_append(m.k[flat], m.v[flat], self.k_cache, self.v_cache, slots)
        o_attn = kda.kda_paged_attention(m.q[flat], self.k_cache, self.v_cache, self.table, cu, seq)
        q, key, v, beta, log_alpha = (x[run].contiguous() for x in m.kda)
        none = torch.zeros(n, dtype=torch.int32, device=run.device)
        o_kda = kda.kda_decode_multi(q, key, v, log_alpha, beta, self.S, commit_len=none)
        target = m.target(o_kda, o_attn.reshape(n, k + 1, HEADS, DIM))
        u = torch.rand(n, k + 1, generator=self.gen, device=run.device)
        tokens, commit = kda.kda_verify_draft(target, dists, drafted.to(torch.int32), u)
        kda.kda_decode_multi(q, key, v, log_alpha, beta, self.S, commit_len=commit, want_o=False)
        self.ctx += commit
        self.last = tokens.gather(1, (commit - 1).long()[:, None])[:, 0].long()
        for text, row in zip(self.text, tokens.tolist()):
            text.extend(t for t in row if t >= 0)
        return commit


def main(steps=8):
    server = Server(Model(torch.device("cuda", 0)), n=6, drafts=4)
    for i in range(steps):
        commit = server.step()
        print(f"step {i}: tokens committed per request {commit.tolist()}")
    print("lengths", server.ctx.tolist())


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
