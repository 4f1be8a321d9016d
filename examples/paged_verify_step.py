"""Greedy tree-speculative decoding of a small random model over a 16-bit paged cache, every step on this library:

  spec_kv_append_rope   the draft tree's keys and values enter the cache, keys and queries rotated by position
  spec_attention        every node attends to the prompt and its ancestors, here with capped scores and a window
  spec_verify_tree      the accepted path and the bonus token
  spec_kv_compact       the path's rows move to their places (keys are rotated for where they land)

  python examples/paged_verify_step.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_72_gb300 as sv  # noqa: E402


class Model:
    """One attention layer between tied embeddings, weights random."""

    def __init__(self, vocab=512, width=256, heads=8, kv_heads=2, head_dim=64, softcap=20.0, window=160, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s, scale: (torch.randn(s, generator=g) * scale).to(device, torch.bfloat16)  # noqa: E731
        self.heads, self.kv_heads, self.head_dim, self.vocab = heads, kv_heads, head_dim, vocab
        self.softcap, self.window = softcap, window
        self.emb = rand(vocab, width, scale=1.0)
        self.w = rand(width, (heads + 2 * kv_heads) * head_dim, scale=2 / width ** 0.5)
        self.wo = rand(heads * head_dim, width, scale=4 / (heads * head_dim) ** 0.5)
        self.inv_freq = 10000.0 ** (-torch.arange(head_dim // 2, device=device) * 2.0 / head_dim)

    def project(self, tokens):
        """Queries, keys and values of tokens [B, N], as slices of one row."""
        B, N = tokens.shape
        y = (self.emb[tokens.long()] @ self.w).view(B, N, -1, self.head_dim)
        return y.split([self.heads, self.kv_heads, self.kv_heads], 2)

    def logits(self, attended):
        B, N = attended.shape[:2]
        return (attended.reshape(B, N, -1) @ self.wo) @ self.emb.t()


class Decoder:
    """A batch of requests, each with `max_len` slots of cache."""

    def __init__(self, model, batch, max_len, page=16, device="cuda"):
        pages = -(-max_len // page)
        self.m = model
        self.cache = sv.paged_cache(batch * pages, model.kv_heads, page, model.head_dim)
        self.table = torch.arange(batch * pages, dtype=torch.int32, device=device).view(batch, pages)
        self.length = torch.zeros(batch, dtype=torch.int32, device=device)

    def forward(self, tokens, parents=None):
        """Logits of new rows behind what the cache holds, and the lengths with them."""
        m = self.m
        q, k, v = m.project(tokens)
        r = sv.spec_kv_append_rope(self.cache, k, v, self.table, self.length, m.inv_freq, q=q, parents=parents)
        att = sv.spec_attention(r["q"], self.cache, self.table, self.length, parents=parents, softcap=m.softcap, window=m.window)
        return m.logits(att["out"]), r["out_len"]

    def prefill(self, tokens):
        """The prompt but its last token, which is the first step's root."""
        _, self.length = self.forward(tokens)

    def step(self, node_tokens, parents, max_depth):
        """One verify pass: the emitted tokens [B, max_depth + 1] (-1 past the last) and how many."""
        logits, _ = self.forward(node_tokens, parents)
        r = sv.spec_verify_tree(logits, node_tokens, parents, max_depth)
        for kv in self.cache:
            n = sv.spec_kv_compact(kv, self.table, self.length, r["nodes"], r["num_accepted"], node_tokens.shape[1])
        self.length = n["out_len"]
        return r["tokens"], r["num_accepted"] + 1


TREE = [-1, 0, 0, 1, 1, 2, 3, 3]   # parents of a tree three deep


def draft(roots, vocab, generator, guess):
    """A tree of random tokens below the roots [B]; the first child at each depth is guess [B, 3] where that is a token."""
    nodes = torch.randint(0, vocab, (roots.shape[0], len(TREE)), generator=generator, dtype=torch.int32).to(roots.device)
    for depth, node in enumerate((1, 3, 6)):
        nodes[:, node] = torch.where(guess[:, depth] >= 0, guess[:, depth], nodes[:, node])
    nodes[:, 0] = roots
    return nodes, torch.tensor(TREE, dtype=torch.int32, device=roots.device).expand(roots.shape[0], -1).contiguous()


def decode(model, prompt, n, guesses=None, seed=1):
    """n tokens after prompt [B, L]; guesses [B, >= n] (a drafter's) are offered to the verify passes. Returns tokens
    [B, n], the number of passes and the decoder."""
    B, L = prompt.shape
    d = Decoder(model, B, L + 4 * n + len(TREE))
    d.prefill(prompt[:, :-1])
    g = torch.Generator().manual_seed(seed)
    out, last, passes = [[] for _ in range(B)], prompt[:, -1].clone(), 0
    while min(map(len, out)) < n:
        guess = torch.full((B, 3), -1, dtype=torch.int32, device=prompt.device)
        if guesses is not None:
            for b in range(B):
                some = guesses[b, len(out[b]):len(out[b]) + 3]
                guess[b, :len(some)] = some
        tokens, count = d.step(*draft(last, model.vocab, g, guess), max_depth=3)
        passes += 1
        for b in range(B):
            out[b] += tokens[b, :int(count[b])].tolist()
            last[b] = out[b][-1]
    return torch.tensor([o[:n] for o in out]), passes, d


def main():
    model = Model()
    prompt = torch.randint(0, model.vocab, (4, 200), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    plain, passes, _ = decode(model, prompt, 40)
    tokens, fewer, _ = decode(model, prompt, 40, guesses=plain.int().cuda())
    print(f"{passes} passes without a drafter, {fewer} with one that knows; {(tokens == plain).float().mean():.0%} the same")


if __name__ == "__main__":
    main()
