"""Greedy tree-speculative decoding of a small random model over an 8-bit paged cache, every step on this library:

  spec_kv_append_q8          the draft tree's keys and values enter the cache
  spec_attention_q8          every node attends to the prompt and its ancestors
  spec_verify_tree           the accepted path and the bonus token
  spec_kv_append_q8          the path's rows, written again over the nodes
  spec_attention_weights_q8  what the accepted rows attended to, kept per slot
  spec_kv_evict_q8           down to a budget once a request outgrows it
  spec_token_logprobs        log-prob, entropy and top alternatives of what was emitted

  python examples/q8_verify_step.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_72_gb300 as sv  # noqa: E402


class Model:
    """One attention layer between tied embeddings, weights random."""

    def __init__(self, vocab=512, width=256, heads=8, kv_heads=2, head_dim=64, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s, scale: (torch.randn(s, generator=g) * scale).to(device, torch.bfloat16)  # noqa: E731
        self.heads, self.kv_heads, self.head_dim, self.vocab = heads, kv_heads, head_dim, vocab
        self.emb = rand(vocab, width, scale=1.0)
        self.wq = rand(width, heads * head_dim, scale=2 / width ** 0.5)
        self.wk = rand(width, kv_heads * head_dim, scale=2 / width ** 0.5)
        self.wv = rand(width, kv_heads * head_dim, scale=4 / width ** 0.5)
        self.wo = rand(heads * head_dim, width, scale=4 / (heads * head_dim) ** 0.5)

    def rows(self, tokens):
        B, N = tokens.shape
        x = self.emb[tokens.long()]
        split = lambda y, h: y.view(B, N, h, self.head_dim)  # noqa: E731
        return x, split(x @ self.wq, self.heads), split(x @ self.wk, self.kv_heads), split(x @ self.wv, self.kv_heads)

    def logits(self, attended):
        B, N = attended.shape[:2]
        return (attended.reshape(B, N, -1) @ self.wo) @ self.emb.t()


class Decoder:
    """A batch of requests, each with `max_len` slots of cache and a budget it is evicted down to."""

    def __init__(self, model, batch, max_len, page=16, budget=None, device="cuda"):
        pages = -(-max_len // page)
        self.m, self.budget, self.max_len = model, budget, pages * page
        self.cache = sv.q8_cache(batch * pages, model.kv_heads, page, model.head_dim)
        self.table = torch.arange(batch * pages, dtype=torch.int32, device=device).view(batch, pages)
        self.length = torch.zeros(batch, dtype=torch.int32, device=device)          # slots in use
        self.seen = torch.zeros(batch, dtype=torch.int32, device=device)            # tokens so far
        shape = (batch, model.kv_heads, self.max_len)
        self.scores = torch.zeros(shape, device=device)
        self.positions = torch.full(shape, -1, dtype=torch.int32, device=device)

    def _note_positions(self, n):
        """Slots length .. length + n - 1 hold the next n tokens of each request."""
        slot = torch.arange(self.max_len, device=n.device)
        new = (slot >= self.length[:, None]) & (slot < (self.length + n)[:, None])
        pos = (self.seen - self.length)[:, None] + slot
        self.positions = torch.where(new[:, None], pos[:, None].int(), self.positions)
        self.seen = self.seen + n

    def prefill(self, tokens):
        """The prompt but its last token (the first step's root), 64 positions at a time."""
        for t in tokens.split(64, 1):
            _, _, k, v = self.m.rows(t)
            n = torch.full_like(self.length, t.shape[1])
            self._note_positions(n)
            self.length = sv.spec_kv_append_q8(self.cache, k, v, self.table, self.length)["out_len"]

    def step(self, node_tokens, parents, max_depth, n_top=5):
        """One verify pass. Returns the emitted tokens [B, max_depth + 1] (-1 past the last), how many, and their
        log-probs."""
        m, base = self.m, self.length
        _, q, k, v = m.rows(node_tokens)
        sv.spec_kv_append_q8(self.cache, k, v, self.table, base)
        att = sv.spec_attention_q8(q, self.cache, self.table, base, parents=parents)
        logits = m.logits(att["out"])
        r = sv.spec_verify_tree(logits, node_tokens, parents, max_depth)
        path, n_acc = r["nodes"], r["num_accepted"]
        new_len = sv.spec_kv_append_q8(self.cache, k, v, self.table, base, path_nodes=path, num_accepted=n_acc)["out_len"]
        self._note_positions(n_acc + 1)
        sv.spec_attention_weights_q8(q, att["lse"], self.cache, self.table, base, self.scores, path_nodes=path,
                                     num_accepted=n_acc, decay=0.95, out=dict(scores=self.scores, status=torch.empty_like(n_acc)))
        self.length = new_len
        if self.budget is not None and int(new_len.max()) > self.budget:
            e = sv.spec_kv_evict_q8(self.cache, self.table, new_len, self.scores, self.positions, self.budget, sinks=4,
                                    protect_from=self.seen - 8)
            self.scores, self.positions, self.length = e["scores"], e["positions"], e["out_len"]
        rows = torch.gather(logits, 1, path.clamp(min=0).long()[:, :, None].expand(-1, -1, m.vocab))
        lp = sv.spec_token_logprobs(rows, r["tokens"], n_top=n_top)
        return r["tokens"], n_acc + 1, lp


TREE = [-1, 0, 0, 1, 1, 2, 3, 3]   # parents of a tree three deep


def draft(tokens, vocab, generator, guess=None):
    """A tree of random tokens below the roots `tokens` [B]; the first child at each depth is guess [B, 3] where given."""
    B = tokens.shape[0]
    nodes = torch.randint(0, vocab, (B, len(TREE)), generator=generator, dtype=torch.int32)
    if guess is not None:
        for depth, node in enumerate((1, 3, 6)):
            nodes[:, node] = torch.where(guess[:, depth].cpu() >= 0, guess[:, depth].cpu().int(), nodes[:, node])
    nodes = nodes.to(tokens.device)
    nodes[:, 0] = tokens
    return nodes, torch.tensor(TREE, dtype=torch.int32, device=tokens.device).expand(B, -1).contiguous()


def decode(model, prompt, n, guesses=None, budget=None, seed=1, report=None):
    """n tokens after prompt [B, L]; guesses [B, >= n] (a drafter's) are offered to the verify passes. Returns tokens
    [B, n], their log-probs and the decoder."""
    B, L = prompt.shape
    # a request may take four tokens a pass while another takes one
    d = Decoder(model, B, L + 4 * n + len(TREE), budget=budget)
    d.prefill(prompt[:, :-1])
    g = torch.Generator().manual_seed(seed)
    out, lps, last = [[] for _ in range(B)], [[] for _ in range(B)], prompt[:, -1].clone()
    while min(map(len, out)) < n:
        guess = None
        if guesses is not None:
            guess = torch.stack([torch.nn.functional.pad(guesses[b, len(out[b]):len(out[b]) + 3], (0, 3), value=-1)[:3]
                                 for b in range(B)])
        nodes, parents = draft(last, model.vocab, g, guess)
        tokens, count, lp = d.step(nodes, parents, max_depth=3)
        for b in range(B):
            c = int(count[b])
            out[b] += tokens[b, :c].tolist()
            lps[b] += lp["logprob"][b, :c].tolist()
            last[b] = out[b][-1]
        if report:
            report(d, count, lp)
    return torch.tensor([o[:n] for o in out]), torch.tensor([x[:n] for x in lps]), d


def main():
    model = Model()
    prompt = torch.randint(0, model.vocab, (4, 200), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    plain, _, _ = decode(model, prompt, 40)
    passes = []
    tokens, lps, d = decode(model, prompt, 40, guesses=plain.int(), report=lambda d, c, lp: passes.append(c.float().mean()))
    same = (tokens == plain).float().mean().item()
    print(f"{len(passes)} verify passes for 40 tokens, {torch.stack(passes).mean():.2f} tokens a pass, {same:.0%} as without drafts, "
          f"mean log-prob {lps.mean():.3f}")
    tokens, lps, d = decode(model, prompt, 40, guesses=plain.int(), budget=128)
    print(f"with a budget of 128 slots: {d.length.tolist()} slots for {d.seen.tolist()} tokens, mean log-prob {lps.mean():.3f}")


if __name__ == "__main__":
    main()
