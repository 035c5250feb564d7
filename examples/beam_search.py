"""Beam search over a paged cache that the beams share.

    python examples/beam_search.py [STEPS]

The model is one attention head over token embeddings (a stand-in: what matters here is what
happens to its logits, its cache and its texts).  A step, for B requests of W beams each:

  attend   each beam's row of the block table is read, its logits come from the cached entries
  process  repetition penalty from the beam's own token counts (process_logits)
  select   the W best of W V continuations, finished beams among them (beam_select)
  reorder  texts and token counts follow their parents, in place (beam_reorder)
  fork     so do the block tables: full pages are shared, the last one is copied where two beams
           go on from one (kv_fork, kv_copy); beams that nobody goes on from give theirs back
  write    the new token's entry

A prompt is written once and forked into its beams.  Requests that are done give their pages back
(kv_free), and the pages that are left move to the front of the pool (kv_compact, kv_copy).
"""
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import speculative_decoding_verification_logits_gb300 as sd  # noqa: E402


class Search:
    """B requests with W beams over a vocabulary of V tokens."""

    def __init__(self, B=4, W=5, V=997, dim=24, prompt=21, room=60, page=8, penalty=1.2, seed=0,
                 device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda *s: torch.randn(s, generator=g, device=device)
        self.B, self.W, self.V, self.dim, self.page, self.eos = B, W, V, dim, page, 1
        self.device = dev = torch.device(device)
        self.emb, self.head = new(V, dim), new(V, dim) * 0.7
        rows, self.length, self.start = B * W, prompt, prompt
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
        # texts, counts and scores of the beams; at first one of a request's is alive
        self.prompts = torch.randint(2, V, (B, prompt), generator=g, device=dev, dtype=torch.int32)
        self.texts = ints(B, W, prompt + room)
        self.texts[:, :, :prompt] = self.prompts[:, None]
        self.scores = torch.full((B, W), -math.inf, device=dev)
        self.scores[:, 0] = 0.0
        self.finished = torch.zeros((B, W), dtype=torch.uint8, device=dev)
        full = torch.full((B,), prompt, dtype=torch.int32, device=dev)
        counts = sd.token_counts(self.prompts, full, V, prompt_lengths=full)
        self.counts = counts[:, None].repeat(1, W, 1)
        self.repetition = torch.full((rows,), penalty, device=dev)
        # the pool; the prompts' rows take pages, are written and forked into W rows each
        max_pages = -(-(prompt + room) // page)
        self.N = rows * max_pages + 8
        self.refs, self.status = ints(self.N), ints(1)
        self.cache = torch.zeros((2, self.N, page, dim), device=dev)   # keys, values
        table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
        n = ints(B)
        sd.kv_extend(table, n, self.refs, page, prompt, status=self.status)
        for i in range(prompt):
            self.write(table, n + i, self.prompts[:, i])
        f = sd.kv_fork(table, n + prompt, ints(B, W), self.refs, page, status=self.status)
        self.copy(f)
        self.table, self.kv_len = f.block_table, f.kv_len

    def copy(self, moves):
        sd.kv_copy(self.cache, moves.src, moves.dst, count=moves.count,
                   fill=getattr(moves, "fill", None), status=self.status)

    def write(self, table, at, tokens):
        """The entries of `tokens` at place `at` of each row."""
        ids = table.gather(1, (at // self.page).long()[:, None])[:, 0].long()
        e = self.emb[tokens.long()]
        slot = (at % self.page).long()
        self.cache[0, ids, slot] = e
        self.cache[1, ids, slot] = torch.tanh(e.roll(1, -1))

    def logits(self):
        """[B W][V] from the entries of each row: one head, the last one's entry asks."""
        n = int(self.length)
        ids = self.table[:, :-(-n // self.page)].clamp(min=0).long()
        k, v = (c[ids].flatten(1, 2)[:, :n] for c in self.cache)
        w = torch.softmax((k * k[:, -1:]).sum(-1) / math.sqrt(self.dim), 1)
        return torch.tanh((w[:, :, None] * v).sum(1) + k[:, -1]) @ self.head.T

    def step(self):
        B, W = self.B, self.W
        x = sd.process_logits(self.logits(), counts=self.counts.view(B * W, -1),
                              repetition=self.repetition)
        b = sd.beam_select(x.view(B, W, -1), self.scores, W, finished=self.finished, eos=self.eos,
                           status=self.status)
        sd.beam_reorder((self.texts, self.counts), b.parents, out=(self.texts, self.counts),
                        status=self.status)
        f = sd.kv_fork(self.table, self.kv_len, b.parents, self.refs, self.page, append=1,
                       status=self.status)
        self.copy(f)
        self.table, self.kv_len = f.block_table, f.kv_len
        self.scores, self.finished = b.scores, b.finished
        tokens = b.tokens.view(-1)
        self.texts[:, :, self.length] = b.tokens
        sd.token_counts_add(self.counts.view(B * W, -1), tokens[:, None],
                            torch.ones_like(tokens), status=self.status)
        self.write(self.table, self.kv_len, tokens)
        self.kv_len = self.kv_len + 1
        self.length += 1
        return b

    def end(self, requests):
        """Requests (flags [B]) give their pages back; the others' move to the pool's front."""
        which = requests.to(torch.uint8)[:, None].expand(self.B, self.W).reshape(-1).contiguous()
        sd.kv_free(self.table, self.refs, which=which, clear=True, status=self.status)
        c = sd.kv_compact(self.refs, self.table, status=self.status)
        self.copy(c)
        return c


def main(steps=40):
    s = Search()
    for _ in range(steps):
        s.step()
    for b in range(s.B):
        text = s.texts[b, 0, s.start:s.length].tolist()
        print(f"request {b}: score {float(s.scores[b, 0]):8.3f}  {text[:12]} ...")
    print(f"pages in use {int((s.refs > 0).sum())} of {s.N} "
          f"({s.B * s.W * -(-s.length // s.page)} if no beam shared one), "
          f"status {int(s.status)}")
    return s


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
