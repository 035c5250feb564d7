"""Speculative decoding that trains its drafter on the rounds it verifies.

    python examples/online_drafter.py [ROUNDS]

Target and drafter are two bigram heads over the same token embeddings (a stand-in for two
models: what matters here is what happens to their logits).  A round:

  draft    the drafter draws K tokens, each from its logits under the request's penalties,
           biases and grammar mask (process_logits, one row at a time: base = j)
  score    the target gives K + 1 rows, processed alike (process_logits, base = 0)
  verify   accepted drafts and the correction or bonus token (verify)
  count    the emitted tokens enter the penalties' state (token_counts_add)
  learn    the target's top logits teach the drafter on the same positions (top_logits,
           distill_grad), one optimizer step

The mean number of tokens per round (tau) grows as the drafter learns.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import speculative_decoding_verification_logits_gb300 as sd  # noqa: E402


class Round:
    """The state of B requests over a vocabulary of V tokens."""

    def __init__(self, B=16, K=4, V=1009, dim=32, top=32, temperature=0.8, lr=0.05, seed=0,
                 device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda *s: torch.randn(s, generator=g, device=device)
        self.B, self.K, self.V, self.top, self.T = B, K, V, top, temperature
        self.gen, self.seed, self.device = g, seed, torch.device(device)
        self.emb = new(V, dim).to(torch.bfloat16)
        self.target = (new(V, dim) * 0.6).to(torch.bfloat16)
        self.drafter = torch.zeros((V, dim), device=device, requires_grad=True)
        self.opt = torch.optim.Adam([self.drafter], lr=lr)
        # prompts, penalties, biases, and a grammar that forbids a tenth of the tokens
        prompt = torch.randint(0, V, (B, 50), generator=g, device=device, dtype=torch.int32)
        full = torch.full((B,), 50, dtype=torch.int32, device=device)
        self.last = prompt[:, -1].contiguous()
        self.counts = sd.token_counts(prompt, full, V, prompt_lengths=full)
        self.temps = torch.full((B,), temperature, device=device)
        bits = torch.rand((B, V), generator=g, device=device) < 0.9
        words = torch.nn.functional.pad(bits, (0, -V % 32)).view(B, -1, 32).to(torch.int64)
        words = (words << torch.arange(32, device=device)).sum(-1)
        self.mask = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
        self.rules = dict(
            repetition=torch.full((B,), 1.1, device=device),
            presence=torch.full((B,), 0.2, device=device),
            frequency=torch.full((B,), 0.1, device=device),
            bias_ids=torch.randint(0, V, (B, 8), generator=g, device=device, dtype=torch.int32),
            bias_vals=torch.full((B, 8), 1.0, device=device), mask=self.mask)
        self.round = 0

    def rows(self, head, tokens):
        """Logits [..., V] (bf16) after each token."""
        return self.emb[tokens.long()] @ head.to(torch.bfloat16).T

    def draft(self):
        """K drafted tokens per request and the processed rows they were drawn from."""
        tokens = torch.zeros((self.B, self.K), dtype=torch.int32, device=self.device)
        drawn, at = [], self.last
        for j in range(self.K):
            row = sd.process_logits(self.rows(self.drafter.detach(), at), counts=self.counts,
                                    prev=tokens, base=j, **self.rules)
            p = torch.softmax(row.float() / self.T, -1)
            at = torch.multinomial(p, 1, generator=self.gen)[:, 0].to(torch.int32)
            tokens[:, j] = at
            drawn.append(row)
        return tokens, torch.stack(drawn, 1)

    def step(self):
        """One round; (tau [B], mean loss)."""
        tokens, drawn = self.draft()
        context = torch.cat([self.last[:, None], tokens], 1)          # [B][K + 1]
        raw = self.rows(self.target, context)
        rows = sd.process_logits(raw, counts=self.counts, prev=tokens, **self.rules)
        r = sd.verify(rows, drawn, tokens, self.temps, self.seed * 1000003 + self.round,
                      check_finite=True)
        sd.token_counts_add(self.counts, r.out_tokens, r.tau)
        self.last = r.out_tokens.gather(1, (r.tau.long() - 1).clamp(min=0)[:, None])[:, 0]
        self.last = self.last.clamp(min=0).contiguous()
        # the drafter learns the target's own rows, of the accepted positions only
        teacher = sd.top_logits(raw, self.top)
        use = torch.arange(self.K + 1, device=self.device) < r.tau[:, None]
        weight = use.float() / use.sum()
        student = self.rows(self.drafter, context)
        loss, grad = sd.distill_grad(student, teacher.ids, teacher.vals, teacher.rest, weight=weight)
        self.opt.zero_grad()
        student.backward(grad)
        self.opt.step()
        self.round += 1
        return r, loss.sum()


def main(rounds=200):
    s = Round()
    taus = []
    for i in range(rounds):
        r, loss = s.step()
        taus.append(r.tau.float().mean())
        if (i + 1) % 25 == 0:
            print(f"round {i + 1:4d}  tau {float(torch.stack(taus[-25:]).mean()):.2f}  "
                  f"loss {float(loss):.3f}")
    return torch.stack(taus).tolist()


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
