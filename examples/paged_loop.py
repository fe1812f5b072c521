"""A speculative decoding loop that never waits for the device: a one-layer
target model over a paged key/value cache, with random weights.

Each step the draft proposes K tokens per request, the target reads the last
token and the drafts in one pass (plan, append, attention), and the verify
step accepts a prefix and plugs the emitted tokens into the sequences.  The
lengths stay on the device: the next step's plan reads what the plug wrote,
takes the pages that the new tokens need and gives back those that rejected
drafts held.

    python examples/paged_loop.py [--batch 8] [--drafts 4] [--steps 16] [--temperature 0]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_verification_25_gb300 import api  # noqa: E402

VOCAB, WIDTH, HQ, HK, D, PAGE = 1024, 512, 8, 2, 64, 16


class Model:
    """Embedding, one attention layer with grouped heads and sinusoidal
    positions beside a linear one, and the embedding again at the output."""

    def __init__(self, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        w = lambda *s: torch.randn(s, generator=g, device=device) * s[-1] ** -0.5
        self.embed = torch.randn(VOCAB, WIDTH, generator=g, device=device)
        self.qkv, self.out, self.mix = w((HQ + 2 * HK) * D, WIDTH), w(WIDTH, HQ * D), w(WIDTH, WIDTH)
        self.rates = torch.logspace(0, -3, WIDTH // 2, device=device)

    def inputs(self, tokens, positions):
        angle = positions.clamp(min=0).unsqueeze(-1) * self.rates
        return self.embed[tokens.long()] + 0.3 * torch.cat([angle.sin(), angle.cos()], -1)

    def project(self, x):
        """Queries, keys and values side by side, [T, HQ + 2 HK, D]."""
        return (x @ self.qkv.T).bfloat16().view(-1, HQ + 2 * HK, D)

    def logits(self, x, attended):
        return (x @ self.mix.T + attended.float().flatten(1) @ self.out.T * 0.5) @ self.embed.T * (4 * WIDTH ** -0.5)

    def draft_logits(self, tokens):
        """The same without positions and attention."""
        return self.embed[tokens.long()] @ self.mix.T @ self.embed.T * (4 * WIDTH ** -0.5)


class Cache:
    """Pages of all requests, and which of them each request holds."""

    def __init__(self, batch, max_len, device):
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)
        per_row = -(-max_len // PAGE)
        n_pages = batch * per_row
        self.k, self.v = (torch.empty(n_pages, HK, PAGE, D, dtype=torch.bfloat16, device=device) for _ in range(2))
        self.table, self.page_count = ints(batch, per_row), ints(batch)
        self.free_pages = torch.arange(n_pages, dtype=torch.int32, device=device)
        self.free_count = torch.full((1,), n_pages, dtype=torch.int32, device=device)

    def plan(self, cached, num_new, max_tokens):
        plan = api.paged_plan(cached, num_new, self.page_count, self.table, self.free_pages, self.free_count,
                              page_size=PAGE, max_tokens=max_tokens)
        self.page_count, self.free_count = plan.page_count, plan.free_count
        return plan


def target_pass(model, cache, tokens, cached, num_new, max_tokens):
    """Logits of the packed new ``tokens`` [max_tokens], which follow the
    ``cached`` ones of every request, and the plan of the pass."""
    plan = cache.plan(cached, num_new, max_tokens)
    x = model.inputs(tokens, plan.positions)
    qkv = model.project(x)
    api.paged_append(qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:], plan.slot_map, cache.k, cache.v)
    attended = api.paged_attention(qkv[:, :HQ], cache.k, cache.v, cache.table, plan.cu_new, plan.kv_len).out
    return model.logits(x, attended), plan


def generate(model, prompts, steps, drafts, temperature, seed=0):
    """Sequences [B, max_len] and their lengths [B], on the device, after
    ``steps`` verified passes over equally long ``prompts`` [B, n]."""
    B, n = prompts.shape
    dev = prompts.device
    max_len = n + 1 + steps * (drafts + 1)
    g = torch.Generator(device=dev).manual_seed(seed)
    cache = Cache(B, max_len, dev)
    T = torch.full((B,), float(temperature), device=dev)
    tokens = torch.zeros(B, max_len, dtype=torch.int32, device=dev)
    tokens[:, :n] = prompts
    seq_len = torch.full((B,), n, dtype=torch.int32, device=dev)
    last = prompts[:, -1].contiguous()
    # the prompt up to its last token, which the first step brings
    if n > 1:
        ahead = torch.full((B,), n - 1, dtype=torch.int32, device=dev)
        target_pass(model, cache, prompts[:, :-1].flatten(), torch.zeros_like(ahead), ahead, B * (n - 1))
    num_new = torch.full((B,), drafts + 1, dtype=torch.int32, device=dev)
    for _ in range(steps):
        # the draft, token by token
        proposal, scores = [last], []
        for _ in range(drafts):
            scores.append(model.draft_logits(proposal[-1]))
            noise = torch.rand(B, VOCAB, generator=g, device=dev).clamp(min=1e-20).log().neg().log().neg()
            proposal.append((scores[-1] + T[:, None] * noise).argmax(-1).to(torch.int32))
        new = torch.stack(proposal, 1)   # [B, drafts + 1]: the last token and the drafts
        logits, _ = target_pass(model, cache, new.flatten(), seq_len - 1, num_new, B * (drafts + 1))
        uniforms = torch.rand(B, drafts + 1, generator=g, device=dev)
        api.spec_verify_and_plug(logits.view(B, drafts + 1, VOCAB), torch.stack(scores, 1), new[:, 1:].contiguous(),
                                 uniforms, T, tokens, seq_len, last_token=last)
    return tokens, seq_len


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--temperature", type=float, default=0.0)
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    prompts = torch.randint(0, VOCAB, (a.batch, 33), dtype=torch.int32, device=dev)
    tokens, seq_len = generate(Model(dev), prompts, a.steps, a.drafts, a.temperature)
    for row, n in zip(tokens.tolist(), seq_len.tolist()):
        print(f"{(n - 33) / a.steps:.2f} tokens per pass:", *row[33:n][:16])


if __name__ == "__main__":
    main()
