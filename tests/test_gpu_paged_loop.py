"""The speculative loop over the paged cache: what it emits is what the target
says of the finished sequence, read in one pass."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def loop():
    spec = importlib.util.spec_from_file_location("paged_loop", os.path.join(ROOT, "examples", "paged_loop.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("batch,prompt,drafts,steps", [(1, 1, 1, 5), (3, 33, 4, 12), (9, 17, 16, 6)])
def test_greedy_tokens_are_the_targets_choice(loop, batch, prompt, drafts, steps):
    import torch
    dev = torch.device("cuda:0")
    model = loop.Model(dev)
    g = torch.Generator(device=dev).manual_seed(batch)
    prompts = torch.randint(0, loop.VOCAB, (batch, prompt), generator=g, dtype=torch.int32, device=dev)
    tokens, seq_len = loop.generate(model, prompts, steps, drafts, 0.0)
    lengths = seq_len.tolist()
    assert all(prompt + steps <= n <= prompt + steps * (drafts + 1) for n in lengths)
    # the finished sequences as one packed batch of prompts
    cache = loop.Cache(batch, max(lengths), dev)
    packed = torch.cat([tokens[b, :n - 1] for b, n in enumerate(lengths)])
    logits, plan = loop.target_pass(model, cache, packed, torch.zeros_like(seq_len), seq_len - 1, packed.numel())
    for b, n in enumerate(lengths):
        at = int(plan.cu_new[b])
        said = logits[at + prompt - 1:at + n - 1]           # what follows each token from the prompt's last on
        chosen = said.gather(1, tokens[b, prompt:n, None].long())[:, 0]
        # queries, keys, probabilities and results are bfloat16: ties may fall either way
        assert bool((chosen >= said.amax(1) - 2 ** -6 * said.abs().amax(1)).all())


def test_sampling_runs_and_gives_pages_back(loop):
    import torch
    dev = torch.device("cuda:0")
    prompts = torch.randint(0, loop.VOCAB, (5, 20), dtype=torch.int32, device=dev)
    tokens, seq_len = loop.generate(loop.Model(dev), prompts, 10, 3, 1.0)
    assert bool((tokens[:, :20] == prompts).all())
    assert all(30 <= n <= 60 for n in seq_len.tolist())
    held = loop.Cache(4, 64, dev)
    five = torch.full((4,), 5, dtype=torch.int32, device=dev)
    held.plan(five * 0, five * 7, 140)
    assert held.page_count.tolist() == [3] * 4 and held.free_count.tolist() == [4]
    held.plan(five, five * 0, 0)
    assert held.page_count.tolist() == [1] * 4 and held.free_count.tolist() == [12]
