"""The example that runs the decode-step operators together: greedy rounds emit what the model would, and the cache
they leave is the one that decoding the same tokens one after the other leaves."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("speculative_round", os.path.join(ROOT, "examples", "speculative_round.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def prompts(model, B, P):
    g = torch.Generator(device="cuda").manual_seed(3)
    return torch.randint(0, model.V, (B, P), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("N,K,P", [(3, 4, 100), (1, 5, 40), (4, 15, 17), (2, 1, 2)])
def test_greedy_rounds_emit_the_models_tokens(N, K, P):
    ex = load()
    model = ex.Decoder()
    presence, forbidden = 0.5, (3, 64, 200, 511)
    x = prompts(model, 4, P)
    done, accepted, (k, v, pages, ctx) = ex.generate(model, x, rounds=5, N=N, K=K, presence=presence, forbidden=forbidden)
    assert accepted.max() <= K
    for b, tokens in enumerate(done):
        assert len(tokens) == P + int((accepted[:, b] + 1).sum()) and int(ctx[b]) == len(tokens) - 1
        # the same tokens one chunk after the other, through a cache of their own
        seq = torch.tensor([tokens[:-1]], dtype=torch.int32, device="cuda")
        n = seq.shape[1]
        k1, v1 = model.cache(-(-n // 16))
        table = torch.arange(-(-n // 16), dtype=torch.int32, device="cuda")[None]
        logits = []
        for t in range(0, n, 64):
            part = seq[:, t:t + 64].contiguous()
            logits.append(model.forward(part, k1, v1, table, torch.tensor([t], dtype=torch.int32, device="cuda")))
        z = torch.cat(logits, 1)[0]
        for i in range(P - 1, n):
            row = z[i].clone()
            made = torch.tensor(sorted(set(tokens[P:i + 1])), dtype=torch.long, device="cuda")
            row[made] -= presence
            row[list(forbidden)] = -float("inf")
            # bf16 products of other shapes may round otherwise: the emitted token is the best or as good
            assert row[tokens[i + 1]] >= row.max() - 0.05, (b, i)
        slots = torch.arange(n, device="cuda")
        for mine, other in ((k, k1), (v, v1)):
            a = mine[:, pages[b].long()[slots // 16], slots % 16].float()
            c = other[:, slots // 16, slots % 16].float()
            assert (a - c).abs().max() <= 0.06 * c.abs().max()


def test_sampled_rounds_run():
    ex = load()
    model = ex.Decoder()
    done, accepted, _ = ex.generate(model, prompts(model, 3, 30), rounds=4, temperature=1.0, forbidden=(7,))
    assert accepted.shape == (4, 3) and all(7 not in t[30:] for t in done)
