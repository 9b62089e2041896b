"""A small decoder that drafts a tree of tokens and verifies it, every round through the library's operators.

Per request and round: N chains of K drafts behind the last emitted token are one tree of 1 + N K new tokens.  In
every layer ``kv_append`` rotates them to their depths and puts their keys and values into the paged cache, and
``paged_attention`` lets each attend to the context and its own chain; ``process_logits`` shapes the logits of every
drafted position by what the request has produced so far and by a grammar; ``verify_multi`` picks a chain and how
far it holds; ``kv_keep`` moves its entries up behind the context.  The weights are random and the draft model is
the target without its layers: the point is the plumbing.

    python examples/speculative_round.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_rejection_verify_gb300 as sv  # noqa: E402

BF16 = torch.bfloat16


class Decoder:
    """Random weights: an embedding, `layers` attention layers with grouped heads, and a head."""

    def __init__(self, V=512, layers=2, q_heads=8, heads=2, D=64, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.V, self.layers, self.Hq, self.H, self.D, self.dev = V, layers, q_heads, heads, D, device
        E = q_heads * D
        rand = lambda *shape: (torch.randn(shape, generator=g, device=device) / shape[-1] ** 0.5).to(BF16)  # noqa: E731
        self.embed, self.head = torch.randn((V, E), generator=g, device=device).to(BF16), rand(V, E)
        self.qkv = [rand((q_heads + 2 * heads) * D, E) for _ in range(layers)]
        self.proj = [2 * rand(E, E) for _ in range(layers)]
        angle = torch.arange(4096, device=device).double()[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device=device).double() / D)
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def cache(self, num_pages, page=16):
        """Keys and values of all layers, [layers, pages, page, heads, D]."""
        return [torch.zeros((self.layers, num_pages, page, self.H, self.D), dtype=BF16, device=self.dev) for _ in range(2)]

    def forward(self, tokens, k, v, pages, ctx_len, positions=None, mask=None, t_per_row=None):
        """Logits [B, T, V] in fp32 of new tokens [B, T], whose keys and values go into the cache."""
        x = self.embed[tokens.long()]
        B, T, E = x.shape
        for i in range(self.layers):
            h = torch.nn.functional.layer_norm(x.float(), (E,)).to(BF16)
            y = (h @ self.qkv[i].T).view(B, T, self.Hq + 2 * self.H, self.D)
            q = sv.kv_append(y[:, :, :self.Hq], y[:, :, self.Hq:self.Hq + self.H], y[:, :, self.Hq + self.H:], k[i], v[i], pages,
                             ctx_len, self.cos, self.sin, t_per_row, positions=positions)
            a = sv.paged_attention(q, k[i], v[i], pages, ctx_len, t_per_row, mask=mask)
            x = x + (a.view(B, T, E) @ self.proj[i].T)
        return self.logits_of(x)

    def logits_of(self, x):
        h = torch.nn.functional.layer_norm(x.float(), x.shape[-1:]).to(BF16)
        return (h @ self.head.T).float() * 3

    def draft_logits(self, tokens):
        """The draft model's logits [rows, V] behind each token: the model without its layers."""
        return self.logits_of(self.embed[tokens.long()])


def tree(N, K, device):
    """Depth and attention bits of a root and N chains of K tokens."""
    depth, bits = [0], [1]
    for n in range(N):
        for j in range(K):
            depth.append(j + 1)
            bits.append(1 | sum(1 << (1 + n * K + i) for i in range(j + 1)))
    return (torch.tensor(depth, dtype=torch.int32, device=device),
            torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64, device=device))


def generate(model, prompts, rounds=6, N=3, K=4, temperature=0.0, presence=0.5, forbidden=(), seed=1, page=16):
    """Decode `rounds` rounds behind prompts [B, P]; returns the tokens of every request (prompt included), the
    accepted counts [rounds, B] and the cache (k, v, pages, ctx_len)."""
    dev, V = model.dev, model.V
    B, P = prompts.shape
    T = 1 + N * K
    i32 = dict(dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(seed)
    max_pages = -(-(P + rounds * (K + 1) + T) // page)
    k, v = model.cache(B * max_pages, page)
    pages = torch.randperm(B * max_pages, generator=g, device=dev).view(B, max_pages).to(torch.int32)
    ctx = torch.zeros(B, **i32)
    for t in range(0, P - 1, sv.decode.MAX_NEW):  # all but the last prompt token, which is the first root
        part = prompts[:, t:min(t + sv.decode.MAX_NEW, P - 1)].contiguous()
        model.forward(part, k, v, pages, ctx)
        ctx += part.shape[1]
    # a grammar that forbids some tokens everywhere: words of allowed tokens
    allowed = torch.ones(V, dtype=torch.bool, device=dev)
    allowed[list(forbidden)] = False
    bits = allowed.view(-1, 32).long() << torch.arange(32, device=dev)
    words = bits.sum(1)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).expand(B * N, K + 1, -1).contiguous()

    history = torch.zeros((B, P + rounds * (K + 1) + 1), **i32)
    history[:, :P] = prompts
    length = torch.full((B,), P, **i32)
    prompt_len = torch.full((B * N,), P, **i32)
    per_chain = lambda x: x.repeat_interleave(N, 0).contiguous()  # noqa: E731
    depth, seen = tree(N, K, dev)
    mask = seen.expand(B, T).contiguous()
    accepted = []
    for _ in range(rounds):
        root = history.gather(1, (length - 1).long()[:, None])  # [B, 1]
        # drafts: every chain samples its own tokens from the draft model
        draft = torch.empty((B, N, K), **i32)
        q = torch.empty((B, N, K, V), device=dev)
        last = per_chain(root).view(-1)
        for j in range(K):
            z = model.draft_logits(last)
            q[:, :, j] = z.view(B, N, V)
            u = torch.rand(B * N, generator=g, device=dev)
            last, _ = sv.sample(z, u, temperature=1.0)
            draft[:, :, j] = last.view(B, N)
        tokens = torch.cat([root, draft.view(B, N * K)], 1)
        logits = model.forward(tokens, k, v, pages, ctx, positions=(ctx[:, None] + depth).contiguous(), mask=mask)
        # position 0 of every chain is the root's row
        rows = torch.cat([logits[:, None, :1].expand(B, N, 1, V), logits[:, 1:].view(B, N, K, V)], 2).reshape(B * N, K + 1, V)
        p = sv.process_logits(rows, history=per_chain(history), history_len=per_chain(length), prompt_len=prompt_len,
                              draft=draft.view(B * N, K), presence=torch.full((B * N,), presence, device=dev), mask=words)
        uniform = None if temperature == 0 else torch.rand((B, N, K), generator=g, device=dev)
        resample = None if temperature == 0 else torch.rand(B, generator=g, device=dev)
        out, n_acc, chain, _ = sv.verify_multi(p.view(B, N, K + 1, V), None if temperature == 0 else q, draft, uniform, resample,
                                               temperature=temperature, draft_temperature=None if temperature == 0 else 1.0)
        # the root and the accepted drafts stay in the cache; the last emitted token is the next root
        steps = torch.arange(K, **i32)
        path = torch.cat([torch.zeros((B, 1), **i32), 1 + chain.clamp(min=0)[:, None] * K + steps], 1).contiguous()
        kept = n_acc + 1
        sv.kv_keep(k, v, pages, ctx, path, kept)
        at = length[:, None] + torch.arange(K + 1, **i32)
        fresh = torch.arange(K + 1, **i32) <= n_acc[:, None]
        history[torch.arange(B, device=dev)[:, None].expand(B, K + 1)[fresh], at[fresh].long()] = out[fresh]
        ctx = ctx + kept
        length = length + kept
        accepted.append(n_acc)
    done = [history[b, :int(length[b])].tolist() for b in range(B)]
    return done, torch.stack(accepted), (k, v, pages, ctx)


def main():
    model = Decoder()
    g = torch.Generator(device="cuda").manual_seed(3)
    prompts = torch.randint(0, model.V, (4, 100), generator=g, device="cuda", dtype=torch.int32)
    for temperature in (0.0, 1.0):
        done, accepted, _ = generate(model, prompts, temperature=temperature)
        print(f"temperature {temperature}: accepted per round {accepted.float().mean(1).tolist()}")
        for b, tokens in enumerate(done):
            print(f"  request {b}: {tokens[100:]}")


if __name__ == "__main__":
    main()
