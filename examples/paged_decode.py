"""Speculative decoding with a paged 8-bit key/value cache: draft, score in one pass, verify, go on.

    python examples/paged_decode.py [--batch 8] [--draft 4] [--rounds 32] [--greedy]

The target is one attention layer with random weights between an embedding and its transpose, small enough to read but
with the real flow of a serving loop: each round feeds K + 1 tokens a sequence (the last emitted one and K drafted ones),
stores their keys and values with `spec_kv_append`, attends over everything stored with `spec_kv_attention`, and hands
the logits of the K + 1 positions to `spec_verify`.  Rejected tokens are dropped by moving the length back; the next
round writes over them.  The draft is the same model with noise on its logits, drawn from with `spec_sample_draft`;
it is stateless (it sees the last token alone), so that the cache is the target's only.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_sampling_verification_spec_gb300 as sv  # noqa: E402


def angles(positions, rot_dim, device, base=10000.0):
    """The cos_sin table of spec_kv_append: [positions, rot_dim], cosines then sines."""
    inv = base ** (-torch.arange(rot_dim // 2, device=device, dtype=torch.float64) / (rot_dim // 2))
    a = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float().contiguous()


class Target:
    """Embedding, one attention layer over a paged cache, unembedding.  dtype: bfloat16 or float32."""

    def __init__(self, vocab=512, heads=8, kv_heads=2, head_dim=64, batch=8, max_tokens=512, page_size=16,
                 dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        d = heads * head_dim

        def w(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[0] ** -0.5).to(dtype)

        self.vocab, self.heads, self.kv_heads, self.head_dim = vocab, heads, kv_heads, head_dim
        self.embed = torch.randn(vocab, d, generator=g, device=device).to(dtype)
        self.wqkv, self.wo = w(d, (heads + 2 * kv_heads) * head_dim), w(d, d)
        self.unembed = w(d, vocab)
        # every sequence owns the pages its table names; which ones they are does not matter
        pages = -(-max_tokens // page_size)
        self.table = torch.randperm(batch * pages, generator=g, device=device).to(torch.int32).view(batch, pages)
        self.cache = sv.PagedKVCache.empty(batch * pages, page_size, kv_heads, head_dim, device)
        self.cos_sin = angles(pages * page_size, head_dim, device)

    def __call__(self, tokens, seq_lens, new_lens=None):
        """tokens [B, T] at positions seq_lens[b] + t -> logits [B, T, vocab] (float32)."""
        B, T = tokens.shape
        h, k, d = self.heads, self.kv_heads, self.head_dim
        x = self.embed[tokens.long()]
        qkv = (x @ self.wqkv).view(B, T, h + 2 * k, d)
        q, keys, values = qkv[:, :, :h], qkv[:, :, h:h + k], qkv[:, :, h + k:]      # views: strides of the fused product
        q = sv.spec_kv_append(q, keys, values, self.cache, self.table, seq_lens, new_lens, cos_sin=self.cos_sin)
        y = sv.spec_kv_attention(q, self.cache, self.table, seq_lens, new_lens)
        return ((x + y.reshape(B, T, h * d) @ self.wo) @ self.unembed).float()

    def draft(self, tokens, noise):
        """Logits of a draft that sees the last token alone: [B, vocab] float32."""
        x = self.embed[tokens.long()]
        return ((x + (x @ self.wqkv[:, :x.shape[-1]]) @ self.wo) @ self.unembed).float() + noise


def decode(target, first, K, rounds, greedy=False, temperature=1.0, seed=0):
    """Rounds of speculative decoding from the first tokens [B]: (tokens emitted, [B, n] with -1 past each sequence's
    own, accepted counts [rounds, B])."""
    dev, B = first.device, first.shape[0]
    g = torch.Generator(device=dev).manual_seed(seed)
    prm = dict(greedy=greedy, temperature=temperature)
    seq = torch.zeros(B, dtype=torch.int32, device=dev)
    last = first.to(torch.int32)
    emitted = torch.full((B, rounds * (K + 1)), -1, dtype=torch.int32, device=dev)
    count = torch.zeros(B, dtype=torch.int64, device=dev)
    accepted = []
    slot = torch.arange(K + 1, device=dev)
    for _ in range(rounds):
        tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
        drafts = torch.empty((B, K, target.vocab), device=dev)
        tokens[:, 0] = last
        for j in range(K):
            noise = torch.randn(B, target.vocab, generator=g, device=dev) * 0.3
            drafts[:, j] = target.draft(tokens[:, j], noise)
            u = None if greedy else torch.rand(B, 1, generator=g, device=dev, dtype=torch.float64)
            tokens[:, j + 1:j + 2] = sv.spec_sample_draft(drafts[:, j:j + 1], u, **prm)
        logits = target(tokens, seq)                     # K + 1 positions in one pass over the cache
        u = None if greedy else torch.rand(B, K + 1, generator=g, device=dev, dtype=torch.float64)
        out, n = sv.spec_verify(logits, None if greedy else drafts, tokens[:, 1:], u, **prm)
        keep = slot[None, :] <= n[:, None]
        at = torch.where(keep, count[:, None] + slot, emitted.shape[1] - 1)
        emitted.scatter_(1, at, torch.where(keep, out, emitted.gather(1, at)))
        last = out.gather(1, n.clamp(min=0).long()[:, None])[:, 0]
        seq = seq + n + 1                                # the rejected tokens' slots are written over next time
        count = count + n + 1
        accepted.append(n)
    return emitted, torch.stack(accepted)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--draft", type=int, default=4, help="drafted tokens a round")
    ap.add_argument("--rounds", type=int, default=32)
    ap.add_argument("--greedy", action="store_true")
    a = ap.parse_args()
    target = Target(batch=a.batch, max_tokens=a.rounds * (a.draft + 1) + a.draft + 1)
    first = torch.arange(a.batch, device="cuda", dtype=torch.int32) % target.vocab
    tokens, accepted = decode(target, first, a.draft, a.rounds, greedy=a.greedy)
    n = accepted.float().mean().item()
    print("%d sequences, %d rounds: %.2f of %d drafted tokens accepted, %.2f tokens a round" % (
        a.batch, a.rounds, n, a.draft, n + 1))
    print("first sequence:", tokens[0][tokens[0] >= 0][:16].tolist())
    print("cache: %.1f KB for %d positions" % (target.cache.nbytes() / 1024, a.batch * target.table.shape[1] * 16))


if __name__ == "__main__":
    main()
