"""Verify steps of speculative decoding over one paged pool, every serving operator of the
package in its place:

    KvPages.reserve / fork / free / compact   whose pages, copy on write, roll back
    Kv8Cache.store                            the drafts' K/V into the 8-bit cache
    indexer_k_prologue, indexer_mqa_logits    the indexer's keys and scores
    PagedTopK                                 the positions each query row attends to
    Kv8Cache.attention_selected               attention over their slots
    verify_drafts                             which drafts stand, and one token more

The "model" is one attention layer with random weights and a random output matrix: what
comes out has no meaning, but the data flow is a serving engine's. Two prompts are stored once;
two samples of each share the prompt's pages and grow apart.

    python examples/speculative_step.py [steps]
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sparse_attention_indexer_gb300 import (Kv8Cache, KvPages, PagedTopK, binding as B,  # noqa: E402
                                            verify_drafts)

PAGE, KV_HEADS, Q_HEADS, DIM, INDEX_HEADS, VOCAB = 64, 2, 16, 128, 64, 1000


def i32(x) -> torch.Tensor:
    return torch.as_tensor(x, dtype=torch.int32, device="cuda").contiguous()


class Layer:
    """One attention layer's weights and caches, and the pool of their pages."""

    def __init__(self, sequences: int, max_len: int, gen: torch.Generator):
        width = -(-max_len // PAGE)
        self.pages = sequences * width + 8
        rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.embed = rand(VOCAB, 256)
        self.wk, self.wv = (rand(256, KV_HEADS * DIM) / 16 for _ in range(2))
        self.wq = rand(256, Q_HEADS * DIM) / 16
        self.wi, self.wg = rand(256, INDEX_HEADS * DIM) / 16, rand(256, INDEX_HEADS) / 16
        self.wik = rand(256, DIM) / 16
        self.out = rand(Q_HEADS * DIM, VOCAB) / 16
        self.cache = Kv8Cache.empty(self.pages, PAGE, KV_HEADS, DIM)
        self.index = torch.zeros((self.pages * PAGE, DIM), dtype=torch.uint8, device="cuda")
        self.index_scale = torch.zeros(self.pages * PAGE, device="cuda")
        self.table = torch.full((sequences, width), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(self.pages, dtype=torch.int32, device="cuda")
        self.pool = KvPages(self.table, self.refs, PAGE,
                            self.cache.planes() + [self.index.view(self.pages, -1),
                                                   self.index_scale.view(self.pages, -1)])
        self.ones, self.zeros = torch.ones(DIM, device="cuda"), torch.zeros(DIM, device="cuda")
        angle = torch.arange(max_len, device="cuda")[:, None] * 0.01 ** torch.linspace(
            0, 1, DIM // 4, device="cuda")
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).contiguous()

    def write(self, tokens: torch.Tensor, rows: torch.Tensor, positions: torch.Tensor) -> None:
        """K, V and indexer keys of tokens into their (writable) pages."""
        x = self.embed[tokens.long()]
        k = (x @ self.wk).to(torch.bfloat16).view(-1, KV_HEADS, DIM)
        v = (x @ self.wv).to(torch.bfloat16).view(-1, KV_HEADS, DIM)
        self.cache.store(k, v, positions, rows, self.table)
        B.indexer_k_prologue((x @ self.wik).to(torch.bfloat16), self.ones, self.zeros, 1e-6,
                             positions, self.rope, DIM // 2, rows, self.table, PAGE, self.index,
                             self.index_scale)

    def probabilities(self, tokens: torch.Tensor, rows: torch.Tensor, lens: torch.Tensor,
                      group: int, max_len: int, k: int) -> torch.Tensor:
        """What each token (a query row; `group` consecutive ones of a sequence) predicts,
        attending to its top k positions among the first lens[t]."""
        n = tokens.shape[0]
        x = self.embed[tokens.long()]
        q8 = (x @ self.wi).view(n, INDEX_HEADS, DIM).to(torch.float8_e4m3fn).view(torch.uint8)
        scores = torch.empty((n, -(-max_len // 4) * 4), device="cuda")
        B.indexer_mqa_logits(q8, (x @ self.wg).contiguous(), lens, max_len, group, rows, self.table,
                             PAGE, self.index, self.index_scale, scores)
        top = PagedTopK(n, max_len)
        top.plan(lens)
        slots, _ = top.select(scores, lens, k, self.table, PAGE, rows.repeat_interleave(group))
        q = (x @ self.wq).to(torch.bfloat16).view(n, Q_HEADS, DIM)
        o, _ = self.cache.attention_selected(q, slots, 1 / math.sqrt(DIM))
        if k >= max_len:  # nothing was left out: the dense form gives the same
            dense, _ = self.cache.attention(q, lens, max_len, self.table, 1 / math.sqrt(DIM), group,
                                            rows)
            assert torch.allclose(o.float(), dense.float(), rtol=2e-2, atol=2e-3)
        return torch.softmax(o.view(n, -1).float() @ self.out, -1)


def main(steps: int = 4, prompt: int = 300, drafts: int = 3, k: int = 2048, seed: int = 0) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    samples, max_len = 4, prompt + 40 + steps * (drafts + 1) + 1
    layer = Layer(2 + samples, max_len, gen)
    rand_tokens = lambda *s: torch.randint(0, VOCAB, s, generator=gen, device="cuda",  # noqa: E731
                                           dtype=torch.int32)
    # the prompts, of different lengths
    prompts = i32([0, 1])
    lens = i32([prompt, prompt + 39])
    layer.pool.reserve(prompts, torch.zeros_like(lens), lens)
    for r in (0, 1):
        n = int(lens[r])
        layer.write(rand_tokens(n), i32([r]).expand(n).contiguous(),
                    torch.arange(n, dtype=torch.int32, device="cuda"))
    # two samples of each share its pages; the prompts' own rows are given up
    rows = i32(range(2, 2 + samples))
    lens = lens.repeat_interleave(2).contiguous()
    layer.pool.fork(prompts.repeat_interleave(2).contiguous(), rows, lens)
    layer.pool.free(prompts)
    shared = int((layer.refs > 1).sum())
    last = rand_tokens(samples)
    texts = [last]
    group = drafts + 1
    for _ in range(steps):
        drafted = rand_tokens(samples, drafts)
        fed = torch.cat([last[:, None], drafted], 1)                 # [samples, drafts + 1]
        layer.pool.reserve(rows, lens, lens + group)                 # the shared tail is copied
        at = (lens[:, None] + torch.arange(group, device="cuda", dtype=torch.int32)).contiguous()
        layer.write(fed.view(-1), rows.repeat_interleave(group).contiguous(), at.view(-1))
        p = layer.probabilities(fed.view(-1), rows, (at + 1).view(-1), group, max_len, k)
        u = torch.rand((samples, group), generator=gen, device="cuda")
        # a draft from nowhere: uniform probabilities
        q = torch.full((samples, drafts, VOCAB), 1 / VOCAB, device="cuda")
        tokens, kept = verify_drafts(p.view(samples, group, VOCAB), q, drafted, u)
        lens = lens + kept + 1
        layer.pool.free(rows, lens)                                  # the refused drafts' pages
        last = tokens.gather(1, kept[:, None].long()).squeeze(1).contiguous()
        texts.append(tokens)
    new_ids, counts = layer.pool.compact()
    owners = torch.bincount(layer.table[layer.table >= 0].long(), minlength=layer.pages)
    status = int(layer.pool.status) | int(layer.cache.status)
    return dict(lens=lens.tolist(), shared=shared, live=int(counts[0]), moved=int(counts[1]),
                owners_match=bool(torch.equal(owners.int(), layer.refs)), status=status,
                texts=[t.tolist() for t in texts], layer=layer)


if __name__ == "__main__":
    r = main(int(sys.argv[1]) if len(sys.argv) > 1 else 4)
    print(f"lengths {r['lens']}, {r['shared']} prompt pages shared by samples, {r['live']} pages live, "
          f"{r['moved']} moved by the compaction, counts match the table: {r['owners_match']}, "
          f"status {r['status']}")
