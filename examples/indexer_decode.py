"""Decode steps of a sparse-attention indexer, from its queries and keys to the rows that it picked.

Each step of a batch of sequences: rotary positions on the queries and the new keys, the keys
quantised into the paged cache, the queries quantised (their scales folded into the heads'
weights), the scores over the whole cache, the exact top-k of each row as cache slots, and the
picked rows read back in 16 bits. The step is captured into one CUDA graph and replayed with new
inputs. Weights are random: the projections that make q, k and the heads' weights are the model's.

    python examples/indexer_decode.py --batch 64 --context 32768 --steps 20
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_sm_gb300 as fw  # noqa: E402

HEADS, DIM, ROT, PAGE = 64, 128, 64, 64


class Indexer:
    """The buffers of a batch that decodes up to `context` keys a sequence."""

    def __init__(self, batch: int, context: int, k: int, device: str = "cuda"):
        pages = -(-context // PAGE)
        self.batch, self.context, self.k = batch, context, k
        self.freqs, self.scale = fw.indexer_rotary_freqs(ROT, scaling="yarn", factor=4.0, original_len=context,
                                                         device=device)
        self.codes = torch.zeros((batch * pages, PAGE, DIM), dtype=torch.float8_e4m3fn, device=device)
        self.scales = torch.zeros((batch * pages, PAGE, 1), device=device)
        self.page_table = torch.randperm(batch * pages, device=device).view(batch, pages).int()
        self.q = torch.zeros((batch, HEADS, DIM), dtype=torch.bfloat16, device=device)
        self.key = torch.zeros((batch, DIM), dtype=torch.bfloat16, device=device)
        self.weights = torch.zeros((batch, HEADS), device=device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)  # keys before this step
        self.rows = torch.arange(batch, device=device)

    def slots(self, positions: torch.Tensor) -> torch.Tensor:
        """The cache slots of one position of each sequence."""
        page = self.page_table[self.rows, (positions // PAGE).long()]
        return page * PAGE + positions % PAGE

    def prefill(self, keys: torch.Tensor) -> None:
        """Writes keys [batch, n, DIM] at positions 0 .. n-1 of an empty cache."""
        n = keys.shape[1]
        at = torch.arange(n, dtype=torch.int32, device=keys.device)
        turned = fw.indexer_rotary(keys.reshape(-1, DIM), at.repeat(self.batch), self.freqs, start=DIM - ROT,
                                   scale=self.scale)
        slots = self.page_table.repeat_interleave(PAGE, 1)[:, :n] * PAGE + at % PAGE
        fw.indexer_cache_write(turned, slots.reshape(-1).contiguous(), self.codes, self.scales)
        self.lens.fill_(n)

    def step(self):
        """One token of each sequence: (scores, picked slots, their rows). Lengths grow by one."""
        q = fw.indexer_rotary(self.q, self.lens, self.freqs, start=DIM - ROT, scale=self.scale)
        key = fw.indexer_rotary(self.key, self.lens, self.freqs, start=DIM - ROT, scale=self.scale)
        fw.indexer_cache_write(key, self.slots(self.lens), self.codes, self.scales)
        self.lens += 1
        q8, w = fw.indexer_quantise(q, weights=self.weights)
        scores = fw.indexer_scores(q8[:, None], w[:, None], self.codes, self.scales, self.page_table,
                                   self.lens[:, None], self.context)
        picked = fw.topk_transform_paged(scores, self.lens, self.page_table, PAGE, self.k)
        return scores, picked, fw.indexer_cache_read(self.codes, self.scales, picked)


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--context", type=int, default=32768)
    ap.add_argument("--k", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    ix = Indexer(a.batch, a.context, a.k)
    first = a.context - a.steps - 1
    if first < 1:
        ap.error("the context must hold the steps and at least two keys more")
    ix.prefill(torch.randn((a.batch, first, DIM), device="cuda").bfloat16())
    ix.step()  # sets the kernels up on this device
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = ix.step()
    begin, end, spent = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True), []
    for _ in range(a.steps):
        ix.q.normal_()
        ix.key.normal_()
        ix.weights.normal_(std=(HEADS * DIM) ** -0.5)
        begin.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        spent.append(begin.elapsed_time(end) * 1e3)
    if fw.indexer_guard_hits() or fw.topk_guard_hits():
        raise RuntimeError("a slot or a page outside the cache")
    us = sorted(spent)[len(spent) // 2]
    print(f"{a.batch} sequences, {int(ix.lens[0])} keys each, top {a.k}: {us:.1f} us a step")
    scores, picked, rows = held
    return {"indexer": ix, "scores": scores, "picked": picked, "rows": rows, "us": us}


if __name__ == "__main__":
    main()
