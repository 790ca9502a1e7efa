"""The attention of a decoder layer over a quantized cache, as a server runs it.

Weights and activations of both projections are INT8, the keys and values are
held in 4 bits: ragged prompts first, all in one call, then single tokens for
every sequence, replayed as one CUDA graph.  (Random weights; no position
encoding, which a model would apply to q and k before they are stored.)

    python examples/attention_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import w4a8_int8_quantized_gb300 as w8  # noqa: E402


class Block:
    """x -> fused q, k, v projection -> cache -> attention -> output projection."""

    def __init__(self, hidden=1024, heads=8, kv_heads=2, head_dim=128, page=64, pages=256, bits=4,
                 device="cuda", seed=0):
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        gen = torch.Generator(device).manual_seed(seed)

        def weight(n, k):
            w = torch.randn(n, k, device=device, generator=gen) * k ** -0.5
            return w8.quantize_weight_int8(w.half())

        self.w_qkv = weight((heads + 2 * kv_heads) * head_dim, hidden)
        self.w_out = weight(hidden, heads * head_dim)
        self.cache = w8.KVCache.empty(pages, kv_heads, page, head_dim, bits, device=device)

    def __call__(self, x, slots, table, lens, offsets=None, max_q=None):
        """x [T, hidden]; slots [T]: where each token is stored; table, lens, offsets: the batch."""
        qkv = w8.linear(x, *self.w_qkv).view(x.shape[0], -1, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        w8.kv_cache_write(k, v, slots, self.cache)
        out = w8.kv_cache_attention(q, self.cache, table, lens, q_offsets=offsets, max_q=max_q)
        return w8.linear(out.view(x.shape[0], -1), *self.w_out), qkv


class Pages:
    """Which pages each sequence holds: a table on the host, copied when it changes."""

    def __init__(self, sequences, width, page, pages, seed=0):
        self.page = page
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.table = torch.zeros(sequences, width, dtype=torch.int32)
        self.lens = [0] * sequences

    def append(self, b, n):
        """n more tokens of sequence b: their slots."""
        slots = []
        for t in range(self.lens[b], self.lens[b] + n):
            if t % self.page == 0:
                self.table[b, t // self.page] = self.free.pop()
            slots.append(int(self.table[b, t // self.page]) * self.page + t % self.page)
        self.lens[b] += n
        return slots


def run(prompts=(700, 33, 257, 1), steps=8, device="cuda", **block):
    """Returns the outputs of the prompts and of each step, and every token's q, k, v."""
    blk = Block(device=device, **block)
    page, pages = blk.cache.page_size, blk.cache.num_pages
    B, hidden = len(prompts), blk.w_out[0].shape[0]
    book = Pages(B, -(-(max(prompts) + steps) // page), page, pages)
    gen = torch.Generator(device).manual_seed(1)

    def tokens(n):
        return torch.randn(n, hidden, device=device, dtype=torch.float16, generator=gen)

    slots = torch.tensor(sum((book.append(b, n) for b, n in enumerate(prompts)), []), device=device)
    offsets = torch.tensor([0, *torch.tensor(prompts).cumsum(0).tolist()], dtype=torch.int32, device=device)
    table, lens = book.table.to(device), torch.tensor(book.lens, dtype=torch.int32, device=device)
    out, qkv = blk(tokens(sum(prompts)), slots, table, lens, offsets, max(prompts))
    outs, qkvs = [out], [list(qkv.split(list(prompts)))]

    # a step's inputs live in fixed buffers, so that one captured graph serves every step
    x, slots = tokens(B), torch.full((B,), -1, dtype=torch.int64, device=device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        blk(x, slots, table, lens)  # slot -1: nothing is stored
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, qkv = blk(x, slots, table, lens)
    for _ in range(steps):
        slots.copy_(torch.tensor([book.append(b, 1)[0] for b in range(B)]))
        table.copy_(book.table)
        lens.add_(1)
        x.copy_(tokens(B))
        graph.replay()
        outs.append(out.clone())
        qkvs.append([row.clone() for row in qkv.split(1)])
    status = w8.w8a8_check_status()
    if status:
        raise RuntimeError(w8.w8a8_status_string(status))
    return blk, outs, qkvs


def exact(blk, qkvs):
    """The same outputs with an unquantized cache and 32-bit attention."""
    h, kvh, d = blk.heads, blk.kv_heads, blk.head_dim
    outs = [[] for _ in qkvs]
    for b in range(len(qkvs[0])):
        seq = torch.cat([step[b] for step in qkvs]).float()
        q, k, v = seq.split([h, kvh, kvh], 1)
        k, v = (t.repeat_interleave(h // kvh, 1) for t in (k, v))
        score = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
        score += torch.full_like(score[0], float("-inf")).triu(1)
        o = torch.einsum("hij,jhd->ihd", score.softmax(-1), v).half().reshape(len(seq), -1)
        o = w8.linear(o, *blk.w_out)
        for step, rows in zip(outs, o.split([len(step[b]) for step in qkvs])):
            step.append(rows)
    return [torch.cat(step) for step in outs]


def main():
    for bits in (8, 4):
        blk, outs, qkvs = run(bits=bits)
        want = exact(blk, qkvs)
        held = sum(t.nbytes for t in (blk.cache.k_codes, blk.cache.v_codes, blk.cache.k_scale, blk.cache.v_scale))
        full = 2 * blk.cache.num_pages * blk.cache.page_size * blk.kv_heads * blk.head_dim * 2
        for name, i in (("prompts", 0), ("last step", -1)):
            err = (outs[i].float() - want[i].float()).norm() / want[i].float().norm()
            print(f"{bits}-bit cache ({held / full:.2f} of fp16's bytes), {name}: "
                  f"relative difference from an unquantized cache {err.item():.4f}")


if __name__ == "__main__":
    main()
