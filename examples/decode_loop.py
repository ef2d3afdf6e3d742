"""A decode loop of a small multi-codebook model, every step one CUDA graph.

The model's weights are random; what it shows is how the calls go together.
Per step, for every stream:

    ts_kv_tables        the stream's next position gets a slot (a new block
                        where its last one is full), a stopped stream's blocks
                        go back
    per layer           qkv = x W; ts_kv_append at the slots;
                        ts_paged_attention over the cached tokens; x += out W'
    ts_lm_head_sample   the frame's logits and tokens, EOS and length stops

The block table, lengths and slot maps are shared by all layers, the stops that
the sampler finds in one step are what the tables release in the next, and
nothing goes through the host.

    python examples/decode_loop.py [--streams 8] [--steps 40] [--cache bf16|e4m3]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import codebook_token_sampling_gb300 as ts  # noqa: E402
import workloads  # noqa: E402


class DecodeLoop:
    def __init__(self, streams=8, steps=40, layers=2, heads=8, kv_heads=4, head_dim=64, block_size=16,
                 vocabs=(256, 128, 128), cache="bf16", seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        dim = heads * head_dim
        q = len(vocabs)

        def weight(rows, cols):
            return (torch.randn((rows, cols), device=device, generator=gen) / rows ** 0.5).bfloat16()
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.w_qkv = [weight(dim, dim + 2 * kv_heads * head_dim) for _ in range(layers)]
        self.w_out = [weight(dim, dim) for _ in range(layers)]
        self.w_codebook = weight(dim, q * dim)  # a hidden state per codebook
        self.embed = torch.randn((max(vocabs) + 1, dim), device=device, generator=gen).bfloat16()

        # the frame: rows are (stream, codebook), logits from the LM head;
        # streams end at an EOS of codebook 0 or at caps of their own
        batch, head = workloads.make_lm_head(0, streams=streams, dim=dim, vocabs=vocabs,
                                             eos_ids=[7] + [-1] * (q - 1))
        batch["seed"] = batch["seed"] + np.uint64(seed)
        self.sampler = ts.Sampler(0)
        self.sampler.reserve_kv(streams)
        self.batch = ts.DeviceBatch(batch, device, advance_steps=True,
                                    finish={"max_steps": steps - 5 * (np.arange(streams) % 4),
                                            "pad_id": max(vocabs)})
        self.head = ts.LmHead(head, device)

        # one block table for all layers; a cache per layer.  There are blocks for every
        # stream's longest run, so no stream is ever refused one (with fewer, a step
        # would have to look at token_starts for streams that got no token)
        wide = -(-steps // block_size)
        self.n_blocks = streams * wide
        self.tables = ts.KvTables(streams, wide, self.n_blocks, block_size, max_tokens=streams,
                                  finished=self.batch.finish_reason, device=device)
        kind = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[cache]
        shape = (self.n_blocks, kv_heads, block_size, head_dim)  # heads before tokens
        self.x = torch.zeros((streams, dim), dtype=torch.bfloat16, device=device)
        self.qkv = torch.zeros((streams, heads + 2 * kv_heads, head_dim), dtype=torch.bfloat16, device=device)
        self.out = torch.zeros((streams, heads, head_dim), dtype=torch.bfloat16, device=device)
        k_new, v_new = self.qkv[:, heads:heads + kv_heads], self.qkv[:, heads + kv_heads:]
        self.tokens = ts.KvTokens(k_new, v_new, self.tables.slots, self.tables.requests)
        self.query = ts.PagedQuery(self.qkv[:, :heads], self.out, self.tables.block_table, self.tables.lens)
        self.caches = []
        for _ in range(layers):
            k, v = (torch.zeros(shape, dtype=torch.bfloat16, device=device).to(kind).permute(0, 2, 1, 3) for _ in range(2))
            scales = [torch.full((kv_heads,), 0.02, device=device) for _ in range(2)] if cache == "e4m3" else (None, None)
            self.caches.append(ts.KvCache(k, v, *scales))
        self.batch.feedback.fill_(0)

    def step(self):
        """One frame of every stream, queued on the current stream."""
        handle, streams = self.sampler.handle, self.x.shape[0]
        ts.ts_kv_tables(handle, self.tables)
        frame = self.batch.feedback.view(streams, -1).long()
        x = self.embed[frame].float().mean(1).bfloat16()
        for cache, w_qkv, w_out in zip(self.caches, self.w_qkv, self.w_out):
            self.qkv.view(streams, -1).copy_(x @ w_qkv)
            ts.ts_kv_append(handle, cache, self.tokens)
            ts.ts_paged_attention(handle, cache, self.query)
            x = x + self.out.view(streams, -1) @ w_out
        x = x / (x.float().square().mean(1, keepdim=True) + 1e-6).sqrt().bfloat16()
        self.head.hidden.view(torch.bfloat16).view(streams, -1).copy_(x @ self.w_codebook)
        ts.ts_lm_head_sample(handle, self.head, self.batch)

    def capture(self):
        """The step as a CUDA graph (after one warm-up on a side stream, whose
        effects are undone)."""
        state = [self.batch.step, self.batch.stop_step, self.batch.finish_reason, self.batch.feedback, self.tables.lens,
                 self.tables.n_free, self.tables.free_blocks, self.tables.block_table]
        saved = [t.clone() for t in state]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
        torch.cuda.current_stream().wait_stream(side)
        for t, s in zip(state, saved):
            t.copy_(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--streams", type=int, default=8)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    a = ap.parse_args()
    loop = DecodeLoop(streams=a.streams, steps=a.steps, cache=a.cache)
    graph = loop.capture()
    for i in range(a.steps + 1):  # the last call releases what stopped at the cap
        graph.replay()
        if i % 10 == 0 or i == a.steps:
            torch.cuda.synchronize()
            print(f"step {i:3d}  tokens held {loop.tables.lens.tolist()}  free blocks {loop.tables.n_free.item()}"
                  f" of {loop.n_blocks}  finish {loop.batch.finish_reason.tolist()}")
    print(f"status {loop.sampler.read_status()}")


if __name__ == "__main__":
    main()
