"""The decode loop example: tables, cache writes, attention, LM head and sampler
in one captured step."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decode_loop
    finally:
        sys.path.pop(0)
    return decode_loop


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_replayed_steps_equal_the_calls(example, cache):
    """Every step's tokens, stops, lengths and free blocks: graph replays against
    plain calls; a stream's length follows its steps until it ends, and in the
    end all blocks are free again, each once."""
    import torch
    steps = 37
    runs = []
    for replay in (False, True):
        loop = example.DecodeLoop(streams=6, steps=steps, cache=cache, seed=3)
        step = loop.capture().replay if replay else loop.step
        seen = []
        for _ in range(steps + 2):
            step()
            seen.append([t.clone() for t in (loop.batch.out_ids, loop.batch.finish_reason, loop.tables.lens,
                                             loop.tables.n_free)])
        torch.cuda.synchronize()
        assert loop.sampler.read_status() == 0
        assert loop.tables.n_free.item() == loop.n_blocks
        assert sorted(loop.tables.free_blocks.tolist()) == list(range(loop.n_blocks))
        runs.append(seen)
    for a, b in zip(*runs):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    done = torch.zeros(6, dtype=torch.bool, device="cuda")
    for i, (_, finish, lens, _) in enumerate(runs[0]):
        assert torch.equal(lens, torch.where(done, 0, i + 1).int())
        done = finish > 0
    assert bool(done.all()) and len({int(r[1].sum()) for r in runs[0]}) > 2  # they end one after another


def test_attention_is_over_the_streams_own_tokens(example):
    """One layer's cache, read back through the block table: a running stream's
    first layer output is the attention over exactly its own frames so far."""
    import torch
    loop = example.DecodeLoop(streams=4, steps=30, layers=1, seed=5)
    keys, values = [], []
    for i in range(21):
        loop.step()
        torch.cuda.synchronize()
        h, kv = loop.heads, loop.kv_heads
        keys.append(loop.qkv[:, h:h + kv].clone())
        values.append(loop.qkv[:, h + kv:].clone())
        running = [s for s in range(4) if int(loop.tables.lens[s]) == i + 1]
        k, v = torch.stack(keys, 1).double(), torch.stack(values, 1).double()  # [stream, token, head, dim]
        q = loop.qkv[:, :h].double().view(4, kv, h // kv, -1)
        p = torch.softmax(torch.einsum("nhgd,nthd->nhgt", q, k) * loop.head_dim ** -0.5, -1)
        want = torch.einsum("nhgt,nthd->nhgd", p, v).reshape(4, h, -1)
        got = loop.out.double()
        for s in running:
            # bf16 outputs of bf16 values: half a unit of 2^-8, and the sums'
            assert bool(((got[s] - want[s]).abs() <= 2.0 ** -8 * want[s].abs() + 2.0 ** -12 * values[0].abs().max()).all())
