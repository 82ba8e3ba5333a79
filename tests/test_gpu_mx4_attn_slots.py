"""The 4-bit attention of batches with more units than SMs, or nearly: one long sequence among short ones, empty ones,
ragged ones, with the slots of one round or of all; one captured call serves both."""
import numpy as np
import pytest
import torch

from test_gpu_mx4_attn import D, built, check, dev, make  # noqa: F401 (built: a fixture)

pytestmark = pytest.mark.gpu


def batch_problem(seed, lens, q_len, Hq, Hkv, P):
    """Sequences with the pages that they need, tables as wide as the longest one's."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int32)
    need = -(-lens // P)
    pages = int(need.sum()) + 2
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(1, int(need.max()))), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    q = rng.standard_normal((len(lens), q_len, Hq, D)).astype(np.float16)
    k, v = (rng.integers(0, 256, (pages, P // 16, Hkv, 2176), dtype=np.uint8) for _ in range(2))
    for pool in (k, v):
        pool[..., 2048:] = rng.integers(124, 127, pool[..., 2048:].shape)
    return dict(q=q, k=k, v=v, table=table, lens=lens, P=P)


def splits(att, lens):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    start, per, act = B.dflash_verify_attn_split_slots(att.plan, [int(n) for n in lens])
    return max(act), int(start[-1])


@pytest.mark.parametrize("batch,heads,q_len,P", [(39, (8, 4), 1, 16), (39, (8, 4), 6, 48), (70, (4, 4), 2, 64),
                                                 (160, (2, 1), 3, 16), (30, (24, 4), 10, 64)])
def test_a_long_sequence_among_many(batch, heads, q_len, P):
    rng = np.random.default_rng(batch + q_len)
    lens = rng.integers(0, 200, batch)
    lens[batch // 2] = 9001
    lens[3] = 0
    pr = batch_problem(batch, lens, q_len, *heads, P)
    att = make(pr)
    longest, used = splits(att, lens)
    assert longest > 8 and used <= att.plan.num_slots
    check(att(*dev(pr)), pr)


@pytest.mark.parametrize("batch,heads,q_len", [(39, (8, 4), 1), (24, (8, 4), 12)])
def test_one_graph_serves_short_and_long_batches(batch, heads, q_len):
    """The rule's choice is made on the device: the slots of one round and of all in the same captured call."""
    rng = np.random.default_rng(7)
    long_lens = rng.integers(1500, 4500, batch)
    short = rng.integers(1, 700, batch)
    one = np.full(batch, 130)
    one[5] = 4499
    pr = batch_problem(3, np.maximum(long_lens, one), q_len, *heads, 16)
    att = make(pr)
    args = dev(pr)
    out, lse = att(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        att(*args, out=out, lse=lse)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att(*args, out=out, lse=lse)
    assert splits(att, short)[1] <= max(att.plan.sm_count // att.plan.row_blocks, batch * heads[1])
    assert splits(att, one)[1] > batch * heads[1]
    for lens in (long_lens, short, one, np.zeros(batch, dtype=int)):
        args[4].copy_(torch.from_numpy(lens.astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        check((out, lse), dict(pr, lens=lens.astype(np.int32)))
