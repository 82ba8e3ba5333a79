"""A decoding loop as it would be used: tables, rotary positions with the cache write, attention
over the shared prefix, step after step, drafts rejected in between. Each step's attention is held to
the FP64 oracle over the codes in the cache, and the cache to a model of it kept on the host."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import compare, to_np
from test_gpu_rope import ARITH, D, exact, nearest_ok, v_codes
from test_paged_step_abi import frequencies

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,P,prefix,graph", [((6, 1), 16, 300, False), ((24, 4), 64, 256, True)],
                         ids=["rank", "model_graph"])
def test_decoding_steps(heads, P, prefix, graph):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import binding as B
    Hq, Hkv = heads
    n, q_len, steps = 5, 4, 6
    mp = -(-(prefix + steps * q_len + q_len) // P) + 1
    shared, num_pages = prefix // P, prefix // P + n * mp + 8
    rng = np.random.default_rng(P)
    g = torch.Generator().manual_seed(P)
    free = rng.permutation(num_pages).astype(np.int32)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    tables = B.PagedTables(n, P, mp, num_pages, mp * P, n * max(q_len, prefix - shared * P + q_len),
                           status=status)
    rotary = B.Rotary(Hq, Hkv, D, 128, base=500000.0, page_size=P, num_pages=num_pages,
                      status=status)
    att = B.SharedPrefixAttention(n, q_len, Hq, Hkv, D, P, mp, num_pages, mp * P, prefix)
    theta = np.array(frequencies(128, 500000.0, "none", 1.0, 1))

    def i32(x):
        return torch.tensor(np.array(x), dtype=torch.int32, device="cuda")
    ks, vs = 0.011, 0.013
    k_scale, v_scale = (torch.tensor([s], device="cuda") for s in (ks, vs))
    pool_shape = (num_pages, P, Hkv, D)
    kp, vp = (torch.randint(0, 256, pool_shape, generator=g, dtype=torch.uint8).cuda()
              for _ in range(2))
    free_t, table = i32(free), i32(np.full((n, mp), -1))

    def rows(t, h):
        return torch.randn((t, h, D), generator=g).to(torch.float16).cuda()

    # the prompt's whole pages, written once: one request, alone
    solo = B.PagedTables(1, P, mp, num_pages, mp * P, shared * P, status=status)
    solo_row = i32(np.full((1, mp), -1))
    first = solo(i32([0]), i32([shared * P]), i32([0]), free_t, i32([0]), solo_row)
    rotary.kv_write(rows(shared * P, Hq), rows(shared * P, Hkv), rows(shared * P, Hkv),
                    first.positions, first.slots, k_scale, v_scale, kp, vp)
    prefix_table = solo_row[0, :shared].contiguous()
    prefix_pages, prefix_len = i32([shared]), i32([prefix])

    # every request forks off it: the rest of the prompt (equal in all) and its own tokens
    cached, held, head = i32([shared * P] * n), i32([0] * n), first.free_head.clone()
    new = i32([prefix - shared * P + q_len] * n)
    T0 = int(new.sum().item())
    out = tables.empty()
    q, k, v = rows(T0, Hq), rows(T0, Hkv), rows(T0, Hkv)
    each = T0 // n
    rest = prefix - shared * P
    for x in (k, v):
        x.view(n, each, Hkv, D)[1:, :rest] = x.view(n, each, Hkv, D)[:1, :rest]
    tables(cached, new, held, free_t, head, table, prefix_table, prefix_pages, out=out)
    q_out = rotary.kv_write(q, k, v, out.positions[:T0], out.slots[:T0], k_scale, v_scale, kp, vp)
    lens = np.full(n, prefix + q_len)

    def attend():
        return att(step_q, kp, vp, prefix_table, prefix_len, table, out.context_lens, k_scale,
                   v_scale, out=step_out, lse=step_lse)
    step_q = q_out.view(n, each, Hq, D)[:, rest:].contiguous()
    step_out = torch.empty_like(step_q)
    step_lse = torch.empty(step_q.shape[:3], device="cuda")
    attend()

    def check_attention(what):
        torch.cuda.synchronize()
        want = oracle.load().verify_attn(to_np(step_q), to_np(kp), to_np(vp), to_np(table),
                                         lens.astype(np.int32), float(np.float32(ks)),
                                         float(np.float32(vs)))
        compare(to_np(step_out), to_np(step_lse), *want, what)
    assert np.array_equal(to_np(out.context_lens), lens)
    check_attention("fork")

    new.fill_(q_len)
    T = n * q_len
    sq, sk, sv = rows(T, Hq), rows(T, Hkv), rows(T, Hkv)

    def step():
        tables(cached, new, held, free_t, head, table, prefix_table, prefix_pages, out=out)
        rotary.kv_write(sq, sk, sv, out.positions[:T], out.slots[:T], k_scale, v_scale, kp, vp,
                        q_out=step_q.view(T, Hq, D))
        attend()
    replay = step
    if graph:
        cached.copy_(i32(lens - 1))
        held.copy_(out.held_pages)
        head.copy_(out.free_head)
        before = [x.clone() for x in (table, kp, vp)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        for x, was in zip((table, kp, vp), before):  # the warm-up step did not happen
            x.copy_(was)
        replay = captured.replay
    else:
        held.copy_(out.held_pages)
        head.copy_(out.free_head)
    for s in range(steps):
        lens = lens - rng.integers(0, q_len, n)  # some of the last block were rejected
        cached.copy_(i32(lens))
        for x, h in ((sq, Hq), (sk, Hkv), (sv, Hkv)):
            x.copy_(rows(T, h))
        was = to_np(table).copy()
        replay()
        lens = lens + q_len
        torch.cuda.synchronize()
        assert np.array_equal(to_np(out.context_lens), lens)
        assert np.array_equal(to_np(out.positions[:T]).reshape(n, q_len),
                              lens[:, None] - q_len + np.arange(q_len))
        now = to_np(table)
        assert (now[was >= 0] == was[was >= 0]).all()  # pages stay where they are
        # the drafted rows are in the cache at their positions, as E4M3 of the rotated values
        pos = to_np(out.positions[:T])
        page = now[np.repeat(np.arange(n), q_len), pos // P]
        at = page.astype(np.int64) * P + pos % P
        assert np.array_equal(at, to_np(out.slots[:T]))
        want_k, mag = exact(sk.double().cpu().numpy(), pos, theta, 1.0, 128, "half")
        assert nearest_ok(kp.cpu().view(-1, Hkv, D)[at], want_k / float(np.float32(ks)),
                          (ARITH * mag + 2.0 ** -23 * np.abs(want_k)) / ks)
        assert np.array_equal(to_np(vp).reshape(-1, Hkv, D)[at], v_codes(sv, vs))
        check_attention(f"step {s}")
        held.copy_(out.held_pages)
        head.copy_(out.free_head)
    own = to_np(table)[:, shared:]
    own = own[own >= 0]
    assert len(own) == len(set(own.tolist())) and not set(own) & set(to_np(prefix_table))
    assert int(status[0].item()) == 0 and att.read_flags() == 0
