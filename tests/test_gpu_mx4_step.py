"""A decoding loop over the 4-bit cache as it would be used: tables, head norms and rotary positions with the
cache write, attention, step after step, drafts rejected in between; eager and captured. Each step's rows
are held to the formulas and its attention to the one in 64 bits over the codes that are in the cache, with
the tolerances that test_gpu_mx4_cache.py and test_gpu_mx4_attn.py derive."""
import numpy as np
import pytest
import torch

import mx4_reference as M
from test_gpu_mx4_attn import check as check_attention
from test_gpu_mx4_cache import D, built, check_codes, check_rows, normed  # noqa: F401 (built: a fixture)
from test_gpu_rope import exact
from test_paged_step_abi import frequencies

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,P,prompts,graph", [((6, 1), 16, [300, 1, 47], False),
                                                   ((24, 4), 64, [130, 64, 5], True),
                                                   ((6, 1), 32, [1100], True)],
                         ids=["rank", "model_graph", "one_graph"])
def test_decoding_steps(heads, P, prompts, graph):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    Hq, Hkv = heads
    n, q_len, steps = len(prompts), 4, 5
    mp = -(-(max(prompts) + (steps + 2) * q_len) // P)
    num_pages = n * mp + 3
    rng = np.random.default_rng(P)
    g = torch.Generator().manual_seed(P)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")

    def i32(x):
        return torch.tensor(np.array(x), dtype=torch.int32, device="cuda")

    def rows(t, h):
        return (torch.randn((t, h, D), generator=g) * 3).to(torch.float16).cuda()
    tables = B.PagedTables(n, P, mp, num_pages, mp * P, max(sum(prompts), n * q_len), status=status)
    rotary = B.Rotary(Hq, Hkv, D, 128, base=500000.0, page_size=P, num_pages=num_pages, status=status)
    cache = B.Mx4Cache(Hkv, D, P, num_pages, status=status)
    att = B.Mx4Attention(n, q_len, Hq, Hkv, D, P, mp, num_pages, mp * P)
    theta = np.array(frequencies(128, 500000.0, "none", 1.0, 1))
    w = (1 + 0.3 * torch.randn((2, D), generator=g)).to(torch.float16).cuda()
    norm = B.HeadNorm(w[0], w[1], 1e-5)
    kp, vp = cache.empty()
    for pool in (kp, vp):  # pages come back from other requests with whatever they held
        pool.copy_(torch.randint(0, 256, pool.shape, generator=g, dtype=torch.uint8))
    free, head = i32(rng.permutation(num_pages)), i32([0])
    table, held, cached, new = i32(np.full((n, mp), -1)), i32([0] * n), i32([0] * n), i32(prompts)
    out = tables.empty()

    def check_written(q, k, v, q_out, T):
        pos, slots = (x[:T].cpu().numpy() for x in (out.positions, out.slots))
        check_rows(q_out, *exact(normed(q, w[0], 1e-5, 0.0), pos, theta, 1.0, 128, "half"), torch.float16)
        check_codes(kp, slots, *exact(normed(k, w[1], 1e-5, 0.0), pos, theta, 1.0, 128, "half"))
        codes, s = M.quantise(v.double().cpu().numpy())
        got_codes, got_s = M.get(vp.cpu().numpy(), slots, True)
        assert np.array_equal(got_codes, codes) and np.array_equal(got_s, s)
        back = cache.read(kp, vp, out.slots[:T], dtype=torch.bfloat16)
        for x, pool, of_v in zip(back, (kp, vp), (False, True)):
            assert np.array_equal(x.double().cpu().numpy(), M.numbers(*M.get(pool.cpu().numpy(), slots, of_v)))

    # the prompts, packed; their last rows attend as a step does
    T0 = sum(prompts)
    q, k, v = rows(T0, Hq), rows(T0, Hkv), rows(T0, Hkv)
    tables(cached, new, held, free, head, table, out=out)
    q_out = rotary.mx4_write(q, k, v, out.positions[:T0], out.slots[:T0], kp, vp, norm=norm)
    torch.cuda.synchronize()
    check_written(q, k, v, q_out, T0)
    lens = np.array(prompts)
    held.copy_(out.held_pages)
    head.copy_(out.free_head)

    T = n * q_len
    new.fill_(q_len)
    cached.copy_(i32(lens))
    sq, sk, sv = rows(T, Hq), rows(T, Hkv), rows(T, Hkv)
    step_q = torch.zeros((n, q_len, Hq, D), dtype=torch.float16, device="cuda")
    step_out, step_lse = torch.zeros_like(step_q), torch.zeros(step_q.shape[:3], device="cuda")

    def step():
        tables(cached, new, held, free, head, table, out=out)
        rotary.mx4_write(sq, sk, sv, out.positions[:T], out.slots[:T], kp, vp, q_out=step_q.view(T, Hq, D),
                         norm=norm, token_starts=out.token_starts)
        att(step_q, kp, vp, table, out.context_lens, out=step_out, lse=step_lse)
    replay = step
    if graph:
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
    for s in range(steps):
        if s:
            lens = lens - rng.integers(0, q_len, n)  # some of the last block were rejected
        cached.copy_(i32(lens))
        for x, h in ((sq, Hq), (sk, Hkv), (sv, Hkv)):
            x.copy_(rows(T, h))
        was = kp.clone(), vp.clone()
        replay()
        lens = lens + q_len
        torch.cuda.synchronize()
        assert np.array_equal(out.context_lens.cpu().numpy(), lens)
        check_written(sq, sk, sv, step_q.view(T, Hq, D), T)
        slots = out.slots[:T].cpu().numpy()
        other = np.setdiff1d(np.arange(num_pages * P), slots)
        for pool, old, of_v in ((kp, was[0], False), (vp, was[1], True)):  # nothing but these slots changed
            for a, b in zip(M.get(pool.cpu().numpy(), other, of_v), M.get(old.cpu().numpy(), other, of_v)):
                assert np.array_equal(a, b)
        pr = dict(q=step_q.cpu().numpy(), k=kp.cpu().numpy(), v=vp.cpu().numpy(),
                  table=table.cpu().numpy(), lens=lens, P=P)
        used = np.unique(pr["table"][pr["table"] >= 0])
        pr["v"][np.setdiff1d(np.arange(num_pages), used)] = 0  # (the tolerance takes V's largest block)
        for b in range(n):
            behind = int(lens[b])
            for j in range(behind, -(-behind // 16) * 16):
                c = pr["v"].reshape(-1, Hkv, 2176)[pr["table"][b, j // P] * (P // 16) + j % P // 16]
                c[:, 2048 + 8 * (j % 16):2056 + 8 * (j % 16)] = 0
            for j in range(-(-behind // 16) * 16, mp * P, 16):
                if pr["table"][b, j // P] >= 0:
                    pr["v"].reshape(-1, Hkv, 2176)[pr["table"][b, j // P] * (P // 16) + j % P // 16] = 0
        check_attention((step_out, step_lse), pr)
        held.copy_(out.held_pages)
        head.copy_(out.free_head)
    assert int(status[0].item()) == 0 and att.read_flags() == 0
