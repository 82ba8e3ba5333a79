"""Requests whose newest token stands inside the shared pages: it has no slot in the cache (its K and V are
there, read only), but a query like any other. The rotary call alone, then the tables, the rotary call and the
attention together, held to the FP64 oracle."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import compare, to_np
from test_gpu_rope import D, check, exact, make, rotary

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(np.array(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,heads", [(1, (6, 1)), (40, (24, 4)), (40, (6, 1)), (1501, (2, 3)), (4801, (1, 1))])
@pytest.mark.parametrize("live", [0, 1, 0.6, 1.0])
def test_tokens_without_a_slot_have_a_query_below_the_live_count(T, heads, live, in_place):
    Hq, Hkv = heads
    live = live if isinstance(live, int) else int(T * live)
    q, k, v, pos = make(T, T, Hq, Hkv, torch.float16, 9000)
    pages = -(-T // 16)
    r, theta, amp = rotary(Hq, Hkv, 64, "half", torch.float16, page_size=16, num_pages=pages)
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * 16, generator=g)[:T]
    slots[::3] = -1
    written = np.zeros(pages * 16, bool)
    written[slots[slots >= 0].numpy()] = True
    one = torch.ones(1, device="cuda")

    def run(**kw):
        pools = [torch.full((pages, 16, Hkv, D), 7, dtype=torch.uint8, device="cuda") for _ in range(2)]
        src = q.clone()
        qo = src if in_place else torch.full((T, Hq, D), 5.0, dtype=torch.float16, device="cuda")
        r.kv_write(src, k, v, pos, slots.cuda(), one, one, *pools, q_out=qo, **kw)
        return [qo] + pools
    without = run()
    got = run(token_starts=i32([0, live // 2, live]))
    for a, b in zip(got[1:], without[1:]):  # the pools do not depend on it
        assert torch.equal(a, b)
        assert (a.view(-1, Hkv, D)[torch.from_numpy(~written).cuda()] == 7).all()
    rotated = (slots >= 0).numpy() | (np.arange(T) < live)
    want, mag = exact(q.double().cpu().numpy(), pos.cpu().numpy(), theta, amp, 64, "half")
    check(got[0][rotated], want[rotated], mag[rotated], torch.float16, 64)
    left = q[~rotated] if in_place else torch.full_like(q[~rotated], 5.0)
    assert torch.equal(got[0][~rotated], left)
    assert r.read_flags() == 0


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("kernel", [1, 2], ids=["rows", "pairs"])
@pytest.mark.parametrize("heads,P", [((6, 1), 16), ((24, 4), 48)])
def test_a_step_of_all_three(heads, P, kernel, graph):
    """One new token each: prompts that are all in the shared pages (one of them a single token), one that
    ends with them, and ones that go past them."""
    from speculative_verify_paged_e4m3_gb300 import binding as B
    Hq, Hkv = heads
    shared, n = 9, 6
    S = shared * P
    cached = [S - 1, 0, S // 2, S, S + 5, P - 1]
    mp, num_pages = shared + 3, shared + 40
    rng = np.random.default_rng(P)
    free = rng.permutation(num_pages)
    prefix_table, free_t = i32(free[:shared]), i32(free[shared:])
    # rows hold the shared pages that they need, and pages of their own past them
    table = np.full((n, mp), -1)
    held = [-(-c // P) for c in cached]
    used = shared
    for b in range(n):
        for lp in range(held[b]):
            if lp < shared:
                table[b, lp] = free[lp]
            else:
                table[b, lp], used = free[used], used + 1
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    tables = B.PagedTables(n, P, mp, num_pages, mp * P, n + 3, status=status)
    rot = B.Rotary(Hq, Hkv, D, 128, page_size=P, num_pages=num_pages, status=status)
    att = B.SharedPrefixAttention(n, 1, Hq, Hkv, D, P, mp, num_pages, mp * P, S, kernel=kernel)
    g = torch.Generator().manual_seed(P)
    shape = (num_pages, P, Hkv, D)
    ks, vs = 0.011, 0.013
    pools = [(torch.randn(shape, generator=g) / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
             .cuda() for s in (ks, vs)]
    before = [p.clone() for p in pools]
    # as many rows as positions and slots: the last three are padding
    q, k, v = (torch.randn((n + 3, h, D), generator=g).half().cuda() for h in (Hq, Hkv, Hkv))
    k_scale, v_scale = (torch.tensor([s], device="cuda") for s in (ks, vs))
    table_t, prefix_pages, prefix_len = i32(table), i32([shared]), i32([S])
    cached_t, new, held_t, head = i32(cached), i32([1] * n), i32(held), i32([used - shared])
    t = tables.empty()
    q_out = torch.full_like(q, float("nan"))  # whatever was there
    out = torch.empty((n, 1, Hq, D), dtype=torch.float16, device="cuda")
    lse = torch.empty((n, 1, Hq), device="cuda")

    def step():
        tables(cached_t, new, held_t, free_t, head, table_t, prefix_table, prefix_pages, out=t)
        rot.kv_write(q, k, v, t.positions, t.slots, k_scale, v_scale, *pools, q_out=q_out,
                     token_starts=t.token_starts)
        att(q_out[:n].view(n, 1, Hq, D), *pools, prefix_table, prefix_len, table_t, t.context_lens, k_scale,
            v_scale, out=out, lse=lse)
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        for p, was in zip(pools, before):
            p.copy_(was)
        q_out.fill_(float("nan"))
        table_t.copy_(i32(table))
        captured.replay()
    else:
        step()
    torch.cuda.synchronize()
    slots = to_np(t.slots)
    assert [s < 0 for s in slots] == [c < S for c in cached] + [True] * 3
    assert np.array_equal(to_np(t.positions), cached + [0] * 3)
    assert torch.isnan(q_out[n:]).all()  # padding is left as it was
    for p, was in zip(pools, before):  # nothing but the new tokens' rows has changed, none of them shared
        same = (p == was).view(-1, Hkv * D).all(1).cpu().numpy()
        assert set(np.flatnonzero(~same)) <= set(slots[slots >= 0])
    lens = np.array(cached, dtype=np.int32) + 1
    qr, _ = rot.apply(q[:n], None, t.positions[:n])
    want = oracle.load().verify_attn(to_np(qr).reshape(n, 1, Hq, D), to_np(pools[0]), to_np(pools[1]),
                                     to_np(table_t), lens, float(np.float32(ks)), float(np.float32(vs)))
    compare(to_np(out), to_np(lse), *want)
    assert int(status[0].item()) == 0


def test_refusals_of_the_token_starts():
    r, _, _ = rotary(6, 2, 64, "half", torch.float16, page_size=16, num_pages=2)
    q, k, v, pos = make(8, 4, 6, 2, torch.float16, 9)
    pools = [torch.zeros((2, 16, 2, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    one, slots = torch.ones(1, device="cuda"), torch.arange(4, device="cuda")
    for bad in (i32([0, 4]).long(), i32([0, 4]).cpu(), i32([]), i32([0, 1, 2, 3])[::2]):
        with pytest.raises(ValueError):
            r.kv_write(q, k, v, pos, slots, one, one, *pools, token_starts=bad)
