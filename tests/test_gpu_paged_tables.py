"""Paged tables against a plain restatement in Python integers, entry by entry. Whole numbers: no
tolerance."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()


CONTEXT_CLAMPED, PAGE_CLAMPED, EXHAUSTED, DROPPED = 0x1, 0x4, 0x10, 0x20


def reference(c):
    """The header's definition, one request and one token at a time."""
    P, mp = c["P"], c["table"].shape[1]
    table = c["table"].copy()
    shared = min(max(c["prefix_pages"], 0), len(c["prefix"])) if c["prefix"] is not None else 0
    head = max(c["head"], 0)
    left = len(c["free"]) - head
    flags, taken = 0, 0
    ctxs, helds, starts, pos, slots = [], [], [], [], []
    for b in range(len(c["cached"])):
        cached, new = max(int(c["cached"][b]), 0), max(int(c["new"][b]), 0)
        if cached + new > c["max_context"]:
            flags |= CONTEXT_CLAMPED
        ctx = min(cached + new, c["max_context"])
        cached = min(cached, c["max_context"])
        held = min(max(int(c["held"][b]), 0), mp)
        need = max(held, -(-ctx // P))
        first = min(max(shared, held), need)
        got = first
        for q in range(held, first):
            table[b, q] = c["prefix"][q]
        for q in range(first, need):
            if taken < left:
                table[b, q] = c["free"][head + taken]
                got = q + 1
            else:
                table[b, q] = -1
                flags |= EXHAUSTED
            taken += 1
        ctxs.append(ctx)
        helds.append(got)
        starts.append(len(pos))
        for p in range(cached, ctx):
            q = p // P
            slot = -1
            if q >= shared and not (q >= held and table[b, q] == -1 and q >= got):
                page = int(table[b, q])
                if 0 <= page < c["num_pages"]:
                    slot = page * P + p % P
                elif len(pos) < c["max_tokens"]:
                    flags |= PAGE_CLAMPED
            pos.append(p)
            slots.append(slot)
    starts.append(len(pos))
    cap = c["max_tokens"]
    if len(pos) > cap:
        flags |= DROPPED
    return dict(table=table, context_lens=np.array(ctxs), held_pages=np.array(helds),
                free_head=np.array([head + min(taken, max(left, 0))]),
                token_starts=np.minimum(starts, cap),
                positions=np.array((pos + [0] * cap)[:cap]),
                slots=np.array((slots + [-1] * cap)[:cap])), flags


def run(c, tables=None):
    from speculative_verify_paged_e4m3_gb300 import binding as B

    def dev(x):
        return torch.tensor(np.array(x), dtype=torch.int32, device="cuda")
    n, mp = c["table"].shape
    t = tables or B.PagedTables(n, c["P"], mp, c["num_pages"], c["max_context"], c["max_tokens"])
    table = dev(c["table"])
    has = c["prefix"] is not None
    out = t(dev(c["cached"]), dev(c["new"]), dev(c["held"]), dev(c["free"]), dev([c["head"]]),
            table, dev(c["prefix"]) if has else None, dev([c["prefix_pages"]]) if has else None)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in out._asdict().items()}
    got["table"] = table.cpu().numpy()
    return got, t.read_flags()


def case(seed, batch, P, mp, new, prefix=0, max_tokens=None, num_free=None, wild=False):
    rng = np.random.default_rng(seed)
    top = mp * P - rng.integers(0, P)
    cached = rng.integers(0, max(1, top - new) + 1, batch)
    news = rng.integers(0, new + 1, batch)
    held = -(-cached // P) + rng.integers(0, 2, batch)
    num_pages = batch * mp + 50
    perm = rng.permutation(num_pages)
    free = perm[:(batch * (new // P + 2) if num_free is None else num_free)]
    if wild:
        cached[rng.integers(0, batch)] = -5
        news[rng.integers(0, batch)] = -3
        news[rng.integers(0, batch)] = 2 ** 31 - 1
        held[rng.integers(0, batch)] = mp + 9
        held[rng.integers(0, batch)] = -2
    table = rng.integers(0, num_pages, (batch, mp))
    if wild:
        table[rng.integers(0, batch, 3), rng.integers(0, mp, 3)] = num_pages + 1
    return dict(P=P, num_pages=num_pages, max_context=top, cached=cached, new=news, held=held,
                free=free, head=int(rng.integers(0, 3)), table=table,
                prefix=perm[::-1][:prefix].copy() if prefix else None, prefix_pages=prefix,
                max_tokens=max_tokens or max(1, int(batch * new)))


CASES = [
    dict(seed=1, batch=1, P=16, mp=8, new=1),
    dict(seed=2, batch=1, P=16, mp=8, new=0),
    dict(seed=3, batch=3, P=1, mp=40, new=5),
    dict(seed=4, batch=7, P=16, mp=64, new=8),
    dict(seed=5, batch=33, P=48, mp=20, new=333),
    dict(seed=6, batch=65, P=7, mp=50, new=29, prefix=9),
    dict(seed=7, batch=511, P=16, mp=40, new=8),
    dict(seed=8, batch=513, P=16, mp=40, new=17, prefix=40),
    dict(seed=9, batch=1025, P=64, mp=6, new=4),
    dict(seed=10, batch=4096, P=16, mp=12, new=3, prefix=3),
    dict(seed=11, batch=5, P=3296, mp=3, new=5000),
    # more tokens than entries, fewer pages than needed, none at all
    dict(seed=12, batch=40, P=16, mp=30, new=50, max_tokens=100),
    dict(seed=13, batch=40, P=16, mp=30, new=50, num_free=20, prefix=4),
    dict(seed=14, batch=9, P=16, mp=30, new=50, num_free=1),
    dict(seed=15, batch=9, P=16, mp=30, new=50, num_free=0),
    # lengths, held counts and table entries outside their ranges
    dict(seed=16, batch=20, P=16, mp=30, new=40, wild=True),
    dict(seed=17, batch=20, P=16, mp=30, new=40, wild=True, prefix=5, num_free=11),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda k: f"b{k['batch']}_p{k['P']}_s{k['seed']}")
def test_tables(kw):
    c = case(**kw)
    want, flags = reference(c)
    got, got_flags = run(c)
    for k, v in want.items():
        assert np.array_equal(got[k], v), k
    assert got_flags == flags


def test_prefix_pages_cut_to_the_table():
    c = case(30, 4, 16, 10, 20, prefix=3)
    c["prefix_pages"] = 99
    want, _ = reference(c)
    got, _ = run(c)
    assert all(np.array_equal(got[k], v) for k, v in want.items())


def test_a_growing_loop_in_one_graph():
    """A captured step replayed with the lengths of the step before: pages left by rejected drafts
    are used again before new ones, and the free list moves on."""
    from speculative_verify_paged_e4m3_gb300 import binding as B
    n, P, mp, q = 6, 16, 12, 8
    t = B.PagedTables(n, P, mp, 200, mp * P, n * q)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    cached, new, held, head = i32([0] * n), i32([q] * n), i32([0] * n), i32([0])
    free, table, out = i32(list(range(199, -1, -1))), i32([[-1] * mp] * n), t.empty()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        t(cached, new, held, free, head, table, out=out)
    side.synchronize()
    table.fill_(-1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t(cached, new, held, free, head, table, out=out)
    rng = np.random.default_rng(0)
    c = dict(P=P, num_pages=200, max_context=mp * P, cached=np.zeros(n, int), new=np.full(n, q),
             held=np.zeros(n, int), free=np.arange(199, -1, -1), head=0,
             table=np.full((n, mp), -1), prefix=None, prefix_pages=0, max_tokens=n * q)
    for _ in range(15):
        g.replay()
        torch.cuda.synchronize()
        want, _ = reference(c)
        for k, v in want.items():
            got = table if k == "table" else getattr(out, k)
            assert np.array_equal(got.cpu().numpy(), v), k
        accepted = rng.integers(1, q + 1, n)
        c.update(cached=c["cached"] + accepted, held=want["held_pages"],
                 head=int(want["free_head"][0]), table=want["table"])
        cached.copy_(i32(c["cached"].tolist()))
        held.copy_(out.held_pages)
        head.copy_(out.free_head)
    used = table[table >= 0]
    assert used.numel() == used.unique().numel()  # no page in two places
    assert t.read_flags() == 0


def test_refusals():
    from speculative_verify_paged_e4m3_gb300 import binding as B
    t = B.PagedTables(2, 16, 4, 8, 64, 16)

    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32, device="cuda")
    ok = dict(cached_lens=i32(2), new_lens=i32(2), held_pages=i32(2), free_pages=i32(8),
              free_head=i32(1), block_table=i32(2, 4))
    t(**ok)
    for k, v in (("cached_lens", i32(3)), ("new_lens", i32(2).long()), ("held_pages", i32(2).cpu()),
                 ("free_head", i32(2)), ("block_table", i32(4, 2).t()),
                 ("prefix_pages", i32(1)), ("block_table", i32(2, 8)[:, ::2])):
        with pytest.raises(ValueError):
            t(**{**ok, k: v})
    with pytest.raises(B.DflashError):  # an output that is an input
        t(**ok, out=t.empty()._replace(context_lens=ok["cached_lens"]))
