"""Attention over a shared prefix against the FP64 oracle over the whole tables (the oracle knows
nothing of the prefix), with the tolerances of the plain attention: max(2e-3, half an FP16 ulp) on
the output, 1e-5 max(1, |lse|) on the log-sum-exp. Unused pool bytes hold random codes, NaN codes
included, and the table entries that must not be read are out of range, which would set a flag."""
import numpy as np
import pytest
import torch

from gpu_helpers import compare, oracle_forward, to_np

pytestmark = pytest.mark.gpu

D = 256
PAGE_CLAMPED, CONTEXT_CLAMPED, SHORT = 0x4, 0x1, 0x2


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()


def make(seed, lens, prefix, q_len=8, heads=(6, 1), P=16, boost=1.0, extra_pages=3):
    """Tables of a batch whose first floor(prefix / P) pages are the same; the page that the
    prefix ends in is copied into a page of every sequence."""
    g = torch.Generator().manual_seed(seed)
    Hq, Hkv = heads
    B, shared = len(lens), prefix // P
    mp = max(1, -(-max(max(lens), prefix) // P))
    num_pages = shared + B * (mp - shared) + extra_pages
    pools = [torch.randint(0, 256, (num_pages, P, Hkv, D), generator=g, dtype=torch.uint8)
             for _ in range(2)]
    perm = torch.randperm(num_pages, generator=g).to(torch.int32)
    table = torch.full((B, mp), num_pages + 9, dtype=torch.int32)
    used = shared
    scales = [0.012 * boost, 0.011]
    pre = [torch.randn((prefix, Hkv, D), generator=g) for _ in range(2)]
    pre[0] = pre[0] * torch.where(torch.rand((prefix, 1, 1), generator=g) < 0.05, boost, 1.0)

    def codes(x, s):
        return (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for w in range(2):
        full = shared * P
        pools[w][perm[:shared].long()] = codes(pre[w][:full], scales[w]).view(shared, P, Hkv, D)
    for b, n in enumerate(lens):
        table[b, :shared] = perm[:shared]
        for lp in range(shared, -(-n // P)):
            table[b, lp] = perm[used]
            used += 1
        x = [torch.randn((max(n - prefix, 0), Hkv, D), generator=g) for _ in range(2)]
        for w in range(2):
            seq = torch.cat([pre[w], x[w]])[:n]
            for lp in range(shared, -(-n // P)):
                part = codes(seq[lp * P:min(n, (lp + 1) * P)], scales[w])
                pools[w][int(table[b, lp]), :part.shape[0]] = part
    q = torch.randn((B, q_len, Hq, D), generator=g).to(torch.float16)
    return dict(q=q, k_pool=pools[0], v_pool=pools[1], block_table=table,
                context_lens=torch.tensor(lens, dtype=torch.int32),
                k_scale=torch.tensor([scales[0]]), v_scale=torch.tensor([scales[1]]),
                prefix_table=perm[:max(1, shared)].clone(),
                prefix_len=torch.tensor([prefix], dtype=torch.int32))


def operator(inp, max_prefix=None, max_context=None, kernel=0):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    n, q_len, Hq, _ = inp["q"].shape
    num_pages, P, Hkv, _ = inp["k_pool"].shape
    mp = inp["block_table"].shape[1]
    mx = int(inp["prefix_len"].item()) if max_prefix is None else max_prefix
    return B.SharedPrefixAttention(n, q_len, Hq, Hkv, D, P, mp, num_pages, max_context or mp * P,
                                   max_prefix=mx, kernel=kernel)


def call(att, dev, **kw):
    return att(dev["q"], dev["k_pool"], dev["v_pool"], dev["prefix_table"], dev["prefix_len"],
               dev["block_table"], dev["context_lens"], dev["k_scale"], dev["v_scale"], **kw)


def hide_prefix_entries(inp):
    """The rows' entries of the shared pages are not read: put them out of range."""
    P = inp["k_pool"].shape[1]
    hidden = dict(inp, block_table=inp["block_table"].clone())
    hidden["block_table"][:, :int(inp["prefix_len"].item()) // P] = -77
    return hidden


def check(inp, kernel, what=""):
    want = oracle_forward(inp)
    dev = {k: v.cuda() for k, v in hide_prefix_entries(inp).items()}
    att = operator(inp, kernel=kernel)
    out, lse = call(att, dev)
    torch.cuda.synchronize()
    compare(to_np(out), to_np(lse), *want, what)
    short = SHORT if (inp["context_lens"] < inp["q"].shape[1]).any() else 0
    assert att.read_flags() == short
    return att


KERNELS = [1, 2]
pytest_kernels = pytest.mark.parametrize("kernel", KERNELS, ids=["rows", "pairs"])


@pytest_kernels
@pytest.mark.parametrize("heads,q_len,lens,prefix,P", [
    ((6, 1), 8, [300, 310, 333], 256, 16),         # whole pages, whole tiles
    ((6, 1), 8, [300, 310, 333], 259, 16),         # the prefix ends inside a page
    ((6, 1), 8, [1400, 1111, 1290, 1283], 1279, 64),
    ((24, 4), 8, [700, 530, 1000], 512, 16),
    ((24, 4), 1, [400] * 7 + [513], 399, 16),      # single tokens
    ((6, 1), 1, [129, 130], 128, 16),              # 12 rows
    ((8, 8), 3, [200, 220], 160, 32),              # one query head per KV head
    ((16, 2), 5, [500, 400, 450, 410, 399], 390, 48),
    ((6, 1), 8, [500], 448, 16),                   # one sequence
    ((6, 1), 16, [420, 700], 401, 16),             # 96 rows per sequence
    ((16, 1), 16, [420, 433], 400, 16),            # 256 rows per sequence
    ((6, 1), 8, [4000, 3500], 3296, 3296),         # pages of 3296 tokens
], ids=str)
def test_against_the_oracle(kernel, heads, q_len, lens, prefix, P):
    check(make(len(lens) + prefix, lens, prefix, q_len, heads, P), kernel)


@pytest_kernels
@pytest.mark.parametrize("prefix", [1, 15, 16, 17, 127, 128, 129, 143, 144, 255, 256, 257, 272,
                                    384, 400, 512, 513, 640])
def test_prefix_lengths_around_tiles(kernel, prefix):
    check(make(prefix, [prefix + 9, prefix + 130, prefix + 64], prefix), kernel)


@pytest_kernels
@pytest.mark.parametrize("batch", [2, 5, 6, 11, 16, 22])
def test_batches_of_many_row_blocks(kernel, batch):
    """96 to 1056 rows per KV head over the prefix, and two KV heads."""
    check(make(batch, [600 + 3 * b for b in range(batch)], 576, 8, (12, 2)), kernel)


@pytest_kernels
def test_long_prefix_in_several_splits(kernel):
    check(make(5, [9000, 8300, 8200], 8192, 8, (6, 1)), kernel)


@pytest_kernels
def test_peaked_scores(kernel):
    check(make(6, [3000, 2900, 2950], 2800, 8, (6, 1), boost=4.0), kernel)


@pytest_kernels
def test_sequences_inside_the_prefix_short_and_empty(kernel):
    """Contexts that end inside the prefix, at its end, right behind it, and padded batch slots."""
    check(make(7, [0, 320, 3, 8, 200, 256, 257, 264, 700, 0], 256), kernel)
    check(make(8, [0, 0, 0], 256), kernel)
    check(make(9, [0, 1, 600], 500, q_len=1), kernel)


@pytest_kernels
def test_prefix_shorter_than_a_page_and_none(kernel):
    inp = make(10, [100, 130], 10)
    check(inp, kernel)
    want = oracle_forward(inp)
    dev = {k: v.cuda() for k, v in inp.items()}
    out, lse = operator(inp, max_prefix=0, kernel=kernel)(
        dev["q"], dev["k_pool"], dev["v_pool"], None, None, dev["block_table"],
        dev["context_lens"], dev["k_scale"], dev["v_scale"])
    compare(to_np(out), to_np(lse), *want)
    inp = make(10, [100, 130], 64)
    dev = {k: v.cuda() for k, v in inp.items()}
    dev["prefix_len"].fill_(-5)  # no prefix at this call: everything is in the rows
    out, lse = call(operator(inp, kernel=kernel), dev)
    compare(to_np(out), to_np(lse), *oracle_forward(inp))


@pytest_kernels
def test_bad_pages_and_lengths_are_cut_and_flagged(kernel):
    inp = make(11, [300, 310], 256)
    dev = {k: v.cuda() for k, v in inp.items()}
    dev["prefix_table"][3] = 10 ** 6
    att = operator(inp, kernel=kernel)
    call(att, dev)
    assert att.read_flags(clear=True) == PAGE_CLAMPED
    dev = {k: v.cuda() for k, v in inp.items()}
    want = oracle_forward(inp)
    dev["prefix_len"].fill_(257 + 10 ** 6)  # cut to max_prefix
    out, lse = call(att, dev)
    compare(to_np(out), to_np(lse), *want)
    assert att.read_flags(clear=True) == CONTEXT_CLAMPED
    dev["prefix_len"].fill_(256)
    dev["context_lens"][1] = 2 ** 31 - 1  # cut to max_context
    call(att, dev)
    assert att.read_flags() & CONTEXT_CLAMPED


@pytest_kernels
def test_padded_slots_may_hold_anything(kernel):
    """Q of a batch slot without a request, or of drafted tokens that see no key, is not looked at."""
    inp = make(16, [700, 0, 640, 3, 650], 600)
    want = oracle_forward(inp)
    inp["q"][1] = float("nan")
    inp["q"][1, :, 0] = float("inf")
    inp["q"][3, :5] = float("-inf")  # 3 tokens in all: the first five rows of the block see none
    dev = {k: v.cuda() for k, v in inp.items()}
    out, lse = call(operator(inp, kernel=kernel), dev)
    compare(to_np(out), to_np(lse), *want)


@pytest_kernels
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_query_that_is_not_finite_spoils_its_own_row_alone(kernel, value):
    inp = make(13, [900, 780, 811], 700)
    want_out, want_lse = oracle_forward(inp)
    bad = dict(inp, q=inp["q"].clone())
    bad["q"][1, 3, 2, ::9] = value
    dev = {k: v.cuda() for k, v in bad.items()}
    out, lse = call(operator(bad, kernel=kernel), dev)
    out, lse = to_np(out), to_np(lse)
    assert np.isnan(out[1, 3, 2]).all() and np.isnan(lse[1, 3, 2])
    keep = np.ones(out.shape[:3], bool)
    keep[1, 3, 2] = False
    out[~keep], lse[~keep] = want_out[~keep], want_lse[~keep]
    compare(out, lse, want_out, want_lse)


@pytest_kernels
@pytest.mark.parametrize("k_scale", [-0.012, 0.0, 1e-6, 0.4])
def test_scales_of_any_size_and_sign(kernel, k_scale):
    inp = make(17, [500, 430], 400)
    inp["k_scale"] = torch.tensor([k_scale])
    inp["v_scale"] = torch.tensor([-0.011])
    check(inp, kernel)


@pytest_kernels
@pytest.mark.parametrize("batch,q_len,heads,longest", [
    (200, 1, (6, 1), 90),    # more sequences than SMs
    (70, 2, (8, 8), 90),     # more (sequence, KV head) units than SMs, one query head each
    (2, 1, (1, 1), 90),      # two rows in all
    (24, 4, (8, 4), 3000),   # two split slots an SM: one long sequence among short ones
], ids=str)
def test_many_and_few_units(kernel, batch, q_len, heads, longest):
    lens = [64 + q_len + (7 * b) % 20 for b in range(batch)]
    lens[batch // 2] = 64 + longest
    check(make(batch, lens, 64, q_len, heads), kernel)


@pytest_kernels
def test_agrees_with_the_plain_attention(kernel):
    from gpu_helpers import gpu_forward
    inp = make(12, [2100, 2300, 2222, 2050], 2048, 8, (24, 4))
    dev = {k: v.cuda() for k, v in inp.items()}
    _, want, want_lse = gpu_forward(dev)
    out, lse = call(operator(inp, kernel=kernel), dev)
    # both sides are within the tolerance of the exact value
    assert (out.float() - want.float()).abs().max().item() <= 4e-3
    assert (lse - want_lse).abs().max().item() <= 2e-5 * max(1.0, want_lse.abs().max().item())


@pytest_kernels
def test_repeats_are_the_same_bits(kernel):
    inp = make(13, [900, 1000, 1100], 800, 8, (24, 4))
    dev = {k: v.cuda() for k, v in inp.items()}
    att = operator(inp, kernel=kernel)
    a = [x.clone() for x in call(att, dev)]
    for _ in range(5):
        b = call(att, dev)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest_kernels
def test_one_graph_serves_changing_lengths(kernel):
    big = make(14, [1500, 1400], 1300)
    att = operator(big, kernel=kernel)
    dev = {k: v.cuda() for k, v in big.items()}
    out, lse = torch.empty_like(dev["q"]), torch.empty(dev["q"].shape[:3], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(att, dev, out=out, lse=lse)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(att, dev, out=out, lse=lse)
    for prefix, lens in ((1300, [1500, 1400]), (640, [1500, 700]), (1296, [1305, 0]),
                         (33, [90, 1400])):
        dev["prefix_len"].fill_(prefix)
        dev["context_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        # the tables share all of the first 1296 tokens' pages, so any shorter prefix is one too
        out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        want = oracle_forward(dict(big), context_override=lens)
        compare(to_np(out), to_np(lse), *want, f"prefix {prefix}")


@pytest_kernels
def test_two_streams_with_a_workspace_each(kernel):
    inps = [make(20 + i, [2000 + i, 1900], 1800, 8, (6, 1)) for i in range(2)]
    devs = [{k: v.cuda() for k, v in i.items()} for i in inps]
    atts = [operator(i, kernel=kernel) for i in inps]
    streams = [torch.cuda.Stream() for _ in inps]
    res = [(torch.empty_like(d["q"]), torch.empty(d["q"].shape[:3], device="cuda")) for d in devs]
    torch.cuda.synchronize()
    for _ in range(4):
        for a, d, s, (o, l) in zip(atts, devs, streams, res):
            call(a, d, out=o, lse=l, stream=s)
    torch.cuda.synchronize()
    for i, (o, l) in zip(inps, res):
        compare(to_np(o), to_np(l), *oracle_forward(i))


def test_refusals():
    inp = make(30, [300, 310], 256)
    dev = {k: v.cuda() for k, v in inp.items()}
    att = operator(inp)
    for k, v in (("q", dev["q"].float()), ("q", dev["q"][:1]), ("k_pool", dev["k_pool"].float()),
                 ("k_pool", dev["k_pool"][:2]), ("prefix_table", dev["prefix_table"][:3]),
                 ("prefix_len", dev["prefix_len"].long()), ("context_lens", inp["context_lens"]),
                 ("block_table", dev["block_table"].t().contiguous().t()),
                 ("v_scale", dev["v_scale"].double())):
        with pytest.raises(ValueError):
            call(att, {**dev, k: v})
    with pytest.raises(ValueError):
        call(att, dev, out=torch.empty((2, 8, 6, 128), dtype=torch.float16, device="cuda"))
