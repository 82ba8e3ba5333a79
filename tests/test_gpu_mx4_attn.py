"""Attention over the 4-bit cache against the formula in 64 bits.

Tolerances, derived. A score is a sum of 256 products q k in FP32 that the tensor core takes 16 at a time:
at most 16 additions that cut the running sum at 2^-23 of the largest partial sum, and the alignment of
each group's products, all below 2^-18 of sum |q k| / 16 =: spread; bringing it to a base-2 exponent
and the exponential add at most 2^-20 (1 + |score|), and |score| <= spread. So a probability is known
to SCORE = 2^-17 spread + 2^-19 relative, and its FP16 rounding adds 2^-11; both sums (numerator and
denominator) take the first. Below 2^-14 of FP16's range it has a fixed step: 2^-33 of the row's
largest at most, half a step lost, the same way for each of n keys. The output's rounding is
2^-11 of itself (2^-25 if subnormal). With weight = sum p |v|:
  |out - exact| <= 2^-11 |exact| + 2^-25 + (2^-11 + 2 SCORE + 2^-20) weight + n 2^-33 vmax
  |lse - exact| <= SCORE + 2^-22 |lse| + 2^-20
"""
import numpy as np
import pytest
import torch

import mx4_reference as M

pytestmark = pytest.mark.gpu

D = 256


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()


def fill(rng, pages, P, Hkv, of_v, gain=1.0, strong=0.0):
    """A pool of quantised normal numbers (packed by arrays: all slots in order)."""
    n = pages * P
    x = rng.standard_normal((n, Hkv, D)) * gain
    if strong:
        x[rng.random(n) < 0.05] *= strong
    codes, s = M.quantise(x)
    if of_v:
        b = codes[..., :128] | codes[..., 128:] << 4
        b = b.reshape(n // 16, 16, Hkv, 128).transpose(0, 2, 3, 1)
    else:
        b = codes[..., 0::2] | codes[..., 1::2] << 4
        b = b.reshape(n // 16, 16, Hkv, 8, 16).transpose(0, 2, 3, 1, 4)
    s = s.reshape(n // 16, 16, Hkv, 8).transpose(0, 2, 1, 3)
    pool = np.concatenate([b.reshape(n // 16, Hkv, 2048), s.reshape(n // 16, Hkv, 128)], -1)
    return np.ascontiguousarray(pool.reshape(pages, P // 16, Hkv, 2176))


def problem(seed, lens, q_len, Hq, Hkv, P, gain=1.0, strong=0.0, spare=2):
    rng = np.random.default_rng(seed)
    B = len(lens)
    mp = max(1, -(-max(lens) // P))
    pages = B * mp + spare
    table = rng.permutation(pages)[:B * mp].reshape(B, mp).astype(np.int32)
    q = rng.standard_normal((B, q_len, Hq, D)).astype(np.float16)
    return dict(q=q, k=fill(rng, pages, P, Hkv, False, gain, strong), v=fill(rng, pages, P, Hkv, True),
                table=table, lens=np.asarray(lens, dtype=np.int32), P=P)


def make(pr, max_context=None, **kw):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    b, q_len, Hq, _ = pr["q"].shape
    return B.Mx4Attention(b, q_len, Hq, pr["k"].shape[2], D, pr["P"], pr["table"].shape[1],
                          pr["k"].shape[0], max_context or pr["table"].shape[1] * pr["P"], **kw)


def dev(pr):
    return [torch.from_numpy(pr[n]).cuda() for n in ("q", "k", "v", "table", "lens")]


def check(got, pr, want=None):
    out, lse, spread, weight = want or M.attention(pr["q"], pr["k"], pr["v"], pr["table"], pr["lens"],
                                                   pr["P"])
    o, l = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    score = 2.0 ** -17 * spread + 2.0 ** -19
    n = max(1, int(pr["lens"].max()))
    vmax = 6 * 2.0 ** (float(pr["v"][..., 2048:].astype(int)[pr["v"][..., 2048:] < 255].max()) - 127)
    tol = (2.0 ** -11 * np.abs(out) + 2.0 ** -25 + n * 2.0 ** -33 * vmax
           + (2.0 ** -11 + 2 * score[..., None] + 2.0 ** -20) * weight)
    assert np.array_equal(np.isnan(o), np.isnan(out)) and np.array_equal(np.isnan(l), np.isnan(lse))
    fine = ~np.isnan(out)
    assert (np.abs(o - out) <= tol)[fine].all(), (np.abs(o - out) / tol)[fine].max()
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(l), empty) and (o[empty] == 0).all()
    fin = np.isfinite(lse)
    ltol = score + 2.0 ** -22 * np.abs(np.where(fin, lse, 0)) + 2.0 ** -20
    assert (np.abs(l - lse)[fin] <= ltol[fin]).all(), (np.abs(l - lse)[fin] / ltol[fin]).max()


CASES = [
    # lens, q_len, Hq, Hkv, page
    ([1], 1, 1, 1, 16), ([1], 1, 6, 1, 16), ([15], 8, 6, 1, 16), ([16], 1, 24, 4, 16),
    ([17], 8, 6, 1, 32), ([127], 8, 6, 1, 16), ([128], 4, 6, 1, 48), ([129], 8, 6, 1, 64),
    ([255, 256, 257], 2, 8, 2, 16), ([300, 0, 5, 1000], 8, 12, 2, 16),
    ([3, 8, 7], 8, 6, 1, 16),  # rows that see nothing
    ([0, 0], 8, 6, 1, 16), ([700], 3, 16, 1, 16),  # 48 rows
    ([650], 7, 7, 1, 16), ([650], 16, 6, 1, 16),  # 49 and 96 rows: row blocks
    ([400], 32, 8, 1, 16),  # 256 rows
    ([1500, 40, 900], 5, 24, 4, 48), ([2500], 1, 24, 4, 64), ([5000], 8, 6, 1, 16),
    ([1100, 777], 2, 17, 1, 16), ([1300], 1, 33, 1, 32),
]


@pytest.mark.parametrize("lens,q_len,Hq,Hkv,P", CASES)
def test_attention(lens, q_len, Hq, Hkv, P):
    pr = problem(len(lens) * 1000 + q_len, lens, q_len, Hq, Hkv, P)
    att = make(pr)
    got = att(*dev(pr))
    check(got, pr)
    from speculative_verify_paged_e4m3_gb300 import binding as B
    short = any(n < q_len for n in lens)
    assert att.read_flags() == (B.DFLASH_FLAG_CONTEXT_SHORT if short else 0)


@pytest.mark.parametrize("splits", [1, 2, 5])
def test_forced_splits(splits):
    pr = problem(splits, [1023, 130], 8, 12, 2, 16)
    check(make(pr, num_splits=splits)(*dev(pr)), pr)


@pytest.mark.parametrize("heads,q_len", [((12, 2), 1), ((4, 2), 30)])
def test_a_long_batch_with_many_units(heads, q_len):
    """More units than half the SMs and room for long contexts: two rounds of slots."""
    rng = np.random.default_rng(q_len)
    lens = rng.integers(0, 400, 41 if q_len == 1 else 20)
    lens[[3, 11]] = 9000, 4099
    lens[5] = 0
    pr = problem(41, lens, q_len, *heads, 64)
    att = make(pr)
    units = len(lens) * heads[1] * att.plan.row_blocks
    assert 2 * units > att.plan.sm_count >= units
    assert att.plan.num_slots == 2 * att.plan.sm_count // att.plan.row_blocks
    check(att(*dev(pr)), pr)


@pytest.mark.parametrize("gain,strong", [(4.0, 0.0), (2.0, 4.0), (0.01, 0.0)])
def test_peaked_and_flat_scores(gain, strong):
    pr = problem(11, [3000, 513], 8, 6, 1, 16, gain, strong)
    check(make(pr)(*dev(pr)), pr)


def test_reference_moves_with_growing_scores():
    """Keys that each draw more than all before them, and then a long flat tail."""
    pr = problem(12, [2600], 8, 6, 1, 16)
    rng = np.random.default_rng(5)
    n = pr["k"].shape[0] * 16
    x = rng.standard_normal((n, 1, D)) * 0.2
    q0 = pr["q"][0, 0, 0].astype(np.float64)
    order = np.empty(n, dtype=int)
    order[:] = 0
    slots = (pr["table"][0][:, None] * 16 + np.arange(16)).reshape(-1)
    for j in range(1500):
        x[slots[j], 0] += q0 * (j / 1500) * 3.0
    codes, s = M.quantise(x)
    pr["k"][:] = 0
    M.put(pr["k"], np.arange(n), codes, s, False)
    pr["q"][0, :, :] = pr["q"][0, 0, 0]
    check(make(pr)(*dev(pr)), pr)


def test_a_strong_key_in_front_of_many():
    """One key of nearly all the weight, 60000 of equal small weights: they must not be lost together."""
    n = 60000
    pr = problem(13, [n], 1, 6, 1, 64)
    rng = np.random.default_rng(6)
    pr["k"][:] = 0
    pr["k"][..., 2048:] = 127
    u = np.zeros((1, 1, D))
    u[..., :32] = 1.0
    for bits in (14.3, 17.7, 20.4):
        q = np.zeros((1, 1, 6, D), dtype=np.float16)
        q[..., :32] = bits * np.log(2) * 16 / 32 / 6
        pr["q"] = q
        codes, s = M.quantise(u * 6.0)
        M.put(pr["k"], [int(pr["table"][0, 0]) * 64], codes, s, False)
        check(make(pr)(*dev(pr)), pr)


def set_scale(pr, name, b, j, h, block, value):
    P = pr["P"]
    s = int(pr["table"][b, j // P]) * P + j % P
    flat = pr[name].reshape((-1,) + pr[name].shape[2:])
    flat[s // 16, h, 2048 + 8 * (s % 16) + block] = value


@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("back", [3, 200])
def test_a_nan_scale_reaches_the_rows_that_see_it(name, back):
    pr = problem(14, [600, 333], 8, 12, 2, 16)
    clean = M.attention(pr["q"], pr["k"], pr["v"], pr["table"], pr["lens"], 16)
    set_scale(pr, name, 0, 600 - back, 1, 5, 255)
    out, lse = (x.copy() for x in clean[:2])
    sees = np.arange(8) >= 8 - back
    out[0, sees, 6:] = np.nan
    lse[0, sees, 6:] = np.nan
    check(make(pr)(*dev(pr)), pr, (out, lse) + clean[2:])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_query_row_that_is_not_finite(value):
    pr = problem(15, [500, 3], 8, 6, 1, 16)
    clean = M.attention(pr["q"], pr["k"], pr["v"], pr["table"], pr["lens"], 16)
    pr["q"][0, 2, 4, 77] = value
    pr["q"][1, 0, 1, 0] = value  # sees no key
    out, lse = (x.copy() for x in clean[:2])
    out[0, 2, 4] = np.nan
    lse[0, 2, 4] = np.nan
    check(make(pr)(*dev(pr)), pr, (out, lse) + clean[2:])


def test_whatever_lies_past_a_length():
    """Codes and scales (NaN among them) behind each length, in its page, tile and beyond."""
    pr = problem(16, [100, 257, 31], 8, 6, 1, 64)
    clean = M.attention(pr["q"], pr["k"], pr["v"], pr["table"], pr["lens"], 64)
    for name in ("k", "v"):
        flat = pr[name].reshape(-1, 2176)
        for b, n in enumerate(pr["lens"]):
            for j in range(n, pr["table"].shape[1] * 64):
                s = int(pr["table"][b, j // 64]) * 64 + j % 64
                flat[s // 16, 2048 + 8 * (s % 16):2056 + 8 * (s % 16)] = 255
    check(make(pr)(*dev(pr)), pr, clean)


@pytest.mark.parametrize("deltas", [(0, 3, 9, 20), (0, 26, 25, 24), (12, 0, 1, 30)])
def test_blocks_of_different_scales(deltas):
    """Blocks of one key far apart: exact down to 2^-26 of the largest, zero below (the reference leaves
    those out)."""
    pr = problem(17, [300], 8, 6, 1, 16)
    for name in ("k", "v"):
        sc = pr[name][..., 2048:].reshape(-1, 16, 8)
        sc[:] = 127
        for i, d in enumerate(deltas):
            sc[..., 2 * i:2 * i + 2] -= d
    want = {n: pr[n].copy() for n in ("k", "v")}
    for p in want.values():
        sc = p[..., 2048:].reshape(-1, 16, 8)
        sc[sc.astype(int) < 127 - 26] = 0
    check(make(pr)(*dev(pr)), pr, M.attention(pr["q"], want["k"], want["v"], pr["table"], pr["lens"], 16))


@pytest.mark.parametrize("shift", [-30, -12, 9, 14])
def test_values_of_any_size(shift):
    """V (and K the other way) far from one: FP16's range is not the cache's."""
    pr = problem(18, [700, 90], 4, 6, 1, 16)
    pr["v"][..., 2048:] += np.uint8(shift % 256)
    pr["k"][..., 2048:] += np.uint8(-shift % 256)
    pr["q"] = (pr["q"].astype(np.float64) * 2.0 ** min(shift, 12)).astype(np.float16)
    want = M.attention(pr["q"], pr["k"], pr["v"], pr["table"], pr["lens"], 16)
    if np.abs(want[0]).max() < 60000:
        check(make(pr)(*dev(pr)), pr, want)


def test_zero_cache():
    pr = problem(19, [200], 8, 6, 1, 16)
    pr["k"][:], pr["v"][:] = 0, 0
    check(make(pr)(*dev(pr)), pr)


def test_flags_of_bad_tables_and_lengths():
    from speculative_verify_paged_e4m3_gb300 import binding as B
    pr = problem(20, [300, 290], 8, 6, 1, 16)
    good = M.attention(pr["q"], pr["k"], pr["v"], pr["table"], pr["lens"], 16)
    att = make(pr)
    bad = dict(pr, table=pr["table"].copy())
    bad["table"][0, 3] = -5
    bad["table"][1, 2] = pr["k"].shape[0] + 9
    clamped = dict(pr, table=np.clip(bad["table"], 0, pr["k"].shape[0] - 1))
    check(att(*dev(bad)), clamped)
    assert att.read_flags(clear=True) == B.DFLASH_FLAG_PAGE_CLAMPED
    small = make(pr, max_context=290)
    got = small(*dev(pr))
    assert small.read_flags() == B.DFLASH_FLAG_CONTEXT_CLAMPED
    check(got, dict(pr, lens=np.array([290, 290], dtype=np.int32)))
    negative = dict(pr, lens=np.array([-7, 290], dtype=np.int32))
    got = att(*dev(negative))
    assert (got[0][0] == 0).all() and got[1][0].isneginf().all()
    assert np.allclose(got[0][1].double().cpu().numpy(), good[0][1], atol=2e-2)


def test_same_bits_every_time_and_nothing_else_written():
    pr = problem(21, [900, 1234, 77], 8, 12, 2, 16)
    att = make(pr)
    args = dev(pr)
    first = [x.clone() for x in att(*args)]
    B_, q_len, Hq = pr["q"].shape[:3]
    wide = torch.full((B_ + 2, q_len, Hq, D), 5.0, dtype=torch.float16, device="cuda")
    lse = torch.full((B_ + 2, q_len, Hq), 5.0, device="cuda")
    for _ in range(20):
        att(*args, out=wide[1:-1], lse=lse[1:-1])
        assert torch.equal(wide[1:-1], first[0]) and torch.equal(lse[1:-1], first[1])
    assert (wide[0] == 5).all() and (wide[-1] == 5).all() and (lse[0] == 5).all() and (lse[-1] == 5).all()
    assert all(np.array_equal(a.cpu().numpy(), pr[n]) for a, n in zip(args, ("q", "k", "v", "table", "lens")))


def test_other_streams_and_two_at_once():
    prs = [problem(22 + i, [2000 + 300 * i, 50], 8, 6, 1, 16) for i in range(2)]
    atts = [make(p) for p in prs]
    args = [dev(p) for p in prs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in prs]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            got[i] = atts[i](*args[i], stream=s)
    torch.cuda.synchronize()
    for g, p in zip(got, prs):
        check(g, p)


def test_a_captured_call_serves_other_lengths():
    pr = problem(24, [1500, 600], 8, 6, 1, 16)
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
    for lens in ([1500, 600], [1, 0], [1007, 599]):
        args[4].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check((out, lse), dict(pr, lens=np.array(lens, dtype=np.int32)))


@pytest.mark.parametrize("pdl", [False, True])
def test_programmatic_launches_back_to_back(pdl):
    """Layer after layer on one workspace, each launch with or without the programmatic attribute."""
    from speculative_verify_paged_e4m3_gb300 import binding as B
    prs = [problem(30 + i, [1800, 900], 8, 6, 1, 16) for i in range(3)]
    att = make(prs[0], flags=B.DFLASH_PROBLEM_PDL if pdl else 0)
    args = [dev(p) for p in prs]
    torch.cuda.synchronize()
    got = [att(*a) for _ in range(4) for a in args][-3:]
    torch.cuda.synchronize()
    for g, p in zip(got, prs):
        check(g, p)


def test_a_pool_past_32_bit_offsets():
    from speculative_verify_paged_e4m3_gb300 import binding as B
    small = problem(26, [500], 8, 12, 4, 64)
    pages = (1 << 32) // (4 * 4 * 2176) + 40
    k, v = (torch.zeros((pages, 4, 4, 2176), dtype=torch.uint8, device="cuda") for _ in range(2))
    n = small["k"].shape[0]
    k[-n:] = torch.from_numpy(small["k"]).cuda()
    v[-n:] = torch.from_numpy(small["v"]).cuda()
    table = torch.from_numpy(small["table"] + (pages - n)).int().cuda()
    att = B.Mx4Attention(1, 8, 12, 4, D, 64, table.shape[1], pages, table.shape[1] * 64)
    got = att(torch.from_numpy(small["q"]).cuda(), k, v, table, torch.from_numpy(small["lens"]).cuda())
    check(got, small)


def test_refusals():
    from speculative_verify_paged_e4m3_gb300 import binding as B
    pr = problem(27, [100], 8, 6, 1, 16)
    att = make(pr)
    q, k, v, table, lens = dev(pr)
    for bad in ((q.float(), k, v, table, lens), (q[:, :4], k, v, table, lens), (q, k[1:], v, table, lens),
                (q, k, v.float(), table, lens), (q, k, v, table.long(), lens), (q, k, v, table, lens.cpu())):
        with pytest.raises(ValueError):
            att(*bad)
    with pytest.raises(ValueError):
        att(q, k, v, table, lens, out=torch.empty_like(q, dtype=torch.float32))
    with pytest.raises(ValueError):
        make(pr, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(B.DflashError):
        make(pr, flags=B.DFLASH_PROBLEM_FUSED_COMBINE)
    with pytest.raises(B.DflashError):
        att(q, k, v, table, lens, out=q)


@pytest.mark.parametrize("power", [6, 14])
def test_a_key_whose_value_is_far_larger_in_one_block(power):
    """Its power stands before its probability: the other keys' weights keep a step of 2^-33 of the largest product of
    both, which the tolerance's last term has as vmax; lse does not know of it."""
    pr = problem(20, [900, 257], 8, 6, 1, 16)
    for b, j in ((0, 300), (1, 10)):
        set_scale(pr, "v", b, j, 0, 3, 127 + power)
    check(make(pr)(*dev(pr)), pr)
