"""One key far above all others of its row (an attention sink), many keys that still matter together.

Every query element is 1, a key's 256 codes are one value c_j and its value's codes one value v_j, so key j
scores 16 c_j k_scale nats and the exact output of a row is a sum over scalars, taken here in 64 bits. The
sink is key 0 with c = 1, v = 0; the other keys stand `gap` bits below it, all of them equal or spread by
random c_j around 0, with v around 1. What the small probabilities lose, all of them in the same
direction, is then the error of the output.

Tolerance, derived. Of the output: half a step of FP16 on the way out and of each probability, 2^-11 each,
and FP32 arithmetic: scores of at most 25 bits (2^-19), the exponential (2^-22), and sums, for which a
truncating accumulator's 2^-24 in each of at most 4096 products over 16 keys gives 2^-12: below 2^-9.
Beside that the fixed grid under the smallest normal probability: step 2^-17, sink at 2^4 or more. Equal
keys are offset within their step by 128 evenly spaced fractions, so that the mean of 128 is within 2^-8 of a step,
65536 * 2^-25 / 2^6 = 2^-15 (16384 keys at 2^4: 2^-15); for random keys the errors are independent, below half a
step each: 6 standard deviations are 6 * 2^8 * 2^-18 / 2^6 < 2^-13 (2^7 and 2^4: 6 * 2^-15 < 2^-12). FP16 (the pair
kernel), step 2^-24, sink at 2^4: 65536 * 2^-25 / 2^4 = 2^-13 if every key errs the same way. So
2^-9 |out| + 2^-12. The log-sum-exp has the plain attention's 1e-5 max(1, |lse|).
"""
import math

import pytest
import torch

from gpu_helpers import MODES, kernel_args

pytestmark = pytest.mark.gpu

D = 256
GAPS = [8.0, 12.0, 13.9, 14.5, 15.5, 15.9, 16.2, 17.9, 19.5, 20.5, 20.9, 21.1, 22.4, 24.0]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()


def keys(n, gap, spread, P, Hkv, stronger=()):
    """Pools of n keys in order (page p holds keys p P .. p P + P - 1), the scale of K, and the scores in
    nats and the values as float64. stronger: more strong keys, (position, c)."""
    g = torch.Generator().manual_seed(int(16 * gap) + n)
    c, v = torch.zeros(n), torch.ones(n)
    if spread:
        c = (0.04 * torch.randn(n, generator=g)).clamp(-0.2, 0.2)
        v = 1.0 + 0.25 * torch.randn(n, generator=g)
    c[0], v[0] = 1.0, 0.0
    for j, x in stronger:
        c[j] = x
    c, v = c.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
    k_scale = torch.tensor([gap * math.log(2.0) / 16.0], device="cuda")
    pages = -(-n // P)

    def pool(x):
        rows = torch.zeros(pages * P, dtype=torch.uint8)
        rows[:n] = x.view(torch.uint8)
        return rows.cuda()[:, None, None].expand(-1, Hkv, D).reshape(pages, P, Hkv, D).contiguous()
    return (pool(c), pool(v), k_scale, c.double().cuda() * 16.0 * k_scale.double(), v.double().cuda())


def check(out, lse, scores, values, n, q_len):
    """Token i of a sequence of n keys sees keys 0 .. n - q_len + i; every sequence and head is the same."""
    for i in range(q_len):
        s = scores[:n - q_len + i + 1]
        z = torch.logsumexp(s, 0)
        want = (torch.exp(s - z) * values[:s.numel()]).sum().item()
        err = (out[:, i].double() - want).abs().max().item()
        assert err <= 2.0 ** -9 * abs(want) + 2.0 ** -12, (i, want, err)
        assert (lse[:, i].double() - z).abs().max().item() <= 1e-5 * max(1.0, abs(z.item()))


@pytest.mark.parametrize("kernel", [1, 2], ids=["rows", "pairs"])
@pytest.mark.parametrize("spread", [False, True], ids=["equal", "spread"])
@pytest.mark.parametrize("gap", GAPS)
def test_over_a_shared_prefix(kernel, spread, gap):
    """65536 shared keys, each row's in a single split or segment."""
    from speculative_verify_paged_e4m3_gb300 import binding as B
    n, P, Hq, Hkv, batch, q_len = 65536, 64, 32, 4, 80, 8
    kp, vp, ks, scores, values = keys(n, gap, spread, P, Hkv)
    pages = n // P
    table = torch.arange(pages, dtype=torch.int32, device="cuda")
    att = B.SharedPrefixAttention(batch, q_len, Hq, Hkv, D, P, pages, pages, n, n, kernel=kernel)
    if kernel == 1:
        assert att.plan.prefix_splits == 1
    else:  # no fewer units than pairs: most segments are whole units
        assert att.plan.prefix_row_blocks * Hkv >= att.plan.prefix_splits
    one = torch.ones(1, device="cuda")
    q = torch.ones((batch, q_len, Hq, D), dtype=torch.float16, device="cuda")
    out, lse = att(q, kp, vp, table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                   table.expand(batch, -1).contiguous(),
                   torch.full((batch,), n, dtype=torch.int32, device="cuda"), ks, one)
    check(out, lse, scores, values, n, q_len)
    assert att.read_flags() == 0


@pytest.mark.parametrize("n,q_len", [(3500, 2), (3500, 5), (16384, 8)])  # 12, 30 and 48 rows
@pytest.mark.parametrize("spread", [False, True], ids=["equal", "spread"])
@pytest.mark.parametrize("gap", GAPS)
def test_over_own_keys(n, q_len, spread, gap):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    P, Hq, Hkv, batch = 64, 6, 1, 320
    kp, vp, ks, scores, values = keys(n, gap, spread, P, Hkv)
    pages = kp.shape[0]
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(batch, -1).contiguous()
    att = B.SharedPrefixAttention(batch, q_len, Hq, Hkv, D, P, pages, pages, n, 0)
    one = torch.ones(1, device="cuda")
    q = torch.ones((batch, q_len, Hq, D), dtype=torch.float16, device="cuda")
    out, lse = att(q, kp, vp, None, None, table,
                   torch.full((batch,), n, dtype=torch.int32, device="cuda"), ks, one)
    check(out, lse, scores, values, n, q_len)
    assert att.read_flags() == 0


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("n,q_len", [(3500, 2), (3500, 5), (16384, 8)])  # 12, 30 and 48 rows
@pytest.mark.parametrize("spread", [False, True], ids=["equal", "spread"])
@pytest.mark.parametrize("gap", GAPS)
def test_in_the_plain_attention(mode, n, q_len, spread, gap):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    P, Hq, Hkv, batch = 64, 6, 1, 140
    kp, vp, ks, scores, values = keys(n, gap, spread, P, Hkv)
    pages = kp.shape[0]
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(batch, -1).contiguous()
    att = B.VerifyAttention(batch, q_len, Hq, Hkv, D, P, pages, pages, n, **kernel_args(mode))
    one = torch.ones(1, device="cuda")
    q = torch.ones((batch, q_len, Hq, D), dtype=torch.float16, device="cuda")
    out, lse = att(q, kp, vp, table, torch.full((batch,), n, dtype=torch.int32, device="cuda"), ks,
                   one)
    check(out, lse, scores, values, n, q_len)


@pytest.mark.parametrize("kernel", [0, 1, 2], ids=["plain", "rows", "pairs"])
@pytest.mark.parametrize("step", [3.0, 9.0, 11.0, 14.0, 15.5, 21.0])
def test_strong_keys_one_after_the_other(kernel, step):
    """Each a quarter to 2 `step`s (bits) above the last: in the tile after it, in the same tile, far behind.
    (Scores of up to 105 bits: 2^-17 of a probability.)"""
    from speculative_verify_paged_e4m3_gb300 import binding as B
    n, P, Hq, Hkv, batch, q_len = 16384, 64, 32, 4, 80, 1
    kp, vp, ks, scores, values = keys(n, step, True, P, Hkv, [
        (97, 2.0), (150, 3.0), (151, 3.25), (400, 3.5), (5000, 4.0), (5001, 0.0), (16383, 5.0)])
    pages = n // P
    table = torch.arange(pages, dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    q = torch.ones((batch, q_len, Hq, D), dtype=torch.float16, device="cuda")
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    lens[::3] = 5003
    rows = table.expand(batch, -1).contiguous()
    if kernel:
        att = B.SharedPrefixAttention(batch, q_len, Hq, Hkv, D, P, pages, pages, n, n, kernel=kernel)
        out, lse = att(q, kp, vp, table, lens[1:2].clone(), rows, lens, ks, one)
    else:
        att = B.VerifyAttention(batch, q_len, Hq, Hkv, D, P, pages, pages, n)
        out, lse = att(q, kp, vp, rows, lens, ks, one)
    for b in (0, 1):
        m = int(lens[b].item())
        some = torch.arange(batch, device="cuda") % 3 == 0 if b == 0 else torch.arange(batch, device="cuda") % 3 > 0
        check(out[some], lse[some], scores[:m], values[:m], m, q_len)
