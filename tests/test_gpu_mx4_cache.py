"""Head norms, the 4-bit cache's write and its read, against the formulas in 64 bits.

Tolerances, derived. A head's norm: the FP32 sum of 256 squares is off by at most 8 + 5 + 1 roundings
(eight a lane, five exchanges, the square) of 2^-24, half of that after the root, which with the
division, the sum with eps, the root and the products x r w' (w' itself rounded) adds 7 more: at most
14 * 2^-24 < 2^-20 of the normed value. The rotation adds 2^-20 (|x| + |y|) amp (test_gpu_rope.py).
So ARITH = 2^-19 of amp (|x| + |y|), x and y the normed pair; the output's type adds eps / 2 of the
value and half the smallest FP16 subnormal. A code of K is the nearest of a number so far off: its
distance is that of the nearest code at most, plus twice that. V is not computed with: its codes and
scales are the formula's, bit for bit, and read() is exact.
"""
import numpy as np
import pytest
import torch

import mx4_reference as M
from test_gpu_rope import exact
from test_paged_step_abi import frequencies

pytestmark = pytest.mark.gpu

D = 256
ARITH = 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()


def normed(x, w, eps, offset):
    x = x.double().cpu().numpy()
    if w is None:
        return x
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
    return x * r * (w.double().cpu().numpy() + offset)


def make(seed, T, Hq, Hkv, dtype, far=100000, fused=False, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=g)
    x = x * torch.exp(spread * torch.randn((T, Hq + 2 * Hkv, 1), generator=g))
    x = x.to(dtype).cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32).cuda()
    w = (1 + 0.5 * torch.randn((2, D), generator=g)).to(dtype).cuda()
    return q, k, v, pos, w[0].contiguous(), w[1].contiguous()


def check_rows(got, want, mag, dtype):
    err = np.abs(got.double().cpu().numpy() - want)
    tol = torch.finfo(dtype).eps / 2 * np.abs(want) * (1 + ARITH) + ARITH * mag + 2.0 ** -25
    assert (err <= tol).all(), (err - tol).max()


def check_codes(pool, slots, want, mag):
    """K's rows in the pool against numbers that are known to ARITH * mag."""
    codes, s = M.get(pool.cpu().numpy(), slots, False)
    off = ARITH * mag
    b = np.abs(want).reshape(want.shape[:-1] + (8, 32))
    d = off.reshape(b.shape)
    unit = np.ldexp(1.0, s.astype(int) - 127)
    assert (((b - d).max(-1) <= 7 * unit) & (((b + d).max(-1) > 3.5 * unit) | (s == 0))).all()
    near = np.min(np.abs(b[..., None] - M.GRID * unit[..., None, None]), -1).reshape(want.shape)
    err = np.abs(M.numbers(codes, s) - want)
    assert (err <= near + 2 * off).all()


SHAPES = [(1, 6, 1), (7, 6, 1), (40, 24, 4), (761, 6, 1), (1530, 4, 2), (4600, 6, 1)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,Hq,Hkv", SHAPES)
def test_norm_rope_apply(T, Hq, Hkv, dtype, layout):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    rot = 64 + 32 * (T % 3) if T != 40 else 256
    q, k, _, pos, qw, kw = make(T, T, Hq, Hkv, dtype, fused=T % 2 == 0)
    r = B.Rotary(Hq, Hkv, D, rot, layout=layout, dtype=dtype, base=500000.0, scaling="yarn", factor=4.0,
                 trained_context=32768)
    theta = np.array(frequencies(rot, 500000.0, "yarn", 4.0, 32768))
    amp = float(r.plan.amplitude)
    qo, ko = r.apply(q, k, pos, norm=B.HeadNorm(qw, kw, 1e-5, 1.0))
    p = pos.cpu().numpy()
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        check_rows(got, *exact(normed(x, w, 1e-5, 1.0), p, theta, amp, rot, layout), dtype)
    # one operand's norm alone; in place
    want_k, mag_k = exact(normed(k, None, 0, 0), p, theta, amp, rot, layout)
    q2, k2 = q.clone(), k.clone()
    r.apply(q2, k2, pos, q_out=q2, k_out=k2, norm=B.HeadNorm(qw, None, 1e-5, 1.0))
    assert torch.equal(q2, qo)
    check_rows(k2, want_k, mag_k, dtype)
    plain = r.apply(q, k, pos)
    none = r.apply(q, k, pos, norm=B.HeadNorm(None, None))
    assert all(torch.equal(a, b) for a, b in zip(plain, none)) and torch.equal(plain[1], k2)
    alone, _ = r.apply(q, None, pos, norm=B.HeadNorm(qw, kw, 1e-5, 1.0))
    assert torch.equal(alone, qo)


def test_norm_of_zeros_tiny_and_not_finite_rows():
    from speculative_verify_paged_e4m3_gb300 import binding as B
    x = torch.zeros((5, 1, D), dtype=torch.float16, device="cuda")
    x[1] = 2.0 ** -24
    x[2, 0, 3] = float("nan")
    x[3, 0, 5] = float("inf")
    x[4] = 65504.0
    w = torch.ones(D, dtype=torch.float16, device="cuda")
    pos = torch.zeros(5, dtype=torch.int32, device="cuda")
    r = B.Rotary(1, 1, D)
    out, _ = r.apply(x, x.clone(), pos, norm=B.HeadNorm(w, w, 1e-6))
    o = out[:, 0].float()
    assert (o[0] == 0).all() and (o[4] == 1).all()
    assert torch.allclose(o[1], torch.full_like(o[1], 2.0 ** -24 / 1e-3), atol=2.0 ** -25, rtol=0)
    assert o[2].isnan().all()
    assert o[3, 5].isnan()
    out, _ = r.apply(x[:1], x[:1].clone(), pos[:1], norm=B.HeadNorm(w, w, 0.0))
    assert out.isnan().all()  # 0 / 0


def test_e4m3_write_takes_the_norm():
    from speculative_verify_paged_e4m3_gb300 import binding as B
    T, Hq, Hkv, P, pages = 37, 24, 4, 16, 5
    q, k, v, pos, qw, kw = make(5, T, Hq, Hkv, torch.float16, fused=True, spread=0.3)
    norm = B.HeadNorm(qw, kw, 1e-6, 0.0)
    r = B.Rotary(Hq, Hkv, D, 128, page_size=P, num_pages=pages)
    slots = torch.randperm(P * pages)[:T].cuda()
    slots[4] = -1
    scale = torch.tensor([0.01], device="cuda")
    kp, vp = (torch.zeros((pages, P, Hkv, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    q_out = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
    r.kv_write(q, k, v, pos, slots, scale, scale, kp, vp, q_out=q_out, norm=norm)
    want_q, want_k = r.apply(q, k, pos, norm=norm)
    live = slots >= 0
    assert torch.equal(q_out[live], want_q[live]) and (q_out[4] == 7).all()
    got = kp.view(torch.float8_e4m3fn).flatten(0, 1)[slots[live]].float() * 0.01
    # a code is off by 2^-4 of itself (below its normal range by half its step, 2^-10), and k's own
    # rounding to FP16 by 2^-11
    err = (got - want_k[live].float()).abs()
    sat = want_k[live].float().abs() > 4.48
    assert (err <= want_k[live].float().abs() * (2 ** -4 + 2 ** -10) + 0.01 * 2 ** -10)[~sat].all()
    assert r.read_flags() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,Hq,Hkv,P", [(1, 6, 1, 16), (8, 6, 1, 16), (61, 24, 4, 64), (803, 6, 1, 48),
                                        (1603, 3, 2, 32), (4601, 2, 1, 16)])
def test_mx4_write(T, Hq, Hkv, P, dtype, layout):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    rot = 16 * (1 + T % 16)
    q, k, v, pos, qw, kw = make(T + 1, T, Hq, Hkv, dtype, fused=T % 2 == 1)
    pages = -(-T // P) + 2
    r = B.Rotary(Hq, Hkv, D, rot, layout=layout, dtype=dtype, page_size=P, num_pages=pages)
    cache = B.Mx4Cache(Hkv, D, P, pages)
    kp, vp = cache.empty()
    kp.fill_(0x11)
    vp.fill_(0x22)
    rng = np.random.default_rng(T)
    at = rng.permutation(pages * P)[:T]
    slots = torch.from_numpy(at.copy()).cuda()
    if T > 8:
        slots[5] = -1
        slots[T - 2] = pages * P  # past the pool
    q_out = torch.full((T, Hq, D), 3.0, dtype=dtype, device="cuda")
    r.mx4_write(q, k, v, pos, slots, kp, vp, q_out=q_out, norm=B.HeadNorm(qw, kw, 1e-6))
    want_q, _ = r.apply(q, k, pos, norm=B.HeadNorm(qw, kw, 1e-6))
    theta = np.array(frequencies(rot, 10000.0, "none", 1.0, 1))
    wk, mag = exact(normed(k, kw, 1e-6, 0.0), pos.cpu().numpy(), theta, 1.0, rot, layout)
    live = slots.cpu().numpy()
    on = (live >= 0) & (live < pages * P)
    assert torch.equal(q_out[torch.from_numpy(live >= 0).cuda()],
                       want_q[torch.from_numpy(live >= 0).cuda()])
    assert (q_out[torch.from_numpy(live < 0).cuda()] == 3).all()
    check_codes(kp, live[on], wk[on], mag[on])
    codes, s = M.quantise(v.double().cpu().numpy()[on])
    want_v = np.full(vp.shape, 0x22, dtype=np.uint8)
    M.put(want_v, live[on], codes, s, True)
    assert np.array_equal(vp.cpu().numpy(), want_v)  # the other slots' bytes too
    rest = np.setdiff1d(np.arange(pages * P), live[on])
    gk, gs = M.get(kp.cpu().numpy(), rest, False)
    assert (gk == 1).all() and (gs == 0x11).all()
    assert r.read_flags() == (B.DFLASH_FLAG_SLOT_RANGE if T > 8 else 0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,Hq,Hkv,P,off", [(1023, 2, 2, 16, 0), (1024, 6, 1, 64, 0), (1025, 24, 4, 64, 5),
                                            (2111, 6, 1, 16, 3), (1500, 8, 8, 48, 13)])
def test_mx4_write_of_prompts(T, Hq, Hkv, P, off, dtype):
    """Runs of slots, as prompts have, that begin anywhere in a page, with padding in between: every byte
    of both pools."""
    from speculative_verify_paged_e4m3_gb300 import binding as B
    q, k, v, pos, qw, kw = make(T + off, T, Hq, Hkv, dtype, fused=T % 2 == 1)
    pages = -(-(T + off) // P) + 2
    rng = np.random.default_rng(T)
    order = rng.permutation(pages)
    at = np.arange(T) + off
    slots = order[at // P] * P + at % P
    slots[rng.random(T) < 0.02] = -1
    slots[T // 2:T // 2 + 20] = -1
    slots[-1] = pages * P + 3
    r = B.Rotary(Hq, Hkv, D, page_size=P, num_pages=pages, dtype=dtype)
    kp, vp = B.Mx4Cache(Hkv, D, P, pages).empty()
    kp.fill_(0x33)
    vp.fill_(0x44)
    zero = torch.zeros_like(pos)
    q_out = torch.full((T, Hq, D), 3.0, dtype=dtype, device="cuda")
    r.mx4_write(q, k, v, zero, torch.from_numpy(slots).cuda(), kp, vp, q_out=q_out)
    on = (slots >= 0) & (slots < pages * P)
    for got, x, of_v, fill in ((kp, k, False, 0x33), (vp, v, True, 0x44)):
        want = np.full(got.shape, fill, dtype=np.uint8)
        codes, s = M.quantise(x.double().cpu().numpy()[on])
        M.put(want, slots[on], codes, s, of_v)
        assert np.array_equal(got.cpu().numpy(), want)
    keep = torch.from_numpy(slots >= 0).cuda()
    assert torch.equal(q_out[keep], q[keep]) and (q_out[~keep] == 3).all()
    assert r.read_flags() == B.DFLASH_FLAG_SLOT_RANGE


def test_mx4_write_without_norm_or_rotation_is_the_formula():
    """Position 0 turns nothing: K's codes are then the formula's, bit for bit. Zeros, ties, numbers
    between 6 and 7 units, subnormal ones, infinities and NaN."""
    from speculative_verify_paged_e4m3_gb300 import binding as B
    g = torch.Generator().manual_seed(3)
    x = torch.randn((32, 2, D), generator=g)
    x[1] = 0
    x[2] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]).repeat(32)
    x[3] = -x[2]
    x[4] = 2.0 ** -24
    x[5] *= 2.0 ** -20
    x[6, :, 40] = float("inf")
    x[7, :, 200] = float("nan")
    x[8, :, 3] = -65504.0
    x[9] = torch.tensor([6.5, 6.0, 6.99, 7.0, 7.01, 3.5, 3.51, 0.1]).repeat_interleave(32)
    x = x.half().cuda()
    r = B.Rotary(1, 2, D, page_size=16, num_pages=2)
    kp, vp = B.Mx4Cache(2, D, 16, 2).empty()
    q = torch.zeros((32, 1, D), dtype=torch.float16, device="cuda")
    zero = torch.zeros(32, dtype=torch.int32, device="cuda")
    slots = torch.arange(32, device="cuda").flip(0).contiguous()
    r.mx4_write(q, x, x.flip(2).contiguous(), zero, slots, kp, vp)
    turned = x.double().cpu().numpy()
    # the partner of an infinity or a NaN is y cos 0 + x sin 0 = y + x * 0: NaN as well
    a, b = turned[..., :128].copy(), turned[..., 128:].copy()
    turned = np.concatenate([np.where(np.isfinite(b), a, np.nan), np.where(np.isfinite(a), b, np.nan)], -1)
    codes, s = M.quantise(turned)
    wk, wv = M.empty_pool(2, 16, 2), M.empty_pool(2, 16, 2)
    M.put(wk, slots.cpu().numpy(), codes, s, False)
    codes, s = M.quantise(x.flip(2).double().cpu().numpy())
    M.put(wv, slots.cpu().numpy(), codes, s, True)
    # (a number that rounds to zero may keep its sign or not)
    for got, want, of_v in ((kp, wk, False), (vp, wv, True)):
        a, b = (M.get(p, np.arange(32), of_v) for p in (got.cpu().numpy(), want))
        assert np.array_equal(a[1], b[1])
        assert np.array_equal(M.numbers(*a), M.numbers(*b), equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float8_e5m2])
@pytest.mark.parametrize("T,Hkv,P", [(1, 1, 16), (17, 3, 48), (130, 4, 16), (1000, 1, 64)])
def test_read(T, Hkv, P, dtype):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    rng = np.random.default_rng(T)
    pages = -(-T // P) + 1
    pools = [rng.integers(0, 256, (pages, P // 16, Hkv, 2176), dtype=np.uint8) for _ in range(2)]
    for p in pools:  # scales near one, a NaN block here and there
        p[..., 2048:] = rng.integers(120, 134, p[..., 2048:].shape)
        p[..., 2048:][rng.random(p[..., 2048:].shape) < 0.01] = 255
    slots = rng.integers(0, pages * P, T)  # some twice
    if T > 1:
        slots[3], slots[T // 2] = -1, pages * P + 7
    cache = B.Mx4Cache(Hkv, D, P, pages)
    kp, vp = (torch.from_numpy(p).cuda() for p in pools)
    big = torch.full((T, 2 * Hkv + 1, D), 1.0, device="cuda").to(dtype)
    k_out, v_out = big[:, :Hkv], big[:, Hkv + 1:]
    cache.read(kp, vp, torch.from_numpy(slots).cuda(), k_out=k_out, v_out=v_out)
    on = (slots >= 0) & (slots < pages * P)
    for got, pool, of_v in ((k_out, pools[0], False), (v_out, pools[1], True)):
        got = got.float().cpu().numpy()
        want = M.numbers(*M.get(pool, slots[on], of_v))
        assert np.array_equal(got[on], want.astype(np.float32), equal_nan=True)
        assert (got[~on] == 1).all()
    assert (big[:, Hkv].float() == 1).all()
    only = cache.read(None, vp, torch.from_numpy(slots).cuda(), dtype=dtype)
    assert only[0] is None
    keep = torch.from_numpy(on).cuda()
    assert np.array_equal(only[1][keep].float().cpu().numpy(), v_out[keep].float().cpu().numpy(),
                          equal_nan=True)
    assert cache.read_flags() == (B.DFLASH_FLAG_SLOT_RANGE if T > 1 else 0)


def test_read_past_a_types_range():
    from speculative_verify_paged_e4m3_gb300 import binding as B
    pool = M.empty_pool(1, 16, 1)
    codes = np.full((3, 1, 256), 7, dtype=np.uint8)
    scales = np.array([[[254] * 8], [[0] * 8], [[127 - 25] * 8]], dtype=np.uint8)
    M.put(pool, [0, 1, 2], codes, scales, False)
    cache = B.Mx4Cache(1, D, 16, 1)
    slots = torch.arange(3, device="cuda")
    p = torch.from_numpy(pool).cuda()
    half = cache.read(p, None, slots)[0].float()
    assert half[0].isinf().all() and (half[1] == 0).all() and (half[2] == 6 * 2.0 ** -24 / 2).all()
    wide = cache.read(p, None, slots, dtype=torch.bfloat16)[0].float()
    assert (wide[1] == 6 * 2.0 ** -127).all() and wide[0].isinf().all()
    assert (cache.read(p, None, slots, dtype=torch.float8_e5m2)[0].float()[0] == 57344).all()


def test_padding_and_prefix_tokens_by_token_starts():
    from speculative_verify_paged_e4m3_gb300 import binding as B
    q, k, v, pos, qw, kw = make(8, 6, 6, 1, torch.float16)
    slots = torch.tensor([-1, 3, -1, 4, -1, -1], device="cuda")
    starts = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    r = B.Rotary(6, 1, D, page_size=16, num_pages=1)
    cache = B.Mx4Cache(1, D, 16, 1)
    kp, vp = cache.empty()
    norm = B.HeadNorm(qw, kw)
    out = torch.full_like(q, 9.0)
    r.mx4_write(q, k, v, pos, slots, kp, vp, q_out=out, norm=norm, token_starts=starts)
    want, _ = r.apply(q, k, pos, norm=norm)
    assert torch.equal(out[:4], want[:4]) and (out[4:] == 9).all()
    assert set(kp.flatten()[2048:].view(16, 8).any(1).nonzero().flatten().tolist()) == {3, 4}


def test_refusals():
    from speculative_verify_paged_e4m3_gb300 import binding as B
    q, k, v, pos, qw, kw = make(9, 4, 6, 1, torch.float16)
    r = B.Rotary(6, 1, D, page_size=16, num_pages=1)
    cache = B.Mx4Cache(1, D, 16, 1)
    kp, vp = cache.empty()
    slots = torch.arange(4, device="cuda")
    for bad in (B.HeadNorm(qw.float(), kw), B.HeadNorm(qw, kw[:128]), B.HeadNorm(qw.cpu(), kw)):
        with pytest.raises(ValueError):
            r.apply(q, k, pos, norm=bad)
        with pytest.raises(ValueError):
            r.mx4_write(q, k, v, pos, slots, kp, vp, norm=bad)
    with pytest.raises(B.DflashError):
        r.apply(q, k, pos, norm=B.HeadNorm(qw, kw, -1.0))
    with pytest.raises(ValueError):
        r.mx4_write(q, k, v, pos, slots, kp[..., :-1].contiguous(), vp)
    with pytest.raises(ValueError):
        r.mx4_write(q, k, v, pos, slots.int(), kp, vp)
    with pytest.raises(B.DflashError):
        r.mx4_write(q, k, v, pos, slots, kp, kp)
    for args in ((1, D, 24, 1), (1, 128, 16, 1)):
        with pytest.raises(B.DflashError):
            B.Mx4Cache(*args)
    with pytest.raises(ValueError):
        B.Mx4Cache(0, D, 16, 1)
    with pytest.raises(ValueError):
        cache.read(kp, vp, slots, dtype=torch.float32)
    with pytest.raises(ValueError):
        cache.read(None, vp, slots, k_out=torch.empty((4, 1, D), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        cache.read(kp, vp, slots, k_out=torch.empty((4, 1, D), dtype=torch.float16, device="cuda"),
                   v_out=torch.empty((4, 1, D), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(B.DflashError):
        cache.read(None, None, slots)


def test_pools_past_32_bit_offsets():
    """The last slots of pools of more than 2^32 bytes."""
    from speculative_verify_paged_e4m3_gb300 import binding as B
    P, Hkv = 64, 4
    pages = (1 << 32) // (4 * Hkv * 2176) + 5
    cache = B.Mx4Cache(Hkv, D, P, pages)
    kp, vp = cache.empty()
    assert kp.numel() > 1 << 32
    q, k, v, pos, _, _ = make(10, 20, 4, Hkv, torch.float16)
    slots = torch.arange(pages * P - 20, pages * P, device="cuda")
    r = B.Rotary(4, Hkv, D, page_size=P, num_pages=pages)
    r.mx4_write(q, k, v, torch.zeros_like(pos), slots, kp, vp)
    gk, gv = cache.read(kp, vp, slots)
    for got, x in ((gk, k), (gv, v)):
        want = M.numbers(*M.quantise(x.double().cpu().numpy()))
        assert np.array_equal(got.double().cpu().numpy(), want)
    assert not kp[:8].any() and r.read_flags() == 0 and cache.read_flags() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,Hq,Hkv", [(1535, 20, 4), (4099, 24, 4), (1024, 7, 2)])
def test_many_tokens_of_many_heads(T, Hq, Hkv, dtype, layout):
    """Held to the formula, and bit for bit to calls of few tokens: each destination, in place, with padding and
    slots past the pool."""
    from speculative_verify_paged_e4m3_gb300 import binding as B
    test_norm_rope_apply(T, Hq, Hkv, dtype, layout)
    P, pages = 16, -(-T // 16) + 3
    q, k, v, pos, qw, kw = make(T + 2, T, Hq, Hkv, dtype, fused=True)
    norm = B.HeadNorm(qw, kw, 1e-5, 0.5)
    r = B.Rotary(Hq, Hkv, D, 64, layout=layout, dtype=dtype, page_size=P, num_pages=pages)
    rng = np.random.default_rng(T)
    slots = rng.permutation(pages * P)[:T]
    slots[[0, 9, 600, T - 1]] = -1
    slots[1000] = pages * P
    slots = torch.from_numpy(slots).cuda()
    starts = torch.tensor([0, 17], dtype=torch.int32, device="cuda")  # tokens 0 and 9 are not padding
    scales = [torch.tensor([x], device="cuda") for x in (0.02, 0.03)]
    cache = B.Mx4Cache(Hkv, D, P, pages)

    def run(step, in_place):
        e = [torch.full((pages, P, Hkv, D), 7, dtype=torch.uint8, device="cuda") for _ in range(2)]
        m = cache.empty()
        outs = [x.clone() if in_place else torch.full_like(x, 9.0) for x in (q, k, q, q)]
        for a in range(0, T, step):
            b = min(a + step, T)
            live = torch.clamp(starts - a, min=0)
            src = outs if in_place else (q, k, q, q)
            r.apply(src[0][a:b], src[1][a:b], pos[a:b], q_out=outs[0][a:b], k_out=outs[1][a:b], norm=norm)
            r.kv_write(src[2][a:b], k[a:b], v[a:b], pos[a:b], slots[a:b], *scales, *e, q_out=outs[2][a:b],
                       norm=norm, token_starts=live)
            r.mx4_write(src[3][a:b], k[a:b], v[a:b], pos[a:b], slots[a:b], *m, q_out=outs[3][a:b],
                        norm=norm, token_starts=live)
        return outs + e + list(m)
    few, many, there = run(300, False), run(T, False), run(T, True)
    for i, (a, b) in enumerate(zip(few, many)):
        assert torch.equal(a, b), i
    padding = (slots < 0).cpu().numpy() & (np.arange(T) >= 17)
    for i, (a, b) in enumerate(zip(many, there)):
        keep = torch.from_numpy(~padding).cuda() if i in (2, 3) else slice(None)
        assert torch.equal(a[keep], b[keep]), i
    assert r.read_flags() == B.DFLASH_FLAG_SLOT_RANGE
