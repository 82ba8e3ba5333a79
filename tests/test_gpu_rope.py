"""Rotary positions, alone and with the E4M3 cache write, against complex arithmetic in 64 bits.

Tolerance of a rotated element of the pair (x, y), derived: the fraction of a turn is off by at most
2^-32 (the bits cut) + 2^-25 (its FP32 rounding, at most half a turn), 2^-24.9 turns or 2.0e-7 rad;
sine and cosine by 2 units of 2^-24; the amplitude and its product by 2^-24 each; the rotation by
three roundings. All are relative to amp (|x| + |y|): below 2.0e-7 + 7 * 2^-24 = 6.2e-7 < 2^-20.
The rounding to the output type adds eps / 2 of the value (and half the smallest FP16 subnormal).
"""
import math

import numpy as np
import pytest
import torch

from test_paged_step_abi import frequencies

pytestmark = pytest.mark.gpu

D = 256
ARITH = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()


def exact(x, pos, theta, amp, d, layout):
    """x [T, H, D] float64 rotated, and amp (|x| + |y|) of each element's pair."""
    z, mag = x.copy(), np.abs(x)
    i = np.arange(d // 2)
    a, b = (i, i + d // 2) if layout == "half" else (2 * i, 2 * i + 1)
    turn = amp * np.exp(1j * np.outer(pos.astype(np.float64), theta))[:, None]
    w = (x[..., a] + 1j * x[..., b]) * turn
    z[..., a], z[..., b] = w.real, w.imag
    mag[..., a] = mag[..., b] = amp * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return z, mag


def check(got, want, mag, dtype, d):
    err = np.abs(got.double().cpu().numpy() - want)
    tol = torch.finfo(dtype).eps / 2 * np.abs(want) * (1 + ARITH) + ARITH * mag + 2.0 ** -25
    assert (err <= tol).all(), (err - tol).max()
    # elements past the rotated part pass through
    assert np.array_equal(got.double().cpu().numpy()[..., d:], want[..., d:])


def make(seed, T, Hq, Hkv, dtype, far, fused=False):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g).to(dtype).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32)
    pos[0] = far - 1
    return q, k, v, pos.cuda()


def rotary(Hq, Hkv, d, layout, dtype, scaling="none", **kw):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    r = B.Rotary(Hq, Hkv, D, d, layout=layout, dtype=dtype, base=500000.0, scaling=scaling,
                 factor=8.0, trained_context=8192, **kw)
    theta = np.array(frequencies(d, 500000.0, scaling, 8.0, 8192))
    return r, theta, 0.1 * math.log(8.0) + 1.0 if scaling == "yarn" else 1.0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d", [16, 48, 64, 128, 240, 256])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
def test_apply(layout, d, dtype):
    T, Hq, Hkv = 37, 6, 1
    q, k, _, pos = make(d, T, Hq, Hkv, dtype, 262144)
    r, theta, amp = rotary(Hq, Hkv, d, layout, dtype)
    qo, ko = r.apply(q, k, pos)
    for x, y in ((q, qo), (k, ko)):
        want, mag = exact(x.double().cpu().numpy(), pos.cpu().numpy(), theta, amp, d, layout)
        check(y, want, mag, dtype, d)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn", "wavelength"])
@pytest.mark.parametrize("far", [1, 20, 2 ** 20, 2 ** 31 - 1])
def test_apply_scaled_and_far(scaling, far):
    q, k, _, pos = make(far % 97, 19, 24, 4, torch.float16, far, fused=True)
    r, theta, amp = rotary(24, 4, 128, "half", torch.float16, scaling)
    qo, ko = r.apply(q, k, pos)
    # 64-bit angles t * theta are themselves off by t * theta * 2^-52 at the farthest position
    slack = far * 2.0 ** -51
    for x, y in ((q, qo), (k, ko)):
        want, mag = exact(x.double().cpu().numpy(), pos.cpu().numpy(), theta, amp, 128, "half")
        check(y, want, mag * (1 + slack / ARITH), torch.float16, 128)


@pytest.mark.parametrize("T", [1, 2, 1000])
@pytest.mark.parametrize("heads", [(1, 1), (24, 4), (16, 16), (9, 3)])
def test_apply_in_place_is_the_same(T, heads):
    q, k, _, pos = make(T, T, *heads, torch.float16, 5000)
    r, _, _ = rotary(*heads, 256, "half", torch.float16)
    qo, ko = r.apply(q, k, pos)
    q2, k2 = q.clone(), k.clone()
    r.apply(q2, k2, pos, q_out=q2, k_out=k2)
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    qo2, none = r.apply(q, None, pos)
    assert torch.equal(qo, qo2) and none is None


def test_unrotated_part_keeps_infinities_and_nan():
    q, k, _, pos = make(3, 5, 2, 1, torch.float16, 100)
    q[:, :, 200] = math.inf
    q[:, :, 255] = math.nan
    for layout in ("half", "interleaved"):
        r, _, _ = rotary(2, 1, 64, layout, torch.float16)
        qo, _ = r.apply(q, k, pos)
        assert torch.isinf(qo[:, :, 200]).all() and torch.isnan(qo[:, :, 255]).all()
        assert torch.isfinite(qo[:, :, :200]).all()


def test_position_zero_is_the_identity():
    q, k, _, _ = make(4, 3, 6, 1, torch.bfloat16, 10)
    r, _, _ = rotary(6, 1, 256, "interleaved", torch.bfloat16)
    qo, ko = r.apply(q, k, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert torch.equal(qo, q) and torch.equal(ko, k)


def test_scores_depend_on_distance_alone():
    """Rotated q and k have the dot product of the same pair moved along together, up to the FP16
    roundings of both: |q||k| 2^-10 bounds their sum."""
    q, k, _, _ = make(6, 1, 1, 1, torch.float16, 10)
    r, _, _ = rotary(1, 1, 256, "half", torch.float16)

    def dot(t):
        p = torch.tensor([t], dtype=torch.int32, device="cuda")
        p2 = torch.tensor([t + 77], dtype=torch.int32, device="cuda")
        return (r.apply(q, None, p2)[0].double() * r.apply(k, None, p)[0].double()).sum().item()
    lim = q.double().norm().item() * k.double().norm().item() * 2.0 ** -10
    assert all(abs(dot(t) - dot(0)) <= lim for t in (1, 1000, 262143))


# ----------------------------------------------------------------------------- cache write

def nearest_ok(codes, u, slack):
    """Every code is the E4M3 value nearest to u (saturated), up to slack in u."""
    got = codes.view(torch.float8_e4m3fn).double().cpu().numpy()
    grid = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    grid = np.unique(grid[np.isfinite(grid)])
    c = np.clip(u, -448, 448)
    hi = np.clip(np.searchsorted(grid, c), 1, len(grid) - 1)
    best = np.minimum(np.abs(grid[hi] - c), np.abs(grid[hi - 1] - c))
    return np.isfinite(got).all() and (np.abs(got - c) <= best + 2 * slack).all()


def v_codes(v, scale):
    """Codes of v / scale: one FP32 division and the library's cast of the saturated value."""
    x = v.float().cpu() / torch.tensor(scale, dtype=torch.float32)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


@pytest.mark.parametrize("layout,d,scaling", [("half", 256, "none"), ("interleaved", 64, "yarn"),
                                              ("half", 112, "linear")])
@pytest.mark.parametrize("T,heads,P,dtype,fused", [
    (1, (6, 1), 16, torch.float16, False), (8, (6, 1), 16, torch.float16, True),
    (131, (24, 4), 48, torch.bfloat16, True), (700, (8, 8), 64, torch.float16, False)])
def test_kv_write(layout, d, scaling, T, heads, P, dtype, fused):
    Hq, Hkv = heads
    q, k, v, pos = make(T + d, T, Hq, Hkv, dtype, 262144, fused)
    num_pages = -(-T // P) + 2
    r, theta, amp = rotary(Hq, Hkv, d, layout, dtype, scaling, page_size=P, num_pages=num_pages)
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(num_pages * P, generator=g)[:T]
    if T > 4:
        slots[::5] = -1
        slots[1] = -2 ** 40
    pools = [torch.randint(0, 256, (num_pages, P, Hkv, D), generator=g, dtype=torch.uint8)
             for _ in range(2)]
    ks, vs = 0.0061, 0.0123  # the largest of a few hundred normal values saturate
    kp, vp = (p.cuda() for p in pools)
    qo = torch.full((T, Hq, D), 7.0, dtype=dtype, device="cuda")

    def one(x):
        return torch.tensor([x], dtype=torch.float32, device="cuda")
    r.kv_write(q, k, v, pos, slots.cuda(), one(ks), one(vs), kp, vp, q_out=qo)
    live = (slots >= 0).numpy()
    at = slots[slots >= 0].numpy()
    want_q, mag_q = exact(q.double().cpu().numpy(), pos.cpu().numpy(), theta, amp, d, layout)
    check(qo[live], want_q[live], mag_q[live], dtype, d)
    assert (qo[~live] == 7.0).all()  # padding is left as it was
    want_k, mag_k = exact(k.double().cpu().numpy(), pos.cpu().numpy(), theta, amp, d, layout)
    s64 = float(np.float32(ks))
    flat = kp.cpu().view(-1, Hkv, D)
    assert nearest_ok(flat[at], want_k[live] / s64, (ARITH * mag_k[live] + 2.0 ** -23 *
                                                     np.abs(want_k[live])) / s64)
    assert np.array_equal(vp.cpu().view(-1, Hkv, D)[at].numpy(), v_codes(v, vs)[live])
    # every other byte of the pools is as it was
    rest = np.ones(num_pages * P, bool)
    rest[at] = False
    for p, was in ((kp, pools[0]), (vp, pools[1])):
        assert np.array_equal(p.cpu().view(-1, Hkv, D)[rest].numpy(),
                              was.view(-1, Hkv, D)[rest].numpy())
    assert r.read_flags() == 0


@pytest.mark.parametrize("T", [759, 760, 761, 762, 4560, 4561, 4563, 9002])
@pytest.mark.parametrize("layout,d,dtype", [("half", 256, torch.float16),
                                            ("interleaved", 48, torch.bfloat16)])
@pytest.mark.parametrize("heads", [(6, 1), (2, 3), (1, 1)])
def test_many_tokens_of_few_heads_are_as_a_few_at_a_time(T, layout, d, dtype, heads):
    Hq, Hkv = heads
    q, k, v, pos = make(T + d, T, Hq, Hkv, dtype, 100000, True)
    pages = -(-T // 16)
    r, _, _ = rotary(Hq, Hkv, d, layout, dtype, page_size=16, num_pages=pages)
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * 16, generator=g)[:T]
    slots[::7] = -1
    slots[T - 2] = pages * 16  # past the pool: no write, a flag
    slots = slots.cuda()
    one = torch.ones(1, device="cuda")

    def run(parts):
        pools = [torch.full((pages, 16, Hkv, D), 7, dtype=torch.uint8, device="cuda")
                 for _ in range(2)]
        qo = torch.full((T, Hq, D), 5.0, dtype=dtype, device="cuda")
        qa = torch.empty((T, Hq, D), dtype=dtype, device="cuda")
        ka = torch.empty((T, Hkv, D), dtype=dtype, device="cuda")
        for part in torch.arange(T).split(parts):
            s = slice(int(part[0]), int(part[-1]) + 1)
            r.kv_write(q[s], k[s], v[s], pos[s], slots[s], one, one, *pools, q_out=qo[s])
            r.apply(q[s], k[s], pos[s], q_out=qa[s], k_out=ka[s])
        assert r.read_flags(clear=True) == 0x40
        return [qo, qa, ka] + pools
    for a, b in zip(run(T), run(500)):
        assert torch.equal(a, b)
    qa, ka = r.apply(q, k, pos)
    qi, ki = q.contiguous().clone(), k.contiguous().clone()
    r.apply(qi, ki, pos, q_out=qi, k_out=ki)
    assert torch.equal(qa, qi) and torch.equal(ka, ki)


def test_kv_write_special_values_and_slots_past_the_pool():
    r, _, _ = rotary(2, 1, 64, "half", torch.float16, page_size=16, num_pages=1)
    q, k, v, pos = make(1, 3, 2, 1, torch.float16, 9)
    v[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 65504.0])
    kp = torch.zeros((1, 16, 1, D), dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    s = torch.tensor([15, 16, 2 ** 33], dtype=torch.int64, device="cuda")
    one = torch.ones(1, device="cuda")
    qo = torch.full_like(q, 9.0)
    r.kv_write(q, k, v, pos, s, one, one, kp, vp, q_out=qo)
    c = vp[0, 15, 0, :4].cpu().tolist()
    assert c[0] == 0x7E and c[1] == 0xFE and c[2] & 0x7F == 0x7F and c[3] == 0x7E
    assert not vp[0, :15].any() and not kp[0, :15].any()
    assert (qo != 9.0).any(-1).all()
    assert r.read_flags(clear=True) == 0x40 and r.read_flags() == 0


def test_kv_write_matches_the_drafted_token_write():
    """At position 0 (no rotation) the bytes are those of the plain attention's KV write."""
    from speculative_verify_paged_e4m3_gb300 import binding as B
    T, P = 8, 16
    q, k, v, _ = make(2, T, 6, 1, torch.float16, 5)
    att = B.VerifyAttention(1, T, 6, 1, D, P, 4, 8, 64)
    table = torch.tensor([[5, 2, 7, 0]], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([40], dtype=torch.int32, device="cuda")
    ks, vs = torch.tensor([0.011], device="cuda"), torch.tensor([0.02], device="cuda")
    a, b = (torch.zeros((8, P, 1, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    att.kv_write(k.view(1, T, 1, D), v.view(1, T, 1, D), table, ctx, ks, vs, a, b)
    r, _, _ = rotary(6, 1, 256, "half", torch.float16, page_size=P, num_pages=8)
    a2, b2 = torch.zeros_like(a), torch.zeros_like(b)
    slots = torch.tensor([7 * P + i for i in range(8)], dtype=torch.int64, device="cuda")
    r.kv_write(q, k, v, torch.zeros(T, dtype=torch.int32, device="cuda"), slots, ks, vs, a2, b2)
    assert torch.equal(a, a2) and torch.equal(b, b2)


def test_refusals():
    r, _, _ = rotary(6, 2, 64, "half", torch.float16)
    q, k, v, pos = make(8, 4, 6, 2, torch.float16, 9)
    r.apply(q, k, pos)
    for a in ((q.bfloat16(), k, pos), (q[:3], k, pos), (q, k, pos.long()), (q, k[:, :1], pos),
              (q.transpose(0, 1), k, pos), (q[..., ::2], k, pos), (q, k, pos.cpu()),
              (q.cpu(), k, pos)):
        with pytest.raises(ValueError):
            r.apply(*a)
    wide = torch.zeros((4, 12, D), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):  # every other head
        r.apply(wide[:, ::2], k, pos)
    assert r.apply(q[:0], k[:0], pos[:0])[0].shape == (0, 6, D)
