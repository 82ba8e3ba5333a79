"""The 4-bit attention's pipeline as long as in use: one split a head, so that a CTA goes over every tile of a
context. Tolerances are those that test_gpu_mx4_attn.py derives; what a test is about (references that move,
weights in FP16's fixed step) is asserted from its scores, worked out here in 64 bits."""
import numpy as np
import pytest
import torch

import mx4_reference as M
from test_gpu_mx4_attn import D, built, check, dev, make, problem  # noqa: F401 (built: a fixture)

pytestmark = pytest.mark.gpu

TILE, SHIFT, MOVE = 128, 8.0, 15.0  # keys a tile, a new reference's exponent, the one that moves it
ROWS = {16: (6, 1, 1), 32: (6, 1, 5), 48: (6, 1, 8)}  # rows a CTA carries: heads, KV heads, tokens


@pytest.mark.parametrize("rows,P,tiles,end", [
    (16, 16, 13, 1), (16, 48, 40, 50), (16, 64, 24, 128), (32, 48, 21, 127), (32, 16, 33, 17),
    (48, 48, 13, 1), (48, 16, 40, 50), (48, 64, 21, 127), (48, 48, 24, 128)])
def test_many_tiles_of_one_split(rows, P, tiles, end):
    Hq, Hkv, q_len = ROWS[rows]
    lens = [(tiles - 1) * TILE + end, (tiles // 2) * TILE + end]
    pr = problem(tiles + rows, lens, q_len, Hq, Hkv, P, gain=1.5)
    att = make(pr, num_splits=1)
    assert att.plan.num_splits == 1 and att.plan.row_blocks == 1
    check(att(*dev(pr)), pr)
    assert att.read_flags() in (0, 2)


def test_many_tiles_of_row_blocks_and_heads():
    pr = problem(5, [3001], 10, 24, 4, 16)  # 60 rows: two blocks of 30
    att = make(pr, num_splits=1)
    assert att.plan.row_blocks == 2
    check(att(*dev(pr)), pr)


def slots_of(pr, b=0):
    n, P = int(pr["lens"][b]), pr["P"]
    j = np.arange(n)
    return pr["table"][b, j // P].astype(np.int64) * P + j % P


def exponents(pr, row):
    """Of the first request's row: each key's score and its V's largest power, in bits."""
    i, hq = row
    slots = slots_of(pr)
    k = M.numbers(*M.get(pr["k"], slots, False))[:, 0]
    ev = M.get(pr["v"], slots, True)[1][:, 0].astype(int).max(-1) - 127
    s = k @ pr["q"][0, i, hq].astype(np.float64) / 16 * np.log2(np.e)
    return s, ev


def moves(s, ev):
    """Tiles past the first that move a row's reference, and what each multiplies its sums by (in bits)."""
    x = s + ev
    ref, got = x[:TILE].max(), []
    for t in range(1, -(-len(x) // TILE)):
        top = x[t * TILE:(t + 1) * TILE].max()
        if top - ref + SHIFT > MOVE:
            got.append((t, ref - top))
            ref = top
    return got


def row_without_a_move(pr, row, skip):
    """The row's output if the sums before tile `skip` were not brought to the new reference."""
    s, ev = exponents(pr, row)
    v = M.numbers(*M.get(pr["v"], slots_of(pr), True))[:, 0]
    bits = dict(moves(s, ev))[skip]
    w = np.exp2(s - s.max())
    w[:skip * TILE] *= 2.0 ** -bits
    return w @ v / w.sum()


@pytest.mark.parametrize("rows", [16, 32, 48])
@pytest.mark.parametrize("growth", [3.0, 7.5, 12.0])
def test_references_that_move_again_and_again(rows, growth):
    """Each tile's best score is `growth` bits above the one's before it, for 20 tiles; then a tail below. Other rows
    have references that move less, or never (their queries point the other way)."""
    Hq, Hkv, q_len = ROWS[rows]
    n = 25 * TILE + 37
    pr = problem(int(growth) + rows, [n], q_len, Hq, Hkv, 16)
    rng = np.random.default_rng(rows)
    q0 = rng.standard_normal(D)
    share = np.linspace(1.0, 0.3, q_len * Hq) * np.where(np.arange(q_len * Hq) % 5 == 4, -1, 1)
    pr["q"] = (share[:, None] * q0).reshape(1, q_len, Hq, D).astype(np.float16)
    bits = np.minimum(np.arange(n) // TILE, 20) * growth + rng.uniform(-2, 0, n)
    bits[21 * TILE:] -= 4
    unit = 16 * np.log(2) / (q0 @ q0)  # a bit of score along q0
    x = rng.standard_normal((pr["k"].shape[0] * 16, 1, D)) * 0.3
    x -= (x @ q0)[..., None] / (q0 @ q0) * q0
    slots = slots_of(pr)
    x[slots, 0] += (bits * unit)[:, None] * q0
    codes, sc = M.quantise(x)
    pr["k"][:] = 0
    M.put(pr["k"], np.arange(len(x)), codes, sc, False)
    row = (q_len - 1, 0) if q_len == 1 else (0, 0)
    late = [t for t, _ in moves(*exponents(pr, row)) if t >= 2]
    assert len(late) >= (5 if growth < 7 else 12), late
    want = M.attention(pr["q"], pr["k"], pr["v"], pr["table"], pr["lens"], 16)
    if growth < 7:  # the tiles before a move still count: without the rescaling the row would be another
        with pytest.raises(AssertionError):
            wrong = want[0].copy()
            wrong[0, row[0], row[1]] = row_without_a_move(pr, row, late[-1])
            check((torch.from_numpy(wrong), torch.from_numpy(want[1])), pr, want)
    check(make(pr, num_splits=1)(*dev(pr)), pr, want)


@pytest.mark.parametrize("rows", [16, 48])
def test_references_that_move_with_growing_values(rows):
    """V's powers grow by a factor of four a tile: the reference of weights moves with them, lse does not know."""
    Hq, Hkv, q_len = ROWS[rows]
    n = 14 * TILE + 5
    pr = problem(rows, [n], q_len, Hq, Hkv, 16)
    slots = slots_of(pr)
    flat = pr["v"].reshape(-1, Hkv, 2176)
    for j, s in enumerate(slots):
        flat[s // 16, 0, 2048 + 8 * (s % 16):2056 + 8 * (s % 16)] += np.uint8((2 * (j // TILE) - 20) % 256)
    late = [t for t, _ in moves(*exponents(pr, (0, 0))) if t >= 2]
    assert len(late) >= 2, late
    check(make(pr, num_splits=1)(*dev(pr)), pr)


@pytest.mark.parametrize("bits", [14.3, 22.6, 25.2, 30.0])
def test_a_strong_key_in_front_of_many_in_one_split(bits):
    """One key of nearly all the weight and 60000 equal small ones, under one reference: the small weights lie
    in FP16's fixed step (below 2^-14 with the shift of 2^8) from 22 bits on."""
    n = 60000
    pr = problem(13, [n], 1, 6, 1, 64)
    pr["k"][:] = 0
    pr["k"][..., 2048:] = 127
    u = np.zeros((1, 1, D))
    u[..., :32] = 1.0
    pr["q"] = np.zeros((1, 1, 6, D), dtype=np.float16)
    pr["q"][..., :32] = bits * np.log(2) * 16 / 32 / 6
    codes, s = M.quantise(u * 6.0)
    M.put(pr["k"], [int(pr["table"][0, 0]) * 64], codes, s, False)
    s, ev = exponents(pr, (0, 0))
    assert abs(s[0] - s[1] - bits) < 0.1 and (s[1:] == s[1]).all()
    small = s[1] + ev[1:].max() - (s[0] + ev[0]) + SHIFT  # exponent of the small weights
    assert (small < -14) == (bits > 23)
    check(make(pr, num_splits=1)(*dev(pr)), pr)


@pytest.mark.parametrize("k_shift,q_shift", [(-12, 12), (10, -10), (5, -5), (20, None)])
@pytest.mark.parametrize("v_shift", [-30, -12, 9, 13])
def test_numbers_of_any_size_with_scores_of_order_one(k_shift, q_shift, v_shift):
    """K's and V's scales far from one, each on its own, and Q's so that scores stay where they matter: FP16's
    subnormal numbers, a few steps of 2^-24, for the largest K."""
    pr = problem(18 + k_shift, [700, 90], 4, 6, 1, 16)
    pr["k"][..., 2048:] += np.uint8(k_shift % 256)
    pr["v"][..., 2048:] += np.uint8(v_shift % 256)
    if q_shift is None:
        steps = np.random.default_rng(1).integers(-16, 17, pr["q"].shape)
        pr["q"] = (steps * 2.0 ** -24).astype(np.float16)
        assert (pr["q"].astype(np.float64) * 2 ** 24 == steps).all()
    else:
        pr["q"] = (pr["q"].astype(np.float64) * 2.0 ** q_shift).astype(np.float16)
    want = M.attention(pr["q"], pr["k"], pr["v"], pr["table"], pr["lens"], 16)
    s, _ = exponents(pr, (0, 0))
    assert 1.0 < s.max() - s.min() < 100.0 and np.abs(want[0]).max() < 60000
    check(make(pr)(*dev(pr)), pr, want)
