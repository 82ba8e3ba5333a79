"""How the 4-bit attention's plans share a batch's slots out, by the host's statement of the rule: no sequence is left
to a single CTA because there are many others, and short batches are not cut up. Without a GPU (152 SMs)."""
import numpy as np
import pytest

SMS = 152


@pytest.fixture(scope="module")
def B():
    from speculative_verify_paged_e4m3_gb300 import binding, build
    build.build()
    return binding


def plan(B, batch, heads, q_len, context, splits=0):
    return B.dflash_mx4_attn_plan(B.make_problem(batch, q_len, *heads, 256, 64, -(-context // 64), 1 << 20,
                                                 context, -1, splits, 0, 0))


def split_tiles(B, p, lens):
    """(tiles of the longest split, CTAs with keys, tiles of all CTAs)"""
    start, per, act = B.dflash_verify_attn_split_slots(p, lens)
    assert start[-1] <= p.num_slots
    n = np.repeat(np.asarray(lens), p.problem.num_kv_heads)
    per, act, count = np.asarray(per), np.asarray(act), np.diff(np.asarray(start))
    assert ((act > 0) == (n > 0)).all() and (act <= count).all()
    assert (per * act >= n).all()  # every key is some split's
    return int(per.max()) // 128, int(act.sum()) * p.row_blocks, int((-(-n // 128)).sum()) * p.row_blocks


@pytest.mark.parametrize("heads,q_len", [((24, 4), 1), ((24, 4), 8), ((6, 1), 8), ((8, 1), 8)])
@pytest.mark.parametrize("batch", [19, 24, 38, 39, 40, 64, 100, 160, 300])
def test_one_long_sequence_among_many(B, batch, heads, q_len):
    context = 262144
    p = plan(B, batch, heads, q_len, context)
    lens = [1000] * batch
    lens[batch // 2] = context
    longest, ctas, tiles = split_tiles(B, p, lens)
    mean = tiles / SMS
    # one SM's fair share and what a unit's own slot takes of the rounds
    assert longest <= 2 * mean + 16, (longest, mean, ctas)


@pytest.mark.parametrize("batch", [24, 39, 48, 64, 96])
@pytest.mark.parametrize("context", [4096, 16384])
def test_ragged_batches_keep_near_an_even_share(B, batch, context):
    lens = np.random.default_rng(batch).integers(context // 3, context + 1, batch)
    for capacity in (context, 262144):  # what a plan has room for does not matter
        longest, ctas, tiles = split_tiles(B, plan(B, batch, (24, 4), 1, capacity), lens.tolist())
        rounds = -(-ctas // SMS)
        assert rounds * (longest + 4) <= 1.6 * (tiles / SMS + 4 * rounds) + 4, (longest, ctas, tiles / SMS)


@pytest.mark.parametrize("batch", [20, 32, 38, 64, 96])
@pytest.mark.parametrize("context", [4096, 262144])
def test_short_sequences_are_not_cut_up(B, batch, context):
    """8 tiles each: one slot a unit, or one round's, whatever the plan has room for."""
    longest, ctas, _ = split_tiles(B, plan(B, batch, (24, 4), 1, context), [1000] * batch)
    assert ctas <= max(SMS, batch * 4)


def test_slots_of_plans(B):
    for batch, slots in ((10, 152), (19, 152), (20, 304), (38, 304), (57, 304), (58, 456), (100, 608)):
        assert plan(B, batch, (24, 4), 1, 262144).num_slots == slots, batch
        assert plan(B, batch, (24, 4), 1, 2048).num_slots == max(152, 4 * batch), batch
        assert plan(B, batch, (24, 4), 1, 4096).num_slots == (152 if batch <= 38 else slots), batch
        assert plan(B, batch, (24, 4), 1, 262144, splits=1).num_slots == 4 * batch
    p = plan(B, 30, (24, 4), 10, 262144)  # row blocks of 30 rows: 76 slots a round, 120 units
    assert p.row_blocks == 2 and p.num_slots == 228
    assert p.workspace_bytes >= p.ws_acc_offset + p.num_slots * p.rows * 1024
    assert p.ws_acc_offset >= p.ws_state_offset + p.num_slots * p.rows * 8


def test_more_units_than_a_grid_takes_are_refused_by_the_plan(B):
    assert plan(B, 16383, (24, 4), 1, 4096).num_slots >= 65532
    for batch, heads in ((16384, (24, 4)), (1, (65536, 65536))):
        with pytest.raises(B.DflashError) as e:
            plan(B, batch, heads, 1, 4096)
        assert e.value.status == B.DFLASH_ERR_UNSUPPORTED


def test_empty_and_single_sequences(B):
    p = plan(B, 64, (24, 4), 1, 32768)
    start, per, act = B.dflash_verify_attn_split_slots(p, [0] * 64)
    assert start[-1] == 0 and not any(act)
    lens = [0] * 64
    lens[40] = 32768
    longest, ctas, tiles = split_tiles(B, p, lens)
    assert ctas >= 128 and longest <= 8
