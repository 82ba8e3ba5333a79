"""Contexts whose key indices would not fit 32 bits are refused by every attention's plan, without a GPU."""
import pytest


@pytest.fixture(scope="module")
def B():
    from speculative_verify_paged_e4m3_gb300 import binding, build
    build.build()
    return binding


PAGE = 1 << 20


def problem(B, context, batch, splits):
    return B.make_problem(batch, 8, 6, 1, 256, PAGE, -(-context // PAGE), 4, context, -1, splits, 0, 0)


@pytest.mark.parametrize("batch,splits", [(1, 0), (1, 65535), (3, 0), (3, 7)])
@pytest.mark.parametrize("plan", ["dflash_verify_attn_plan", "dflash_mx4_attn_plan"])
def test_largest_context(B, plan, batch, splits):
    make = getattr(B, plan)
    for context, fine in ((1 << 30, True), ((1 << 30) + 1, False), ((1 << 31) - 1, False)):
        if fine:
            p = make(problem(B, context, batch, splits))
            # the furthest key that an index reaches: behind the last split, some tiles on
            per = max(-(-context // p.num_splits), p.min_split_keys) + p.tile_keys
            assert p.num_splits * per + 16 * p.tile_keys < 1 << 31
        else:
            with pytest.raises(B.DflashError) as e:
                make(problem(B, context, batch, splits))
            assert e.value.status == B.DFLASH_ERR_UNSUPPORTED


def test_largest_context_of_a_shared_prefix(B):
    for context, fine in ((1 << 30, True), ((1 << 30) + 1, False)):
        pr = B.make_prefix_problem(4, 8, 6, 1, 256, PAGE, -(-context // PAGE), 4, context, PAGE, -1)
        if fine:
            B.dflash_prefix_attn_plan(pr)
        else:
            with pytest.raises(B.DflashError) as e:
                B.dflash_prefix_attn_plan(pr)
            assert e.value.status == B.DFLASH_ERR_UNSUPPORTED
