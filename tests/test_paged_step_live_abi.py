"""The cache write with a count of live tokens, its C ABI without a GPU: refusals before any launch."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def B():
    from speculative_verify_paged_e4m3_gb300 import binding, build
    build.build()
    return binding


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), 0), (dict(T=-1), -1), (dict(live=0xd0002), -1), (dict(q=0), -1), (dict(slots=0x50004), -1),
    (dict(status=0), -1), (dict(qs=1528), -1), (dict(kp=0xd0000), -1), (dict(status=0xd0000), -1),
    (dict(qo=0xd0000), -1), (dict(vp=0x30000), -1)])
def test_refusals(B, bad, status):
    plan, _ = B.dflash_rope_plan(B.make_rope_problem(6, 2, 256, 128, page_size=16, num_pages=4))
    a = dict(T=4, q=0x10000, qs=1536, k=0x20000, v=0x30000, pos=0x40000, slots=0x50000, ph=0x60000,
             ks_=0x70000, vs_=0x80000, qo=0x90000, kp=0xa0000, vp=0xb0000, status=0xc0000, live=0xd0000)
    a.update(bad)
    assert B.load_library().dflash_rope_kv_write_live(
        ctypes.byref(plan), a["T"], a["q"], a["qs"], a["k"], 512, a["v"], 512, a["pos"], a["slots"],
        a["live"], a["ph"], a["ks_"], a["vs_"], a["qo"], 1536, a["kp"], a["vp"], a["status"], None) == status


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("max_prefix,page,table,length,status", [
    (16, 16, 0, 1, -1), (15, 16, 0, 0, -1), (15, 16, 0, 1, -3), (0, 16, 0, 0, -3), (16, 16, 1, 1, -3)])
def test_a_prefix_without_a_whole_page_needs_no_table(B, kernel, max_prefix, page, table, length, status):
    """(Calls that pass the pointer checks are refused for their workspace, before any launch.)"""
    plan = B.dflash_prefix_attn_plan(B.make_prefix_problem(4, 8, 6, 1, 256, page, 64, 256, 1024, max_prefix, -1,
                                                           kernel))
    at = [0x100000 * (i + 1) for i in range(12)]
    assert B.load_library().dflash_prefix_attn_forward(
        ctypes.byref(plan), at[0], at[1], at[2], at[3] * table, at[4] * length, at[5], at[6], at[7], at[8],
        at[9], 1024, at[10], at[11], None) == status
