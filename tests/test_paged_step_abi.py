"""The paged step's C ABI without a GPU: struct layouts, plans, rotary frequencies and refusals."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    from speculative_verify_paged_e4m3_gb300 import binding, build
    build.build()
    return binding


def test_struct_layouts_match_c(B, tmp_path):
    pairs = [("dflash_paged_tables_problem", B.PagedTablesProblem),
             ("dflash_rope_problem", B.RopeProblem), ("dflash_rope_plan_t", B.RopePlan),
             ("dflash_prefix_attn_problem", B.PrefixAttnProblem),
             ("dflash_prefix_attn_plan_t", B.PrefixAttnPlan)]
    lines = []
    for c, py in pairs:
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        lines += [f'printf("%zu\\n", offsetof({c}, {f[0]}));' for f in py._fields_]
    prog = tmp_path / "sizes.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dflash_paged_step.h"\n'
                    "int main(void){" + "".join(lines) + "return 0;}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = []
    for _, py in pairs:
        want.append(ctypes.sizeof(py))
        want += [getattr(py, f[0]).offset for f in py._fields_]
    assert got == want


# ------------------------------------------------------------------------------------ tables

def tables_call(B, bad=None, **kw):
    """dflash_paged_tables with host addresses that are never followed: every call here is refused
    before a launch."""
    args = dict(version=1, batch=4, page_size=16, max_pages_per_seq=8, num_pages=64,
                max_context=128, max_tokens=32, num_free=16, prefix_capacity=2)
    args.update(kw)
    pr = B.PagedTablesProblem(*[args[f[0]] for f in B.PagedTablesProblem._fields_])
    names = ["cached", "new", "held", "free", "head", "ptable", "ppages", "table", "ctx",
             "held_out", "head_out", "starts", "positions", "slots", "status"]
    ptrs = {n: 0x10000 + 0x1000 * i for i, n in enumerate(names)}
    ptrs.update(bad or {})
    return B.load_library().dflash_paged_tables(ctypes.byref(pr), *[ptrs[n] for n in names], None)


@pytest.mark.parametrize("kw,status", [
    (dict(version=7), -1), (dict(batch=0), -1), (dict(batch=4097), -2), (dict(page_size=0), -1),
    (dict(max_context=129), -1), (dict(max_context=0), -1), (dict(max_tokens=0), -1),
    (dict(num_free=-1), -1), (dict(num_pages=0), -1), (dict(prefix_capacity=9), -1),
    (dict(prefix_capacity=-1), -1),
    (dict(prefix_capacity=0), -1),  # a prefix table for no prefix
    (dict(bad=dict(ptable=0)), -1), (dict(bad=dict(ppages=0)), -1),
    (dict(bad=dict(cached=0)), -1), (dict(bad=dict(free=0)), -1), (dict(bad=dict(status=0)), -1),
    (dict(bad=dict(slots=0x10004)), -1), (dict(bad=dict(table=0x10002)), -1),
    # outputs that are inputs
    (dict(bad=dict(ctx=0x10000)), -1), (dict(bad=dict(held_out=0x12000)), -1),
    (dict(bad=dict(head_out=0x14000)), -1),
])
def test_tables_refusals(B, kw, status):
    assert tables_call(B, **kw) == status


TABLES_IN = ["cached", "new", "held", "free", "head", "ptable", "ppages"]
TABLES_OUT = ["ctx", "held_out", "head_out", "starts", "positions", "slots", "status", "table"]


@pytest.mark.parametrize("out", TABLES_OUT)
@pytest.mark.parametrize("other", TABLES_IN + TABLES_OUT)
def test_tables_refuse_an_output_that_is_another_buffer(B, out, other):
    # (the table's first row may be the prefix's owner: its entries are read, not written)
    if out == other or (out, other) == ("table", "ptable"):
        return
    names = ["cached", "new", "held", "free", "head", "ptable", "ppages", "table", "ctx",
             "held_out", "head_out", "starts", "positions", "slots", "status"]
    assert tables_call(B, bad={out: 0x10000 + 0x1000 * names.index(other)}) == -1


def test_tables_null_problem(B):
    assert B.load_library().dflash_paged_tables(None, *([None] * 16)) == -1


# ------------------------------------------------------------------------------------ rotary

def frequencies(d, base, scaling, s, trained, fast=32.0, slow=1.0, low=1.0, high=4.0):
    """theta_i by the header's formulas, in Python floats, one pair at a time."""
    out = []
    if scaling == "ntk":
        base = base * s ** (d / (d - 2))
    for i in range(d // 2):
        th = base ** (-2.0 * i / d)
        if scaling == "linear":
            th /= s
        elif scaling == "yarn":
            def c(n):
                return d * math.log(trained / (2 * math.pi * n)) / (2 * math.log(base))
            lo, hi = max(0, math.floor(c(fast))), min(d - 1, math.ceil(c(slow)))
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            th = th * (1 - r) + th / s * r
        elif scaling == "wavelength":
            g = min(1.0, max(0.0, (trained * th / (2 * math.pi) - low) / (high - low)))
            th = th * g + th / s * (1 - g)
        out.append(th)
    return out


SCALES = ["none", "linear", "ntk", "yarn", "wavelength"]


@pytest.mark.parametrize("scaling", SCALES)
@pytest.mark.parametrize("d,base", [(256, 500000.0), (16, 10000.0), (128, 1000000.0), (48, 1.5)])
def test_rope_frequencies(B, scaling, d, base):
    pr = B.make_rope_problem(6, 1, 256, d, base=base, scaling=SCALES.index(scaling), factor=8.0,
                             trained_context=4096)
    plan, phases = B.dflash_rope_plan(pr)
    want = frequencies(d, base, scaling, 8.0, 4096)
    got = np.array([p * 2.0 ** -64 * 2 * math.pi for p in phases])
    # a handful of roundings of 2^-53 each, a power of an exponent up to ln(500000) among them
    assert np.allclose(got, want, rtol=64 * 2.0 ** -53, atol=2.0 ** -60)
    amp = 0.1 * math.log(8.0) + 1.0 if scaling == "yarn" else 1.0
    assert plan.amplitude == np.float32(amp)
    assert max(phases) < 2 ** 62


@pytest.mark.parametrize("kw,status", [
    (dict(version=0), -1), (dict(num_q_heads=0), -1), (dict(num_kv_heads=257), -1),
    (dict(rotary_dim=0), -1), (dict(rotary_dim=272), -1), (dict(rotary_dim=24), -2),
    (dict(head_dim=128, rotary_dim=64), -2), (dict(layout=2), -1), (dict(dtype=2), -1),
    (dict(scaling=5), -1), (dict(base=1.0), -1), (dict(base=float("nan")), -1),
    (dict(base=float("inf")), -1), (dict(scaling=1, factor=0.5), -1),
    (dict(scaling=2, factor=float("nan")), -1), (dict(scaling=3, trained_context=0), -1),
    (dict(scaling=3, beta_slow=0.0), -1), (dict(scaling=4, low_turns=4.0), -1),
    (dict(reserved=1), -1), (dict(page_size=0), -1), (dict(num_pages=0), -1),
])
def test_rope_plan_refusals(B, kw, status):
    pr = B.make_rope_problem(6, 1, 256, 128)
    for k, v in kw.items():
        setattr(pr, k, v)
    plan = B.RopePlan()
    phases = (ctypes.c_uint64 * 256)()
    assert B.load_library().dflash_rope_plan(ctypes.byref(pr), ctypes.byref(plan), phases) == status


def rope_apply_status(B, **bad):
    plan, _ = B.dflash_rope_plan(B.make_rope_problem(6, 2, 256, 128))
    a = dict(T=4, q=0x10000, qs=6 * 256, k=0x20000, ks=2 * 256, pos=0x30000, ph=0x40000,
             qo=0x50000, qos=6 * 256, ko=0x60000, kos=2 * 256)
    a.update(bad)
    if "version" in a:
        plan.version = a["version"]
    return B.load_library().dflash_rope_apply(
        ctypes.byref(plan), a["T"], a["q"], a["qs"], a["k"], a["ks"], a["pos"], a["ph"], a["qo"],
        a["qos"], a["ko"], a["kos"], None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(q=0), dict(q=0x10008), dict(qs=6 * 256 - 8), dict(qs=6 * 256 + 4),
    dict(k=0), dict(ko=0), dict(ks=256), dict(pos=0), dict(pos=0x30002), dict(ph=0x40004),
    dict(ph=0), dict(qo=0x10000, qos=7 * 256), dict(ko=0x20000, kos=3 * 256), dict(version=0)])
def test_rope_apply_refusals(B, bad):
    assert rope_apply_status(B, **bad) == -1


def test_rope_no_tokens(B):
    assert rope_apply_status(B, T=0) == 0


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(q=0), dict(k=0), dict(v=0), dict(v=0x30008), dict(vs=256), dict(slots=0),
    dict(slots=0x50004), dict(ks_=0), dict(vs_=0x80002), dict(kp=0), dict(vp=0xb0004),
    dict(status=0), dict(qo=0x10008)])
def test_rope_write_refusals(B, bad):
    plan, _ = B.dflash_rope_plan(B.make_rope_problem(6, 2, 256, 128, page_size=16, num_pages=4))
    a = dict(T=4, q=0x10000, k=0x20000, v=0x30000, vs=512, pos=0x40000, slots=0x50000, ph=0x60000,
             ks_=0x70000, vs_=0x80000, qo=0x90000, kp=0xa0000, vp=0xb0000, status=0xc0000)
    a.update(bad)
    assert B.load_library().dflash_rope_kv_write(
        ctypes.byref(plan), a["T"], a["q"], 1536, a["k"], 512, a["v"], a["vs"], a["pos"],
        a["slots"], a["ph"], a["ks_"], a["vs_"], a["qo"], 1536, a["kp"], a["vp"], a["status"],
        None) == -1


@pytest.mark.parametrize("bad", [dict(ko=0x10000, kos=6 * 256), dict(qo=0x20000),
                                 dict(ko=0x50000, kos=6 * 256), dict(qo=0x30000),
                                 dict(ko=0x40000)])
def test_rope_apply_refuses_an_output_that_is_another_buffer(B, bad):
    assert rope_apply_status(B, **bad) == -1


@pytest.mark.parametrize("bad", [dict(qo=0x20000), dict(qo=0x30000), dict(kp=0xb0000),
                                 dict(kp=0x90000), dict(vp=0x90000), dict(kp=0x10000),
                                 dict(kp=0x20000), dict(vp=0x30000), dict(vp=0x10000),
                                 dict(status=0x40000), dict(status=0x50000)])
def test_rope_write_refuses_an_output_that_is_another_buffer(B, bad):
    test_rope_write_refusals(B, bad)


# ---------------------------------------------------------------------------- shared prefix

def prefix_problem(B, **kw):
    args = dict(batch=4, q_len=8, num_q_heads=6, num_kv_heads=1, head_dim=256, page_size=16,
                max_pages_per_seq=512, num_pages=4096, max_context=8192, max_prefix=4096,
                device=-1)
    args.update(kw)
    return B.make_prefix_problem(**args)


@pytest.mark.parametrize("kw,status", [
    (dict(version=0), -1), (dict(batch=0), -1), (dict(batch=4097), -2), (dict(q_len=0), -1),
    (dict(num_q_heads=5, num_kv_heads=2), -1), (dict(head_dim=128), -2), (dict(page_size=24), -2),
    (dict(max_pages_per_seq=8), -1), (dict(max_prefix=8193), -1), (dict(max_prefix=-1), -1),
    (dict(kernel=3), -1), (dict(flags=1), -1), (dict(q_len=43), -2),
])
def test_prefix_plan_refusals(B, kw, status):
    pr = prefix_problem(B, **{k: v for k, v in kw.items() if k != "version"})
    if "version" in kw:
        pr.version = kw["version"]
    plan = B.PrefixAttnPlan()
    assert B.load_library().dflash_prefix_attn_plan(ctypes.byref(pr), ctypes.byref(plan)) == status


@pytest.mark.parametrize("kw", [dict(), dict(batch=1), dict(batch=40, num_q_heads=24,
                                                            num_kv_heads=4, max_prefix=8000),
                                dict(q_len=1, batch=4096), dict(max_prefix=0)])
def test_prefix_plan_workspace(B, kw):
    plan = B.dflash_prefix_attn_plan(prefix_problem(B, **kw))
    pr = plan.problem
    rows = pr.batch * pr.q_len * pr.num_q_heads // pr.num_kv_heads
    assert plan.prefix_rows == rows and plan.suffix.rows * pr.batch == rows
    # every row of every KV head has a place in some split state; the parts do not overlap
    if pr.max_prefix:
        assert plan.prefix_slots * plan.prefix_slot_rows >= rows * pr.num_kv_heads
    states = plan.prefix_slots * plan.prefix_slot_rows
    assert plan.suffix.workspace_bytes <= plan.ws_prefix_state_offset
    assert plan.ws_prefix_state_offset + 8 * states <= plan.ws_prefix_acc_offset
    assert plan.ws_prefix_acc_offset + 1024 * states <= plan.ws_unit_offset
    assert plan.workspace_bytes >= plan.ws_unit_offset + 16 * pr.batch * pr.num_kv_heads
    assert plan.ws_unit_offset % 16 == 0
    assert plan.ws_prefix_state_offset % 256 == 0 and plan.ws_prefix_acc_offset % 256 == 0


def prefix_forward_status(B, plan, ws_bytes=None, **bad):
    a = {n: 0x100000 * (i + 1) for i, n in enumerate(
        ("q", "k", "v", "ptable", "plen", "table", "lens", "ks", "vs", "ws", "out", "lse"))}
    a.update(bad)
    return B.load_library().dflash_prefix_attn_forward(
        ctypes.byref(plan), a["q"], a["k"], a["v"], a["ptable"], a["plen"], a["table"], a["lens"],
        a["ks"], a["vs"], a["ws"], plan.workspace_bytes if ws_bytes is None else ws_bytes,
        a["out"], a["lse"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=0), -1), (dict(ptable=0), -1), (dict(plen=0), -1), (dict(out=0), -1), (dict(lse=0), -1),
    (dict(q=0x100008), -1), (dict(k=0x200008), -1), (dict(ws=0xa00010), -1),
    (dict(table=0x600002), -1), (dict(ws_bytes=1024), -3)])
def test_prefix_forward_refusals(B, bad, status):
    plan = B.dflash_prefix_attn_plan(prefix_problem(B))
    assert prefix_forward_status(B, plan, **bad) == status


@pytest.mark.parametrize("field,value", [
    ("version", 0), ("prefix_splits", 10000), ("prefix_slots", 1), ("prefix_rows", 8),
    ("prefix_kernel", 9), ("ws_prefix_acc_offset", 0), ("workspace_bytes", 256)])
def test_prefix_forward_refuses_a_changed_plan(B, field, value):
    plan = B.dflash_prefix_attn_plan(prefix_problem(B))
    setattr(plan, field, value)
    assert prefix_forward_status(B, plan, ws_bytes=1 << 40) == -1
    plan = B.dflash_prefix_attn_plan(prefix_problem(B))
    plan.suffix.num_slots += 1
    assert prefix_forward_status(B, plan, ws_bytes=1 << 40) == -1


@pytest.mark.parametrize("out", ["out", "lse", "ws"])
@pytest.mark.parametrize("other", ["q", "k", "v", "ptable", "plen", "table", "lens", "ks", "vs",
                                   "out", "lse"])
def test_prefix_forward_refuses_an_output_that_is_another_buffer(B, out, other):
    if out == other:
        return
    plan = B.dflash_prefix_attn_plan(prefix_problem(B))
    at = dict(zip(("q", "k", "v", "ptable", "plen", "table", "lens", "ks", "vs", "ws", "out", "lse"),
                  range(0x100000, 0xd00000, 0x100000)))[other]
    assert prefix_forward_status(B, plan, **{out: at}) == -1


@pytest.mark.parametrize("splits", [0, -1, 77, 152, 2 ** 31 - 1])
def test_prefix_forward_refuses_more_pairs_than_the_gpu_has(B, splits):
    plan = B.dflash_prefix_attn_plan(prefix_problem(B, kernel=2))
    assert plan.prefix_kernel == 2 and 0 < plan.prefix_splits <= 76
    plan.prefix_splits = splits
    assert prefix_forward_status(B, plan, ws_bytes=1 << 40) == -1
    plan = B.dflash_prefix_attn_plan(prefix_problem(B, kernel=2))
    plan.prefix_kernel = 1  # not the kernel that the problem asks for
    assert prefix_forward_status(B, plan, ws_bytes=1 << 40) == -1


@pytest.mark.parametrize("batch,q_len,heads,prefix,kernel", [
    (3, 8, (6, 1), 4099, 1), (2, 1, (24, 4), 300, 1), (40, 8, (24, 4), 131000, 2),
    (32, 1, (24, 4), 65536, 2), (12, 8, (24, 4), 0, 1)])
def test_prefix_kernel_is_chosen(B, batch, q_len, heads, prefix, kernel):
    plan = B.dflash_prefix_attn_plan(prefix_problem(
        B, batch=batch, q_len=q_len, num_q_heads=heads[0], num_kv_heads=heads[1],
        max_pages_per_seq=9000, num_pages=9000, max_context=prefix + 500, max_prefix=prefix))
    assert plan.prefix_kernel == kernel
