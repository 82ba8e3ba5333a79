"""The tests' own 4-bit format, held to what the header states; the C structs and every refusal of the
4-bit cache's and the head norms' entry points, without a GPU."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import mx4_reference as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
rng = np.random.default_rng


@pytest.fixture(scope="module")
def B():
    from speculative_verify_paged_e4m3_gb300 import binding, build
    build.build()
    return binding


# ------------------------------------------------------------------------------------ the format

def test_every_code_and_scale_survives():
    codes = np.tile(np.arange(16, dtype=np.uint8), 16)[None, None]
    codes[..., 8::16] = 0  # (minus zero is written for a negative number only)
    for s in (1, 100, 127, 200, 252):
        sc = np.full((1, 1, 8), s, dtype=np.uint8)
        got, sc2 = M.quantise(M.numbers(codes, sc))
        assert np.array_equal(sc, sc2) and np.array_equal(got, codes)


@pytest.mark.parametrize("x,want", [(0.25, 0.0), (0.2500001, 0.5), (0.75, 1.0), (1.25, 1.0),
                                    (1.75, 2.0), (2.5, 2.0), (3.5, 4.0), (5.0, 4.0), (5.1, 6.0),
                                    (6.9, 6.0), (-5.0, -4.0), (-0.2, 0.0)])
def test_nearest_ties_to_even(x, want):
    row = np.zeros((1, 1, 256))
    row[..., 0], row[..., 1] = x, 7.0  # the scale is 1
    assert M.numbers(*M.quantise(row))[0, 0, 0] == want


@pytest.mark.parametrize("top,e", [(7.0, 0), (7.0001, 1), (3.5, -1), (3.51, 0), (2.0 ** -140, -127),
                                   (65504.0, 14), (57344.0, 13), (3.3e38, 126)])
def test_least_scale(top, e):
    assert M.least_scale(np.array(top)) == e + 127


def test_rounding_is_off_by_half_a_step_at_most():
    x = rng(0).standard_normal((50, 2, 256)) * np.exp(rng(1).standard_normal((50, 2, 1)))
    codes, s = M.quantise(x)
    step = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, -1)
    y = np.abs(x) / step
    half = np.where(y < 2, 0.25, np.where(y < 4, 0.5, 1.0))
    assert (np.abs(M.numbers(codes, s) - x) <= half * step).all()


def test_put_and_get_are_one_layout():
    codes = rng(2).integers(0, 16, (40, 3, 256), dtype=np.uint8)
    scales = rng(3).integers(0, 255, (40, 3, 8), dtype=np.uint8)
    slots = rng(4).permutation(64)[:40]
    for of_v in (False, True):
        pool = M.empty_pool(2, 32, 3)
        M.put(pool, slots, codes, scales, of_v)
        got = M.get(pool, slots, of_v)
        assert np.array_equal(got[0], codes) and np.array_equal(got[1], scales)


def test_layout_as_the_header_states():
    codes = np.zeros((1, 1, 256), dtype=np.uint8)
    codes[0, 0, 2 * 32 + 2 * 5 + 1] = 9
    codes[0, 0, 130] = 3
    scales = np.arange(8, dtype=np.uint8)[None, None]
    k, v = M.empty_pool(1, 16, 1), M.empty_pool(1, 16, 1)
    M.put(k, [7], codes, scales, False)
    M.put(v, [7], codes, scales, True)
    assert k[0, 0, 0, 256 * 2 + 16 * 7 + 5] == 9 << 4
    assert v[0, 0, 0, 16 * 2 + 7] == 3 << 4
    assert k[0, 0, 0, 2048 + 8 * 7 + 4] == 4 == v[0, 0, 0, 2048 + 8 * 7 + 4]


# --------------------------------------------------------------------------------- the C side

def test_struct_layout_and_constants_match_c(B, tmp_path):
    prog = tmp_path / "sizes.c"
    fields = [f[0] for f in B.HeadNormArgs._fields_]
    lines = ['printf("%zu\\n", sizeof(dflash_head_norm));']
    lines += [f'printf("%zu\\n", offsetof(dflash_head_norm, {f}));' for f in fields]
    consts = ["DFLASH_E5M2", "DFLASH_KERNEL_MX4", "DFLASH_MX4_CHUNK_TOKENS", "DFLASH_MX4_CHUNK_BYTES"]
    lines += [f'printf("%d\\n", {c});' for c in consts]
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dflash_mx4_cache.h"\n'
                    "int main(void){" + "".join(lines) + "return 0;}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(prog),
                    "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == ([ctypes.sizeof(B.HeadNormArgs)] + [getattr(B.HeadNormArgs, f).offset
                                                      for f in fields]
                   + [getattr(B, c) for c in consts])


# Addresses that are never followed: every call here is refused before a launch.
def address(names, bad):
    at = {n: 0x100000 + 0x1000 * i for i, n in enumerate(names)}
    at.update(bad)
    return at


def norm_args(B, at, eps=1e-6, offset=0.0):
    return ctypes.byref(B.HeadNormArgs(at["qw"], at["kw"], eps, offset))


def write_call(B, fn="dflash_mx4_kv_write", plan=None, tokens=4, strides=(6 * 256, 256, 256, 6 * 256),
               eps=1e-6, offset=0.0, norm=True, page=16, **bad):
    names = ["q", "k", "v", "pos", "slots", "live", "phases", "ks", "vs", "q_out", "k_pool",
             "v_pool", "status", "qw", "kw"]
    at = address(names, bad)
    if plan is None:
        plan, _ = B.dflash_rope_plan(B.make_rope_problem(6, 1, 256, 256, page_size=page,
                                                         num_pages=8))
    n = norm_args(B, at, eps, offset) if norm else None
    scales = [at["ks"], at["vs"]] if fn == "dflash_norm_rope_kv_write" else []
    return getattr(B.load_library(), fn)(
        ctypes.byref(plan), n, tokens, at["q"], strides[0], at["k"], strides[1], at["v"],
        strides[2], at["pos"], at["slots"], at["live"], at["phases"], *scales, at["q_out"],
        strides[3], at["k_pool"], at["v_pool"], at["status"], None)


WRITES = ["dflash_mx4_kv_write", "dflash_norm_rope_kv_write"]


@pytest.mark.parametrize("fn", WRITES)
@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), -1), (dict(tokens=1 << 31), -1), (dict(tokens=0), 0),
    (dict(strides=(6 * 256 - 8, 256, 256, 1536)), -1), (dict(strides=(1536, 260, 256, 1536)), -1),
    (dict(strides=(1536, 256, 128, 1536)), -1), (dict(strides=(1536, 256, 256, 1540)), -1),
    (dict(q=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(pos=0), -1), (dict(slots=0), -1),
    (dict(phases=0), -1), (dict(q_out=0), -1), (dict(k_pool=0), -1), (dict(v_pool=0), -1),
    (dict(status=0), -1), (dict(q=0x100008), -1), (dict(slots=0x104004), -1),
    (dict(k_pool=0x10A004), -1), (dict(status=0x10C002), -1), (dict(live=0x105002), -1),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
    (dict(offset=float("inf")), -1), (dict(qw=0x10D008), -1), (dict(kw=0x10E002), -1),
])
def test_write_refusals(B, fn, kw, status):
    assert write_call(B, fn, **kw) == status


@pytest.mark.parametrize("fn", WRITES)
@pytest.mark.parametrize("out", ["q_out", "k_pool", "v_pool", "status"])
@pytest.mark.parametrize("other", ["k", "v", "pos", "slots", "live", "phases", "q_out", "k_pool",
                                   "v_pool", "status", "qw", "kw"])
def test_write_refuses_an_output_that_is_another_buffer(B, fn, out, other):
    if out == other:
        return
    names = ["q", "k", "v", "pos", "slots", "live", "phases", "ks", "vs", "q_out", "k_pool",
             "v_pool", "status", "qw", "kw"]
    assert write_call(B, fn, **{out: 0x100000 + 0x1000 * names.index(other)}) == -1


def test_write_wants_pages_of_whole_chunks(B):
    assert write_call(B, page=24) == -2
    assert write_call(B, page=24, tokens=0) == -2
    assert write_call(B, k_pool=0x10A008) == -1  # 16-byte aligned


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), -1), (dict(pos=0), -1), (dict(phases=0), -1), (dict(eps=-1.0), -1),
    (dict(offset=float("nan")), -1), (dict(qw=0x106008), -1), (dict(kw=0x107004), -1),
    (dict(q_out=0x106000), -1), (dict(k_out=0x107000), -1), (dict(k_out=0), -1),
    (dict(q_out=0x101000), -1), (dict(tokens=0), 0), (dict(tokens=-1), -1),
])
def test_norm_rope_apply_refusals(B, kw, status):
    kw = dict(kw)
    tokens, eps, offset = kw.pop("tokens", 4), kw.pop("eps", 1e-6), kw.pop("offset", 0.0)
    at = address(["q", "k", "pos", "phases", "q_out", "k_out", "qw", "kw"], kw)
    plan, _ = B.dflash_rope_plan(B.make_rope_problem(6, 1, 256, 256))
    assert B.load_library().dflash_norm_rope_apply(
        ctypes.byref(plan), norm_args(B, at, eps, offset), tokens, at["q"], 1536, at["k"], 256,
        at["pos"], at["phases"], at["q_out"], 1536, at["k_out"], 256, None) == status


def read_call(B, heads=2, dim=256, page=16, pages=8, tokens=4, dtype=0, ks=512, vs=512, **bad):
    at = address(["k_pool", "v_pool", "slots", "k_out", "v_out", "status"], bad)
    return B.load_library().dflash_mx4_read(heads, dim, page, pages, at["k_pool"], at["v_pool"], tokens,
                                            at["slots"], dtype, at["k_out"], ks, at["v_out"], vs,
                                            at["status"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), -1), (dict(heads=257), -1), (dict(dim=128), -2), (dict(dim=0), -1),
    (dict(page=8), -2), (dict(page=0), -1), (dict(pages=0), -1), (dict(tokens=-1), -1),
    (dict(tokens=1 << 31), -1), (dict(tokens=0), 0), (dict(dtype=3), -1), (dict(dtype=-1), -1),
    (dict(ks=511), -1), (dict(ks=256), -1), (dict(vs=520), -1), (dict(slots=0), -1),
    (dict(slots=0x102004), -1), (dict(status=0), -1), (dict(k_pool=0), -1), (dict(v_out=0), -1),
    (dict(k_pool=0, v_pool=0, k_out=0, v_out=0), -1), (dict(k_out=0x103008), -1),
    (dict(v_pool=0x101004), -1), (dict(k_out=0x104000), -1), (dict(k_out=0x100000), -1),
    (dict(v_out=0x100000), -1), (dict(k_out=0x102000), -1), (dict(status=0x101000), -1),
    (dict(status=0x103000), -1),
])
def test_read_refusals(B, kw, status):
    assert read_call(B, **kw) == status


def attn_problem(B, **kw):
    a = dict(batch=2, q_len=8, num_q_heads=12, num_kv_heads=2, head_dim=256, page_size=16,
             max_pages_per_seq=64, num_pages=128, max_context=1024, device=-1)
    a.update(kw)
    return B.make_problem(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), -1), (dict(q_len=0), -1), (dict(num_q_heads=5), -1), (dict(head_dim=128), -2),
    (dict(page_size=8, max_context=512), -2), (dict(page_size=24), -2), (dict(max_context=1025), -1),
    (dict(q_len=43), -2), (dict(kernel=7), -1), (dict(kernel=1), -2), (dict(kernel=2), -2),
    (dict(flags=1), -2), (dict(flags=4), -2), (dict(num_splits=-1), -1),
])
def test_attention_plan_refusals(B, kw, status):
    plan = B.Plan()
    pr = attn_problem(B, **kw)
    assert B.load_library().dflash_mx4_attn_plan(ctypes.byref(pr), ctypes.byref(plan)) == status


def test_attention_plan(B):
    plan = B.dflash_mx4_attn_plan(attn_problem(B, flags=B.DFLASH_PROBLEM_PDL))
    assert plan.kernel == B.DFLASH_KERNEL_MX4 and plan.rows == 48 and plan.row_blocks == 1
    assert plan.num_slots <= 152 and plan.problem.flags == B.DFLASH_PROBLEM_PDL
    assert B.dflash_mx4_attn_plan(attn_problem(B, q_len=16)).row_blocks == 2
    assert B.load_library().dflash_mx4_attn_plan(None, ctypes.byref(plan)) == -1


def attn_call(B, plan=None, ws_bytes=None, **bad):
    names = ["q", "k_pool", "v_pool", "table", "lens", "ws", "out", "lse"]
    at = address(names, bad)
    plan = plan or B.dflash_mx4_attn_plan(attn_problem(B))
    return B.load_library().dflash_mx4_attn_forward(
        ctypes.byref(plan), at["q"], at["k_pool"], at["v_pool"], at["table"], at["lens"], at["ws"],
        plan.workspace_bytes if ws_bytes is None else ws_bytes, at["out"], at["lse"], None)


@pytest.mark.parametrize("kw,status", [
    *[({n: 0}, -1) for n in ("q", "k_pool", "v_pool", "table", "lens", "ws", "out", "lse")],
    (dict(q=0x100008), -1), (dict(k_pool=0x101008), -1), (dict(v_pool=0x102004), -1),
    (dict(table=0x103002), -1), (dict(lens=0x104001), -1), (dict(ws=0x105010), -1),
    (dict(out=0x106004), -1), (dict(lse=0x107002), -1), (dict(ws_bytes=100), -3),
    (dict(out=0x100000), -1), (dict(out=0x101000), -1), (dict(lse=0x104000), -1),
    (dict(ws=0x102000), -1), (dict(out=0x107000), -1), (dict(lse=0x105000), -1),
])
def test_attention_refusals(B, kw, status):
    assert attn_call(B, **kw) == status


def test_plans_of_the_two_caches_are_not_taken_for_each_other(B):
    pr = attn_problem(B)
    e4m3 = B.dflash_verify_attn_plan(pr)
    assert attn_call(B, plan=e4m3) == -1
    mx4 = B.dflash_mx4_attn_plan(pr)
    args = [0x100000 + 0x1000 * i for i in range(10)]
    assert B.load_library().dflash_verify_attn_forward(
        ctypes.byref(mx4), *args[:8], mx4.workspace_bytes, args[8], args[9], None) == -1
    mx4.num_splits = 0
    assert attn_call(B, plan=mx4) == -1
