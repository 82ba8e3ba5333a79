"""What the tensor-core kernels must do and no call can show: read from their sources."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def source(name="mx4_attn.cu"):
    path = os.path.join(ROOT, "speculative_verify_paged_e4m3_gb300", "csrc", name)
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_products_are_through_before_tensor_memory_is_given_back():
    """After a wait that gave up no other wait sees the products through: the one in front of the release goes on
    when the CTA has given up (`never` stays 0), and both issuing threads arrive on its barrier whatever happened."""
    s = source()
    end = s[s.rindex("__syncthreads();"):s.index("tmem_dealloc(tmem")]
    assert re.search(r"mbar_wait\(smem_u32\(&sm\.odone\), 0, &sm\.never, kWaitLimitNs\)", end)
    assert s.count("if (issuer) mma_commit(smem_u32(&sm.odone));") == 1
    assert "mbar_init(smem_u32(&sm.odone), 2)" in s
    assert not re.search(r"never\s*=\s*[^0;]", s.replace("sm.abort = sm.never = 0", ""))


def body(s, head):
    """The text of the braces that follow `head`."""
    at = s.index("{", s.index(head))
    depth = 0
    for i in range(at, len(s)):
        depth += {"{": 1, "}": -1}.get(s[i], 0)
        if not depth:
            return s[at:i]
    raise AssertionError(head)


def test_lanes_are_together_where_instructions_want_a_whole_warp():
    """A wait's first try may succeed for some lanes of a warp only, and masks differ between lanes: tensor-memory
    loads and stores and the groups' barriers come behind a __syncwarp()."""
    s = source()
    assert re.search(r"__all_sync\(.*?\);\s*__syncwarp\(\);", body(s, "bool wait_warp("), re.S)
    for head in ("bool group_vote(", "void group_bar("):
        b = body(s, head)
        assert b.index("__syncwarp()") < b.index("asm volatile")
    assert re.search(r"__syncwarp\(\);\s*tc_fence_after\(\);\s*tmem_dealloc\(", s)


def test_the_e4m3_kernels_see_copies_and_products_through():
    s = source("tc_partial.cu")
    assert re.search(r"mma_commit\(smem_u32\(&sm\.odone\)\);\s*"
                     r"mbar_wait\(smem_u32\(&sm\.odone\), 0, &sm\.never, kWaitLimitNs\);", s)
    assert s.count("mma_commit(smem_u32(&sm.odone))") == 1
    drains = re.findall(r"mbar_wait\(smem_u32\(&sm\.(\w+)(?:\[[^]]*\])?\),[^;]*?&sm\.(\w+),", s)
    assert sorted(drains) == [("kfull", "never"), ("odone", "never"), ("vfull", "never"), ("vtail", "never")]
    assert not re.search(r"never\s*=\s*[^0;]", s.replace("sm.abort = sm.never = 0", ""))
    s = source("prefix_pairs.cu")
    end = s[s.index("ctx.wait_warp(&sm.done, 0)"):s.index("tcgen05.dealloc")]
    assert end.index("drain(&sm.done, 0)") < end.index("__syncthreads()") < end.index("cluster_wait()")
    assert s.count("commit_pair(smem_u32(&sm.done));") == 2 and "mbar_init(smem_u32(&sm.done), 2)" in s
