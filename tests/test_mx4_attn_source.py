"""What the 4-bit attention's kernel must do and no call can show: read from its source."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def source():
    path = os.path.join(ROOT, "speculative_verify_paged_e4m3_gb300", "csrc", "mx4_attn.cu")
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
