"""A prefix too short for a whole page: the shared table has no entries, and may be missing or empty."""
import pytest
import torch

from gpu_helpers import compare, oracle_forward, to_np
from test_gpu_prefix_attn import make, operator

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel", [1, 2], ids=["rows", "pairs"])
@pytest.mark.parametrize("prefix,P", [(1, 16), (63, 64)])
@pytest.mark.parametrize("empty", [False, True])
def test_no_whole_page(kernel, prefix, P, empty):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()
    inp = make(prefix, [prefix + 90, prefix + 8, 0], prefix, P=P)
    want = oracle_forward(inp)
    d = {k: v.cuda() for k, v in inp.items()}
    table = d["prefix_table"][:0] if empty else None
    att = operator(inp, kernel=kernel)
    out, lse = att(d["q"], d["k_pool"], d["v_pool"], table, d["prefix_len"], d["block_table"],
                   d["context_lens"], d["k_scale"], d["v_scale"])
    compare(to_np(out), to_np(lse), *want)
    assert att.read_flags() == 0x2  # a sequence shorter than its block, nothing else
    with pytest.raises(ValueError):  # a plan whose prefix fills a page
        operator(inp, max_prefix=P, kernel=kernel)(
            d["q"], d["k_pool"], d["v_pool"], table, d["prefix_len"], d["block_table"], d["context_lens"],
            d["k_scale"], d["v_scale"])
