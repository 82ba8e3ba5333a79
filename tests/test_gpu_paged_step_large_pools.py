"""Pools of more than 2^32 bytes: pages at their far end give the same bits as the same pages of a
small pool, and nothing lands where a 32-bit offset would wrap to."""
import pytest
import torch

from test_gpu_prefix_attn import call, make, operator

pytestmark = pytest.mark.gpu

P, HKV, D = 64, 4, 256
PAGES = 2 ** 32 // (P * HKV * D) + 500


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs two pools of 4.3 GB")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()


def test_kv_write():
    from speculative_verify_paged_e4m3_gb300 import binding as B
    T, few = 300, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn((T, h, D), device="cuda", generator=g).half() for h in (24, HKV, HKV))
    pos = torch.randint(0, 1000, (T,), device="cuda", generator=g).int()
    slots = torch.randperm(few * P, device="cuda", generator=g)[:T]
    one = torch.ones(1, device="cuda")

    def write(pages, first):
        pools = [torch.zeros((pages, P, HKV, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
        r = B.Rotary(24, HKV, D, page_size=P, num_pages=pages)
        qo = r.kv_write(q, k, v, pos, slots + first * P, one, one, *pools)
        assert r.read_flags() == 0
        return qo, pools
    want, small = write(few, 0)
    got, large = write(PAGES, PAGES - few)
    assert torch.equal(want, got)
    for s, l in zip(small, large):
        assert torch.equal(s, l[PAGES - few:]) and s.any()
        assert not any(part.any() for part in l[:PAGES - few].split(1 << 12))


@pytest.mark.parametrize("kernel", [1, 2], ids=["rows", "pairs"])
def test_shared_prefix(kernel):
    inp = make(77, [900, 650, 700], 600, 8, (24, HKV), P)
    dev = {k: v.cuda() for k, v in inp.items()}
    n = inp["k_pool"].shape[0]
    want = call(operator(inp, kernel=kernel), dev)
    far = dict(dev)
    for name in ("k_pool", "v_pool"):
        far[name] = torch.zeros((PAGES, P, HKV, D), dtype=torch.uint8, device="cuda")
        far[name][PAGES - n:] = dev[name]
    far["prefix_table"] = dev["prefix_table"] + (PAGES - n)
    # (make's entries past a sequence's end are out of range and not read)
    far["block_table"] = dev["block_table"] + (PAGES - n)
    att = operator(far, kernel=kernel)
    got = call(att, far)
    torch.cuda.synchronize()
    assert att.read_flags() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))
