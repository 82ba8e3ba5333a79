"""The status word of calls on a stream that is not the current one: read behind them on request."""
import pytest
import torch

from test_gpu_paged_step_streams import CLOCKS, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()


def exhausted(B):
    t = B.PagedTables(2, 16, 4, 8, 64, 64)
    args = (i32(0, 0), i32(40, 40), i32(0, 0), i32(1, 2), i32(0), torch.zeros((2, 4), dtype=torch.int32,
                                                                             device="cuda"))
    return t, 0x30, lambda s: t(*args, stream=s)  # (80 tokens for 64 entries, too)


def slot_past_the_pool(B):
    r = B.Rotary(2, 1, 256, num_pages=2)
    q, k = (torch.zeros((3, h, 256), dtype=torch.float16, device="cuda") for h in (2, 1))
    pools = [torch.zeros((2, 16, 1, 256), dtype=torch.uint8, device="cuda") for _ in range(2)]
    one, slots = torch.ones(1, device="cuda"), torch.tensor([0, 32, 1], device="cuda")
    return r, 0x40, lambda s: r.kv_write(q, k, k, i32(0, 1, 2), slots, one, one, *pools, stream=s)


def length_past_the_plan(B):
    a = B.SharedPrefixAttention(1, 1, 6, 1, 256, 16, 4, 8, 64, 32)
    q = torch.zeros((1, 1, 6, 256), dtype=torch.float16, device="cuda")
    pool = torch.zeros((8, 16, 1, 256), dtype=torch.uint8, device="cuda")
    table, one = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4), torch.ones(1, device="cuda")
    prefix, n, ctx = table[0, :2].contiguous(), i32(32), i32(65)
    return a, 0x1, lambda s: a(q, pool, pool, prefix, n, table, ctx, one, one, stream=s)


@pytest.mark.parametrize("make", [exhausted, slot_past_the_pool, length_past_the_plan])
@pytest.mark.parametrize("handle", [False, True])
def test_flags_are_read_behind_the_calls_of_a_stream(make, handle):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    op, flag, call = make(B)
    side = torch.cuda.Stream()
    s = side.cuda_stream if handle else side
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CLOCKS)
    call(s)
    assert op.read_flags(clear=True, stream=s) == flag
    assert side.query()
    assert op.read_flags(stream=s) == 0 and op.read_flags() == 0
