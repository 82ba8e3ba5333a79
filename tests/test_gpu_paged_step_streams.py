"""The paged step's operators on a stream that is not the current one: results made by the call come
from that stream's memory, and an operator is ready when its constructor returns."""
import pytest
import torch

pytestmark = pytest.mark.gpu

CLOCKS = 200_000_000  # about 0.1 s of the GPU


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def tables(B):
    t = B.PagedTables(2, 16, 256, 600, 4096, 5000)
    args = (i32(5, 40), i32(1000, 3000), i32(1, 3), torch.arange(600, dtype=torch.int32,
                                                                device="cuda"), i32(7),
            torch.zeros((2, 256), dtype=torch.int32, device="cuda"))
    return lambda **kw: t(*args, **kw)[3:]


def rotary(B):
    r = B.Rotary(6, 1, 256)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.randn((700, h, 256), device="cuda", generator=g).half() for h in (6, 1))
    pos = torch.arange(700, dtype=torch.int32, device="cuda")
    return lambda **kw: r.apply(q, k, pos, **kw)


def write(B):
    r = B.Rotary(6, 1, 256, num_pages=50)
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn((700, h, 256), device="cuda", generator=g).half() for h in (6, 1, 1))
    pos = torch.arange(700, dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    pools = [torch.zeros((50, 16, 1, 256), dtype=torch.uint8, device="cuda") for _ in range(2)]
    return lambda **kw: (r.kv_write(q, k, v, pos, pos.long(), one, one, *pools, **kw),)


def attention(B):
    a = B.SharedPrefixAttention(2, 8, 6, 1, 256, 16, 64, 128, 1024, 512)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((2, 8, 6, 256), device="cuda", generator=g).half()
    pools = [torch.randint(0, 100, (128, 16, 1, 256), device="cuda", generator=g).to(torch.uint8)
             for _ in range(2)]
    table = torch.arange(128, dtype=torch.int32, device="cuda").view(2, 64)
    table[1, :32] = table[0, :32]
    args = (q, *pools, table[0, :32].contiguous(), i32(512), table, i32(700, 900),
            torch.full((1,), 0.01, device="cuda"), torch.full((1,), 0.1, device="cuda"))
    return lambda **kw: a(*args, **kw)


@pytest.mark.parametrize("make", [tables, rotary, write, attention])
@pytest.mark.parametrize("handle", [False, True])
def test_results_are_not_memory_that_the_current_stream_still_writes(make, handle):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    call = make(B)
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(t) for t in want for _ in range(4)]
    torch.cuda._sleep(CLOCKS)
    for t in old:
        t.fill_(3)
    del old, t  # freed here, written when the sleep ends
    got = call(stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_results_on_the_default_stream_by_its_handle():
    from speculative_verify_paged_e4m3_gb300 import binding as B
    call = rotary(B)
    want = call()
    got = call(stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("make", [tables, rotary, write, attention])
def test_an_operator_is_ready_when_it_is_made(make):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    made = []

    class Made(Exception):
        pass

    class Spy:  # the operator's class, the stream looked at as its constructor returns
        def __getattr__(self, name):
            def construct(*args, **kw):
                torch.cuda._sleep(CLOCKS)
                op = getattr(B, name)(*args, **kw)
                made.append((op, torch.cuda.current_stream().query()))
                raise Made
            return construct
    torch.cuda.synchronize()
    with pytest.raises(Made):
        make(Spy())
    assert made[0][1]
    assert made[0][0].read_flags() == 0
