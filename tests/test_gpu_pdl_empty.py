"""Programmatic launches when a call has nothing to do: every CTA of its partial kernel is idle, and its combine must
still come after everything before it on the stream. Two calls write the same outputs, a long one and then one
whose sequences are all empty: what is left is the second's (zeros, lse -inf), every time, eager and captured."""
import pytest
import torch

from test_gpu_mx4_attn import D, built, dev, make, problem  # noqa: F401 (built: a fixture)

pytestmark = pytest.mark.gpu


def calls(kind, batch):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    n, P = 3000, 16
    pr = problem(51, [n] * batch, 8, 6, 1, P)
    q, k, v, table, lens = dev(pr)
    none = torch.zeros_like(lens)
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], device="cuda")
    if kind == "mx4":
        att = make(pr, flags=B.DFLASH_PROBLEM_PDL)

        def run(lengths):
            att(q, k, v, table, lengths, out=out, lse=lse)
    else:
        g = torch.Generator(device="cuda").manual_seed(1)
        pools = [torch.randint(0, 96, (k.shape[0], P, 1, D), generator=g, device="cuda", dtype=torch.uint8)
                 for _ in range(2)]
        one = torch.ones(1, device="cuda")
        att = B.VerifyAttention(batch, 8, 6, 1, D, P, table.shape[1], k.shape[0], table.shape[1] * P,
                                kernel=kind, flags=B.DFLASH_PROBLEM_PDL)

        def run(lengths):
            att(q, *pools, table, lengths, one, one, out=out, lse=lse)
    return run, lens, none, out, lse, att


@pytest.mark.parametrize("batch", [1, 4])
@pytest.mark.parametrize("kind", ["mx4", 1, 2], ids=["mx4", "simt", "tcgen05"])
def test_an_empty_call_comes_after_the_one_before_it(kind, batch):
    run, lens, none, out, lse, att = calls(kind, batch)

    def both():
        run(lens)
        run(none)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for once in [both] * 100 + [graph.replay] * 100:
        out.fill_(7.0)
        lse.fill_(7.0)
        once()
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    run(lens)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(lse).all())
    flags = int(att.workspace[:4].view(torch.int32).item())
    assert flags & ~0x2 == 0  # (the empty call is shorter than its drafted tokens)
