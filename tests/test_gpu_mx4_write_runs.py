"""The 4-bit cache's write of batches whose tokens lie in many runs of slots: single tokens, drafted blocks and
pieces of prompts side by side, whole chunks among them and parts. Every byte of both pools."""
import numpy as np
import pytest
import torch

import mx4_reference as M
from test_gpu_mx4_cache import D, built, make  # noqa: F401 (built: a fixture)

pytestmark = pytest.mark.gpu


def run_slots(rng, T, P, lengths):
    """(slots of T tokens in runs of these lengths, each at a place of its own in some pages; pages)."""
    slots, page = [], 0
    while len(slots) < T:
        n = int(rng.choice(lengths))
        off = int(rng.integers(0, P))
        slots.append(page * P + off + np.arange(n))
        page += -(-(off + n) // P)
        if sum(map(len, slots)) >= T:
            break
    order = rng.permutation(len(slots))
    return np.concatenate([slots[i] for i in order])[:T], page


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,Hq,Hkv,P,lengths", [
    (384, 24, 4, 16, [1]), (769, 24, 4, 16, [1]), (512, 24, 4, 64, [8]), (2049, 6, 1, 48, [1, 8]),
    (2301, 6, 1, 32, [15, 16, 17]),
    (1700, 8, 2, 16, [1, 3, 16, 33, 64]), (1000, 12, 4, 64, [31, 32, 47, 130]), (2100, 2, 1, 16, [16, 32]),
])
def test_write_of_many_runs(T, Hq, Hkv, P, lengths, dtype):
    from speculative_verify_paged_e4m3_gb300 import binding as B
    rng = np.random.default_rng(T)
    slots, pages = run_slots(rng, T, P, lengths)
    slots = slots.copy()
    slots[rng.random(T) < 0.01] = -1
    slots[T // 3] = pages * P + 7  # past the pool
    q, k, v, pos, qw, kw = make(T, T, Hq, Hkv, dtype, fused=T % 2 == 1)
    r = B.Rotary(Hq, Hkv, D, page_size=P, num_pages=pages, dtype=dtype)
    kp, vp = B.Mx4Cache(Hkv, D, P, pages).empty()
    kp.fill_(0x33)
    vp.fill_(0x44)
    r.mx4_write(q, k, v, torch.zeros_like(pos), torch.from_numpy(slots).cuda(), kp, vp)  # (nothing turned)
    on = (slots >= 0) & (slots < pages * P)
    for got, x, of_v, fill in ((kp, k, False, 0x33), (vp, v, True, 0x44)):
        want = np.full(got.shape, fill, dtype=np.uint8)
        codes, s = M.quantise(x.double().cpu().numpy()[on])
        M.put(want, slots[on], codes, s, of_v)
        assert np.array_equal(got.cpu().numpy(), want)
    assert r.read_flags() == B.DFLASH_FLAG_SLOT_RANGE
