"""Shared-prefix attention with values that are not finite where the softmax could take them for an empty row:
a row that sees a key gives NaN, in its own place alone, whichever kernel has the prefix."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import compare, oracle_forward, to_np
from test_gpu_prefix_attn import call, make, operator

pytestmark = pytest.mark.gpu

both = pytest.mark.parametrize("kernel", [1, 2], ids=["rows", "pairs"])


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()


@both
@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("element", [0, 77, 255])
@pytest.mark.parametrize("length", [1, 2, 30, 256, 400], ids=lambda n: f"n{n}")
def test_one_infinite_element(kernel, value, element, length):
    """Sequence 1 ends inside the prefix (or has own keys too), and every key that it sees has the same sign in
    the element: its scores are all +inf, or all -inf."""
    inp = make(length + element, [500, length, 444], 432, q_len=1)
    k = inp["k_pool"]
    k[..., element] = (k[..., element] & 0x7F).clamp(8, 0x7E)  # positive and finite
    want_out, want_lse = oracle_forward(inp)
    bad = dict(inp, q=inp["q"].clone())
    bad["q"][1, 0, 4, element] = value
    out, lse = call(operator(bad, kernel=kernel), {k: v.cuda() for k, v in bad.items()})
    out, lse = to_np(out), to_np(lse)
    assert np.isnan(out[1, 0, 4]).all() and np.isnan(lse[1, 0, 4])
    out[1, 0, 4], lse[1, 0, 4] = want_out[1, 0, 4], want_lse[1, 0, 4]
    compare(out, lse, want_out, want_lse)


@both
@pytest.mark.parametrize("lens", [[256, 100, 0, 1], [500, 300, 0, 3]], ids=["prefix_alone", "own_keys_too"])
@pytest.mark.parametrize("k_scale", [math.nan, math.inf, -math.inf])
def test_a_scale_that_is_not_finite(kernel, lens, k_scale):
    """Every row that sees a key is NaN; the others are empty as ever."""
    inp = make(3, lens, 256, q_len=2)
    inp["k_scale"] = torch.tensor([k_scale])
    out, lse = call(operator(inp, kernel=kernel), {k: v.cuda() for k, v in inp.items()})
    out, lse = to_np(out), to_np(lse)
    for b, n in enumerate(lens):
        for i in range(2):
            if n - 2 + i + 1 > 0:
                assert np.isnan(out[b, i]).all() and np.isnan(lse[b, i]).all(), (b, i)
            else:
                assert (out[b, i] == 0).all() and np.isneginf(lse[b, i]).all(), (b, i)


@both
def test_a_value_scale_that_is_not_a_number(kernel):
    inp = make(5, [256, 300, 0], 256, q_len=2)
    want_lse = oracle_forward(inp)[1]
    inp["v_scale"] = torch.tensor([math.nan])
    out, lse = call(operator(inp, kernel=kernel), {k: v.cuda() for k, v in inp.items()})
    out, lse = to_np(out), to_np(lse)
    assert np.isnan(out[:2]).all() and (out[2] == 0).all()
    compare(np.zeros_like(out), lse, np.zeros(out.shape), want_lse)
