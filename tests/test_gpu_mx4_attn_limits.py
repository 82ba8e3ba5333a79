"""The 4-bit attention at the ends of its numbers' range. Rows are made so that one key has all the weight: the
output is that key's V, exactly (its weight is a power of two, and so is the sum), and lse its score."""
import numpy as np
import pytest
import torch

import mx4_reference as M
from test_gpu_mx4_attn import D, built, dev, make, problem  # noqa: F401 (built: a fixture)

pytestmark = pytest.mark.gpu


def one_element_keys(pr, sizes, scales):
    """Key j of the first request: its element 0 is sizes[j] (of the grid) times 2^(scales[j] - 127)."""
    n, P = len(sizes), pr["P"]
    codes = np.zeros((n, 1, D), dtype=np.uint8)
    codes[:, 0, 0] = [np.flatnonzero(M.GRID == abs(x))[0] + (8 if x < 0 else 0) for x in sizes]
    sc = np.zeros((n, 1, D // 32), dtype=np.uint8)
    sc[:, 0, 0] = scales
    slots = [int(pr["table"][0, j // P]) * P + j % P for j in range(n)]
    M.put(pr["k"], slots, codes, sc, False)
    return slots


@pytest.mark.parametrize("scale", [127 + 90, 127 + 100, 127 + 101, 254])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_of_the_largest_scales_are_numbers(scale, sign):
    """A single key is seen whatever its score, and among keys the largest score wins; a scale above 2^100 counts
    as 2^100."""
    pr = problem(41, [3], 3, 6, 1, 16)
    pr["q"][:] = 0
    pr["q"][..., 0] = sign * 60000.0
    slots = one_element_keys(pr, [-6.0, 4.0, -4.0], [scale] * 3)
    out, lse = (x.double().cpu().numpy() for x in make(pr)(*dev(pr)))
    v = M.numbers(*M.get(pr["v"], slots, True))[:, 0]
    k = np.array([-6.0, 4.0, -4.0]) * 2.0 ** (min(scale, 227) - 127)
    score = float(pr["q"][0, 0, 0, 0]) * k / 16
    for i in range(3):  # token i sees keys 0 .. i
        best = int(np.argmax(score[:i + 1]))
        assert (out[0, i] == v[best]).all(), i
        assert (np.abs(lse[0, i] / score[best] - 1) <= 2.0 ** -17).all(), i
