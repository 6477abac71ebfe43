"""The rotated append over blocks that a cache filled by other means gave scales
below 2^-126."""
import numpy as np
import pytest
import torch

from oracle import e4m3
from tests._e4m3 import D, Pool, check_attention, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("old", [2.0 ** -126, 2.0 ** -127, 1.5 * 2.0 ** -130, 2.0 ** -149])
@pytest.mark.parametrize("new", [0.0, 2.0 ** -130, 1e-38, 1.0])
def test_scales_below_the_least(old, new):
    """Codes stay finite, older rows follow the scale, and the rows are as the model has them."""
    p = Pool(2, 8, 2, 64)
    cached = [20, 3]
    p.fill(cached)
    at = [int(p.order[b, c // 16]) for b, c in enumerate(cached)]
    p.ks[0, at], p.vs[0, at] = old, old
    state = p.host()
    rows = p.normal(4, 2, D, tag="rows") * new
    rows[1] = 0
    p.kvc.check(p.kvc.kvc_append_packed(p.h, 0, rows, rows, ints([0, 3, 4]), ints(cached), 4))
    for b, (c, lo, hi) in enumerate(((20, 0, 3), (3, 3, 4))):
        part = rows[lo:hi].float().cpu().numpy()
        e4m3.append(state[0], state[1], p.order[b], c, part)
        e4m3.append(state[2], state[3], p.order[b], c, part)
    p.same(state)
    for x, c in ((state[0], cached), (state[2], cached)):
        for b, n in ((0, 23), (1, 4)):
            assert np.isfinite(e4m3.gather(x, state[1], p.order[b], n).numpy()).all()
    q = p.normal(2, 8, D, tag="q")
    out = torch.zeros_like(q)
    p.kvc.check(p.kvc.kvc_packed_attn(p.h, 0, q, None, ints([22, 3]), 2, 0, out))
    # (values' scales below 2^-90 may be taken as that: sequence 1 has no others, but where new is 1)
    least = float(p.vs[0, at[1]].min()) < 2.0 ** -90
    check_attention(p, q, out, [0, 1, 2], [22, 3], skip=(1,) if least else ())
    assert not least or float(out[1].abs().max()) <= 448 * 2.0 ** -90
    assert p.error() == 0 and p.intact()
