"""The 8-bit paged cache where a row with an infinity or NaN comes and is taken back."""
import numpy as np
import pytest
import torch

from oracle import e4m3
from tests._e4m3 import D, Pool, check_attention, ints

pytestmark = pytest.mark.gpu


def _same_bits(p, state):
    p.same(state)
    got = p.host()
    for i in (1, 3):
        assert np.array_equal(got[i].view(np.uint32), state[i].view(np.uint32))


@pytest.mark.parametrize("cached", [(0, 1, 15, 16), (3, 17, 30, 28)])
@pytest.mark.parametrize("odd_scales", [False, True])
def test_a_rejected_draft_leaves_no_trace(cached, odd_scales):
    """Drafts with bad rows in some heads, K or V, then rows in their place: bit for bit as the
    model has it, and where scales are powers of two as without the bad rows."""
    p = Pool(4, 8, 2, 64, seed=sum(cached))
    p.fill(cached)
    if odd_scales:
        p.ks.mul_(1.5), p.vs.mul_(1.25)
    state, before, kvc = p.host(), p.host(), p.kvc

    def store(k, v, c, to):
        n = len(k) // 4
        kvc.check(kvc.kvc_append_packed(p.h, 0, k, v, ints([n * b for b in range(5)]), ints(c), 4 * n))
        for b in range(4):
            for i, x in ((0, k), (2, v)):
                for s in to:
                    e4m3.append(s[i], s[i + 1], p.order[b], c[b], x[n * b:n * b + n].float().cpu().numpy())

    k, v = p.normal(20, 2, D, tag="draft k"), p.normal(20, 2, D, tag="draft v")
    k[0, 0, 5], k[7, 1, 127], v[6, 0, 0], v[12, 1, 77], k[19] = np.inf, np.nan, -np.inf, np.inf, np.nan
    store(k, v, cached, [state])
    _same_bits(p, state)
    assert np.isnan(state[1]).any() and np.isnan(state[3]).any()
    # the first bad rows are 0, 1, 2 and 4 of the drafts
    for b, good in enumerate((0, 1, 2, 4)):
        for i, x in ((0, k), (2, v)):
            e4m3.append(before[i], before[i + 1], p.order[b], cached[b], x[5 * b:5 * b + good].float().cpu().numpy())
    c = [a + good for a, good in zip(cached, (0, 1, 2, 4))]
    k2, v2 = p.normal(8, 2, D, tag="next k"), p.normal(8, 2, D, tag="next v")
    store(k2, v2, c, [state, before])
    _same_bits(p, state)
    rows = [a + 2 for a in c]
    for b in range(4):
        blocks = p.order[b, :-(-rows[b] // 16)]
        assert np.isfinite(state[1][blocks]).all() and np.isfinite(state[3][blocks]).all()
        if not odd_scales:
            for i in (0, 2):
                assert torch.equal(e4m3.gather(state[i], state[i + 1], p.order[b], rows[b]), e4m3.gather(before[i], before[i + 1], p.order[b], rows[b]))
    q = p.normal(4, 8, D, tag="q")
    out = torch.zeros_like(q)
    kvc.check(kvc.kvc_packed_attn(p.h, 0, q, None, ints([r - 1 for r in rows]), 4, 0, out))
    check_attention(p, q, out, [0, 1, 2, 3, 4], [r - 1 for r in rows])
    assert p.error() == 0 and p.intact()


def test_rows_behind_a_bad_one_are_lost():
    """They read as NaN, and so does a block whose NaN keeps nothing, until its first row is stored."""
    p = Pool(1, 8, 2, 64, seed=3)
    kvc, state = p.kvc, p.host()
    x = p.normal(10, 2, D, tag="x")
    x[4, 1, 3] = np.nan
    q = p.normal(1, 8, D, tag="q")
    out = torch.zeros_like(q)

    def store(part, at):
        kvc.check(kvc.kvc_append_packed(p.h, 0, part, part, ints([0, len(part)]), ints([at]), len(part)))
        for i in (0, 2):
            e4m3.append(state[i], state[i + 1], p.order[0], at, part.float().cpu().numpy())
        _same_bits(p, state)
        kvc.check(kvc.kvc_packed_attn(p.h, 0, q, None, ints([at + len(part) - 1]), 1, 0, out))
        return out[0, :4].isfinite().all().item(), out[0, 4:].isfinite().all().item()
    assert store(x[:10], 0) == (True, False)
    assert store(x[:3], 10) == (True, False)
    assert store(x[5:7], 5) == (True, False)
    assert store(x[5:6], 4) == (True, True)
    p.ks[0, int(p.order[0, 0])] = state[1][int(p.order[0, 0])] = np.nan
    assert store(x[:2], 5) == (False, False)
    assert store(x[:1], 0) == (True, True)
    assert p.error() == 0 and p.intact()
