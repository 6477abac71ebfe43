"""Waits of the attention over the 8-bit paged cache that run out: every role of
the block leaves, the error is reported, and the handle works on.

Nothing is broken for it: the limit of the kernels' waits (kvc_set_wait_timeout_ns)
is made shorter than a copy takes to arrive.  The waits for copies and products in
flight before a block leaves keep their limit of 1 s.
"""
import pytest
import torch

from tests._e4m3 import D, DT, Pool, check_attention, cumulative, ints

pytestmark = pytest.mark.gpu

TICKETS = slice(256, 256 + 4 * 160)   # the workspace's counters


# several heads of a tile, one, 32 query rows (two warps per key), 64 (two groups), query rows on M
@pytest.mark.parametrize("H, G, n, cached", [(8, 2, (1, 1, 1), (1500, 700, 3)), (24, 8, (1, 1, 1), (1000, 900, 15)), (32, 1, (1, 1, 1), (1400, 20, 900)),
                                             (64, 1, (1, 1, 1), (1400, 20, 900)), (32, 8, (200, 65, 333), (800, 0, 128))])
def test_short_limits(H, G, n, cached):
    p = Pool(3, H, G, 1536, seed=H)
    p.fill([c + x for c, x in zip(cached, n)])
    q = p.normal(sum(n), H, D, tag="q")
    out = torch.zeros(sum(n), H, D, dtype=DT[p.dtype], device="cuda")
    cu, c = ints(cumulative(n)), ints(cached)
    state, seen = p.host(), set()
    kvc = p.kvc
    for limit in (1, 300, 1000, 3000, 10000, 1):
        kvc.check(kvc.kvc_set_wait_timeout_ns(p.h, limit))
        for _ in range(4):
            out.zero_()
            kvc.check(kvc.kvc_packed_attn(p.h, 0, q, cu, c, sum(n), 0, out))
            e = p.error()
            seen.add(e)
            assert e in (kvc.KVC_OK, kvc.KVC_ERR_TIMEOUT)
            assert not p.ws.data[TICKETS].any() and p.error() == kvc.KVC_OK
            if e == kvc.KVC_OK:
                check_attention(p, q, out, cumulative(n), cached)
    assert kvc.KVC_ERR_TIMEOUT in seen, "a limit of 1 ns is shorter than a copy"
    kvc.check(kvc.kvc_set_wait_timeout_ns(p.h, 0))
    for _ in range(2):
        out.zero_()
        kvc.check(kvc.kvc_packed_attn(p.h, 0, q, cu, c, sum(n), 0, out))
        assert p.error() == kvc.KVC_OK
        check_attention(p, q, out, cumulative(n), cached)
    p.same(state)
    assert p.intact()


@pytest.mark.parametrize("H, G, n, cached", [(8, 2, (1, 1, 1), (1500, 700, 3)), (32, 8, (200, 65, 333), (800, 0, 128))])
def test_short_limit_behind_another_error(H, G, n, cached):
    """A bad sequence's error is the first; the counters that a wait left are cleared all the same."""
    p = Pool(3, H, G, 1536, seed=H)
    p.fill([c + x for c, x in zip(cached, n)])
    q = p.normal(sum(n), H, D, tag="q")
    out = torch.zeros(sum(n), H, D, dtype=DT[p.dtype], device="cuda")
    cu, kvc = ints(cumulative(n)), p.kvc
    for _ in range(4):
        kvc.check(kvc.kvc_set_wait_timeout_ns(p.h, 1))
        kvc.check(kvc.kvc_packed_attn(p.h, 0, q, cu, ints([cached[0], -1, cached[2]]), sum(n), 0, out))
        assert p.error() in (kvc.KVC_ERR_DEVICE_INDEX, kvc.KVC_ERR_TIMEOUT) and not p.ws.data[TICKETS].any()
        kvc.check(kvc.kvc_set_wait_timeout_ns(p.h, 0))
        kvc.check(kvc.kvc_packed_attn(p.h, 0, q, cu, ints(cached), sum(n), 0, out))
        assert p.error() == kvc.KVC_OK
        check_attention(p, q, out, cumulative(n), cached)
    assert p.intact()
