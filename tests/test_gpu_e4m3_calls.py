"""The 8-bit paged cache: calls that are refused leave nothing behind."""
import pytest
import torch

from tests._e4m3 import D, Pool, ints

pytestmark = pytest.mark.gpu


def test_refused_attention_calls():
    """An output over the queries, or not aligned: refused before the step's append."""
    p = Pool(2, 4, 2, 64)
    p.fill([20, 0])
    kvc, state = p.kvc, p.host()
    x = torch.zeros(3, 4, D, dtype=torch.bfloat16, device="cuda")
    q, k, v = p.normal(2, 4, D, tag="q"), p.normal(2, 2, D, tag="k"), p.normal(2, 2, D, tag="v")
    valid, cached, row = ints([21, 1]), ints([20, 0]), 4 * D * 2
    calls = (lambda a, b: kvc.kvc_decode_step(p.h, 0, a, k, v, valid, 0, b), lambda a, b: kvc.kvc_decode_attn(p.h, 0, a, valid, 0, b),
             lambda a, b: kvc.kvc_packed_attn(p.h, 0, a, None, cached, 2, 0, b))
    for call in calls:
        assert call(x, x) == kvc.KVC_ERR_INVALID
        assert call(x, x.data_ptr() + row) == kvc.KVC_ERR_INVALID and call(x.data_ptr() + row, x) == kvc.KVC_ERR_INVALID
        for off in (2, 4, 8):
            assert call(q, x.data_ptr() + off) == kvc.KVC_ERR_ALIGNMENT
    p.same(state)
    assert not x.any() and p.error() == 0
    y = torch.zeros(4, 4, D, dtype=torch.bfloat16, device="cuda")  # side by side
    y[:2] = q
    kvc.check(kvc.kvc_decode_step(p.h, 0, y, k, v, valid, 0, y[2:]))
    assert y[2:].any() and torch.equal(y[:2], q) and p.error() == 0 and p.intact()
