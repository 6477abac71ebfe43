"""The 8-bit paged cache: calls that are refused leave nothing behind."""
import pytest
import torch

from tests import _rows
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


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_rope_outputs_over_other_inputs(cache):
    """Warps write outputs while others still read: refused, but for q and k in their own place."""
    p = Pool(2, 4, 2, 64) if cache == "e4m3" else _rows.Cache("bf16", 1, 2, 4, 2, D, 64)
    kvc = p.kvc
    K = p.K.clone()
    buf = torch.zeros(64 * D, dtype=torch.bfloat16, device="cuda")
    q, k, v, out, far = (buf.data_ptr() + 2 * D * x for x in (0, 12, 18, 24, 36))  # 3 tokens: 12, 6, 6 rows; outputs 12, 6
    fused = buf.data_ptr() + 2 * D * 40                                         # 3 tokens of 4 + 2 + 2 rows
    c, cu, row = ints([5, 0]), ints([0, 1, 3]), 2 * D

    def call(q_out, k_out, q=q, k=k, v=v, qs=4, ks=2, vs=2):
        return kvc.kvc_append_rope(p.h, 0, None, q, qs * D, k, ks * D, v, vs * D, cu, c, 3, q_out, k_out)
    for q_out, k_out in ((k, None), (v, None), (q + row, None), (k - 11 * row, None), (v + 5 * row, None), (out, out), (out, out + 11 * row),
                         (out, v), (out, q), (out, q + 11 * row), (out, k + row), (out, v + 5 * row)):
        assert call(q_out, k_out) == kvc.KVC_ERR_INVALID, (q_out, k_out)
    for at in (0, 4, 6, 23):
        assert call(fused + at * row, None, fused, fused + 4 * row, fused + 6 * row, 8, 8, 8) == kvc.KVC_ERR_INVALID
        assert call(out, fused + at * row, fused, fused + 4 * row, fused + 6 * row, 8, 8, 8) == kvc.KVC_ERR_INVALID
    view = torch.int16 if cache == "bf16" else torch.uint8
    assert torch.equal(p.K.view(view), K.view(view)) and not buf.any()
    for q_out, k_out in ((out, None), (out, far), (q, None), (q, far)):  # side by side, and q in its place
        kvc.check(call(q_out, k_out))
    assert call(q, k) == (kvc.KVC_ERR_INVALID if cache == "e4m3" else kvc.KVC_OK)
    kvc.check(kvc.kvc_append_rope(p.h, 0, None, None, 0, k, 2 * D, v, 2 * D, cu, c, 3, None, far))
    assert p.error() == 0 and p.intact()
