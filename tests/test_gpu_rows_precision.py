"""Prompt and tree attention: sums in which small terms count."""
import pytest
import torch

from oracle import rows
from tests import _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [900, 32000])
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("paged", [False, True])
def test_many_faint_keys_beside_a_dominant_one(m, T, paged):
    """fp16, one key whose probability is nearly 1 and m others of 2^-25.25 each,
    less than half of fp16's least step: together they still count.

    The dominant key's V is 0, the others' 1, so that the output is the faint
    keys' mass.  A probability is rounded to fp16 after it was scaled by 2^7
    (the reference maximum's stays below 2^15): off by half a unit, or by half of
    the least step, 2^-25 2^-7 of the reference's; m of them are off by m 2^-32."""
    B, G, D, score = 8, 8, 64, 17.5
    c = _rows.Cache("fp16", 1, B, 2 * G, G, D, 32000, paged=paged, seed=96)
    lead = torch.zeros(G, 1, D, dtype=torch.float16, device="cuda")
    lead[..., 0] = score * D ** 0.5 / 8
    for b in range(B):
        c.put(c.K, 0, b, range(m), torch.zeros(G, m, D, dtype=torch.float16, device="cuda"))
        c.put(c.V, 0, b, range(m), torch.ones(G, m, D, dtype=torch.float16, device="cuda"))
        c.put(c.K, 0, b, [m * b // B], lead)
        c.put(c.V, 0, b, [m * b // B], 0 * lead)
    q = torch.zeros(B, 2 * G, T, D, dtype=torch.float16, device="cuda")
    q[..., 0] = 8
    k = torch.zeros(B, G, T, D, dtype=torch.float16, device="cuda")
    seen = torch.zeros(B, T, T, dtype=torch.bool)   # cached rows alone
    out = torch.full_like(q, 7.0)
    assert c.kvc.kvc_tree_attn(c.h, 0, q, k, k, _rows.ints([m] * B), None, _rows.words(seen), T, 0, c.scratch.data,
                               c.scratch.nbytes, out, None) == 0
    assert c.error() == 0
    for b in range(B):
        ref, mass, reach = rows.attend(q[b], c.at(c.K, 0, b, range(m)), c.at(c.V, 0, b, range(m)), k[b], k[b], seen[b])
        assert (ref > 2.4e-8 * m).all()
        tol = rows.tolerance(ref, mass, reach, "fp16", D, m) + m * 2.0 ** -32
        err = (out[b].double() - ref).abs()
        assert (err <= tol).all(), (b, float(err.max()), float(tol.min()))
