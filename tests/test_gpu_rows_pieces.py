"""Prompt and tree attention where CTA boundaries cut items: the pieces' merge
in every form, and the kernels' instances that test_gpu_rows.py leaves out.

An item is cut where it has more than four key tiles and its call's longest more
than eight; here one or two sequences of 2,048 cached rows and few KV heads
spread over the GPU's SMs, so that every item is cut into several pieces.
"""
import pytest
import torch

from oracle import rows
from tests import _rows
from tests.test_gpu_rows import check_prompt, check_tree, drafts

pytestmark = pytest.mark.gpu

# groups that divide 128, groups that leave rows of a query tile empty, and a
# group of one, in both widths and both types
CUT = [("bf16", 2, 2, 128), ("fp16", 1, 1, 64), ("bf16", 4, 2, 64), ("fp16", 8, 2, 128), ("bf16", 3, 1, 128),
       ("fp16", 5, 1, 64), ("bf16", 6, 1, 64), ("fp16", 7, 1, 128), ("bf16", 16, 1, 128), ("fp16", 32, 1, 64),
       ("bf16", 64, 1, 128), ("fp16", 128, 2, 64)]


@pytest.mark.parametrize("dtype,H,G,D", CUT)
@pytest.mark.parametrize("paged", [False, True])
def test_cut_prompts(dtype, H, G, D, paged):
    if paged and H == G:
        pytest.skip("paged caches have at least two query heads per KV head")
    c = _rows.Cache(dtype, 1, 2, H, G, D, 2048, paged=paged, seed=90)
    cached = [2048, 1403]
    c.fill(0, cached)
    check_prompt(c, [3, 75], cached)
    check_prompt(c, [260, 1], cached)


@pytest.mark.parametrize("dtype,H,G,D", CUT)
@pytest.mark.parametrize("T", [2, 45, 300])
def test_cut_trees(dtype, H, G, D, T):
    """T = 2 fits one query tile (folded pieces) for every group, 300 fills two."""
    c = _rows.Cache(dtype, 1, 2, H, G, D, 2048, seed=91)
    cached = [2011, 1152]
    c.fill(0, cached)
    check_tree(c, T, cached, [T, T - 1], torch.stack([_rows.tree(T, s) for s in range(2)]))


@pytest.mark.parametrize("dtype,H,G,D", [("bf16", 8, 2, 64), ("fp16", 6, 2, 128), ("bf16", 16, 1, 128)])
@pytest.mark.parametrize("T", [7, 70, 140])
def test_infinities_and_nan_in_cut_items(dtype, H, G, D, T):
    """In V rows of drafted tokens, folded (T = 7) or not; K of a token that
    nobody sees holds NaN."""
    c = _rows.Cache(dtype, 1, 2, H, G, D, 2048, seed=92 + T)
    cached = [2048, 1300]
    c.fill(0, cached)
    seen = torch.stack([_rows.tree(T, T), _rows.tree(T, T + 1)])
    dead = T - 2
    seen[:, :, dead] = False
    q, k, v = drafts(c, [T, T], None, T)
    k[:, :, dead] = float("nan")
    v[:, :, dead, 3] = float("inf")
    v[0, 0, 1, 5], v[0, G - 1, T // 2, 0], v[1, 0, 2, D - 1], v[1, 0, 4, D - 1] = (float(x) for x in ("inf", "nan", "inf", "-inf"))
    out = torch.zeros_like(q)
    assert c.kvc.kvc_tree_attn(c.h, 0, q, k, v, _rows.ints(cached), None, _rows.words(seen), T, 0, c.scratch.data,
                               c.scratch.nbytes, out, None) == 0
    assert c.error() == 0
    for b in range(2):
        m = cached[b]
        ref = rows.attend(q[b], c.at(c.K, 0, b, range(m)), c.at(c.V, 0, b, range(m)), k[b], v[b], seen[b])
        assert not torch.isfinite(ref[0]).all()
        _rows.close(out[b], *ref, dtype, D, m + T)


@pytest.mark.parametrize("dtype,G,D", [("bf16", 1, 128), ("fp16", 2, 64)])
@pytest.mark.parametrize("way", ["up", "down"])
def test_pieces_with_maxima_far_apart(dtype, G, D, way):
    """Scores that grow, or shrink, along the cached rows: each piece's maximum
    is far from its neighbours', and the last or the first piece decides."""
    c = _rows.Cache(dtype, 1, 1, 4 * G, G, D, 2048, seed=94)
    c.fill(0, [2048])
    ramp = torch.linspace(0.2, 12, 2048, device="cuda")
    c.K[0, 0] *= (ramp if way == "up" else ramp.flip(0))[:, None].to(c.tdt)
    check_tree(c, 20, [2048], None, torch.stack([_rows.tree(20, 3)]))
    check_prompt(c, [200], [2048])


# the widths and types that run on the CUDA cores
@pytest.mark.parametrize("dtype,H,G,D", [("fp32", 4, 2, 256), ("fp32", 6, 2, 32), ("bf16", 4, 1, 256), ("fp16", 8, 1, 32)])
def test_the_other_widths(dtype, H, G, D):
    c = _rows.Cache(dtype, 2, 3, H, G, D, 320, seed=95)
    cached = [300, 0, 129]
    c.fill(1, cached)
    check_prompt(c, [70, 1, 33], cached, layer=1, gap=(2, 3))
    check_prompt(c, [70, 0, 33], None)
    check_tree(c, 21, cached, [21, 0, 13], torch.stack([_rows.tree(21, s) for s in range(3)]), layer=1)
