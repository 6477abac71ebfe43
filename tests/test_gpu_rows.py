"""Prompt and tree attention on the GPU against their 64-bit definition.

Cached rows past cache_index, new rows past a sequence's own, and packed rows
outside every sequence hold NaN, outputs that must stay unwritten a canary
value.  Tolerances are derived in oracle.rows.tolerance.
"""
import numpy as np
import pytest
import torch

from oracle import rows
from static_kv_cache_gb300 import synth
from tests import _rows

pytestmark = pytest.mark.gpu

UNTOUCHED = 7.0


def prompt(c, lens, cached, layer=0, gap=(0, 0), stream=None):
    """Run kvc_prompt_attn; returns (packed q, k, v, cu, out buffer, out)."""
    total = gap[0] + sum(lens) + gap[1]
    cu = gap[0] + np.concatenate([[0], np.cumsum(lens)])
    q, k, v = c.draw(total, c.H, c.D, tag="q"), c.draw(total, c.G, c.D, tag="k"), c.draw(total, c.G, c.D, tag="v")
    for x in (q, k, v):
        x[:gap[0]] = float("nan")
        x[total - gap[1]:] = float("nan")
    kb, k = _rows.guarded(k)
    vb, v = _rows.guarded(v)
    ob, out = _rows.guarded(torch.full_like(q, UNTOUCHED))
    st = c.kvc.kvc_prompt_attn(c.h, layer, q, k, v, _rows.ints(cu), None if cached is None else _rows.ints(cached), total,
                               c.scratch.data, c.scratch.nbytes, out, stream)
    return st, q, k, v, cu, (kb, vb, ob), out


def check_prompt(c, lens, cached, layer=0, gap=(0, 0), skip=()):
    st, q, k, v, cu, bufs, out = prompt(c, lens, cached, layer, gap)
    assert st == 0
    assert c.error() == (c.kvc.KVC_ERR_DEVICE_INDEX if skip else 0)
    written = torch.zeros(len(q), dtype=torch.bool)
    for b, n in enumerate(lens):
        if b in skip or n == 0:
            continue
        a, m = int(cu[b]), cached[b] if cached is not None else 0
        written[a:a + n] = True
        keys, vals = c.at(c.K, layer, b, range(m)), c.at(c.V, layer, b, range(m))
        ref = rows.attend(q[a:a + n].transpose(0, 1), keys, vals, k[a:a + n].transpose(0, 1), v[a:a + n].transpose(0, 1),
                          torch.ones(n, n, dtype=torch.bool).tril())
        _rows.close(out[a:a + n].transpose(0, 1), *ref, c.dtype, c.D, m + n, f"sequence {b}")
    assert (out.cpu()[~written] == UNTOUCHED).all()
    assert c.intact() and all(x.canaries_intact() for x in bufs)


def drafts(c, nodes, seen, T, gen_tag="t"):
    q, k, v = c.draw(c.B, c.H, T, c.D, tag=gen_tag), c.draw(c.B, c.G, T, c.D, tag=gen_tag + "k"), c.draw(c.B, c.G, T, c.D, tag=gen_tag + "v")
    for b, n in enumerate(nodes):
        for x in (q, k, v):
            x[b, :, n:] = float("nan")
    return q, k, v


def check_tree(c, T, cached, nodes, seen, layer=0, chain=False, hint=None, skip=(), stated_nodes=None, stated_cached=None):
    n_of = [T] * c.B if nodes is None else nodes
    q, k, v = drafts(c, n_of, seen, T)
    kb, k = _rows.guarded(k)
    vb, v = _rows.guarded(v)
    ob, out = _rows.guarded(torch.full_like(q, UNTOUCHED))
    said = stated_nodes if stated_nodes is not None else nodes
    st = c.kvc.kvc_tree_attn(c.h, layer, q, k, v, _rows.ints(stated_cached if stated_cached is not None else cached),
                             None if said is None else _rows.ints(said), None if chain else _rows.words(seen), T,
                             max(cached) if hint is None else hint, c.scratch.data, c.scratch.nbytes, out, None)
    assert st == 0
    assert c.error() == (c.kvc.KVC_ERR_DEVICE_INDEX if skip else 0)
    for b, n in enumerate(n_of):
        if b in skip:
            assert (out[b] == UNTOUCHED).all()
            continue
        assert (out[b, :, n:] == UNTOUCHED).all()
        if n == 0:
            continue
        m = cached[b]
        ref = rows.attend(q[b, :, :n], c.at(c.K, layer, b, range(m)), c.at(c.V, layer, b, range(m)), k[b, :, :n], v[b, :, :n],
                          seen[b, :n, :n])
        _rows.close(out[b, :, :n], *ref, c.dtype, c.D, m + n, f"sequence {b}")
    assert c.intact() and all(x.canaries_intact() for x in (kb, vb, ob))


# dtype, H, G, D: every kernel, groups that divide 128 and groups that do not
SHAPES = [("bf16", 8, 2, 128), ("fp16", 6, 2, 128), ("bf16", 7, 1, 64), ("fp16", 2, 2, 64), ("bf16", 16, 1, 128),
          ("fp16", 32, 1, 128), ("bf16", 64, 1, 64), ("bf16", 5, 1, 128), ("fp32", 4, 2, 64), ("bf16", 8, 2, 32),
          ("fp16", 4, 1, 256), ("fp32", 2, 2, 128)]


@pytest.mark.parametrize("dtype,H,G,D", SHAPES)
def test_prompts_of_different_lengths(dtype, H, G, D):
    c = _rows.Cache(dtype, 2, 6, H, G, D, 320, seed=1)
    lens = [1, 0, 130, 17, 65, 2]
    cached = [0, 40, 200, 3, 0, 129]
    c.fill(1, cached)
    check_prompt(c, lens, cached, layer=1, gap=(3, 5))
    check_prompt(c, lens, None)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_prompt_lengths_around_the_tiles(n):
    c = _rows.Cache("bf16", 1, 2, 4, 1, 128, 16, seed=n)
    check_prompt(c, [n, 3], None)


@pytest.mark.parametrize("m", [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 383])
@pytest.mark.parametrize("paged", [False, True])
def test_prefix_lengths_around_the_tiles(m, paged):
    c = _rows.Cache("fp16", 1, 2, 4, 1, 128, 400, paged=paged, seed=m)
    c.fill(0, [m, 400])
    check_prompt(c, [5, 40], [m, 400])


@pytest.mark.parametrize("dtype,H,G,D", [("bf16", 8, 2, 128), ("fp16", 6, 2, 64), ("bf16", 32, 1, 128), ("fp16", 64, 1, 64), ("bf16", 7, 1, 128)])
def test_paged_prompts(dtype, H, G, D):
    c = _rows.Cache(dtype, 2, 4, H, G, D, 320, paged=True, seed=2)
    cached = [320, 0, 33, 144]
    c.fill(1, cached)
    check_prompt(c, [20, 70, 150, 1], cached, layer=1)


def test_one_prompt_split_over_the_gpu():
    """One KV head and many key tiles: several CTAs share the rows."""
    c = _rows.Cache("bf16", 1, 1, 4, 1, 128, 2048, seed=4)
    c.fill(0, [2048])
    check_prompt(c, [70], [2048])


def test_bad_ranges_are_skipped():
    c = _rows.Cache("bf16", 1, 4, 4, 2, 64, 64, seed=5)
    c.fill(0, [10, 64, 20, 0])
    q = c.draw(60, 4, 64, tag="q")
    k, v = c.draw(60, 2, 64, tag="k"), c.draw(60, 2, 64, tag="v")
    ob, out = _rows.guarded(torch.full_like(q, UNTOUCHED))
    # sequence 0: cached rows out of range; 1: reversed; 2: past the end; 3 fine
    for cu, cached, fine in (([0, 10, 20, 30, 60], [65, 64, -1, 0], (1, 3)), ([30, 40, 20, 61, 61], [0] * 4, (0,)),
                             ([-1, 5, 60, 60, 59], [0] * 4, (1, 2))):
        out.fill_(UNTOUCHED)
        st = c.kvc.kvc_prompt_attn(c.h, 0, q, k, v, _rows.ints(cu), _rows.ints(cached), 60, c.scratch.data, c.scratch.nbytes, out, None)
        assert st == 0 and c.error() == c.kvc.KVC_ERR_DEVICE_INDEX and c.error() == 0
        written = torch.zeros(60, dtype=torch.bool)
        for b in fine:
            written[cu[b]:cu[b + 1]] = True
        assert (out.cpu()[~written] == UNTOUCHED).all() and torch.isfinite(out.float()).all()
        assert (out.cpu()[written] != UNTOUCHED).any(-1).all()
    assert c.intact() and ob.canaries_intact()


@pytest.mark.parametrize("dtype,H,G,D", SHAPES)
def test_trees(dtype, H, G, D):
    T = 21
    c = _rows.Cache(dtype, 2, 5, H, G, D, 304, seed=6)
    cached, nodes = [300, 0, 129, 64, 1], [21, 20, 0, 1, 13]
    c.fill(1, cached)
    seen = torch.stack([_rows.tree(T, s) for s in range(5)])
    check_tree(c, T, cached, nodes, seen, layer=1)


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 100, 128, 129, 200, 260])
def test_tree_sizes(T):
    c = _rows.Cache("fp16", 1, 2, 4, 2, 64, 272, paged=True, seed=T)
    c.fill(0, [130, 16])
    seen = torch.stack([_rows.tree(T, T), _rows.tree(T, T + 1)])
    check_tree(c, T, [130, 16], [T, max(1, T - 3)], seen, hint=0)


@pytest.mark.parametrize("dtype,H,G,D", [("bf16", 8, 2, 128), ("fp16", 12, 2, 128), ("bf16", 32, 1, 64)])
def test_paged_trees(dtype, H, G, D):
    T = 40
    c = _rows.Cache(dtype, 1, 3, H, G, D, 640, paged=True, seed=8)
    c.fill(0, [640, 15, 333])
    check_tree(c, T, [640, 15, 333], None, torch.stack([_rows.tree(T, s) for s in range(3)]))


@pytest.mark.parametrize("dtype,D,paged", [("bf16", 128, True), ("fp16", 64, False), ("fp32", 64, False)])
def test_more_drafts_than_the_cache_has_rows(dtype, D, paged):
    c = _rows.Cache(dtype, 1, 2, 4, 2, D, 16, paged=paged, seed=35)
    c.fill(0, [16, 5])
    check_tree(c, 150, [16, 5], [150, 140], torch.stack([_rows.tree(150, i) for i in range(2)]))


def test_a_chain_needs_no_mask():
    c = _rows.Cache("bf16", 1, 2, 4, 1, 128, 300, seed=9)
    c.fill(0, [300, 7])
    seen = torch.stack([_rows.tree(50, 0, chain=True)] * 2)
    check_tree(c, 50, [300, 7], [50, 33], seen, chain=True)


def test_one_token_is_the_decode_step():
    """T = 1: the decode attention of the row, were it appended."""
    c = _rows.Cache("bf16", 1, 3, 8, 2, 128, 200, seed=10)
    c.fill(0, [150, 1, 64])
    check_tree(c, 1, [150, 1, 64], None, torch.ones(3, 1, 1, dtype=torch.bool))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_that_see_nothing_are_zero(dtype):
    """Any mask: rows without a bit, rows that do not see themselves, bits of
    tokens a sequence does not have."""
    T = 37
    c = _rows.Cache(dtype, 1, 3, 4, 2, 64, 64, seed=11)
    c.fill(0, [0, 20, 0])
    rng = np.random.default_rng(12)
    seen = torch.from_numpy(rng.random((3, T, T)) < 0.2)
    seen[:, 5] = False
    seen[0, 30:] = False
    seen[:, 36, 36] = False
    check_tree(c, T, [0, 20, 0], [37, 37, 30], seen)


@pytest.mark.parametrize("dtype,paged", [("bf16", False), ("fp16", True), ("fp32", False)])
@pytest.mark.parametrize("T", [7, 70, 140])
def test_infinities_and_nan_reach_the_tokens_that_see_them(dtype, paged, T):
    """In V rows of drafted tokens; K rows of tokens that nobody sees hold NaN."""
    c = _rows.Cache(dtype, 1, 2, 8, 2, 64, 320, paged=paged, seed=40 + T)
    cached = [300, 0]
    c.fill(0, cached)
    seen = torch.stack([_rows.tree(T, T), _rows.tree(T, T + 1)])
    dead = T - 2
    seen[:, :, dead] = False
    q, k, v = drafts(c, [T, T], None, T)
    k[:, :, dead] = float("nan")
    v[:, :, dead, 3] = float("inf")
    v[0, 0, 1, 5], v[0, 1, T // 2, 0], v[1, 0, 2, 63], v[1, 0, 4, 63] = (float(x) for x in ("inf", "nan", "inf", "-inf"))
    out = torch.zeros_like(q)
    assert c.kvc.kvc_tree_attn(c.h, 0, q, k, v, _rows.ints(cached), None, _rows.words(seen), T, 0, c.scratch.data,
                               c.scratch.nbytes, out, None) == 0
    assert c.error() == 0
    for b in range(2):
        m = cached[b]
        ref = rows.attend(q[b], c.at(c.K, 0, b, range(m)), c.at(c.V, 0, b, range(m)), k[b], v[b], seen[b])
        assert not torch.isfinite(ref[0]).all()
        _rows.close(out[b], *ref, dtype, 64, m + T)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_prompts_infinities_reach_later_tokens_only(dtype):
    c = _rows.Cache(dtype, 1, 3, 4, 1, 128, 64, seed=50)
    lens = [150, 30, 77]
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = c.draw(257, 4, 128, tag="q"), c.draw(257, 1, 128, tag="k"), c.draw(257, 1, 128, tag="v")
    v[140, 0, 7], v[150, 0, 0], v[256, 0, 1] = float("nan"), float("inf"), float("-inf")
    out = torch.zeros_like(q)
    assert c.kvc.kvc_prompt_attn(c.h, 0, q, k, v, _rows.ints(cu), None, 257, c.scratch.data, c.scratch.nbytes, out, None) == 0
    assert c.error() == 0
    empty = torch.zeros(1, 0, 128, device="cuda")
    for b, n in enumerate(lens):
        a = int(cu[b])
        ref = rows.attend(q[a:a + n].transpose(0, 1), empty, empty, k[a:a + n].transpose(0, 1), v[a:a + n].transpose(0, 1),
                          torch.ones(n, n, dtype=torch.bool).tril())
        _rows.close(out[a:a + n].transpose(0, 1), *ref, dtype, 128, n)


@pytest.mark.parametrize("dtype,D,paged", [("bf16", 64, True), ("fp16", 128, False), ("fp32", 64, False)])
@pytest.mark.parametrize("T", [7, 70, 140])
def test_infinite_and_nan_scores_in_a_tree(dtype, D, paged, T):
    """In K rows of drafted tokens (an infinite element's score is +inf or -inf by
    the sign of q) and in a cached one, which every token sees."""
    c = _rows.Cache(dtype, 1, 3, 8, 2, D, 320, paged=paged, seed=70 + T)
    cached = [300, 0, 200]
    c.fill(0, cached)
    c.put(c.K, 0, 2, [130], torch.full((2, 1, D), float("nan"), dtype=c.tdt, device="cuda"))
    seen = torch.stack([_rows.tree(T, T + i) for i in range(3)])
    q, k, v = drafts(c, [T] * 3, None, T)
    k[0, 0, 3, 5], k[0, 1, T // 2, 0], k[1, 0, 4, 63], k[1, 1, T - 2, 1] = (float(x) for x in ("inf", "nan", "nan", "nan"))
    out = torch.zeros_like(q)
    assert c.kvc.kvc_tree_attn(c.h, 0, q, k, v, _rows.ints(cached), None, _rows.words(seen), T, 0, c.scratch.data,
                               c.scratch.nbytes, out, None) == 0
    assert c.error() == 0
    for b in range(3):
        m = cached[b]
        ref = rows.attend(q[b], c.at(c.K, 0, b, range(m)), c.at(c.V, 0, b, range(m)), k[b], v[b], seen[b])
        assert ref[0].isnan().all() if b == 2 else ref[0].isnan().any() and not ref[0].isnan().all()
        _rows.close(out[b], *ref, dtype, D, m + T)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m", [0, 2048])
def test_infinite_and_nan_scores_in_a_prompt(dtype, m):
    """Without cached rows, and with so many that the keys are split: the tokens
    from the bad key on are NaN, also where a piece holds nothing else."""
    c = _rows.Cache(dtype, 1, 1, 4, 1, 128, 2048, seed=80)
    c.fill(0, [m])
    n = 300
    q, k, v = c.draw(n, 4, 128, tag="q"), c.draw(n, 1, 128, tag="k"), c.draw(n, 1, 128, tag="v")
    k[200] = float("nan")
    k[250, 0, 3] = float("inf")
    out = torch.zeros_like(q)
    assert c.kvc.kvc_prompt_attn(c.h, 0, q, k, v, _rows.ints([0, n]), _rows.ints([m]), n, c.scratch.data, c.scratch.nbytes, out, None) == 0
    assert c.error() == 0
    ref = rows.attend(q.transpose(0, 1), c.at(c.K, 0, 0, range(m)), c.at(c.V, 0, 0, range(m)), k.transpose(0, 1), v.transpose(0, 1),
                      torch.ones(n, n, dtype=torch.bool).tril())
    assert ref[0][:, 200:].isnan().all() and torch.isfinite(ref[0][:, :200]).all()
    _rows.close(out.transpose(0, 1), *ref, dtype, 128, m + n)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_large_scores(dtype):
    """Scores far apart: the reference maximum moves from tile to tile."""
    c = _rows.Cache(dtype, 1, 1, 4, 2, 128, 700, seed=60)
    c.fill(0, [700])
    ramp = torch.linspace(0.2, 12, 700, device="cuda")[torch.randperm(700, generator=torch.Generator().manual_seed(1)).cuda()]
    c.K[0, 0] *= ramp[:, None].to(c.tdt)
    check_tree(c, 40, [700], None, torch.stack([_rows.tree(40, 3)]))
    check_prompt(c, [200], [700])


def test_bad_tree_arguments_are_skipped():
    c = _rows.Cache("bf16", 1, 4, 4, 2, 64, 64, seed=13)
    c.fill(0, [10, 64, 20, 5])
    seen = torch.stack([_rows.tree(9, s) for s in range(4)])
    check_tree(c, 9, [10, 64, 20, 5], [9, 9, 4, 9], seen, skip=(1, 3), stated_nodes=[9, -1, 4, 10])
    check_tree(c, 9, [10, 64, 20, 5], None, seen, skip=(0, 2), stated_cached=[65, 64, -1, 5])


def test_a_page_out_of_range_is_recorded():
    c = _rows.Cache("bf16", 1, 2, 8, 2, 128, 64, paged=True, seed=14)
    c.fill(0, [60, 60])
    good = c.table.clone()
    for wrong in (-1, c.blocks, 2 ** 31 - 1):
        c.table.copy_(good)
        c.table[0, 2] = wrong
        q, k, v = drafts(c, [4, 4], None, 4)
        out = torch.zeros_like(q)
        seen = torch.stack([_rows.tree(4, 1)] * 2)
        assert c.kvc.kvc_tree_attn(c.h, 0, q, k, v, _rows.ints([60, 60]), None, _rows.words(seen), 4, 0, c.scratch.data,
                                   c.scratch.nbytes, out, None) == 0
        assert c.error() == c.kvc.KVC_ERR_DEVICE_INDEX
        ref = rows.attend(q[1], c.at(c.K, 0, 1, range(60)), c.at(c.V, 0, 1, range(60)), k[1], v[1], seen[1])
        _rows.close(out[1], *ref, "bf16", 128, 64)
        # entries behind the cached rows are not looked at
        c.table.copy_(good)
        c.table[0, 2:] = wrong
        assert c.kvc.kvc_tree_attn(c.h, 0, q, k, v, _rows.ints([32, 60]), None, _rows.words(seen), 4, 0, c.scratch.data,
                                   c.scratch.nbytes, out, None) == 0
        assert c.error() == 0
    c.table.copy_(good)


def test_refusals():
    c = _rows.Cache("bf16", 2, 2, 4, 2, 64, 64, seed=15)
    k, p = c.kvc, 256
    big = 1 << 40
    call = lambda **kw: k.kvc_prompt_attn(c.h, *[{**dict(layer=0, q=p, k=p, v=p, cu=p, c=None, total=8, ws=p, n=big, out=p), **kw}[x]  # noqa: E731
                                                 for x in ("layer", "q", "k", "v", "cu", "c", "total", "ws", "n", "out")])
    assert call(layer=2) == call(layer=-1) == call(total=-1) == call(q=None) == call(k=None) == call(v=None) == k.KVC_ERR_INVALID
    assert call(cu=None) == call(out=None) == k.KVC_ERR_INVALID
    assert call(q=p + 8) == call(k=p + 2) == call(v=p + 4) == call(out=p + 8) == call(ws=p + 16) == k.KVC_ERR_ALIGNMENT
    assert call(ws=None) == call(n=k.kvc_rows_workspace_bytes(c.cfg) - 1) == k.KVC_ERR_WORKSPACE
    assert call(total=0) == 0
    call = lambda **kw: k.kvc_tree_attn(c.h, *[{**dict(layer=0, q=p, k=p, v=p, c=p, n=None, m=None, T=4, hint=0, ws=p, nb=big, out=p), **kw}[x]  # noqa: E731
                                               for x in ("layer", "q", "k", "v", "c", "n", "m", "T", "hint", "ws", "nb", "out")])
    assert call(layer=2) == call(T=0) == call(T=-1) == call(hint=-1) == call(hint=65) == call(c=None) == k.KVC_ERR_INVALID
    assert call(q=p + 8) == call(out=p + 2) == k.KVC_ERR_ALIGNMENT
    assert call(ws=None) == call(nb=0) == k.KVC_ERR_WORKSPACE
    assert k.kvc_append_packed(c.h, 2, p, p, p, p, 1) == k.kvc_append_packed(c.h, 0, p, p, None, p, 1) == k.KVC_ERR_INVALID
    assert k.kvc_append_packed(c.h, 0, p + 8, p, p, p, 1) == k.KVC_ERR_ALIGNMENT
    assert k.kvc_append_packed(c.h, 0, p, p, p, p, 0) == 0
    for bad in ((0, 3, 4, 4), (1, 2, 4, 4), (0, 0, 4, 4), (0, 1, 0, 4), (0, 1, 4, 0)):
        assert k.kvc_tree_commit(c.h, bad[0], bad[1], p, p, p, p, p, bad[2], bad[3]) == k.KVC_ERR_INVALID
    assert k.kvc_tree_commit(c.h, 0, 1, p, p + 8, p, p, p, 4, 4) == k.KVC_ERR_ALIGNMENT
    q8 = _rows.Cache("int8", 1, 2, 4, 2, 128, 64)
    assert k.kvc_prompt_attn(q8.h, 0, p, p, p, p, None, 8, p, big, p) == k.KVC_ERR_UNSUPPORTED
    assert k.kvc_tree_attn(q8.h, 0, p, p, p, p, None, None, 4, 0, p, big, p) == k.KVC_ERR_UNSUPPORTED


@pytest.mark.parametrize("paged", [False, True])
def test_many_sequences(paged):
    """More sequences than a warp has lanes, a third of them without tokens."""
    c = _rows.Cache("bf16", 1, 75, 4, 2, 64, 160, paged=paged, seed=33)
    rng = np.random.default_rng(33)
    cached = [int(x) for x in rng.integers(0, 161, 75)]
    lens = [int(x) if i % 3 else 0 for i, x in enumerate(rng.integers(1, 200, 75))]
    c.fill(0, cached)
    check_prompt(c, lens, cached)
    T = 9
    check_tree(c, T, cached, [min(n, T) for n in lens], torch.stack([_rows.tree(T, i) for i in range(75)]))


def test_two_streams_at_once():
    """Calls on one handle that overlap, each with its own workspace."""
    c = _rows.Cache("bf16", 1, 2, 8, 2, 128, 1024, seed=34)
    c.fill(0, [1000, 700])
    ws = [c.scratch, _rows._gpu.Guarded(c.kvc.kvc_rows_workspace_bytes(c.cfg))]
    lens, cu = [300, 150], _rows.ints([0, 300, 450])
    m = _rows.ints([1000, 700])
    q = [c.draw(450, 8, 128, tag=("q", i)) for i in range(2)]
    k, v = c.draw(450, 2, 128, tag="k"), c.draw(450, 2, 128, tag="v")

    def call(i, out, stream):
        assert c.kvc.kvc_prompt_attn(c.h, 0, q[i], k, v, cu, m, 450, ws[i].data, ws[i].nbytes, out, stream) == 0

    alone = [torch.zeros_like(x) for x in q]
    for i in range(2):
        call(i, alone[i], None)
        torch.cuda.synchronize()
    assert torch.isfinite(alone[0].float()).all() and (alone[0] != alone[1]).any()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(x) for x in q] for _ in range(20)]
    torch.cuda.synchronize()
    for o in outs:
        for i in range(2):
            call(i, o[i], streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o[i], alone[i]) for o in outs for i in range(2))
    assert c.error() == 0 and c.intact() and ws[1].canaries_intact()


def test_sequences_that_share_rows():
    """Ranges 0..n, n..0, 0..n, ...: the reversed ones are recorded; the others
    have no cached rows here, so that each gives the same output."""
    n = 300
    c = _rows.Cache("bf16", 1, 6, 4, 2, 64, 64, seed=31)
    q, k, v = c.draw(n, 4, 64, tag="q"), c.draw(n, 2, 64, tag="k"), c.draw(n, 2, 64, tag="v")
    ob, out = _rows.guarded(torch.full_like(q, UNTOUCHED))
    assert c.kvc.kvc_prompt_attn(c.h, 0, q, k, v, _rows.ints([0, n] * 3 + [0]), None, n, c.scratch.data, c.scratch.nbytes, out, None) == 0
    assert c.error() == c.kvc.KVC_ERR_DEVICE_INDEX and c.error() == 0
    ref = rows.attend(q.transpose(0, 1), k[:0].transpose(0, 1), v[:0].transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1),
                      torch.ones(n, n, dtype=torch.bool).tril())
    _rows.close(out.transpose(0, 1), *ref, c.dtype, c.D, n)
    assert ob.canaries_intact()


def test_sequences_that_share_rows_past_the_limit():
    """2048 sequences of 8192 query blocks with 256 key tiles on average pass 2^31
    together, though none does alone: nothing is written."""
    n, B = 65536, 4096
    c = _rows.Cache("bf16", 1, B, 32, 1, 64, 16, seed=32)
    q, k = torch.zeros(n, 32, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(n, 1, 64, device="cuda", dtype=torch.bfloat16)
    out = torch.full_like(q, UNTOUCHED)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda").repeat(B // 2 + 1)[:B + 1].contiguous()
    assert c.kvc.kvc_prompt_attn(c.h, 0, q, k, k, cu, None, n, c.scratch.data, c.scratch.nbytes, out, None) == 0
    assert c.error() == c.kvc.KVC_ERR_DEVICE_INDEX and c.error() == 0
    assert (out == UNTOUCHED).all() and c.intact()


@pytest.mark.parametrize("what", ["prompt", "tree"])
def test_captured_and_replayed_on_another_stream(what):
    """Two handles' calls in one graph, on a side stream, with one workspace in
    stream order; the replay reads the inputs of the replay."""
    a, b = (_rows.Cache("bf16", 1, 2, 8, 2, 128, 512, seed=s, paged=s == 21) for s in (20, 21))
    for c in (a, b):
        c.fill(0, [512, 77])
    T = 24
    seen = torch.stack([_rows.tree(T, 1), _rows.tree(T, 2)])
    w, lens, cached = _rows.words(seen), _rows.ints([0, T, 2 * T]), _rows.ints([512, 77])
    data = {}
    for c in (a, b):
        if what == "tree":
            q, k, v = drafts(c, [T, T], None, T)
        else:
            q, k, v = c.draw(2 * T, c.H, c.D, tag="q"), c.draw(2 * T, c.G, c.D, tag="k"), c.draw(2 * T, c.G, c.D, tag="v")
        data[c] = (q, k, v, torch.zeros_like(q))

    def call(c, stream):
        q, k, v, out = data[c]
        if what == "tree":
            st = c.kvc.kvc_tree_attn(c.h, 0, q, k, v, cached, None, w, T, 0, a.scratch.data, a.scratch.nbytes, out, stream)
        else:
            st = c.kvc.kvc_prompt_attn(c.h, 0, q, k, v, lens, cached, 2 * T, a.scratch.data, a.scratch.nbytes, out, stream)
        assert st == 0

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(a, side)
            call(b, side)
    for c in (a, b):
        data[c][0].mul_(0.5)
        data[c][3].fill_(UNTOUCHED)
    torch.cuda.synchronize()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for c in (a, b):
        q, k, v, out = data[c]
        for s in range(2):
            n = [512, 77][s]
            if what == "tree":
                x = (q[s], k[s], v[s], out[s], seen[s])
            else:
                x = [t[s * T:(s + 1) * T].transpose(0, 1) for t in (q, k, v, out)] + [torch.ones(T, T, dtype=torch.bool).tril()]
            ref = rows.attend(x[0], c.at(c.K, 0, s, range(n)), c.at(c.V, 0, s, range(n)), x[1], x[2], x[4])
            _rows.close(x[3], *ref, "bf16", 128, n + T)
        assert c.error() == 0 and c.intact()


def test_the_same_call_gives_the_same_bits():
    c = _rows.Cache("bf16", 1, 3, 8, 2, 128, 1500, seed=30)
    c.fill(0, [1500, 700, 3])
    seen = torch.stack([_rows.tree(30, s) for s in range(3)])
    q, k, v = drafts(c, [30] * 3, None, 30)
    outs = []
    for _ in range(5):
        out = torch.zeros_like(q)
        assert c.kvc.kvc_tree_attn(c.h, 0, q, k, v, _rows.ints([1500, 700, 3]), None, _rows.words(seen), 30, 0, c.scratch.data,
                                   c.scratch.nbytes, out, None) == 0
        outs.append(out.view(torch.int16).clone())
    assert all(torch.equal(outs[0], x) for x in outs[1:])


@pytest.mark.parametrize("paged", [False, True])
def test_offsets_past_32_bits(paged):
    """A layer of 5 GB per tensor: the last sequence's rows lie past 2^32 bytes,
    the second layer's past 2^32 elements."""
    G, D, T, L = 8, 128, 81920, 2
    B = 30
    c = _rows.Cache("bf16", L, B, 16, G, D, T, paged=paged, spare=0, seed=70)
    assert c.K[0].numel() * 2 > 1 << 32 and c.K.numel() > 1 << 32
    cached = [0] * (B - 2) + [300, 4000]
    if paged:   # the last blocks of the pool, in descending order
        c.table[B - 1] = torch.arange(c.blocks - 1, c.blocks - 1 - T // 16, -1, device="cuda", dtype=torch.int32)
        c.table[B - 2] = torch.arange(T // 16, device="cuda", dtype=torch.int32)
    c.fill(1, cached)
    nodes = [0] * (B - 2) + [5, 20]
    seen = torch.stack([_rows.tree(20, s) for s in range(B)])
    check_tree(c, 20, cached, nodes, seen, layer=1)
    lens = [0] * (B - 2) + [40, 70]
    check_prompt(c, lens, cached, layer=1)
    # rows stored there by both calls
    k, v = c.draw(70, G, D, tag="ak"), c.draw(70, G, D, tag="av")
    cu = [0] * B + [70]
    assert c.kvc.kvc_append_packed(c.h, 1, k, v, _rows.ints(cu), _rows.ints([0] * (B - 1) + [T - 70]), 70, None) == 0
    kt, vt = c.draw(1, B, G, 9, D, tag="ck"), c.draw(1, B, G, 9, D, tag="cv")
    path, n = np.tile(np.arange(4) * 2, (B, 1)), [0] * (B - 1) + [4]
    assert c.kvc.kvc_tree_commit(c.h, 1, 1, kt, vt, _rows.ints([0] * (B - 1) + [T - 90]), _rows.ints(path), _rows.ints(n), 9, 4, None) == 0
    assert c.error() == 0
    assert torch.equal(c.at(c.K, 1, B - 1, range(T - 70, T)), k.transpose(0, 1)) and torch.equal(c.at(c.V, 1, B - 1, range(T - 70, T)), v.transpose(0, 1))
    assert torch.equal(c.at(c.K, 1, B - 1, range(T - 90, T - 86)), kt[0, B - 1][:, ::2][:, :4])
    assert torch.equal(c.at(c.V, 1, B - 1, range(T - 90, T - 86)), vt[0, B - 1][:, ::2][:, :4])
    assert c.intact()


def test_a_prompt_then_drafts_then_decoding():
    """The calls as a server makes them, over pages: prompts of different
    lengths attended and stored, a tree verified, its accepted path stored, a
    decode step -- every output is the dense attention of the history so far."""
    import oracle
    from tests.test_gpu_pages import Pool
    p = Pool(L=1, B=4, G=2, D=128, per=12, blocks=60, H=8)
    k = p.kvc
    ws = torch.empty(k.kvc_rows_workspace_bytes(p.cfg), dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    hist = [torch.zeros(2, 2, 0, 128, device="cuda", dtype=torch.bfloat16) for _ in range(4)]   # [K or V, head, row, D]
    length = [0] * 4
    for lens in ([37, 1, 100, 0], [5, 60, 0, 3]):      # the second prompts continue the first ones
        total = sum(lens)
        cu = np.concatenate([[0], np.cumsum(lens)])
        q, kk, vv = draw(total, 8, 128), draw(total, 2, 128), draw(total, 2, 128)
        grown = [a + b for a, b in zip(length, lens)]
        p.reserve(length, grown)
        out = torch.zeros_like(q)
        assert k.kvc_prompt_attn(p.h, 0, q, kk, vv, _rows.ints(cu), _rows.ints(length), total, ws, ws.numel(), out, None) == 0
        assert k.kvc_append_packed(p.h, 0, kk, vv, _rows.ints(cu), _rows.ints(length), total, None) == 0
        for b, n in enumerate(lens):
            new = torch.stack([kk, vv])[:, cu[b]:cu[b + 1]].transpose(1, 2)
            if n:
                ref = rows.attend(q[cu[b]:cu[b + 1]].transpose(0, 1), hist[b][0], hist[b][1], new[0], new[1], torch.ones(n, n, dtype=torch.bool).tril())
                _rows.close(out[cu[b]:cu[b + 1]].transpose(0, 1), *ref, "bf16", 128, grown[b])
            hist[b] = torch.cat([hist[b], new], 2)
        length = grown
    for step in range(3):
        T = 11
        seen = torch.stack([_rows.tree(T, 10 * step + b) for b in range(4)])
        q, kk, vv = draw(4, 8, T, 128), draw(4, 2, T, 128), draw(4, 2, T, 128)
        out = torch.zeros_like(q)
        assert k.kvc_tree_attn(p.h, 0, q, kk, vv, _rows.ints(length), None, _rows.words(seen), T, max(length), ws, ws.numel(), out, None) == 0
        for b in range(4):
            _rows.close(out[b], *rows.attend(q[b], hist[b][0], hist[b][1], kk[b], vv[b], seen[b]), "bf16", 128, length[b] + T)
        last = [4 + b + step for b in range(4)]           # the accepted leaf of each tree, and its path
        paths = [seen[b, last[b]].nonzero()[:, 0].tolist() for b in range(4)]
        grown = [n + len(x) for n, x in zip(length, paths)]
        p.reserve(length, grown)
        path = np.zeros((4, T), int)
        for b, x in enumerate(paths):
            path[b, :len(x)] = x
        assert k.kvc_tree_commit(p.h, 0, 1, kk, vv, _rows.ints(length), _rows.ints(path), _rows.ints([len(x) for x in paths]), T, T, None) == 0
        for b, x in enumerate(paths):
            hist[b] = torch.cat([hist[b], torch.stack([kk[b], vv[b]])[:, :, x]], 2)
        length = grown
        q1, k1, v1 = draw(4, 8, 128), draw(4, 2, 1, 128), draw(4, 2, 1, 128)
        p.reserve(length, [n + 1 for n in length])
        length = [n + 1 for n in length]
        out = torch.zeros_like(q1)
        assert k.kvc_decode_step(p.h, 0, q1, k1, v1, _rows.ints(length), max(length), out, None) == 0
        for b in range(4):
            hist[b] = torch.cat([hist[b], torch.stack([k1[b], v1[b]])], 2)
            want = oracle.decode_attn(synth.to_bits(q1[b:b + 1]), synth.to_bits(hist[b][0][None].contiguous()),
                                      synth.to_bits(hist[b][1][None].contiguous()), np.array([length[b]], np.int32), "bf16")
            assert np.abs(out[b].float().cpu().numpy() - want[0]).max() <= 2e-2
    assert k.kvc_get_error(p.h, None) == 0
