"""Packed rows and accepted paths into the cache, bit for bit; every other
cache row stays as it was."""
import numpy as np
import pytest
import torch

import oracle
from static_kv_cache_gb300 import synth
from tests import _rows

pytestmark = pytest.mark.gpu

KINDS = [("bf16", 2, 128, False), ("fp16", 3, 64, False), ("fp32", 2, 32, False), ("bf16", 1, 256, False),
         ("bf16", 2, 128, True), ("fp16", 2, 64, True), ("int8", 2, 128, False)]


def _snapshot(c):
    return [x.clone().view(torch.uint8) for x in ((c.K, c.V, c.ks, c.vs) if c.dtype == "int8" else (c.K, c.V))]


def _expect(c, before, layer, b, at, krows, vrows):
    """Write the rows [G, n, D] into the snapshot the way the append defines it."""
    for X, S, r, i in ((c.K, getattr(c, "ks", None), krows, 0), (c.V, getattr(c, "vs", None), vrows, 1)):
        snap = before[i].view(X.dtype).view(X.shape)
        if c.dtype == "int8":
            codes, scale = oracle.quantize_rows(synth.to_bits(r.contiguous()), "bf16")
            snap[layer, b][:, at] = torch.from_numpy(codes).cuda()
            before[2 + i].view(torch.float32).view(S.shape)[layer, b][:, at] = torch.from_numpy(scale).cuda()
        else:
            c.put(snap, layer, b, at, r)


@pytest.mark.parametrize("dtype,G,D,paged", KINDS)
@pytest.mark.parametrize("prefix", [False, True])
def test_packed_append(dtype, G, D, paged, prefix):
    c = _rows.Cache(dtype, 2, 5, 2 * G, G, D, 160, paged=paged, seed=1)
    lens, at = [7, 0, 100, 1, 33], [0, 160, 60, 159, 16] if prefix else [0] * 5
    cu = 2 + np.concatenate([[0], np.cumsum(lens)])
    k, v = c.draw(sum(lens) + 6, G, D, tag="k"), c.draw(sum(lens) + 6, G, D, tag="v")
    want = _snapshot(c)
    for b, n in enumerate(lens):
        if n:
            r = slice(int(cu[b]), int(cu[b]) + n)
            _expect(c, want, 1, b, list(range(at[b], at[b] + n)), k[r].transpose(0, 1), v[r].transpose(0, 1))
    assert c.kvc.kvc_append_packed(c.h, 1, k, v, _rows.ints(cu), _rows.ints(at) if prefix else None, len(k), None) == 0
    assert c.error() == 0
    assert all(torch.equal(x, y) for x, y in zip(_snapshot(c), want)) and c.intact()


@pytest.mark.parametrize("dtype,paged", [("bf16", False), ("bf16", True), ("int8", False)])
def test_packed_append_skips_what_does_not_fit(dtype, paged):
    c = _rows.Cache(dtype, 1, 4, 4, 2, 128, 64, paged=paged, seed=2)
    k, v = c.draw(40, 2, 128, tag="k"), c.draw(40, 2, 128, tag="v")
    for cu, at, fine in (([0, 10, 20, 30, 40], [55, 54, -1, 0], (1, 3)), ([0, 10, 5, 41, 41], [0] * 4, (0,)),
                         ([-3, 4, 40, 40, 40], [0, 65, 0, 0], ())):
        want = _snapshot(c)
        for b in fine:
            n = cu[b + 1] - cu[b]
            r = slice(cu[b], cu[b + 1])
            _expect(c, want, 0, b, list(range(at[b], at[b] + n)), k[r].transpose(0, 1), v[r].transpose(0, 1))
        assert c.kvc.kvc_append_packed(c.h, 0, k, v, _rows.ints(cu), _rows.ints(at), 40, None) == 0
        assert c.error() == c.kvc.KVC_ERR_DEVICE_INDEX
        assert all(torch.equal(x, y) for x, y in zip(_snapshot(c), want)) and c.intact()


@pytest.mark.parametrize("dtype,G,D,paged", KINDS)
@pytest.mark.parametrize("P", [1, 9])
def test_path_commit(dtype, G, D, paged, P):
    c = _rows.Cache(dtype, 3, 4, 2 * G, G, D, 96, paged=paged, seed=3)
    T = 20
    at, n = [0, 96, 87, 31], [P, 0, P, min(P, 5)]
    path = np.full((4, P), -77)   # entries behind n_accept are not looked at
    rng = np.random.default_rng(4)
    for b in range(4):
        path[b, :n[b]] = np.sort(rng.choice(T, n[b], replace=False))
    path[3, :2] = path[3, 0]      # the same token twice
    k, v = c.draw(2, 4, G, T, D, tag="k"), c.draw(2, 4, G, T, D, tag="v")
    want = _snapshot(c)
    for layer in range(2):
        for b in range(4):
            if n[b]:
                sel = torch.as_tensor(path[b, :n[b]], device="cuda")
                _expect(c, want, 1 + layer, b, list(range(at[b], at[b] + n[b])), k[layer, b][:, sel], v[layer, b][:, sel])
    path[3, n[3]:] = 10 ** 6
    assert c.kvc.kvc_tree_commit(c.h, 1, 2, k, v, _rows.ints(at), _rows.ints(path), _rows.ints(n), T, P, None) == 0
    assert c.error() == 0
    assert all(torch.equal(x, y) for x, y in zip(_snapshot(c), want)) and c.intact()


@pytest.mark.parametrize("dtype,paged", [("fp16", False), ("fp16", True), ("int8", False)])
def test_path_commit_skips_bad_sequences(dtype, paged):
    c = _rows.Cache(dtype, 1, 6, 4, 2, 128, 64, paged=paged, seed=5)
    k, v = c.draw(1, 6, 2, 8, 128, tag="k"), c.draw(1, 6, 2, 8, 128, tag="v")
    path = np.tile(np.arange(4), (6, 1))
    path[0, 3], path[1, 0] = 8, -1
    at, n = [0, 0, 61, -1, 7, 0], [4, 4, 4, 1, 4, 5]
    want = _snapshot(c)
    _expect(c, want, 0, 4, list(range(7, 11)), k[0, 4][:, :4], v[0, 4][:, :4])
    assert c.kvc.kvc_tree_commit(c.h, 0, 1, k, v, _rows.ints(at), _rows.ints(path), _rows.ints(n), 8, 4, None) == 0
    assert c.error() == c.kvc.KVC_ERR_DEVICE_INDEX and c.error() == 0
    assert all(torch.equal(x, y) for x, y in zip(_snapshot(c), want)) and c.intact()


def test_a_missing_page_is_recorded_and_not_written():
    c = _rows.Cache("bf16", 1, 2, 4, 2, 64, 64, paged=True, seed=6)
    k, v = c.draw(40, 2, 64, tag="k"), c.draw(40, 2, 64, tag="v")
    good = c.table.clone()
    c.table[0, 1] = -1
    want = _snapshot(c)
    table, c.table = c.table, good
    for rows_ in (range(0, 16), range(32, 40)):
        _expect(c, want, 0, 0, list(rows_), k[rows_.start:rows_.stop].transpose(0, 1), v[rows_.start:rows_.stop].transpose(0, 1))
    assert c.kvc.kvc_append_packed(c.h, 0, k, v, _rows.ints([0, 40, 40]), None, 40, None) == 0
    assert c.error() == c.kvc.KVC_ERR_DEVICE_INDEX
    assert all(torch.equal(x, y) for x, y in zip(_snapshot(c), want)) and c.intact()
    table.copy_(good)
