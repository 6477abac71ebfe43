"""The 64-bit definition of several new tokens' attention, and the host model
of the pages, pinned on the CPU before anything is compared with them."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import pages, rows
from static_kv_cache_gb300 import synth


def _draw(H, G, c, n, D, seed=5):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64).float()  # noqa: E731
    return r(H, n, D), r(G, c, D), r(G, c, D), r(G, n, D), r(G, n, D)


@pytest.mark.parametrize("H,G,c,n,D", [(4, 2, 7, 5, 32), (3, 3, 0, 6, 32), (8, 1, 33, 1, 64)])
def test_a_chain_is_the_prefill_oracle(H, G, c, n, D):
    q, k, v, kn, vn = _draw(H, G, c, n, D)
    out, mass, reach = rows.attend(q, k, v, kn, vn, torch.ones(n, n, dtype=torch.bool).tril())
    K = torch.cat([k, kn], 1).numpy()[None]
    V = torch.cat([v, vn], 1).numpy()[None]
    for t in range(n):
        want = oracle.decode_attn(synth.to_bits(q[None, :, t].contiguous()), K, V, np.array([c + t + 1], np.int32), "fp32")
        assert np.abs(out[:, t].numpy() - want[0]).max() < 1e-12
    assert (mass >= out.abs() - 1e-12).all() and (reach > 0).all()


def test_marks_choose_the_rows():
    """A token that sees one row gets that row; none: zeros; the others do not matter."""
    q, k, v, kn, vn = _draw(2, 1, 0, 4, 32)
    marks = torch.zeros(4, 4, dtype=torch.bool)
    marks[0, 2] = marks[2, 1] = marks[3, 1] = marks[3, 3] = True
    kn[:, 0] = math.nan
    vn[:, 0] = math.inf
    out, _, _ = rows.attend(q, k, v, kn, vn, marks)
    assert torch.equal(out[:, 0], vn[:, 2].expand(2, -1).double()) and torch.equal(out[:, 2], vn[:, 1].expand(2, -1).double())
    assert (out[:, 1] == 0).all()
    x = q[0, 3].double() @ kn[0, [1, 3]].double().T / 32 ** 0.5
    w = 1 / (1 + math.exp(float(x[1] - x[0])))
    assert (out[0, 3] - (w * vn[0, 1].double() + (1 - w) * vn[0, 3].double())).abs().max() < 1e-12


def test_tolerance_covers_an_fp32_evaluation():
    q, k, v, kn, vn = _draw(2, 1, 40, 3, 64)
    marks = torch.ones(3, 3, dtype=torch.bool).tril()
    out, mass, reach = rows.attend(q, k, v, kn, vn, marks)
    s = q @ torch.cat([k, kn], 1)[0].T / 8
    s = s.masked_fill(~torch.cat([torch.ones(3, 40, dtype=torch.bool), marks], 1), -math.inf)
    got = torch.softmax(s, -1) @ torch.cat([v, vn], 1)[0]
    assert ((got.double() - out).abs() <= rows.tolerance(out, mass, reach, "fp32", 64, 43)).all()
    wrong = torch.softmax(s * 1.01, -1) @ torch.cat([v, vn], 1)[0]  # a slightly wrong scale is seen
    assert not ((wrong.double() - out).abs() <= rows.tolerance(out, mass, reach, "fp32", 64, 43)).all()


def _pool(B, per, blocks):
    return pages.Pages([[-1] * per for _ in range(B)], [0] * blocks)


def test_pages_by_hand():
    p = _pool(3, 4, 8)
    assert p.reserve([0, 0, 0], [20, 16, 0]) == []
    assert p.table == [[0, 1, -1, -1], [2, -1, -1, -1], [-1] * 4] and p.check()
    p.fork([0, 0, 0])      # three beams of sequence 0
    assert p.refs[:3] == [3, 3, 0] and p.check()
    # rows 20.. of all three: two split page 1 (4 live rows), the last keeps it
    assert p.reserve([20] * 3, [21] * 3) == [(1, 2, 4), (1, 3, 4)]
    assert [row[1] for row in p.table] == [2, 3, 1] and p.check()
    p.free([0, 17, 16])
    assert p.table == [[-1] * 4, [0, 3, -1, -1], [0, -1, -1, -1]] and p.check()
    assert p.compact() == ([(3, 1)], 2) and p.table[1] == [0, 1, -1, -1] and p.check()
    assert p.reserve([0, 17, 16], [64, 64, 64]) is None and p.table[1] == [0, 1, -1, -1]


def test_pages_hold_what_a_dense_cache_holds():
    """Random forks, growth, rewinds and compactions: every sequence's rows,
    read through the table, are those of a plain copy per sequence."""
    rng = np.random.default_rng(3)
    B, per, blocks = 5, 6, 40
    p = _pool(B, per, blocks)
    store, dense = {}, [[] for _ in range(B)]
    for step in range(200):
        what = rng.integers(4)
        if what == 0:
            par = rng.integers(-1, B, B)
            p.fork(par)
            dense = [list(dense[x]) if x >= 0 else [] for x in par]
        elif what == 1:
            grow = [min(96, len(d) + int(rng.integers(0, 20))) for d in dense]
            got = p.reserve([len(d) for d in dense], grow)
            if got is None:
                continue
            for a, b, n in got:
                for i in range(n):
                    store[b, i] = store[a, i]
            for b, d in enumerate(dense):
                while len(d) < grow[b]:
                    store[p.table[b][len(d) // 16], len(d) % 16] = (step, b, len(d))
                    d.append((step, b, len(d)))
        elif what == 2:
            keep = [int(rng.integers(0, len(d) + 1)) if rng.random() < 0.4 else len(d) for d in dense]
            p.free(keep)
            dense = [d[:n] for d, n in zip(dense, keep)]
        else:
            moves, live = p.compact()
            for a, b in moves:
                for i in range(16):
                    if (a, i) in store:
                        store[b, i] = store[a, i]
            assert all(x < live for row in p.table for x in row)
        assert p.check()
        for b, d in enumerate(dense):
            assert [store[p.table[b][i // 16], i % 16] for i in range(len(d))] == d
