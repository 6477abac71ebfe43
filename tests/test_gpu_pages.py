"""The page calls on the GPU against the host model (oracle.pages): tables,
counts and every row of the pools, exactly."""
import numpy as np
import pytest
import torch

from oracle import pages
from static_kv_cache_gb300 import synth
from tests import _gpu, _rows

pytestmark = pytest.mark.gpu


class Pool:
    """A paged cache with its counts, and the host model beside it."""

    def __init__(self, L=2, B=6, G=2, D=64, per=5, blocks=40, dtype="bf16", seed=0, H=None):
        from static_kv_cache_gb300 import kvc
        self.kvc, self.L, self.B, self.per, self.blocks = kvc, L, B, per, blocks
        self.cfg = kvc.make_config(L, B, H or 2 * G, G, D, 16 * per, dtype)
        shape = (L, blocks, G, 16, D)
        self.kb, self.K = _rows.guarded(synth.normal(shape, dtype, seed * 2 + 1, "cuda"))
        self.vb, self.V = _rows.guarded(synth.normal(shape, dtype, seed * 2 + 2, "cuda"))
        self.tb, self.table = _rows.guarded(torch.full((B, per), -1, dtype=torch.int32, device="cuda"))
        self.rb, self.refs = _rows.guarded(torch.zeros(blocks, dtype=torch.int32, device="cuda"))
        self.lb, self.live = _rows.guarded(torch.zeros(1, dtype=torch.int32, device="cuda"))
        self.ws = _gpu.Guarded(kvc.kvc_workspace_bytes(self.cfg))
        self.scratch = _gpu.Guarded(kvc.kvc_pages_workspace_bytes(self.cfg, blocks))
        self.scratch.data.fill_(0xA5)   # nothing is expected of it
        st, self.h = kvc.kvc_alloc_paged(self.cfg, self.K, self.V, blocks, self.table, self.ws.ptr(), self.ws.nbytes)
        kvc.check(st, "alloc")
        self.model = pages.Pages(self.table.tolist(), self.refs.tolist())
        self.k_want, self.v_want = self.K.clone(), self.V.clone()

    def __del__(self):
        if getattr(self, "h", None):
            self.kvc.kvc_free(self.h)

    def _moved(self, pairs):
        for X in (self.k_want, self.v_want):
            old = X.clone()
            for a, b, n in pairs:
                X[:, b, :, :n] = old[:, a, :, :n]

    def fork(self, parent, stream=None):
        assert self.kvc.kvc_pages_fork(self.h, self.table, self.refs, _rows.ints(parent), stream) == 0
        self.model.fork(parent)

    def reserve(self, n, m, stream=None):
        assert self.kvc.kvc_pages_reserve(self.h, self.table, self.refs, _rows.ints(n), _rows.ints(m), self.scratch.data,
                                          self.scratch.nbytes, stream) == 0
        got = self.model.reserve(n, m)
        self._moved(got or [])
        return got

    def free(self, keep, stream=None):
        assert self.kvc.kvc_pages_free(self.h, self.table, self.refs, _rows.ints(keep), stream) == 0
        self.model.free(keep)

    def compact(self, block_map=None, stream=None):
        assert self.kvc.kvc_pages_compact(self.h, self.table, self.refs, block_map, self.live, self.scratch.data,
                                          self.scratch.nbytes, stream) == 0
        moves, live = self.model.compact()
        self._moved([(a, b, 16) for a, b in moves])
        return moves, live

    def check(self, error=0):
        assert self.kvc.kvc_get_error(self.h, None) == error
        assert self.table.tolist() == self.model.table and self.refs.tolist() == self.model.refs
        assert torch.equal(self.K, self.k_want) and torch.equal(self.V, self.v_want)
        assert all(x.canaries_intact() for x in (self.kb, self.vb, self.tb, self.rb, self.lb, self.ws, self.scratch))


@pytest.mark.parametrize("kw", [dict(), dict(L=1, B=1, per=1, blocks=1), dict(L=3, B=7, G=3, D=128, per=9, blocks=50, dtype="fp16"),
                                dict(L=1, B=33, G=1, D=64, per=37, blocks=700)])
def test_a_random_life(kw):
    """Forks, growth, rewinds and compactions in any order."""
    p = Pool(seed=3, **kw)
    rng = np.random.default_rng(p.B)
    length = np.zeros(p.B, int)
    for _ in range(60):
        what = rng.integers(4)
        if what == 0:
            par = rng.integers(-1, p.B, p.B)
            p.fork(par.tolist())
            length = np.where(par >= 0, length[par.clip(0)], 0)
        elif what == 1:
            new = np.minimum(16 * p.per, length + rng.integers(0, 40, p.B) * (rng.random(p.B) < 0.7))
            full = p.reserve(length.tolist(), new.tolist()) is None
            p.check(p.kvc.KVC_ERR_CAPACITY if full else 0)
            length = length if full else new
            continue
        elif what == 2:
            keep = np.where(rng.random(p.B) < 0.5, (length * rng.random(p.B)).astype(int), length)
            p.free(keep.tolist())
            length = keep
        else:
            _, live = p.compact()
            assert int(p.live) == live
        p.check()


def test_beams_share_until_they_write():
    p = Pool(B=8, per=4, blocks=40)
    p.reserve([0] * 8, [40, 23, 32, 0, 1, 16, 17, 64])
    p.check()
    p.fork([0, 0, 0, 1, 1, 2, 2, 7])
    p.check()
    assert p.model.refs.count(3) == 3   # the three pages of 40 rows
    # two of the three holders of a page write: both leave it, the third still holds it
    p.reserve([40, 40, 40, 23, 23, 32, 32, 64], [41, 41, 40, 24, 40, 33, 32, 64])
    p.check()
    # pages reserved ahead of the rows are shared by a fork too, and split without copies
    p.reserve([41, 41, 40, 24, 24, 33, 32, 64], [64, 64, 64, 64, 24, 33, 32, 64])
    p.fork([0, 0, 2, 3, 4, 5, 6, 7])
    p.reserve([41, 41, 40, 24, 24, 33, 32, 64], [60, 60, 40, 24, 24, 33, 32, 64])
    p.check()


def test_a_pinned_page_is_split_by_every_writer():
    p = Pool(B=3, per=3, blocks=12)
    p.reserve([0, 0, 0], [20, 0, 0])
    page = p.model.table[0][1]
    p.refs[page] += 1
    p.model.refs[page] += 1
    p.fork([0, 0, 0])
    assert len(p.reserve([20] * 3, [21] * 3)) == 3
    p.check()
    # and a compaction says where it went
    p.free([0, 0, 0])
    _, m = _rows.guarded(torch.zeros(12, dtype=torch.int32, device="cuda"))
    moves, live = p.compact(m)
    p.check()
    want = list(range(12))
    for a, b in moves:
        want[a] = b
    assert m.tolist() == want and live == 1 and want[page] == 0


def test_too_few_blocks_change_nothing():
    p = Pool(B=4, per=4, blocks=9)
    p.reserve([0] * 4, [40, 16, 1, 0])
    p.check()
    p.fork([0, 0, 2, 3])
    assert p.reserve([40, 40, 1, 0], [50, 64, 33, 33]) is None
    p.check(p.kvc.KVC_ERR_CAPACITY)
    assert p.reserve([40, 40, 1, 0], [50, 48, 17, 16]) is not None
    p.check()


def test_bad_arguments_leave_a_sequence_alone():
    p = Pool(B=5, per=3, blocks=20)
    p.reserve([0, -1, 5, 0, 0], [49, 4, 4, 48, 7])     # too long; negative; shrinking; fine; fine
    p.check(p.kvc.KVC_ERR_DEVICE_INDEX)
    p.reserve([0, 0, 3, 48, 7], [1, 0, 9, 48, 9])      # sequence 2 has no page for its 3 rows
    p.check(p.kvc.KVC_ERR_DEVICE_INDEX)
    p.fork([5, 3, -2, 3, 2 ** 31 - 1])
    p.check(p.kvc.KVC_ERR_DEVICE_INDEX)
    p.free([-1, 49, 48, 20, 2 ** 31 - 1])
    p.check(p.kvc.KVC_ERR_DEVICE_INDEX)


def test_entries_out_of_range_are_no_pages():
    p = Pool(B=3, per=3, blocks=10)
    p.reserve([0, 0, 0], [30, 30, 30])
    p.check()
    for bad in (10, -2, 2 ** 31 - 1, -2 ** 31):
        p.table[0, 2] = bad
        p.reserve([32, 30, 30], [33, 30, 30])
        p.check(p.kvc.KVC_ERR_DEVICE_INDEX)
        p.free([32, 48, 48])
        p.check()
        p.table[0, 2] = bad
        p.free([32, 48, 48])
        p.check(p.kvc.KVC_ERR_DEVICE_INDEX)
        p.table[1, 2] = bad
        p.fork([0, 1, 1])
        p.table[1, 2] = -1
        p.check(p.kvc.KVC_ERR_DEVICE_INDEX)
        p.table[0, 2] = bad
        p.compact()
        p.table[0, 2] = -1
        p.check(p.kvc.KVC_ERR_DEVICE_INDEX)


def test_copies_of_listed_blocks():
    p = Pool(L=3, G=3, D=128, blocks=30, H=6)
    src, dst = [4, 9, 4, 30, 2, -1, 7], [11, 12, 13, 1, -1, 3, 30]
    assert p.kvc.kvc_pages_copy(p.h, _rows.ints(src), _rows.ints(dst), 7, None) == 0
    p._moved([(4, 11, 16), (9, 12, 16), (4, 13, 16)])
    p.check(p.kvc.KVC_ERR_DEVICE_INDEX)


def test_many_sequences_and_blocks():
    """More sequences than a block has threads, more blocks than a scan step."""
    p = Pool(L=1, B=1500, G=1, D=64, per=7, blocks=9001)
    rng = np.random.default_rng(8)
    length = rng.integers(0, 90, 1500)
    p.reserve([0] * 1500, length.tolist())
    p.check()
    par = rng.integers(0, 1500, 1500)
    p.fork(par.tolist())
    length = length[par]
    p.reserve(length.tolist(), (length + 1).tolist())
    p.check()
    keep = np.where(rng.random(1500) < 0.3, 0, length)
    p.free(keep.tolist())
    p.compact()
    p.check()


def test_decoding_over_forked_pages():
    """Fork, reserve and decode steps together: each beam's output is the dense
    attention over its own history."""
    import oracle
    p = Pool(L=1, B=4, G=2, D=128, per=4, blocks=20, H=8)
    k = p.kvc
    rng = np.random.default_rng(9)
    hist = [[] for _ in range(4)]
    n = 0
    for step in range(40):
        if step in (18, 19, 33):
            par = rng.integers(0, 4, 4).tolist()
            p.fork(par)
            hist = [list(hist[x]) for x in par]
        p.reserve([n] * 4, [n + 1] * 4)
        q, kn, vn = (synth.normal(s, "bf16", 100 * step + i, "cuda") for i, s in enumerate([(4, 8, 128), (4, 2, 1, 128), (4, 2, 1, 128)]))
        n += 1
        for b in range(4):
            hist[b].append((synth.to_bits(kn)[b, :, 0], synth.to_bits(vn)[b, :, 0]))
        out = torch.empty_like(q)
        assert k.kvc_decode_step(p.h, 0, q, kn, vn, _rows.ints([n] * 4), n, out, None) == 0
        assert k.kvc_get_error(p.h, None) == 0
        K, V = (np.stack([np.stack([r[i] for r in h], 1) for h in hist]) for i in (0, 1))
        _gpu.compare(out, oracle.decode_attn(synth.to_bits(q), K, V, np.full(4, n, np.int32), "bf16"), "bf16", f"step {step}")


def test_captured_and_replayed():
    p = Pool(B=4, per=4, blocks=30)
    p.reserve([0] * 4, [20, 30, 40, 50])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    parent, n, m, keep = (_rows.ints(x) for x in ([0, 0, 2, 2], [20, 20, 40, 40], [25, 36, 41, 64], [25, 0, 41, 30]))
    args = (p.h, p.table, p.refs)
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            assert p.kvc.kvc_pages_fork(*args, parent, side) == 0
            assert p.kvc.kvc_pages_reserve(*args, n, m, p.scratch.data, p.scratch.nbytes, side) == 0
            assert p.kvc.kvc_pages_free(*args, keep, side) == 0
            assert p.kvc.kvc_pages_compact(*args, None, p.live, p.scratch.data, p.scratch.nbytes, side) == 0
    torch.cuda.synchronize()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        p.model.fork([0, 0, 2, 2])
        p._moved(p.model.reserve([20, 20, 40, 40], [25, 36, 41, 64]))
        p.model.free([25, 0, 41, 30])
        moves, live = p.model.compact()
        p._moved([(a, b, 16) for a, b in moves])
        p.check()
        assert int(p.live) == live


def test_refusals():
    p, q = Pool(), 256
    k, a = p.kvc, (p.h, p.table, p.refs)
    assert k.kvc_pages_fork(p.h, p.refs, p.refs, q) == k.kvc_pages_fork(*a, None) == k.KVC_ERR_INVALID
    assert k.kvc_pages_fork(p.h, p.table, None, q) == k.kvc_pages_free(*a, None) == k.KVC_ERR_INVALID
    assert k.kvc_pages_fork(p.h, p.table, p.refs.data_ptr() + 4, q) == k.KVC_ERR_ALIGNMENT
    n = p.scratch.nbytes
    assert k.kvc_pages_reserve(*a, q, None, p.scratch.data, n) == k.kvc_pages_reserve(*a, None, q, p.scratch.data, n) == k.KVC_ERR_INVALID
    assert k.kvc_pages_reserve(*a, q, q, None, n) == k.kvc_pages_reserve(*a, q, q, p.scratch.data, n - 1) == k.KVC_ERR_WORKSPACE
    assert k.kvc_pages_reserve(*a, q, q, p.scratch.ptr() + 8, n) == k.KVC_ERR_ALIGNMENT
    assert k.kvc_pages_compact(*a, None, None, p.scratch.data, n) == k.KVC_ERR_INVALID
    assert k.kvc_pages_compact(*a, None, p.live, p.scratch.data, 0) == k.KVC_ERR_WORKSPACE
    assert k.kvc_pages_copy(p.h, q, q, -1) == k.kvc_pages_copy(p.h, None, q, 1) == k.KVC_ERR_INVALID
    assert k.kvc_pages_copy(p.h, None, None, 0) == 0
    c = _rows.Cache("bf16", 1, 2, 4, 2, 64, 64)
    assert k.kvc_pages_fork(c.h, q, q, q) == k.kvc_pages_copy(c.h, q, q, 1) == k.KVC_ERR_UNSUPPORTED
    p.check()
