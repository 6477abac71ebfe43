"""The serving calls with many sequences, more than one step of a kernel's
search takes, and at the limits of what a call may be."""
import numpy as np
import pytest
import torch

from oracle import rows
from tests import _rows
from tests.test_gpu_ingest import _expect, _snapshot

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,paged", [("bf16", False), ("bf16", True), ("int8", False)])
@pytest.mark.parametrize("wrong", ["range", "index", "room"])
def test_packed_append_records_a_late_bad_sequence(dtype, paged, wrong):
    """600 sequences with valid rows on both sides of a bad one that is not among
    the first 256: it is skipped and recorded, the others are stored."""
    B, bad = 600, 300
    c = _rows.Cache(dtype, 1, B, 4, 2, 128, 32, paged=paged, seed=7)
    rng = np.random.default_rng(17)
    lens = rng.integers(0, 12, B)
    at = rng.integers(0, 21, B)
    lens[:3], lens[bad], lens[bad + 1], lens[-1] = 5, 0 if wrong == "range" else 9, 4, 6
    cu = np.concatenate([[0], np.cumsum(lens)])
    total = int(cu[-1])
    fine = set(range(B)) - {bad}
    if wrong == "range":      # reversed; the sequence before it then ends past the packed rows
        cu[bad] = total + 1
        fine -= {bad - 1}
    elif wrong == "index":
        at[bad] = -1
    else:
        at[bad] = 24
    k, v = c.draw(total, 2, 128, tag="k"), c.draw(total, 2, 128, tag="v")
    want = _snapshot(c)
    for b in sorted(fine):
        n = int(cu[b + 1] - cu[b])
        if n:
            r = slice(int(cu[b]), int(cu[b + 1]))
            _expect(c, want, 0, b, list(range(at[b], at[b] + n)), k[r].transpose(0, 1), v[r].transpose(0, 1))
    assert c.kvc.kvc_append_packed(c.h, 0, k, v, _rows.ints(cu), _rows.ints(at), total, None) == 0
    assert c.error() == c.kvc.KVC_ERR_DEVICE_INDEX and c.error() == 0
    assert all(torch.equal(x, y) for x, y in zip(_snapshot(c), want)) and c.intact()


@pytest.mark.parametrize("B", [1000, 6120, 6130, 6143, 6144, 8192])
def test_reserve_at_every_count_of_sequences(B):
    """The ranges of all sequences are in shared memory: below, between and past
    the sizes at which they need more than a block has without asking."""
    from tests.test_gpu_pages import Pool
    p = Pool(L=1, B=B, G=1, D=64, per=1, blocks=B + 3)
    n = np.random.default_rng(B).integers(0, 17, B)
    p.reserve([0] * B, n.tolist())
    p.check()


def test_tables_past_32_bits_are_refused():
    """8,192 sequences of 262,144 pages are 2^31 table entries."""
    from static_kv_cache_gb300 import kvc
    B, T = 8192, 16 * 262144
    cfg = kvc.make_config(1, B, 4, 2, 64, T, "bf16")
    K = torch.zeros(1, 4, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
    x = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(kvc.kvc_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    st, h = kvc.kvc_alloc_paged(cfg, K, K.clone(), 4, x, ws, ws.numel())
    kvc.check(st, "alloc")
    try:
        s = torch.empty(kvc.kvc_pages_workspace_bytes(cfg, 4), dtype=torch.uint8, device="cuda")
        refused = kvc.KVC_ERR_UNSUPPORTED
        assert kvc.kvc_pages_reserve(h, x, x, x, x, s, s.numel()) == refused
        assert kvc.kvc_pages_fork(h, x, x, x) == kvc.kvc_pages_free(h, x, x, x) == refused
        assert kvc.kvc_pages_compact(h, x, x, None, x, s, s.numel()) == refused
        assert kvc.kvc_get_error(h, None) == 0 and not x.any()
    finally:
        kvc.kvc_free(h)


def _wide():
    """8,192 sequences that could hold 524,288 rows each, over 64 KV heads, in a
    pool of few pages: by their limits alone the calls would pass the line's."""
    B, H, G, D, T = 8192, 128, 64, 64, 524288
    from static_kv_cache_gb300 import kvc
    cfg = kvc.make_config(1, B, H, G, D, T, "bf16")
    blocks = 64
    K, V = (torch.randn(1, blocks, G, 16, D, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).bfloat16() for i in (1, 2))
    table = torch.full((B, T // 16), -1, dtype=torch.int32, device="cuda")
    cached = np.zeros(B, int)
    at = 0
    for b, n in ((0, 17), (100, 300), (5000, 1), (8191, 130)):
        pages = -(-n // 16)
        table[b, :pages] = torch.arange(at, at + pages, dtype=torch.int32, device="cuda")
        cached[b], at = n, at + pages
    ws = torch.empty(kvc.kvc_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    st, h = kvc.kvc_alloc_paged(cfg, K, V, blocks, table, ws, ws.numel())
    kvc.check(st, "alloc")
    return kvc, cfg, h, (K, V, table, ws), cached


@pytest.mark.parametrize("what", ["tree", "prompt"])
def test_short_calls_on_a_cache_with_long_limits(what):
    """One new token per sequence; almost all see it alone and return its V row."""
    kvc, cfg, h, (K, V, table, ws), cached = _wide()
    try:
        B, H, G, D = 8192, 128, 64, 64
        gen = torch.Generator("cuda").manual_seed(5)
        q, k, v = (torch.randn(B, n, D, device="cuda", generator=gen).bfloat16() for n in (H, G, G))
        out = torch.full_like(q, 7.0)
        scratch = torch.empty(kvc.kvc_rows_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
        if what == "tree":
            st = kvc.kvc_tree_attn(h, 0, q, k, v, _rows.ints(cached), None, None, 1, 0, scratch, scratch.numel(), out)
        else:
            st = kvc.kvc_prompt_attn(h, 0, q, k, v, _rows.ints(np.arange(B + 1)), _rows.ints(cached), B, scratch, scratch.numel(), out)
        assert st == 0 and kvc.kvc_get_error(h, None) == 0
        alone = torch.from_numpy(cached == 0).cuda()
        assert torch.equal(out[alone], v.repeat_interleave(2, 1)[alone])
        for b in cached.nonzero()[0].tolist():
            n = int(cached[b])
            pages = table[b, :-(-n // 16)].long()
            old = [X[0, pages].transpose(0, 1).reshape(G, -1, D)[:, :n] for X in (K, V)]
            ref = rows.attend(q[b][:, None], *old, k[b][:, None], v[b][:, None], torch.ones(1, 1, dtype=torch.bool))
            _rows.close(out[b][:, None], *ref, "bf16", D, n + 1, f"sequence {b}")
    finally:
        kvc.kvc_free(h)


def test_a_call_past_the_limit_is_recorded():
    """One sequence that says it has 2^30 cached rows: 8 query blocks over 64 KV
    heads with 2^23 key tiles each are 2^32 places.  Nothing is read or written."""
    from static_kv_cache_gb300 import kvc
    H, G, D, T, n = 128, 64, 64, 1 << 30, 1024
    cfg = kvc.make_config(1, 1, H, G, D, T, "bf16")
    K = torch.zeros(1, 4, G, 16, D, device="cuda", dtype=torch.bfloat16)
    table = torch.full((1, T // 16), -1, dtype=torch.int32, device="cuda")
    ws = torch.empty(kvc.kvc_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    st, h = kvc.kvc_alloc_paged(cfg, K, K.clone(), 4, table, ws, ws.numel())
    kvc.check(st, "alloc")
    try:
        scratch = torch.empty(kvc.kvc_rows_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
        q, k = torch.zeros(1, H, n, D, device="cuda", dtype=torch.bfloat16), torch.zeros(1, G, n, D, device="cuda", dtype=torch.bfloat16)
        out = torch.full_like(q, 7.0)
        for m in (T, T - T // 4):   # 2^32 places (0 in 32 bits) and 3 2^30 (negative)
            assert kvc.kvc_tree_attn(h, 0, q, k, k, _rows.ints([m]), None, None, n, 0, scratch, scratch.numel(), out) == 0
            assert kvc.kvc_get_error(h, None) == kvc.KVC_ERR_DEVICE_INDEX and kvc.kvc_get_error(h, None) == 0
            assert (out == 7.0).all()
    finally:
        kvc.kvc_free(h)


def test_a_capacity_past_32_bits_is_refused():
    from static_kv_cache_gb300 import kvc
    cfg = kvc.make_config(1, 1, 4, 2, 64, 2 ** 31 - 16, "bf16")
    K = torch.zeros(1, 4, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
    x = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(kvc.kvc_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    st, h = kvc.kvc_alloc_paged(cfg, K, K.clone(), 4, x, ws, ws.numel())
    kvc.check(st, "alloc")
    try:
        scratch = torch.empty(kvc.kvc_rows_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
        q, k = torch.zeros(1, 4, 1, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(1, 2, 1, 64, device="cuda", dtype=torch.bfloat16)
        assert kvc.kvc_tree_attn(h, 0, q, k, k, x, None, None, 1, 0, scratch, scratch.numel(), q) == kvc.KVC_ERR_UNSUPPORTED
        assert kvc.kvc_prompt_attn(h, 0, q, k, k, x, x, 1, scratch, scratch.numel(), q) == kvc.KVC_ERR_UNSUPPORTED
    finally:
        kvc.kvc_free(h)
