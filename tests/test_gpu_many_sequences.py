"""The serving calls with many sequences: more than one step of a kernel's
search takes."""
import numpy as np
import pytest
import torch

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
