"""Host side of the prompt, tree and page calls: sizes, and refusals that need
no GPU."""
import pytest


@pytest.fixture()
def kvc(kvc_library_path):
    from static_kv_cache_gb300 import kvc
    return kvc


def test_workspace_sizes(kvc):
    cfg = kvc.make_config(2, 4, 32, 8, 128, 1024, "bf16")
    assert kvc.kvc_rows_workspace_bytes(cfg) > 0
    assert kvc.kvc_pages_workspace_bytes(cfg, 100) >= 4 * 4 * 100
    assert kvc.kvc_pages_workspace_bytes(cfg, 0) == 0 and kvc.kvc_pages_workspace_bytes(cfg, -5) == 0
    bad = kvc.make_config(2, 4, 32, 7, 128, 1024, "bf16")
    assert kvc.kvc_rows_workspace_bytes(bad) == 0 and kvc.kvc_pages_workspace_bytes(bad, 100) == 0


def test_calls_reject_a_missing_handle(kvc):
    p = 256
    bad = kvc.KVC_ERR_INVALID
    assert kvc.kvc_prompt_attn(None, 0, p, p, p, p, p, 1, p, 1 << 30, p) == bad
    assert kvc.kvc_append_packed(None, 0, p, p, p, p, 1) == bad
    assert kvc.kvc_tree_attn(None, 0, p, p, p, p, p, p, 1, 0, p, 1 << 30, p) == bad
    assert kvc.kvc_tree_commit(None, 0, 1, p, p, p, p, p, 1, 1) == bad
    assert kvc.kvc_pages_fork(None, p, p, p) == bad
    assert kvc.kvc_pages_reserve(None, p, p, p, p, p, 1 << 30) == bad
    assert kvc.kvc_pages_free(None, p, p, p) == bad
    assert kvc.kvc_pages_copy(None, p, p, 1) == bad
    assert kvc.kvc_pages_compact(None, p, p, None, p, p, 1 << 30) == bad
