"""Host checks of the speculative-step entry points that need no GPU: a null
context is refused, and the size queries say 0."""
import pytest

from hybrid_sliding_window_gb300 import api


def test_null_context():
    L = api.lib()
    bad = api.SWA_ERR_INVALID
    assert L.swa_tree_bytes(None, 4, 4) == 0
    assert L.swa_attn_tree_ws_bytes(None, 0, 1, 4, 4, 100) == 0
    assert L.swa_tree_plan(None, 1, None, None, None, 1, 1, None, None, 0, None) == bad
    assert L.swa_attn_tree(None, 0, 1, None, 0, None, None, None, 1, 1, 1, None, None, None, None, 1.0,
                           1.0, 1.0, None, None, 0, None) == bad
    assert L.swa_qk_norm_rope_store(None, 0, None, 0, None, 0, None, 0, 1, None, None, None, 0.0, None, 0,
                                    0, 0, None, None, 1.0, 1.0, None, None) == bad
    assert L.swa_commit_tree(None, 1, None, 0, None, None, None, 1, None, None) == bad
    assert L.swa_copy_kv(None, None, None, 1, None) == bad


def test_header_and_binding_agree_on_the_tree_limit():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    txt = open(os.path.join(root, "include", "swa.h")).read()
    assert int(re.search(r"SWA_TREE_MAX_NODES = (\d+)", txt).group(1)) == api.TREE_MAX_NODES
