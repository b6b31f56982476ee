"""Keeping accepted nodes: the two caches and the new lengths must not share memory. No GPU."""
import pytest

import flash_attention_gb300 as fa
from tests.test_draft_abi import KEPT, at, lib, struct  # noqa: F401
from tests.test_rows_in_place import no_gpu

SIZE = KEPT["num_pages"] * KEPT["n_kv_heads"] * KEPT["page_size"] * KEPT["head_dim"] * 2  # bytes


@pytest.mark.parametrize("kw", [
    dict(v_cache=at(0)), dict(v_cache=at(0) + 16), dict(v_cache=at(0) + SIZE - 16),
    dict(k_cache=at(1) + SIZE - 16), dict(new_lengths=at(0)), dict(new_lengths=at(1) + SIZE - 4),
], ids=str)
def test_caches_that_share_memory_are_refused(lib, kw):
    """(Rows of the one would be moved while the other's are read.)"""
    assert lib.fa_paged_keep(struct(fa.FaPagedKept, KEPT, **kw), None) == fa.FA_ERR_INVALID


def test_caches_side_by_side_are_taken(lib):
    no_gpu()
    for kw in (dict(v_cache=at(0) + SIZE), dict(k_cache=at(1) + SIZE), dict(new_lengths=at(0) + SIZE)):
        rc = lib.fa_paged_keep(struct(fa.FaPagedKept, KEPT, **kw), None)
        assert rc not in (fa.FA_OK, fa.FA_ERR_INVALID), kw
