"""Limits of drafted decoding's calls: the list of key tiles that tree attention cuts has to fit 30 bits,
counted by the table's room. No GPU."""
import pytest

import flash_attention_gb300 as fa
from tests.test_draft_abi import FAKE, lib, params  # noqa: F401
from tests.test_rows_in_place import no_gpu

ROOM = dict(page_size=256, max_pages=1 << 14)  # 2^22 keys: 65536 tiles, and 5 for a unit's ends


def units(head_dim, rows):
    """The largest batch * n_kv_heads that the header's rule allows with such a table."""
    block = 128 if head_dim == 256 else 256
    return ((1 << 30) - 1) // ((65536 + 5) * -(-rows // block))


@pytest.mark.parametrize("head_dim,heads,nodes", [(64, 1, 8), (128, 1, 8), (128, 1, 256), (128, 2, 150),
                                                  (256, 1, 128), (256, 1, 129), (64, 9, 250)])
def test_room_of_the_table(lib, head_dim, heads, nodes):
    no_gpu()
    n = units(head_dim, heads * nodes)
    for kv in (1, 2):
        for batch, good in ((n // kv, True), (n // kv + 1, False)):
            p = params(batch=batch, n_heads=heads * kv, n_kv_heads=kv, q_len=nodes, head_dim=head_dim,
                       num_pages=64, **ROOM)
            rc = lib.fa_paged_tree_attention(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, FAKE, None, p, None)
            assert (rc != fa.FA_ERR_INVALID) == good, (batch, kv)
