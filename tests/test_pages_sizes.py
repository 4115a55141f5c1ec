"""The largest page tables (no kernel is launched)."""
import pytest

import causal_gqa_attention_rope_gb300 as na
from causal_gqa_attention_rope_gb300 import _build


@pytest.mark.parametrize("batch,per_seq,page", [(4096, 1 << 20, 16), (4096, 1 << 19, 128),
                                                (65, (1 << 25) - 1, 64), (17, (1 << 27) - 1, 16)])
def test_fork_of_more_entries_than_32_bits_count(batch, per_seq, page):
    """All of them may be missing: their number would have wrapped round, and pages have been handed to
    entries behind a row."""
    _build.build()
    rc = na.load_library().na_pages_fork(batch, 4, 16, None, 16, 16, per_seq, page, 16, 100, 16, 16, 16, 16, 16,
                                         None, None)
    assert rc == na.NA_ERR_UNSUPPORTED
