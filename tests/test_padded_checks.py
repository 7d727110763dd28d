"""The debug checks of batches with rows behind the last request's."""
import numpy as np
import pytest

from paged_kv_cache_varlen_gb300 import debug_checks as dc

TABLE = np.array([[3, 1, -1, 7], [2, 0, 4, -1]])
SIZES = dict(max_query_len=3, num_blocks=8, block_size=16)


def test_padded_batches_pass_where_they_are_allowed():
    cu, lens = [0, 1, 4], [20, 40]
    for t in (4, 5, 100):
        dc.check_append_tables(cu, lens, TABLE, num_tokens=t, **SIZES)
        dc.check_attention_tables(cu, lens, TABLE, num_tokens=t, max_seq_len=40, padded=True,
                                  **SIZES)
    with pytest.raises(ValueError, match="num_tokens"):
        dc.check_attention_tables(cu, lens, TABLE, num_tokens=5, max_seq_len=40, **SIZES)
    with pytest.raises(ValueError, match="num_tokens"):
        dc.check_append_tables(cu, lens, TABLE, num_tokens=3, **SIZES)
    with pytest.raises(ValueError, match="num_tokens"):
        dc.check_attention_tables(cu, lens, TABLE, num_tokens=3, max_seq_len=40, padded=True,
                                  **SIZES)
