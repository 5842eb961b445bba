"""Numbers that do not fit in 32 bits are refused (no GPU), not cut to those that do."""
import pytest

import rank_kv_cache_isvd_b200 as iskv

D = 128
ROWS = iskv.iskv_exact_rows(k=256, v=256, seq_stride=512 * D, head_stride=512 * D, row_stride=D, batch=1,
                            n_kv_heads=1, rows=512, dtype=iskv.ISKV_BF16, lens=None)
QUERIES = iskv.iskv_exact_queries(q=256, out=256, q_seq_stride=D, q_head_stride=D, q_tok_stride=D,
                                  o_seq_stride=D, o_head_stride=D, o_tok_stride=D, n_q_heads=1, m=1,
                                  dtype=iskv.ISKV_BF16, q_lens=None)
BIG = [2 ** 32 + 64, 2 ** 31, -2 ** 31 - 1, -2 ** 32 + 64]


@pytest.mark.parametrize("x", BIG)
def test_numbers_past_32_bits(x):
    calls = [
        lambda: iskv.iskv_window_attn_workspace(ROWS, QUERIES, x, 0),
        lambda: iskv.iskv_window_attn_workspace(ROWS, QUERIES, 64, x),
        lambda: iskv.iskv_window_attn(ROWS, QUERIES, x, 0, 256, 0, stream=0),
        lambda: iskv.iskv_window_attn(ROWS, QUERIES, 64, x, 256, 0, stream=0),
        lambda: iskv.iskv_evict_workspace(ROWS, x),
        lambda: iskv.iskv_evict(ROWS, 256, 256, 256, 256, 256, x, 1, 0, 256, 0, stream=0),
        lambda: iskv.iskv_evict(ROWS, 256, 256, 256, 256, 256, 64, x, 0, 256, 0, stream=0),
        lambda: iskv.iskv_evict(ROWS, 256, 256, 256, 256, 256, 64, 1, x, 256, 0, stream=0),
        lambda: iskv.iskv_exact_wait_limit(x),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_the_largest_numbers_pass():
    assert iskv.iskv_evict_workspace(ROWS, 2 ** 31 - 1)[0] == 0
    assert iskv.iskv_window_attn_workspace(ROWS, QUERIES, 2 ** 31 - 1, 2 ** 31 - 1)[0] in (0, iskv.ISKV_ERR_CUDA)
