"""Which sizes the calls on exact caches refuse (no GPU): what one of their kernels cannot count is refused
for the calls that take that kernel alone."""
import pytest

import rank_kv_cache_isvd_b200 as iskv

UNSUPPORTED = iskv.ISKV_ERR_UNSUPPORTED
D = 128


def _rows(batch, n_kv, rows, dtype):
    return iskv.iskv_exact_rows(k=256, v=256, seq_stride=n_kv * rows * D, head_stride=rows * D, row_stride=D,
                                batch=batch, n_kv_heads=n_kv, rows=rows, dtype=dtype, lens=None)


def _queries(n_q, m, dtype):
    return iskv.iskv_exact_queries(q=256, out=256, q_seq_stride=n_q * m * D, q_head_stride=m * D,
                                   q_tok_stride=D, o_seq_stride=n_q * m * D, o_head_stride=m * D,
                                   o_tok_stride=D, n_q_heads=n_q, m=m, dtype=dtype, q_lens=None)


@pytest.mark.parametrize("dtype", [iskv.ISKV_BF16, iskv.ISKV_F32])
@pytest.mark.parametrize("batch,n_kv,n_q,tokens", [(1, 8, 32, 131072), (4, 8, 64, 32768), (1, 8, 8, 1 << 20)])
def test_long_prompts_are_not_refused(batch, n_kv, n_q, tokens, dtype):
    """Their tokens times their rows pass 2^31 tiles of 8 query rows times steps, which only the split kernel
    counts; prompts never take it."""
    r, q = _rows(batch, n_kv, tokens, dtype), _queries(n_q, tokens, dtype)
    code, need = iskv.iskv_window_attn_workspace(r, q, tokens, 0)
    assert code in (iskv.ISKV_OK, iskv.ISKV_ERR_CUDA)          # (without a GPU there is no workspace size)
    assert code == iskv.ISKV_ERR_CUDA or need > 0


def test_what_the_split_kernel_cannot_count_is_refused():
    r, q = _rows(512, 64, 1 << 24, iskv.ISKV_BF16), _queries(64, 1, iskv.ISKV_BF16)
    assert iskv.iskv_window_attn_workspace(r, q, 1 << 24, 0)[0] == UNSUPPORTED
    assert iskv.iskv_mass_decode_workspace(r, q)[0] == UNSUPPORTED
    p = iskv.iskv_exact_prefix(k=256, v=256, head_stride=D, row_stride=D, rows=1)
    assert iskv.iskv_prefix_decode_workspace(r, q, p)[0] == UNSUPPORTED


def test_more_blocks_than_a_grid_has_are_refused():
    """Queries that many sequences and kv-heads share by zero strides."""
    r = _rows(1024, 63, 16, iskv.ISKV_F32)
    q = _queries(63 * 8, 1 << 24, iskv.ISKV_F32)
    assert iskv.iskv_window_attn_workspace(r, q, 16, 0)[0] == UNSUPPORTED
