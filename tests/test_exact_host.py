"""Host-side checks of the exact-cache entry points (no GPU): what they refuse, before any CUDA
call, and the 64-bit reference that the GPU tests compare with."""
import math

import numpy as np
import pytest
import torch

import rank_kv_cache_isvd_b200 as iskv
from exact_reference import Attended, evicted, visible

INVALID, UNSUPPORTED = iskv.ISKV_ERR_INVALID_ARG, iskv.ISKV_ERR_UNSUPPORTED


def _rows(**kw):
    base = dict(k=256, v=256, seq_stride=8 * 512 * 128, head_stride=512 * 128, row_stride=128,
                batch=2, n_kv_heads=8, rows=512, dtype=iskv.ISKV_BF16, lens=None)
    base.update(kw)
    return iskv.iskv_exact_rows(**base)


def _queries(**kw):
    base = dict(q=256, out=256, q_seq_stride=32 * 128, q_head_stride=128, q_tok_stride=128,
                o_seq_stride=32 * 128, o_head_stride=128, o_tok_stride=128, n_q_heads=32, m=1,
                dtype=iskv.ISKV_BF16, q_lens=None)
    base.update(kw)
    return iskv.iskv_exact_queries(**base)


def _prefix(**kw):
    base = dict(k=256, v=256, head_stride=512 * 128, row_stride=128, rows=512)
    base.update(kw)
    return iskv.iskv_exact_prefix(**base)


WS = (256, 1 << 40)      # a workspace that is never touched: every call here is refused before

BAD_ROWS = [
    (dict(k=0), INVALID), (dict(v=264), INVALID), (dict(rows=-1), INVALID),
    (dict(rows=(1 << 24) + 1), INVALID), (dict(batch=0), INVALID), (dict(n_kv_heads=0), INVALID),
    (dict(dtype=3), INVALID), (dict(row_stride=132), INVALID), (dict(head_stride=-128), INVALID),
    (dict(batch=10000), UNSUPPORTED),
]
BAD_QUERIES = [
    (dict(q=0), INVALID), (dict(out=0), INVALID), (dict(q=264), INVALID), (dict(m=0), INVALID),
    (dict(n_q_heads=12), INVALID), (dict(n_q_heads=72), INVALID), (dict(dtype=5), INVALID),
    (dict(q_head_stride=130), INVALID), (dict(o_head_stride=0), INVALID),
    (dict(o_seq_stride=64), INVALID),
]


@pytest.mark.parametrize("bad,code", BAD_ROWS)
def test_bad_rows_are_refused_by_every_call(bad, code):
    r, q = _rows(**bad), _queries()
    assert iskv.iskv_window_attn(r, q, 64, 4, *WS, stream=0) == code
    assert iskv.iskv_mass_decode(r, q, 256, 256, *WS, stream=0) == code
    assert iskv.iskv_prefix_decode(r, q, _prefix(), *WS, stream=0) == code
    assert iskv.iskv_evict(r, 256, 256, 256, 256, 256, 64, 1, 0, *WS, stream=0) == code


@pytest.mark.parametrize("bad,code", BAD_QUERIES)
def test_bad_queries_are_refused_by_every_attention(bad, code):
    r, q = _rows(), _queries(**bad)
    assert iskv.iskv_window_attn(r, q, 64, 4, *WS, stream=0) == code
    assert iskv.iskv_mass_decode(r, q, 256, 256, *WS, stream=0) == code
    assert iskv.iskv_prefix_decode(r, q, _prefix(), *WS, stream=0) == code


def test_float32_rows_need_float32_queries():
    r, q = _rows(dtype=iskv.ISKV_F32), _queries()
    assert iskv.iskv_window_attn(r, q, 64, 4, *WS, stream=0) == UNSUPPORTED
    assert iskv.iskv_mass_decode(r, q, 256, 256, *WS, stream=0) == UNSUPPORTED
    assert iskv.iskv_prefix_decode(r, q, _prefix(), *WS, stream=0) == UNSUPPORTED


def test_window_and_workspace_are_checked():
    r, q = _rows(), _queries()
    assert iskv.iskv_window_attn(r, q, 0, 4, *WS, stream=0) == INVALID
    assert iskv.iskv_window_attn(r, q, 64, -1, *WS, stream=0) == INVALID
    assert iskv.iskv_window_attn(r, q, 64, 4, None, 1 << 40, stream=0) == INVALID
    assert iskv.iskv_window_attn(r, q, 64, 4, 260, 1 << 40, stream=0) == INVALID
    assert iskv.iskv_window_attn(None, q, 64, 4, *WS, stream=0) == INVALID
    assert iskv.iskv_window_attn(r, None, 64, 4, *WS, stream=0) == INVALID
    assert iskv.lib.iskv_window_attn_workspace(None, None, 64, 4, None) == INVALID


def test_decode_takes_one_token_per_sequence():
    r = _rows()
    for bad in (dict(m=2), dict(q_lens=256)):
        q = _queries(**bad)
        assert iskv.iskv_mass_decode(r, q, 256, 256, *WS, stream=0) == INVALID
        assert iskv.iskv_prefix_decode(r, q, _prefix(), *WS, stream=0) == INVALID


@pytest.mark.parametrize("bad", [dict(k=0), dict(v=8), dict(rows=-1), dict(row_stride=4),
                                 dict(head_stride=-8)])
def test_bad_prefixes_are_refused(bad):
    assert iskv.iskv_prefix_decode(_rows(), _queries(), _prefix(**bad), *WS, stream=0) == INVALID
    assert iskv.iskv_prefix_decode(_rows(), _queries(), None, *WS, stream=0) == INVALID


def test_prefixes_of_more_steps_than_32_bits_are_refused():
    """A prefix that the split kernel takes by itself, one tile of query rows for each of many
    kv-heads that share it."""
    r = _rows(batch=1, n_kv_heads=4096, rows=1)
    q = _queries(n_q_heads=4096)
    p = _prefix(head_stride=0, rows=1 << 24)
    assert iskv.iskv_prefix_decode_workspace(r, q, p)[0] == UNSUPPORTED
    assert iskv.iskv_prefix_decode(r, q, p, *WS, stream=0) == UNSUPPORTED


def test_eviction_refuses_what_it_cannot_keep_or_move():
    ok = (256, 256, 256, 256, 256)
    r = _rows()
    assert iskv.iskv_evict(r, *ok, 0, 0, 0, *WS, stream=0) == INVALID
    assert iskv.iskv_evict(r, *ok, 64, 60, 5, *WS, stream=0) == INVALID       # more fixed than kept
    assert iskv.iskv_evict(r, *ok, 64, -1, 0, *WS, stream=0) == INVALID
    assert iskv.iskv_evict(r, 256, 256, 256, 256, None, 64, 1, 0, *WS, stream=0) == INVALID
    assert iskv.iskv_evict(r, None, 256, 256, 256, 256, 64, 1, 0, *WS, stream=0) == INVALID
    for shared in (dict(seq_stride=0), dict(head_stride=0), dict(row_stride=0)):
        assert iskv.iskv_evict(_rows(**shared), *ok, 64, 1, 0, *WS, stream=0) == INVALID
    code, need = iskv.iskv_evict_workspace(r, 64)
    assert code == 0 and need > 0
    assert iskv.iskv_evict(r, *ok, 64, 1, 0, 256, need - 1, stream=0) == iskv.ISKV_ERR_CAPACITY


def test_the_wrapper_wants_cuda_tensors():
    x = torch.zeros((1, 1, 4, 128))
    with pytest.raises(ValueError):
        iskv.ExactKVCache(x, x)
    with pytest.raises(ValueError):
        iskv.ExactKVCache(x[..., :64], x[..., :64])


# -- the reference itself ---------------------------------------------------------------------
def test_reference_visibility_by_hand():
    see = visible(6, 3, 4, window=2, sinks=1)          # tokens at positions 3, 4, 5, and a padded one
    want = [[1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1], [0] * 6]
    assert np.array_equal(see, np.array(want, bool))
    assert not visible(1, 3, 3, window=4, sinks=0)[:2].any()      # positions -2 and -1


def test_reference_attention_closed_forms():
    v = torch.arange(3 * 128, dtype=torch.float64).view(3, 128)
    k = torch.ones((3, 128))
    q = torch.randn((2, 128), generator=torch.Generator().manual_seed(1))
    a = Attended(q, k, v, np.array([[1, 1, 0], [0, 0, 0]], bool))
    assert torch.allclose(a.o[0], v[:2].mean(0)) and not a.o[1].any()
    # two keys: the weight is a logistic function of the score difference
    k = torch.stack([q[0], torch.zeros(128)])
    d = float(q[0].double() @ q[0].double()) / math.sqrt(128)
    a = Attended(q[:1], k, v[:2], np.ones((1, 2), bool))
    assert abs(float(a.w[0, 0]) - 1 / (1 + math.exp(-d))) < 1e-12


def test_reference_eviction_by_hand():
    mass, pos = [5, 1, 9, 9, 0, 2], [0, 1, 2, 3, 4, 5]
    slots, keep = evicted(mass, pos, 6, 4, recent=1, sinks=1)
    assert keep == 4 and slots.tolist() == [0, 5, 2, 3]          # slot 1 freed, row 5 moved there
    slots, keep = evicted([1, 1, 1, 1], [3, 2, 1, 0], 4, 2, recent=0, sinks=0)
    assert slots.tolist() == [0, 1]                              # ties: the lowest slots
    slots, keep = evicted(mass, pos, 3, 4, recent=1, sinks=1)
    assert keep == 3 and slots.tolist() == [0, 1, 2]
