"""Whether queries and outputs share memory (no GPU): against sets of bytes."""
import random

import pytest
import torch

from rank_kv_cache_isvd_b200.exact import _overlap, _rows_of, _span


def _bytes(x, base):
    at = (x.data_ptr() - base) // x.element_size()
    starts = [at]
    for s, e in zip(x.stride()[:-1], x.shape[:-1]):
        starts = [a + i * s for a in starts for i in range(e)]
    return {a + c for a in starts for c in range(x.shape[-1])}


def _shares(q, out):
    return _overlap(out.data_ptr() - q.data_ptr(), _rows_of(q), _rows_of(out), q.shape[-1] * q.element_size())


def test_interleaved_views_are_apart_and_shifted_ones_are_not():
    x = torch.zeros((2, 10, 3, 4, 16))                       # batch, tokens, (q, out, other), heads, channels
    q, out = x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2)
    assert not _shares(q, out) and not _shares(out, q)
    assert _shares(q, q)
    y = torch.zeros((2, 6, 12, 16))
    assert _shares(y[:, :4], y[:, 1:5])                      # one head further
    assert not _shares(y[:, :3], y[:, 3:])
    assert _shares(y[:, :, :8], y[:, :, 3:11])               # three tokens further
    assert not _shares(y[:, :, :6], y[:, :, 6:])
    z = torch.zeros(2 * 3 * 16 + 8)
    assert _shares(z[:96].view(2, 3, 16), z[8:].view(2, 3, 16))      # half a row further
    e = torch.zeros((1, 3, 4, 16))
    assert _shares(e.expand(5, 3, 4, 16), e.expand(5, 3, 4, 16)[:, :1])
    assert _span(y[:, :4]) == 4 * (y.numel() - 2 * 12 * 16)


@pytest.mark.parametrize("seed", range(4))
def test_random_views(seed):
    """Slices and permutations of one buffer, and buffers cut in two, as random programs make them."""
    rng = random.Random(seed)
    seen = {True: 0, False: 0}
    for _ in range(400):
        dims = [rng.randint(1, 5) for _ in range(3)]
        big = torch.zeros([d + rng.randint(0, 4) for d in dims] + [8])

        def view():
            x = big
            for i, d in enumerate(dims):
                step = 2 if big.shape[i] >= 2 * d and rng.random() < 0.4 else 1
                lo = rng.randint(0, big.shape[i] - (d - 1) * step - 1)
                x = x.narrow(i, lo, (d - 1) * step + 1)[tuple([slice(None)] * i + [slice(None, None, step)])]
            return x

        q, out = view(), view()
        if rng.random() < 0.5:                               # dimensions of one extent in another order
            order = [0, 1, 2]
            rng.shuffle(order)
            out = out.permute(*order, 3)
        base = big.data_ptr()
        want = bool(_bytes(q, base) & _bytes(out, base))
        seen[want] += 1
        assert _shares(q, out) == want, (q.stride(), q.shape, out.stride(), out.shape)
    assert min(seen.values()) > 40


def test_tensors_are_read_only():
    from rank_kv_cache_isvd_b200 import ExactKVCache
    for name in ("k", "v", "lens"):
        assert getattr(ExactKVCache, name).fset is None
