"""Numbers of a call that do not fit in 32 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

D = 128


def test_numbers_past_32_bits_are_refused():
    from rank_kv_cache_isvd_b200 import ExactKVCache
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((1, 2, 300, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((1, 4, 1, D), generator=g, device="cuda")
    lens = torch.full((1,), 300, dtype=torch.int32, device="cuda")
    mass = torch.rand((1, 2, 300), generator=g, device="cuda")
    pos = torch.arange(300, dtype=torch.int32, device="cuda").expand(1, 2, 300).contiguous()
    cache = ExactKVCache(k, v, lens=lens)
    for bad in (dict(window=2 ** 32 + 64), dict(window=64, sinks=2 ** 32)):
        with pytest.raises(ValueError):
            cache.window_attn(q, **bad)
    for bad in (dict(budget=2 ** 32 + 50, recent=1), dict(budget=50, recent=2 ** 32),
                dict(budget=50, recent=1, sinks=2 ** 32)):
        for _ in range(2):
            with pytest.raises(ValueError):
                cache.evict(mass, pos, **bad)
    assert lens.item() == 300
    whole = cache.window_attn(q, window=300)
    assert torch.equal(cache.window_attn(q, window=2 ** 31 - 1, sinks=2 ** 31 - 1), whole)
