"""Outputs that overlap what a call reads are refused; outputs that lie between queries are not."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

D = 128


def _cache(B=2, H=2, n=200):
    from rank_kv_cache_isvd_b200 import ExactKVCache
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((B, H, n, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    return ExactKVCache(k, v, lens=torch.full((B,), n, dtype=torch.int32, device="cuda")), g


@pytest.mark.parametrize("m", [1, 20])
def test_outputs_over_queries_are_refused(m):
    cache, g = _cache()
    big = torch.randn((2, m + 3, 9, D), generator=g, device="cuda").bfloat16().transpose(1, 2)
    q = big[:, :4, :m]
    for out in (q, big[:, 1:5, :m], big[:, :4, 1:m + 1] if m > 1 else big[:, 3:7, :m]):
        before = big.clone()
        with pytest.raises(ValueError):
            cache.window_attn(q, window=50, out=out)
        assert torch.equal(big, before)
    want = cache.window_attn(q, window=50)
    got = cache.window_attn(q, window=50, out=big[:, 4:8, :m])           # the heads behind the queries'
    assert torch.equal(got, want) and torch.equal(big[:, 4:8, :m], want)


def test_decode_outputs_over_queries_are_refused():
    cache, g = _cache()
    big = torch.randn((2, 6, D), generator=g, device="cuda")
    mass = torch.zeros((2, 2, 200), device="cuda")
    pk, pv = cache.k[0].clone(), cache.v[0].clone()
    with pytest.raises(ValueError):
        cache.mass_decode(big[:, :4], mass, out=big[:, 1:5])
    with pytest.raises(ValueError):
        cache.prefix_decode(big[:, :4], pk, pv, out=big[:, 2:])
    assert not mass.any()


def test_arrays_that_overlap_in_part_are_refused():
    cache, g = _cache()
    q = torch.randn((2, 4, D), generator=g, device="cuda")
    n = 2 * 2 * 200
    mass = torch.rand((n + 8,), generator=g, device="cuda")
    pos = torch.arange(n + 8, dtype=torch.int32, device="cuda")
    lens = torch.zeros((3,), dtype=torch.int32, device="cuda")
    m0, m1, p0, p1 = (x.view(2, 2, 200) for x in (mass[:n], mass[8:], pos[:n], pos[8:]))
    from rank_kv_cache_isvd_b200 import ExactKVCache
    with pytest.raises(ValueError):
        cache.mass_decode(q, m0, mass_out=m1)
    with pytest.raises(ValueError):
        cache.evict(m0, p0, budget=100, recent=10, mass_out=m1)
    with pytest.raises(ValueError):
        cache.evict(m0, p0, budget=100, recent=10, pos_out=p1)
    other = ExactKVCache(cache.k, cache.v, lens=lens[:2])
    with pytest.raises(ValueError):
        other.evict(m0, p0, budget=100, recent=10, lens_out=lens[1:])


def test_tensors_of_an_object_cannot_be_replaced():
    """The C structs hold their addresses, so ``cache.lens = cache.lens + 1`` would go on reading what the old
    tensor held, or what is there when it is gone."""
    cache, _ = _cache()
    for name in ("k", "v", "lens"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name).clone())
    cache.lens.sub_(1)                                       # in place: the object sees it
    assert cache.lens.tolist() == [199, 199]
