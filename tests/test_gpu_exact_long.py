"""Prompts whose tokens times rows pass what 32 bits count."""
import pytest

torch = pytest.importorskip("torch")

from exact_reference import Attended, out_bound  # noqa: E402

pytestmark = pytest.mark.gpu

D = 128


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_of_65537_tokens(dtype):
    """8 kv-heads of 8 q-heads: 2^31 pairs of a token's tile and 16 rows. On a sample of its tokens."""
    from rank_kv_cache_isvd_b200 import ExactKVCache
    g = torch.Generator(device="cuda").manual_seed(1)
    H, G, n, window, sinks = 8, 8, 65537, 100, 4
    k, v = (torch.randn((1, H, n, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((1, n, H * G, D), generator=g, device="cuda", dtype=dtype).transpose(1, 2)
    out = ExactKVCache(k, v).window_attn(q, window=window, sinks=sinks)
    assert torch.isfinite(out).all()
    for h in (0, 3, 7):
        for a in (0, 7):
            for t0 in (0, 90, 32760, 65440, n - 20):
                some = torch.arange(t0, min(n, t0 + 20))
                lo = max(sinks, t0 - window)
                cols = torch.cat([torch.arange(min(sinks, n)), torch.arange(lo, int(some[-1]) + 1)])
                p, j = some[:, None], cols[None]
                see = (j <= p) & ((j < sinks) | (j > p - window))
                ref = Attended(q[0, h * G + a, some.cuda()], k[0, h, cols.cuda()], v[0, h, cols.cuda()], see)
                err = (out[0, h * G + a, some.cuda()].double().cpu() - ref.o).abs()
                assert (err <= out_bound(ref, dtype, dtype)).all()
