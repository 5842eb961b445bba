"""Window attention with sinks over float32 rows, whose steps are half as long as those of bf16 rows: few and
many (sequence, kv-head) items, so that teams of every size work by items and by steps."""
import pytest

torch = pytest.importorskip("torch")

from exact_reference import Attended, out_bound  # noqa: E402

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    from rank_kv_cache_isvd_b200 import iskv_exact_status
    assert iskv_exact_status() == 0


def _attended(q, k, v, see):
    """64-bit attention of q [b][h][r][128] over k, v [b][h][n][128] under see [b][1][r][n], on the device,
    with what ``out_bound`` asks of an ``Attended``. Rows that are not seen are zeros."""
    ref = Attended.__new__(Attended)
    q, k, v = (x.double() for x in (q, k, v))
    s = torch.where(see, q @ k.transpose(-1, -2) * D ** -0.5, -torch.inf)
    ref.w = torch.softmax(s, -1).nan_to_num(0.0)                 # (rows without any: 0)
    ref.o, ref.spread = ref.w @ v, ref.w @ v.abs()
    sizes = torch.where(see, q.abs() @ k.abs().transpose(-1, -2) * D ** -0.5, 0.0)
    ref.terms = sizes.amax(-1, keepdim=True)
    ref.n = int(see.sum(-1).max())
    return ref


def _check(B, H, G, n, m, window, sinks, lens, seed, rt=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn((B, H, n, D), generator=g, device="cuda") for _ in range(2))
    at = torch.arange(n, device="cuda")
    v[:, :, at % 16 >= 12] *= 30                     # a row that gets lost in a step's last rows shows
    k, v = k.to(rt), v.to(rt)
    q = torch.randn((B, H * G, m, D), generator=g, device="cuda")
    nl = torch.tensor(lens, device="cuda")
    p = nl[:, None] - m + torch.arange(m, device="cuda")                       # [B][m]
    j, p = at[None, None], p[:, :, None]
    see = (j <= p) & ((j < sinks) | (j > p - window))                          # [B][m][n]
    unseen = ~see.any(1)[:, None, :, None]
    k.masked_fill_(unseen, float("nan"))
    v.masked_fill_(unseen, float("nan"))
    from rank_kv_cache_isvd_b200 import ExactKVCache
    cache = ExactKVCache(k, v, lens=None if min(lens) == n else nl.int())
    outs = [cache.window_attn(q, window=window, sinks=sinks) for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    for b in range(0, B, 8):
        part = slice(b, b + 8)
        cols = see[part].any(0).any(0)                                         # rows that any of them sees
        kk, vv = k[part][:, :, cols].nan_to_num(0.0), v[part][:, :, cols].nan_to_num(0.0)
        mask = see[part][:, None, :, cols]
        mask = mask[:, :, None].expand(-1, -1, G, -1, -1).reshape(mask.shape[0], 1, G * m, -1)
        qq = q[part].reshape(-1, H, G * m, D)
        ref = _attended(qq, kk, vv, mask)
        err = (outs[0][part].double().reshape(ref.o.shape) - ref.o).abs()
        bound = out_bound(ref, torch.float32)
        assert (err <= bound).all(), (b, float((err / bound).max()))


@pytest.mark.parametrize("sinks", [1, 4, 15, 17, 130])
@pytest.mark.parametrize("B,window", [(1, 40), (1, 300), (1, 1000), (4, 1000), (10, 2000), (16, 1000), (40, 40),
                                      (40, 300), (40, 1000), (80, 40), (80, 1000), (128, 40), (128, 1000)])
def test_single_tokens_over_float32_rows(B, window, sinks):
    n = window + 333
    _check(B, 8, 1, n, 1, window, sinks, [n] * B, seed=B + sinks)


@pytest.mark.parametrize("sinks", [3, 16, 33])
@pytest.mark.parametrize("B,G,m,window", [(3, 2, 3, 200), (60, 1, 5, 90), (100, 4, 2, 300), (100, 8, 1, 700)])
def test_ragged_tokens_over_float32_rows(B, G, m, window, sinks):
    n = window + 200
    lens = [max(0, n - 37 * b % (n + 1)) for b in range(B)]
    _check(B, 4, G, n, m, window, sinks, lens, seed=B + sinks)


@pytest.mark.parametrize("sinks", [4, 17])
@pytest.mark.parametrize("rt", [torch.float32, torch.bfloat16])
def test_chunks_of_float32_queries(rt, sinks):
    """More than 8 query rows: the rows kernel, which fills up its sinks in the same way."""
    _check(2, 3, 4, 900, 70, 150, sinks, [900, 333], seed=sinks, rt=rt)
