"""Attention over exact rows (window with sinks, accumulated weights, shared prefix) and eviction on
the GPU, against 64-bit references. Bounds are derived in ``exact_reference``."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from exact_reference import Attended, evicted, out_bound, visible, weight_bound  # noqa: E402

pytestmark = pytest.mark.gpu

D = 128
T = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    from rank_kv_cache_isvd_b200 import iskv_exact_status
    assert iskv_exact_status() == 0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _kv(g, B, H, n, dtype, tokens_first=False, k_scale=1.0):
    shape = (B, n, H, D) if tokens_first else (B, H, n, D)
    k, v = (torch.randn(shape, generator=g, device="cuda") for _ in range(2))
    k, v = (k * k_scale).to(T[dtype]), v.to(T[dtype])
    return (k.transpose(1, 2), v.transpose(1, 2)) if tokens_first else (k, v)


def _cache(k, v, lens=None):
    from rank_kv_cache_isvd_b200 import ExactKVCache
    return ExactKVCache(k, v, lens=lens)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _check_window(k, v, q, out, lens, q_lens, window, sinks, p_dtype, before):
    B, H, n, _ = k.shape
    G, m = q.shape[1] // H, q.shape[2]
    got = out.double().cpu()
    for b in range(B):
        nb, qb = lens[b], q_lens[b]
        see = visible(nb, qb, m, window, sinks)
        for h in range(H):
            for g in range(G):
                ref = Attended(q[b, h * G + g], k[b, h, :nb], v[b, h, :nb], see)
                err = (got[b, h * G + g] - ref.o).abs()[:qb]
                bound = out_bound(ref, q.dtype, p_dtype)[:qb]
                assert (err <= bound).all(), (b, h, g, float((err / bound).max()))
        assert torch.equal(out[b, :, qb:], before[b, :, qb:])      # padded tokens: not written


WINDOW_CASES = [
    # B, H, G, rows, m, window, sinks, io, rows_type, lens, q_lens, tokens_first
    (1, 2, 4, 300, 1, 64, 4, "f32", "bf16", None, None, False),
    (2, 2, 4, 257, 1, 1000, 0, "bf16", "bf16", [257, 1], None, False),
    (3, 1, 8, 130, 1, 1, 0, "f32", "f32", [130, 0, 7], None, False),
    (2, 3, 1, 97, 3, 5, 2, "f32", "f32", [97, 2], [3, 3], True),
    (2, 2, 5, 200, 2, 64, 9, "f32", "bf16", [200, 65], [2, 0], True),
    (2, 1, 3, 70, 70, 16, 1, "f32", "bf16", [70, 33], [70, 33], False),
    (1, 2, 4, 256, 256, 1 << 30, 0, "bf16", "bf16", None, None, True),
    (1, 1, 4, 1, 1, 1, 0, "bf16", "bf16", None, None, False),
    (2, 2, 2, 515, 129, 200, 130, "bf16", "bf16", [515, 400], [129, 77], True),
    (1, 2, 4, 1000, 1000, 100, 4, "bf16", "bf16", None, None, True),
    (3, 1, 5, 333, 111, 77, 3, "bf16", "bf16", [333, 100, 0], [111, 111, 50], False),
    (1, 1, 8, 700, 700, 700, 0, "bf16", "bf16", None, None, False),
    (2, 1, 7, 260, 130, 64, 0, "bf16", "bf16", [260, 131], [130, 1], True),
    (1, 1, 1, 900, 300, 128, 128, "bf16", "bf16", None, None, False),
    (1, 3, 6, 150, 40, 150, 200, "bf16", "bf16", None, None, True),
    (1, 2, 4, 600, 600, 90, 5, "f32", "bf16", None, None, True),
    (2, 1, 8, 333, 200, 77, 40, "f32", "f32", [333, 150], [200, 150], False),
    (1, 1, 5, 3000, 30, 1 << 24, 0, "f32", "bf16", None, None, False),
    (1, 1, 4, 5000, 9, 4000, 100, "bf16", "bf16", None, None, False),
    (70, 8, 2, 700, 1, 300, 40, "bf16", "bf16", list(range(1, 701, 10)), None, False),
    (160, 2, 4, 90, 2, 1000, 0, "f32", "bf16", [90] * 160, [2, 0] * 80, True),
    # more pairs of tiles than SMs, the last round nearly empty; odd and missing tokens
    (3, 8, 4, 420, 420, 100, 3, "bf16", "bf16", None, None, True),
    (4, 13, 8, 96, 90, 1000, 0, "bf16", "bf16", [96, 80, 5, 0], [90, 31, 9, 0], False),
    (13, 12, 1, 200, 130, 70, 5, "bf16", "bf16", list(range(188, 201)), list(range(0, 130, 10)), True),
]


@pytest.mark.parametrize("B,H,G,n,m,window,sinks,io,rt,lens,q_lens,tf", WINDOW_CASES)
def test_window_attention(B, H, G, n, m, window, sinks, io, rt, lens, q_lens, tf):
    g = _gen(1)
    k, v = _kv(g, B, H, n, rt, tf, k_scale=2.0)
    shape = (B, m, H * G, D) if tf else (B, H * G, m, D)
    q = torch.randn(shape, generator=g, device="cuda").to(T[io])
    before = torch.full(shape, 7.0, device="cuda").to(T[io])
    if tf:
        q, before = q.transpose(1, 2), before.transpose(1, 2)
    nl, ml = lens or [n] * B, q_lens or [m] * B
    for b in range(B):               # rows behind the last: never used, so they may be anything
        k[b, :, nl[b]:] = float("nan")
        v[b, :, nl[b]:] = float("inf")
    out = before.clone()
    cache = _cache(k, v, None if lens is None else _i32(lens))
    res = cache.window_attn(q, window=window, sinks=sinks, out=out,
                            q_lens=None if q_lens is None else _i32(q_lens))
    assert res is out
    _check_window(k, v, q, out, nl, ml, window, sinks, torch.bfloat16 if io == "bf16" else
                  torch.float32, before)


@pytest.mark.parametrize("io,rt", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
def test_window_never_reads_what_no_token_sees(io, rt):
    """Single tokens of a long cache: rows between the sinks and the window hold NaN."""
    g = _gen(2)
    B, H, G, n, window, sinks = 2, 2, 4, 1500, 200, 3
    lens = [1500, 900]
    k, v = _kv(g, B, H, n, rt)
    for b in range(B):
        k[b, :, sinks:lens[b] - window] = float("nan")
        v[b, :, sinks:lens[b] - window] = float("nan")
    q = torch.randn((B, H * G, 1, D), generator=g, device="cuda").to(T[io])
    out = _cache(k, v, _i32(lens)).window_attn(q, window=window, sinks=sinks)
    _check_window(k, v, q, out, lens, [1, 1], window, sinks, T[io], out.clone())


@pytest.mark.parametrize("G,io", [(4, "bf16"), (1, "bf16"), (4, "f32")])
def test_values_that_are_not_finite_stay_near_their_window(G, io):
    """One NaN among the values of a prompt: tokens more than 256 positions away from all that see it
    come out as if it were not there."""
    g = _gen(12)
    n, window, at = 1400, 100, 600
    k, v = _kv(g, 1, 1, n, "bf16")
    q = torch.randn((1, G, n, D), generator=g, device="cuda").to(T[io])
    v[0, 0, at] = float("nan")
    out = _cache(k, v).window_attn(q, window=window)[0].double().cpu()
    far = [i for i in range(n) if i < at - 256 or i >= at + window + 256]
    see = visible(n, n, n, window, 0)[far]
    for a in range(G):
        ref = Attended(q[0, a, far], k[0, 0], v[0, 0], see)
        assert ((out[a, far] - ref.o).abs() <= out_bound(ref, T[io], T[io])).all()
    assert torch.isnan(out[:, at:at + window]).all()


@pytest.mark.parametrize("sharp", [1.0, 12.0])
def test_window_prompt_of_many_blocks(sharp):
    """A prompt of several thousand tokens, on a sample of its tokens; sharp: logits of about 50."""
    g = _gen(3)
    H, G, n, window, sinks = 2, 4, 2500, 900, 5
    k, v = _kv(g, 1, H, n, "bf16", True, k_scale=sharp)
    q = torch.randn((1, n, H * G, D), generator=g, device="cuda").bfloat16().transpose(1, 2)
    out = _cache(k, v).window_attn(q, window=window, sinks=sinks).double().cpu()
    see = visible(n, n, n, window, sinks)
    some = [0, 1, 4, 5, 6, 127, 128, 899, 900, 901, 1023, 1024, 2047, 2498, 2499] + \
        list(range(3, n, 97))
    for h in range(H):
        for a in range(G):
            ref = Attended(q[0, h * G + a, some], k[0, h], v[0, h], see[some])
            err = (out[0, h * G + a, some] - ref.o).abs()
            assert (err <= out_bound(ref, torch.bfloat16, torch.bfloat16)).all()


MASS_CASES = [
    (1, 1, 1, 1, "f32", "bf16", None), (2, 2, 4, 300, "f32", "bf16", [300, 17]),
    (2, 2, 2, 515, "bf16", "bf16", [515, 0]), (3, 2, 5, 129, "f32", "f32", [1, 129, 64]),
    (1, 3, 8, 2100, "f32", "bf16", None), (1, 1, 3, 4097, "bf16", "bf16", None),
    (40, 1, 7, 70, "f32", "bf16", list(range(31, 71))),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,H,G,n,io,rt,lens", MASS_CASES)
def test_mass_decode(B, H, G, n, io, rt, lens, in_place):
    g = _gen(4)
    k, v = _kv(g, B, H, n, rt, k_scale=2.0)
    q = torch.randn((B, H * G, D), generator=g, device="cuda").to(T[io])
    mass = torch.rand((B, H, n), generator=g, device="cuda")
    old = mass.clone()
    nl = lens or [n] * B
    for b in range(B):
        k[b, :, nl[b]:] = float("nan")
        v[b, :, nl[b]:] = float("nan")
    cache = _cache(k, v, None if lens is None else _i32(lens))
    given = mass if in_place else torch.full_like(mass, -3.0)
    out, new = cache.mass_decode(q, mass, mass_out=None if in_place else given)
    assert new is given
    for b in range(B):
        for h in range(H):
            ref = Attended(q[b, h * G:(h + 1) * G], k[b, h, :nl[b]], v[b, h, :nl[b]],
                           np.ones((G, nl[b]), bool))
            err = (out[b, h * G:(h + 1) * G].double().cpu() - ref.o).abs()
            assert (err <= out_bound(ref, q.dtype)).all()
            if nl[b]:
                w = ref.w.sum(0)
                want = old[b, h, :nl[b]].double().cpu() + w
                bound = (ref.w * weight_bound(ref)).sum(0) + G * 2.0 ** -24 * w + \
                    2.0 ** -23 * want
                assert ((new[b, h, :nl[b]].double().cpu() - want).abs() <= bound).all()
        rest = old if in_place else torch.full_like(old, -3.0)
        assert torch.equal(new[b, :, nl[b]:], rest[b, :, nl[b]:])


PREFIX_CASES = [
    # B, H, G, P, rows, io, rows_type, lens
    (1, 1, 1, 1, 1, "f32", "bf16", None), (2, 2, 4, 300, 0, "f32", "bf16", None),
    (3, 2, 4, 0, 40, "bf16", "bf16", [40, 0, 1]), (9, 1, 8, 257, 130, "f32", "f32", None),
    (33, 2, 4, 500, 77, "bf16", "bf16", list(range(33))),
    (17, 2, 5, 129, 64, "f32", "bf16", [0] * 17), (130, 1, 4, 1000, 20, "bf16", "bf16", None),
    (70, 2, 1, 333, 9, "bf16", "bf16", None), (65, 1, 7, 640, 3, "bf16", "bf16", None),
    (16, 1, 8, 2100, 5, "bf16", "bf16", None), (300, 1, 2, 128, 1, "bf16", "bf16", None),
    (5, 2, 3, 4000, 33, "bf16", "bf16", [33, 0, 2, 3, 4]),
    (9, 1, 8, 500, 1500, "bf16", "bf16", None), (40, 1, 4, 1100, 600, "f32", "bf16", None),
    (150, 1, 2, 257, 40, "f32", "f32", None), (40, 1, 4, 300, 60000, "bf16", "bf16",
                                               [60000] + [0] * 38 + [7]), (20, 2, 4, 900, 300, "f32", "f32", [300, 1] * 10),
]


@pytest.mark.parametrize("B,H,G,P,n,io,rt,lens", PREFIX_CASES)
def test_prefix_decode(B, H, G, P, n, io, rt, lens):
    g = _gen(5)
    k, v = _kv(g, B, H, n, rt, k_scale=2.0)
    pk, pv = _kv(g, 1, H, P, rt, tokens_first=True, k_scale=2.0)
    pk, pv = pk[0], pv[0]
    q = torch.randn((B, H * G, D), generator=g, device="cuda").to(T[io])
    nl = lens or [n] * B
    for b in range(B):
        k[b, :, nl[b]:] = float("nan")
        v[b, :, nl[b]:] = float("nan")
    out = _cache(k, v, None if lens is None else _i32(lens)).prefix_decode(q, pk, pv)
    p_dtype = T[io]
    for b in range(B):
        for h in range(H):
            kk, vv = torch.cat([pk[h], k[b, h, :nl[b]]]), torch.cat([pv[h], v[b, h, :nl[b]]])
            ref = Attended(q[b, h * G:(h + 1) * G], kk, vv, np.ones((G, P + nl[b]), bool))
            err = (out[b, h * G:(h + 1) * G].double().cpu() - ref.o).abs()
            bound = out_bound(ref, q.dtype, p_dtype)
            assert (err <= bound).all(), (b, h, float((err / bound).max()))


EVICT_CASES = [
    # B, H, rows, budget, recent, sinks, rows_type, lens
    (1, 1, 2, 1, 0, 0, "bf16", None), (2, 3, 300, 200, 32, 4, "bf16", None),
    (3, 2, 1000, 500, 1, 0, "f32", [1000, 500, 501]), (2, 1, 257, 256, 256, 0, "bf16", None),
    (2, 2, 64, 64, 8, 8, "bf16", [64, 0]), (1, 2, 5000, 100, 64, 36, "bf16", None),
    (2, 2, 4099, 4000, 100, 4, "f32", [4099, 4050]), (1, 1, 60000, 59000, 64, 4, "bf16", None),
    (2, 2, 33000, 16001, 64, 4, "bf16", [33000, 20000]), (40, 2, 17000, 16500, 1, 0, "bf16", None),
    (1, 2, 140000, 70000, 64, 4, "bf16", None),
]


def _evict_inputs(g, B, H, n, rt, ties):
    k, v = _kv(g, B, H, n, rt)
    mass = torch.rand((B, H, n), generator=g, device="cuda")
    if ties:
        mass = (mass * 4).floor()                    # many equal weights, zeros among them
        mass[mass == 1] = -0.0
    pos = torch.argsort(torch.rand((B, H, n), generator=g, device="cuda"), dim=-1).int() * 2
    return k, v, mass, pos


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,H,n,budget,recent,sinks,rt,lens", EVICT_CASES)
def test_evict(B, H, n, budget, recent, sinks, rt, lens, in_place, ties):
    k, v, mass, pos = _evict_inputs(_gen(6), B, H, n, rt, ties)
    k0, v0, m0, p0 = (x.cpu().clone() for x in (k, v, mass, pos))
    nl = lens or [n] * B
    ls = _i32(nl)
    cache = _cache(k, v, ls)
    if in_place:
        cache.evict(mass, pos, budget=budget, recent=recent, sinks=sinks)
        mo, po, lo = mass, pos, ls
    else:
        mo, po, lo = torch.full_like(mass, 9.0), torch.full_like(pos, -9), _i32([-9] * B)
        cache.evict(mass, pos, budget=budget, recent=recent, sinks=sinks, mass_out=mo, pos_out=po,
                    lens_out=lo)
        assert torch.equal(mass.cpu(), m0) and torch.equal(pos.cpu(), p0)
    assert lo.tolist() == [min(x, budget) for x in nl]
    for b in range(B):
        for h in range(H):
            slots, keep = evicted(m0[b, h].numpy(), p0[b, h].numpy(), nl[b], budget, recent, sinks)
            want_k, want_v = k0[b, h].clone(), v0[b, h].clone()
            want_k[:keep], want_v[:keep] = k0[b, h][slots], v0[b, h][slots]
            assert torch.equal(k[b, h].cpu(), want_k) and torch.equal(v[b, h].cpu(), want_v)
            rest_m = m0[b, h] if in_place else torch.full((n,), 9.0)
            rest_p = p0[b, h] if in_place else torch.full((n,), -9, dtype=torch.int32)
            assert torch.equal(mo[b, h].cpu()[:keep], m0[b, h][slots])
            assert torch.equal(po[b, h].cpu()[:keep], p0[b, h][slots])
            assert torch.equal(mo[b, h].cpu()[keep:], rest_m[keep:])
            assert torch.equal(po[b, h].cpu()[keep:], rest_p[keep:])


def test_evict_of_single_heads_replaces_lengths_in_place():
    """One launch, one block per sequence: no warp may read a length that another has replaced."""
    B, n, budget = 200, 900, 600
    k, v, mass, pos = _evict_inputs(_gen(16), B, 1, n, "bf16", False)
    m0, p0 = mass.cpu().numpy().copy(), pos.cpu().numpy().copy()
    nl = [n - 2 * b for b in range(B)]
    want = [evicted(m0[b, 0], p0[b, 0], nl[b], budget, 32, 4) for b in range(B)]
    for _ in range(20):
        m, p, ls = torch.from_numpy(m0).cuda(), torch.from_numpy(p0).cuda(), _i32(nl)
        _cache(k, v, ls).evict(m, p, budget=budget, recent=32, sinks=4)
        assert ls.tolist() == [min(x, budget) for x in nl]
        for b, (slots, keep) in enumerate(want):
            assert np.array_equal(m[b, 0].cpu().numpy()[:keep], m0[b, 0][slots])
            assert np.array_equal(p[b, 0].cpu().numpy()[:keep], p0[b, 0][slots])


def test_evict_weights_that_are_not_finite():
    """NaN and infinite weights order above finite ones and never lose a fixed row."""
    k, v, mass, pos = _evict_inputs(_gen(7), 1, 1, 200, "bf16", False)
    mass[0, 0, 10:20] = float("inf")
    mass[0, 0, 30:33] = float("nan")
    p0, k0, v0 = pos.cpu().numpy()[0, 0], k.cpu().clone(), v.cpu().clone()
    m0 = mass.cpu().numpy()[0, 0]
    cache = _cache(k, v, _i32([200]))
    cache.evict(mass, pos, budget=40, recent=10, sinks=4)
    fixed = set(np.flatnonzero((p0 < 4) | (p0 > p0.max() - 10)).tolist())
    odd = set(range(10, 20)) | set(range(30, 33))
    at = {int(x): i for i, x in enumerate(p0)}
    got = {at[int(x)] for x in pos[0, 0, :40].cpu()}
    assert len(got) == 40 and fixed | odd <= got
    light = sorted((float(m0[i]) for i in set(range(200)) - fixed - odd), reverse=True)
    kept_light = sorted((float(m0[i]) for i in got - fixed - odd), reverse=True)
    assert kept_light == light[:len(kept_light)]


def test_shared_rows_and_queries_by_zero_strides():
    """Heads that share one row stream, and a batch that shares its queries."""
    g = _gen(8)
    k, v = _kv(g, 2, 1, 300, "bf16")
    ke, ve = k.expand(2, 3, 300, D), v.expand(2, 3, 300, D)
    q = torch.randn((1, 6, 5, D), generator=g, device="cuda").bfloat16().expand(2, 6, 5, D)
    out = torch.empty((2, 6, 5, D), dtype=torch.bfloat16, device="cuda")
    _cache(ke, ve).window_attn(q, window=90, sinks=2, out=out)
    _check_window(ke, ve, q, out, [300] * 2, [5] * 2, 90, 2, torch.bfloat16, out.clone())


def test_calls_on_another_stream_and_in_graphs():
    """The same bits eagerly, on a side stream, and from two graphs captured on objects of their
    own and replayed on two streams at once."""
    g = _gen(9)
    B, H, G, n = 4, 2, 4, 700
    k, v = _kv(g, B, H, n, "bf16")
    lens = _i32([700, 650, 3, 128])
    q = torch.randn((B, H * G, 1, D), generator=g, device="cuda")
    want = _cache(k, v, lens).window_attn(q, window=300, sinks=4)
    mass = torch.zeros((B, H, n), device="cuda")
    want_o, want_m = _cache(k, v, lens).mass_decode(q[:, :, 0].contiguous(), mass,
                                                    mass_out=torch.zeros_like(mass))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _cache(k, v, lens).window_attn(q, window=300, sinks=4, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    caches = [_cache(k, v, lens) for _ in range(2)]
    q1 = q[:, :, 0].contiguous()
    outs = [torch.zeros_like(q) for _ in range(2)]
    masses = [torch.zeros_like(mass) for _ in range(2)]
    graphs = []
    for c, o, mo in zip(caches, outs, masses):
        c.window_attn(q, window=300, sinks=4, out=o)         # sizes the workspace
        c.mass_decode(q1, mass, mass_out=mo)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.window_attn(q, window=300, sinks=4, out=o)
            c.mass_decode(q1, mass, mass_out=mo)
        graphs.append(gr)
    for o, mo in zip(outs, masses):
        o.zero_()
        mo.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for o, mo in zip(outs, masses):
        assert torch.equal(o, want) and torch.equal(mo, want_m)


def _workspace_of(cache):
    return cache._ws.data_ptr(), cache._ws.numel()


@pytest.mark.parametrize("by_argument", [False, True])
def test_a_workspace_in_use_on_another_stream_is_not_handed_out(by_argument):
    """An object that goes while its last call is still due on another stream: the memory of its
    workspace must not come back from the allocator before that call has run."""
    g = _gen(17)
    k, v = _kv(g, 2, 2, 600, "bf16")
    q = torch.randn((2, 4, D), generator=g, device="cuda")
    mass = torch.zeros((2, 2, 600), device="cuda")
    want = _cache(k, v).mass_decode(q, mass, mass_out=torch.zeros_like(mass))[1]
    out, got = torch.zeros_like(q), torch.zeros_like(mass)
    cache = _cache(k, v)
    cache.mass_decode(q, mass, mass_out=torch.zeros_like(mass), out=out)     # sized on this stream
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)                                       # some 50 ms
    if by_argument:
        cache.mass_decode(q, mass, mass_out=got, out=out, stream=side)
    else:
        with torch.cuda.stream(side):
            cache.mass_decode(q, mass, mass_out=got, out=out)
    at, size = _workspace_of(cache)
    del cache
    again = torch.empty((size,), dtype=torch.uint8, device="cuda")
    assert not side.query()                              # the call has not run yet
    assert again.data_ptr() != at
    again.fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_what_a_call_allocates_belongs_to_its_stream():
    """With `stream`, outputs and workspace come from that stream's memory, not from what the
    current one may still be using."""
    g = _gen(18)
    k, v = _kv(g, 1, 2, 300, "bf16")
    q = torch.randn((1, 4, 1, D), generator=g, device="cuda")
    want = _cache(k, v).window_attn(q, window=300)
    torch.cuda.synchronize()
    need = 4 * (1 << 20)
    busy = torch.empty((need,), dtype=torch.uint8, device="cuda")
    out_busy = torch.empty_like(q)
    torch.cuda._sleep(100_000_000)
    held = {busy.data_ptr(): need, out_busy.data_ptr(): out_busy.numel() * 4}
    del busy, out_busy                                   # free to this stream, behind its sleep
    side, cache = torch.cuda.Stream(), _cache(k, v)
    out = cache.window_attn(q, window=300, stream=side)
    assert not torch.cuda.current_stream().query()       # this stream is not through
    at, size = _workspace_of(cache)
    for lo, n in held.items():
        assert not (lo <= at < lo + n or at <= lo < at + size)
        assert out.data_ptr() != lo
    side.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()


def test_every_call_captured_without_a_first_one():
    """All calls in one graph of a fresh object (its workspace and plans are made while capturing),
    replayed on new contents: the same bits as eager calls."""
    g = _gen(13)
    B, H, G, n, P, budget = 20, 2, 4, 400, 300, 350
    k, v = _kv(g, B, H, n, "bf16")
    pk, pv = (x[0] for x in _kv(g, 1, H, P, "bf16"))
    q = torch.randn((B, H * G, 30, D), generator=g, device="cuda").bfloat16()
    q1 = torch.randn((B, H * G, D), generator=g, device="cuda")
    mass = torch.rand((B, H, n), generator=g, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(B, H, n).contiguous()
    lens = _i32([n - b for b in range(B)])
    start = [x.clone() for x in (k, v, mass, pos, lens, q, q1)]

    def calls(c):
        a = c.window_attn(q, window=64, sinks=3)
        b = c.mass_decode(q1, mass)[0]
        p = c.prefix_decode(q1, pk, pv)
        p2 = c.prefix_decode(q1.bfloat16(), pk, pv)
        c.evict(mass, pos, budget=budget, recent=16, sinks=2)
        return a, b, p, p2

    c = _cache(k, v, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(c)
    for scale in (1.0, -0.5):
        for x, y in zip((k, v, mass, pos, lens, q, q1), start):
            x.copy_(y)
        q.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        seen = [x.clone() for x in (*got, k, v, mass, pos, lens)]
        for x, y in zip((k, v, mass, pos, lens, q, q1), start):
            x.copy_(y)
        q.mul_(scale)
        eager = calls(_cache(k, v, lens))
        torch.cuda.synchronize()
        for x, y in zip(seen, (*eager, k, v, mass, pos, lens)):
            assert torch.equal(x, y)
        assert lens.tolist() == [min(n - b, budget) for b in range(B)]


def test_prompt_then_decode_with_eviction():
    """The operators together, as a bounded cache uses them: a prompt's attention, decode steps
    that append a row and accumulate weights, an eviction at each overflow, and a shared-prefix
    step over what is left. Every step against the 64-bit forms on the same rows."""
    g = _gen(10)
    B, H, G, cap, budget, prompt = 2, 2, 4, 160, 144, 150
    k, v = _kv(g, B, H, cap, "bf16")
    lens = _i32([prompt] * B)
    cache = _cache(k, v, lens)
    q = torch.randn((B, H * G, prompt, D), generator=g, device="cuda").bfloat16()
    out = cache.window_attn(q, window=cap, sinks=0)
    _check_window(k, v, q, out, [prompt] * B, [prompt] * B, cap, 0, torch.bfloat16, out.clone())
    mass = torch.zeros((B, H, cap), device="cuda")
    pos = torch.arange(cap, dtype=torch.int32, device="cuda").expand(B, H, cap).contiguous()
    evictions = 0
    for step in range(25):
        n = int(lens[0])
        if n == cap:
            m0, p0, k0 = mass.cpu().clone(), pos.cpu().clone(), k.cpu().clone()
            cache.evict(mass, pos, budget=budget, recent=8, sinks=2)
            evictions += 1
            for b in range(B):
                for h in range(H):
                    slots, keep = evicted(m0[b, h].numpy(), p0[b, h].numpy(), cap, budget, 8, 2)
                    assert torch.equal(pos[b, h, :keep].cpu(), p0[b, h][slots])
                    assert torch.equal(k[b, h, :keep].cpu(), k0[b, h][slots])
            n = int(lens[0])
            assert n == budget
        k[:, :, n], v[:, :, n] = (torch.randn((B, H, D), generator=g, device="cuda").bfloat16()
                                  for _ in range(2))
        mass[:, :, n] = 0
        pos[:, :, n] = prompt + step
        lens += 1
        qs = torch.randn((B, H * G, D), generator=g, device="cuda")
        before = mass.double().cpu()
        o, _ = cache.mass_decode(qs, mass)
        for b in range(B):
            for h in range(H):
                ref = Attended(qs[b, h * G:(h + 1) * G], k[b, h, :n + 1], v[b, h, :n + 1],
                               np.ones((G, n + 1), bool))
                assert ((o[b, h * G:(h + 1) * G].double().cpu() - ref.o).abs() <=
                        out_bound(ref, torch.float32)).all()
                want = before[b, h, :n + 1] + ref.w.sum(0)
                assert torch.allclose(mass[b, h, :n + 1].double().cpu(), want, rtol=1e-5, atol=0)
    assert evictions >= 1
    n = int(lens[0])
    pk, pv = k[0, :, :budget].clone(), v[0, :, :budget].clone()
    o = cache.prefix_decode(qs, pk, pv)
    for b in range(B):
        for h in range(H):
            kk, vv = torch.cat([pk[h], k[b, h, :n]]), torch.cat([pv[h], v[b, h, :n]])
            ref = Attended(qs[b, h * G:(h + 1) * G], kk, vv, np.ones((G, budget + n), bool))
            assert ((o[b, h * G:(h + 1) * G].double().cpu() - ref.o).abs() <=
                    out_bound(ref, torch.float32)).all()


def test_small_workspaces_and_wrong_tensors_are_refused():
    import rank_kv_cache_isvd_b200 as iskv
    k, v = _kv(_gen(11), 1, 2, 64, "bf16")
    c = _cache(k, v)
    q = torch.zeros((1, 8, 1, D), device="cuda")
    ok = torch.empty_like(q)
    assert c.window_attn(q, window=8, out=ok) is ok
    with pytest.raises(iskv.IsKVError):
        c.window_attn(q, window=0)
    with pytest.raises(iskv.IsKVError):
        c.window_attn(q[:, :7], window=8)                    # 7 q-heads over 2 kv-heads
    with pytest.raises(ValueError):
        c.window_attn(q.half(), window=8)
    with pytest.raises(ValueError):
        c.window_attn(q[0], window=8)
    with pytest.raises(ValueError):
        c.window_attn(q, window=8, q_lens=torch.ones(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        c.mass_decode(q[:, :, 0], torch.zeros((1, 2, 63), device="cuda"))
    with pytest.raises(ValueError):
        c.evict(torch.zeros((1, 2, 64), device="cuda"),
                torch.zeros((1, 2, 64), dtype=torch.int32, device="cuda"), budget=8, recent=1)
    with pytest.raises(ValueError):
        c.prefix_decode(q[:, :, 0], k[0].float(), v[0].float())
    form = iskv.iskv_exact_queries(0, 0, 8 * D, D, D, 8 * D, D, D, 8, 1, iskv.ISKV_F32, None)
    form.q, form.out = q.data_ptr(), ok.data_ptr()
    code, need = iskv.iskv_window_attn_workspace(c._rows, form, 8, 0)
    assert code == 0
    assert iskv.iskv_window_attn(c._rows, form, 8, 0, c._ws, need - 1) == iskv.ISKV_ERR_CAPACITY


def test_outputs_in_place_of_queries_are_refused():
    k, v = _kv(_gen(19), 1, 1, 64, "bf16")
    q, pk, pv = torch.zeros((1, 1, 1, D), device="cuda"), k[0].clone(), v[0].clone()
    mass = torch.zeros((1, 1, 64), device="cuda")
    cache = _cache(k, v)
    with pytest.raises(ValueError):
        cache.window_attn(q, window=8, out=q)
    with pytest.raises(ValueError):
        cache.mass_decode(q[:, :, 0], mass, out=q[:, :, 0])
    with pytest.raises(ValueError):
        cache.prefix_decode(q[:, :, 0], pk, pv, out=q[:, :, 0])


def _whole(q, k, v):
    """64-bit attention of q [r][128] over all of k, v [n][128], on the device in chunks: weights
    [r][n], outputs, and what ``out_bound`` asks of an ``Attended``."""
    ref, chunk = Attended.__new__(Attended), 1 << 20
    q = q.double()
    s = torch.empty((q.shape[0], k.shape[0]), dtype=torch.float64, device=k.device)
    ref.terms = torch.zeros((q.shape[0], 1), dtype=torch.float64, device=k.device)
    for i in range(0, k.shape[0], chunk):
        x = k[i:i + chunk].double()
        s[:, i:i + chunk] = (q @ x.T) * D ** -0.5
        size = (q.abs() @ x.abs().T) * D ** -0.5
        ref.terms = torch.maximum(ref.terms, size.amax(-1, keepdim=True))
    ref.w = torch.softmax(s, -1)
    ref.o, ref.spread = (torch.zeros_like(q) for _ in range(2))
    for i in range(0, k.shape[0], chunk):
        x = v[i:i + chunk].double()
        ref.o += ref.w[:, i:i + chunk] @ x
        ref.spread += ref.w[:, i:i + chunk] @ x.abs()
    ref.n = k.shape[0]
    return ref


def test_offsets_past_32_bits():
    """Rows of one cache past 2^31 elements (2^32 bytes), by every call: the last rows count."""
    g = _gen(20)
    H, G, n = 2, 2, (1 << 23) + 5
    k, v = (torch.randn((1, n, H, D), generator=g, device="cuda", dtype=torch.bfloat16).transpose(1, 2)
            for _ in range(2))
    assert (n - 1) * k.stride(2) + D > 1 << 31
    cache = _cache(k, v, _i32([n]))
    # window: single token (split kernel) and a chunk (tile kernel); near rows and three sinks
    for m in (1, 70):
        q = torch.randn((1, H * G, m, D), generator=g, device="cuda").bfloat16()
        out = cache.window_attn(q, window=200, sinks=3)
        near = 300
        pick = torch.cat([torch.arange(3), torch.arange(n - near, n)]).cuda()
        j, p = pick.cpu().numpy()[None], (n - m + np.arange(m))[:, None]
        see = (j <= p) & ((j < 3) | (j > p - 200))
        for x in range(H * G):
            ref = Attended(q[0, x], k[0, x // G][pick], v[0, x // G][pick], see)
            err = (out[0, x].double().cpu() - ref.o).abs()
            assert (err <= out_bound(ref, q.dtype, torch.bfloat16)).all()
    # accumulated weights over all rows, the last of them made to stand out
    q = torch.randn((1, H * G, D), generator=g, device="cuda")
    k[0, :, n - 1] = 4 * q[0, ::G].bfloat16()
    mass = torch.zeros((1, H, n), device="cuda")
    out, mass = cache.mass_decode(q, mass)
    for h in range(H):
        ref = _whole(q[0, h * G:(h + 1) * G], k[0, h], v[0, h])
        err = (out[0, h * G:(h + 1) * G].double() - ref.o).abs()
        assert (err <= out_bound(ref, q.dtype)).all()
        err = (mass[0, h].double() - ref.w.sum(0)).abs()
        assert (err <= (ref.w * weight_bound(ref)).sum(0) + ref.w.sum(0) * G * 2.0 ** -24 + 1e-30).all()
        assert mass[0, h, n - 1] > 0.01
        del ref, err
    # the rows as a prefix of three sequences
    q = torch.randn((3, H * G, D), generator=g, device="cuda").bfloat16()
    own_k, own_v = _kv(g, 3, H, 4, "bf16")
    out = _cache(own_k, own_v, _i32([0, 0, 0])).prefix_decode(q, k[0], v[0])
    for h in range(H):
        ref = _whole(q[:, h * G:(h + 1) * G].reshape(3 * G, D), k[0, h], v[0, h])
        err = (out[:, h * G:(h + 1) * G].reshape(3 * G, D).double() - ref.o).abs()
        assert (err <= out_bound(ref, q.dtype, torch.bfloat16)).all()
        del ref, err
    # eviction: rows from the far end move down
    budget = n - 3000
    mass = torch.rand((1, H, n), generator=g, device="cuda")
    pos = torch.arange(n, device="cuda", dtype=torch.int32).expand(1, H, n).contiguous()
    k0, v0, m0, p0 = k[0].clone(), v[0].clone(), mass.cpu().numpy(), pos.cpu().numpy()
    cache.evict(mass, pos, budget=budget, recent=100, sinks=4)
    assert cache.lens.tolist() == [budget]
    for h in range(H):
        slots, keep = evicted(m0[0, h], p0[0, h], n, budget, 100, 4)
        at = torch.from_numpy(slots).cuda()
        assert int((at != torch.arange(keep, device="cuda")).sum()) > 1000
        assert torch.equal(pos[0, h, :keep].long(), at)
        for i in range(0, keep, 1 << 20):
            part = slice(i, min(keep, i + (1 << 20)))
            assert torch.equal(k[0, h, part], k0[h][at[part]])
            assert torch.equal(v[0, h, part], v0[h][at[part]])
