"""Workspaces of an object of exact caches: an earlier one is kept only for graphs that may use it, and those
kept stay few."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

D, N = 128, 3000


class _Evictions:
    """Evictions whose lists of moves, and so their workspaces, grow with the number of rows that go."""

    def __init__(self):
        from rank_kv_cache_isvd_b200 import ExactKVCache
        g = torch.Generator(device="cuda").manual_seed(1)
        k, v = (torch.randn((8, 2, N, D), generator=g, device="cuda").bfloat16() for _ in range(2))
        self.mass = torch.rand((8, 2, N), generator=g, device="cuda")
        self.pos = torch.arange(N, dtype=torch.int32, device="cuda").expand(8, 2, N).contiguous()
        self.cache = ExactKVCache(k, v)

    def outputs(self):
        return (torch.zeros_like(self.mass), torch.zeros_like(self.pos),
                torch.zeros((8,), dtype=torch.int32, device="cuda"))

    def call(self, gone, outs, stream=None):
        self.cache.evict(self.mass, self.pos, budget=N - gone, recent=1, mass_out=outs[0], pos_out=outs[1],
                         lens_out=outs[2], stream=stream)

    def needs(self):
        return [plan.need for plan in self.cache._plans.values()]


def test_forms_that_grow_keep_no_workspaces():
    e = _Evictions()
    outs, made, last = e.outputs(), 0, 0
    for gone in range(1, 1400, 3):
        e.call(gone, outs)
        made += e.cache._ws.numel() != last
        last = e.cache._ws.numel()
        assert not e.cache._old_ws
    assert max(e.needs()) > 100 * min(e.needs()) and len(e.needs()) > 400    # they did grow
    assert e.cache._ws.numel() <= 1.5 * max(e.needs()) and made < 20


@pytest.mark.parametrize("by_argument", [False, True])
def test_graphs_keep_their_workspace_when_it_grows(by_argument):
    e, ref = _Evictions(), _Evictions()
    graphs, outs, wants = [], [], []
    for gone in range(1, 1400, 40):
        out = e.outputs()
        wants.append(ref.outputs())
        ref.call(gone, wants[-1])
        e.call(gone, out)                                    # eager: this one alone keeps nothing
        for x in out:
            x.zero_()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            e.call(gone, out, torch.cuda.current_stream().cuda_stream if by_argument else None)
        graphs.append(graph)
        outs.append(out)
    assert 0 < len(e.cache._old_ws) < 20
    assert sum(x.numel() for x in e.cache._old_ws) <= 3 * e.cache._ws.numel()
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (600, 4000, 40000, 200000) * 50]
    torch.cuda.synchronize()
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        for x, y in zip(out, want):
            assert torch.equal(x, y)
    assert all(bool((x == 255).all()) for x in junk)         # no graph wrote where others live now
