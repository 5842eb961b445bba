"""Calls on exact caches whose device-side waits give up: they return, say so once in the status, write
nothing but their outputs, and leave the next call as it would be."""
import time

import pytest

torch = pytest.importorskip("torch")

import rank_kv_cache_isvd_b200 as iskv  # noqa: E402

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert iskv.iskv_exact_status() == 0
    yield
    assert iskv.iskv_exact_wait_limit() == 0
    assert iskv.iskv_exact_status() == 0


CASES = [
    # call, B, H, G, rows, m (prefix: its rows), window, sinks, io, rows_type
    ("window", 1, 2, 4, 3000, 1, 2000, 4, "f32", "bf16"),        # items, shared by clusters
    ("window", 130, 8, 1, 90, 1, 60, 4, "bf16", "bf16"),         # items, teams of few warps
    ("window", 40, 8, 1, 1300, 1, 1000, 4, "f32", "f32"),        # steps and their merge
    ("mass", 2, 4, 4, 2500, 1, 0, 0, "f32", "bf16"),
    ("mass", 19, 8, 2, 3000, 1, 0, 0, "f32", "f32"),
    ("window", 1, 2, 4, 600, 600, 100, 3, "bf16", "bf16"),       # pairs of tiles
    ("window", 2, 2, 4, 900, 30, 500, 3, "bf16", "bf16"),        # one tile, its rows split
    ("window", 1, 2, 4, 700, 300, 200, 20, "f32", "bf16"),       # rows kernel
    ("window", 1, 2, 4, 700, 60, 500, 20, "f32", "f32"),
    ("prefix", 40, 2, 4, 300, 1500, 0, 0, "bf16", "bf16"),       # tile kernel, then the own rows
    ("prefix", 40, 2, 4, 300, 1500, 0, 0, "f32", "f32"),         # rows kernel, then the own rows
    ("prefix", 2, 2, 4, 300, 1500, 0, 0, "bf16", "bf16"),        # all by steps
]


@pytest.mark.parametrize("call,B,H,G,n,m,window,sinks,io,rt", CASES)
def test_waits_that_give_up(call, B, H, G, n, m, window, sinks, io, rt):
    types = {"bf16": torch.bfloat16, "f32": torch.float32}
    g = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    k, v = rand(B, H, n, D).to(types[rt]), rand(B, H, n, D).to(types[rt])
    cache = iskv.ExactKVCache(k, v, lens=torch.full((B,), n, dtype=torch.int32, device="cuda"))
    shape = (B, H * G, m, D) if call == "window" else (B, H * G, D)
    q = rand(*shape).to(types[io])
    around = torch.full((q.numel() + 256,), 7.0, device="cuda").to(types[io])
    out = around[128:-128].view(shape)
    mass, mass_out = torch.zeros((B, H, n), device="cuda"), torch.zeros((B, H, n), device="cuda")
    pk, pv = rand(H, m, D).to(types[rt]), rand(H, m, D).to(types[rt])

    def run():
        out.zero_()
        if call == "window":
            cache.window_attn(q, window=window, sinks=sinks, out=out)
        elif call == "mass":
            cache.mass_decode(q, mass, mass_out=mass_out, out=out)
        else:
            cache.prefix_decode(q, pk, pv, out=out)
        return out.clone(), mass_out.clone()

    want = run()
    assert iskv.iskv_exact_status() == 0 and torch.isfinite(want[0]).all() and want[0].any()
    assert iskv.iskv_exact_wait_limit(0) == 0
    begun = time.monotonic()
    run()
    torch.cuda.synchronize()
    took = time.monotonic() - begun
    assert iskv.iskv_exact_status() == iskv.ISKV_ERR_TIMEOUT
    assert iskv.iskv_exact_status() == 0                         # once
    assert took < 1.0                                            # its copies had arrived or did soon
    assert (around[:128] == 7).all() and (around[-128:] == 7).all() and not mass.any()
    assert iskv.iskv_exact_wait_limit() == 0
    got = run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
