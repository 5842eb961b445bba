"""Attention over an exact KV cache, and the cache's eviction: what is measured of them.

Four operators over exact rows (keys as attended, so already rotated; values) of ``[batch][n_kv]
[rows][128]``, each sequence holding its first ``lens[b]`` rows:

* ``window``: attention of the last ``m`` tokens with a sliding window and a few first tokens that
  stay visible. Token i of sequence b sits at position p = lens[b] - q_lens[b] + i and sees the
  rows j <= p with j < sinks or j > p - window.
* ``mass``: decode attention of one token per sequence over all its rows, which adds every row's
  attention weight (summed over the q-heads of its kv-head) to ``mass``.
* ``evict``: keeps ``budget`` rows per (sequence, kv-head): the first ``sinks`` positions, the
  ``recent`` latest positions and the heaviest of the rest (ties: the lowest slot). Kept rows from
  slots >= budget move into the freed slots below it, both in ascending order.
* ``prefix``: decode attention of one token per sequence over one prefix that all sequences share
  and then the sequence's own rows.

``own`` chooses between the plain forms (float32 torch operations) and the framework's calls.
"""
import math

import numpy as np
import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a prompt of the Llama-shaped layer, prefilled in one call: activations in [token][head]
        dict(name="window prompt 4096", op="window", batch=1, kv=8, group=4, rows=4096, m=4096,
             window=1024, sinks=4, ragged=False, io="bf16", rows_type="bf16", tokens_first=True),
        # a long prompt whose window covers it all: plain causal attention
        dict(name="window causal 8192", op="window", batch=1, kv=8, group=4, rows=8192, m=8192,
             window=8192, sinks=0, ragged=False, io="bf16", rows_type="bf16", tokens_first=True),
        # a padded batch of odd lengths, its next chunk of at most 511 tokens after cached ones
        dict(name="window chunks ragged", op="window", batch=5, kv=4, group=5, rows=2047, m=511,
             window=700, sinks=9, ragged=True, io="bf16", rows_type="bf16", tokens_first=True),
        # one decode step of the long-context batch: window and sinks of long caches
        dict(name="window decode 4x65536", op="window", batch=4, kv=8, group=4, rows=65536, m=1,
             window=4096, sinks=64, ragged=True, io="f32", rows_type="bf16", tokens_first=False),
        # the smallest: one sequence of the Llama-shaped layer, a window of 256
        dict(name="window decode 1x4096", op="window", batch=1, kv=8, group=4, rows=4096, m=1,
             window=256, sinks=4, ragged=False, io="f32", rows_type="bf16", tokens_first=False),
        # a decode step of the Qwen3-shaped layer on an uncompressed cache
        dict(name="mass 8x32768", op="mass", batch=8, kv=8, group=4, rows=32768, ragged=False,
             io="f32", rows_type="bf16"),
        # odd ragged lengths in float32, groups of two
        dict(name="mass f32 ragged", op="mass", batch=3, kv=5, group=2, rows=5001, ragged=True,
             io="f32", rows_type="f32"),
        # an eviction of one eighth of the Qwen3-shaped cache
        dict(name="evict 8x32768", op="evict", batch=8, kv=8, rows=32768, budget=28672, recent=256,
             sinks=4, ragged=False, rows_type="bf16"),
        # a short cache that is held at 4096 rows by evicting a block of 64
        dict(name="evict 1x4160", op="evict", batch=1, kv=8, rows=4160, budget=4096, recent=256,
             sinks=4, ragged=False, rows_type="bf16"),
        # 32 samples of one long prompt, some way into their answers
        dict(name="prefix 32x32768", op="prefix", batch=32, kv=8, group=4, prefix=32768, rows=1024,
             ragged=True, io="bf16", rows_type="bf16"),
        # a large batch over a system prompt of odd length
        dict(name="prefix 130x4001", op="prefix", batch=130, kv=8, group=4, prefix=4001, rows=513,
             ragged=True, io="bf16", rows_type="bf16"),
        # a few samples in the types of the compressed cache's decode (float32 queries and outputs)
        dict(name="prefix f32 8x4096", op="prefix", batch=8, kv=8, group=4, prefix=4096, rows=256,
             ragged=False, io="f32", rows_type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window prompt", "window step", "mass", "evict", "prefix"])
    group = rng.choice([1, 2, 4, 4, 5, 8])
    kv = rng.choice([1, 2, 4, 5, 8, 8])
    batch = _log(rng, 1, 8)
    io, rows_type = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
    ragged = rng.random() < 0.5
    if op == "window prompt":
        m = _log(rng, 17, 8192)
        rows = min(8192, m + rng.choice([0, _log(rng, 1, 4096)]))
        batch = max(1, min(batch, 2048 // rows))
        kv = max(1, min(kv, 32 // group))
        return dict(op="window", batch=batch, kv=kv, group=group, rows=rows, m=min(m, rows),
                    window=_log(rng, 64, 8192), sinks=rng.choice([0, 1, 4, 64, 130]),
                    ragged=ragged, io="bf16", rows_type="bf16", tokens_first=rng.random() < 0.7)
    if op == "window step":
        return dict(op="window", batch=min(batch, 4), kv=kv, group=group,
                    rows=_log(rng, 256, 65536), m=rng.choice([1, 1, 1, 2, 3]),
                    window=_log(rng, 64, 8192), sinks=rng.choice([0, 1, 4, 64, 130]),
                    ragged=ragged, io=io, rows_type=rows_type, tokens_first=rng.random() < 0.3)
    if op == "mass":
        return dict(op="mass", batch=batch, kv=kv, group=group,
                    rows=_log(rng, 128, 32768 if rows_type == "bf16" else 16384), ragged=ragged,
                    io=io, rows_type=rows_type)
    if op == "evict":
        rows = _log(rng, 300, 32768)
        budget = max(80, int(rows * rng.uniform(0.5, 0.995)))
        return dict(op="evict", batch=batch, kv=kv, rows=rows, budget=budget,
                    recent=rng.choice([1, 32, 64]), sinks=rng.choice([0, 4]), ragged=ragged,
                    rows_type=rows_type)
    prefix = _log(rng, 100, 32768)
    return dict(op="prefix", batch=_log(rng, 2, 130), kv=kv, group=group,
                prefix=min(prefix, 16384 if io == "f32" else prefix), rows=_log(rng, 1, 600),
                ragged=ragged, io=io, rows_type=rows_type)


# -- inputs -------------------------------------------------------------------------------------
def _rows(gen, shape, dtype, channels):
    """Rows with lognormal channel scales (shared along each row stream)."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    return x.mul_(channels.to(dtype)) if channels is not None else x


def _lens(gen, batch, rows, ragged):
    lens = torch.full((batch,), rows, dtype=torch.int32, device="cuda")
    if ragged:
        lens -= (torch.rand((batch,), generator=gen, device="cuda") * (rows // 2 + 1)).int()
        lens[0] = rows
    return lens


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, H, n = case["batch"], case["kv"], case["rows"]
    rt = TYPES[case["rows_type"]]
    s = {"case": case}
    ck = torch.exp(0.5 * torch.randn((1, H, 1, D), generator=gen, device="cuda"))
    cv = torch.exp(0.5 * torch.randn((1, H, 1, D), generator=gen, device="cuda"))
    if case.get("tokens_first"):
        s["k"] = _rows(gen, (B, n, H, D), rt, ck.transpose(1, 2)).transpose(1, 2)
        s["v"] = _rows(gen, (B, n, H, D), rt, cv.transpose(1, 2)).transpose(1, 2)
    else:
        s["k"] = _rows(gen, (B, H, n, D), rt, ck)
        s["v"] = _rows(gen, (B, H, n, D), rt, cv)
    s["lens"] = _lens(gen, B, n, case["ragged"])
    if case["op"] == "window":
        m, nq, it = case["m"], H * case["group"], TYPES[case["io"]]
        shape = (B, m, nq, D) if case["tokens_first"] else (B, nq, m, D)
        q = _rows(gen, shape, it, None)
        out = torch.zeros_like(q)
        s["q"], s["out"] = (q.transpose(1, 2), out.transpose(1, 2)) if case["tokens_first"] else (
            q, out)
        s["q_lens"] = torch.minimum(_lens(gen, B, m, case["ragged"]), s["lens"])
    elif case["op"] == "mass":
        s["q"] = _rows(gen, (B, H * case["group"], D), TYPES[case["io"]], None)
        s["out"] = torch.zeros_like(s["q"])
        s["mass"] = torch.rand((B, H, n), generator=gen, device="cuda")
        s["mass_out"] = torch.zeros_like(s["mass"])
    elif case["op"] == "evict":
        # weights of very different sizes, some rows never attended (equal weights: 0); slots out
        # of order, as earlier evictions left them
        mass = torch.exp(2 * torch.randn((B, H, n), generator=gen, device="cuda") - 4)
        mass[torch.rand((B, H, n), generator=gen, device="cuda") < 0.05] = 0.0
        s["mass"] = mass
        order = torch.argsort(torch.rand((B, H, n), generator=gen, device="cuda"), dim=-1)
        gaps = torch.rand((B, H, n), generator=gen, device="cuda") < 0.3
        s["pos"] = torch.gather(torch.cumsum(1 + gaps.int(), -1).int() - 1, -1, order)
        s["pos"] = s["pos"].int().contiguous()
        s["mass_out"], s["pos_out"] = torch.zeros_like(s["mass"]), torch.zeros_like(s["pos"])
        s["lens_out"] = torch.zeros_like(s["lens"])
    else:
        s["pk"] = _rows(gen, (H, case["prefix"], D), rt, ck[0])
        s["pv"] = _rows(gen, (H, case["prefix"], D), rt, cv[0])
        s["q"] = _rows(gen, (B, H * case["group"], D), TYPES[case["io"]], None)
        s["out"] = torch.zeros_like(s["q"])
    return s


# -- the framework's calls -----------------------------------------------------------------------
def _cache(s):
    """The cache object that a program keeps next to its buffers."""
    if "cache" not in s:
        from rank_kv_cache_isvd_b200 import ExactKVCache
        s["cache"] = ExactKVCache(s["k"], s["v"], lens=s["lens"])
    return s["cache"]


def _own(s):
    case, cache = s["case"], _cache(s)
    if case["op"] == "window":
        return cache.window_attn(s["q"], window=case["window"], sinks=case["sinks"],
                                 q_lens=s["q_lens"], out=s["out"])
    if case["op"] == "mass":
        return cache.mass_decode(s["q"], s["mass"], mass_out=s["mass_out"], out=s["out"])
    if case["op"] == "evict":
        cache.evict(s["mass"], s["pos"], budget=case["budget"], recent=case["recent"],
                    sinks=case["sinks"], mass_out=s["mass_out"], pos_out=s["pos_out"],
                    lens_out=s["lens_out"])
        return s["k"], s["v"], s["mass_out"], s["pos_out"], s["lens_out"]
    return cache.prefix_decode(s["q"], s["pk"], s["pv"], out=s["out"])


# -- the plain forms -----------------------------------------------------------------------------
def _softmax(x):
    """Softmax along the last axis in place; rows of -inf become rows of 0."""
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    return x.div_(torch.where(total == 0, torch.ones_like(total), total))


def _plain_window(s):
    case, k, v = s["case"], s["k"], s["v"]
    B, H, n, _ = k.shape
    m, G = case["m"], case["group"]
    i = torch.arange(m, device=k.device)[None, :, None]
    j = torch.arange(n, device=k.device)[None, None, :]
    ql = s["q_lens"].long()[:, None, None]
    p = s["lens"].long()[:, None, None] - ql + i
    hidden = (j > p) | ((j >= case["sinks"]) & (j <= p - case["window"]))         # [B][m][n]
    q = s["q"].float().reshape(B, H, G * m, D)
    x = torch.matmul(q, k.float().transpose(-1, -2)).mul_(SCALE).view(B, H, G, m, n)
    x.masked_fill_(hidden[:, None, None], -math.inf)
    w = _softmax(x).view(B, H, G * m, n)
    o = torch.matmul(w, v.float()).view(B, H * G, m, D)
    s["out"].copy_(torch.where((i < ql)[:, None], o.to(s["out"].dtype), s["out"]))
    return s["out"]


def _plain_mass(s):
    case, k, v = s["case"], s["k"], s["v"]
    B, H, n, _ = k.shape
    j = torch.arange(n, device=k.device)
    held = (j < s["lens"][:, None])[:, None]                                     # [B][1][n]
    x = torch.matmul(s["q"].float().view(B, H, -1, D), k.float().transpose(-1, -2)).mul_(SCALE)
    w = _softmax(x.masked_fill_(~held[:, :, None], -math.inf))
    s["out"].copy_(torch.matmul(w, v.float()).view(s["out"].shape))
    s["mass_out"].copy_(torch.where(held, s["mass"] + w.sum(2), s["mass_out"]))
    return s["out"], s["mass_out"]


def _plain_evict(s):
    case, k, v = s["case"], s["k"], s["v"]
    n, R = k.shape[2], case["budget"]
    slot = torch.arange(n, device=k.device)
    lens = s["lens"][:, None, None]
    held = slot < lens
    keep = torch.minimum(lens, torch.full_like(lens, R))
    pos = torch.where(held, s["pos"], torch.full_like(s["pos"], -1))
    fixed = held & ((pos < case["sinks"]) | (pos > pos.amax(-1, keepdim=True) - case["recent"]))
    value = torch.where(held, s["mass"], torch.full_like(s["mass"], -1.0))
    value = torch.where(fixed, torch.full_like(value, math.inf), value)
    order = torch.sort(value, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order))
    kept = rank < keep
    free = (~kept & (slot < keep)).nonzero(as_tuple=True)
    move = (kept & (slot >= keep)).nonzero(as_tuple=True)
    k[free], v[free] = k[move], v[move]
    mass, at = s["mass"].clone(), s["pos"].clone()
    mass[free], at[free] = mass[move], at[move]
    left = slot < keep
    s["mass_out"].copy_(torch.where(left, mass, s["mass_out"]))
    s["pos_out"].copy_(torch.where(left, at, s["pos_out"]))
    s["lens_out"].copy_(keep[:, 0, 0])
    return k, v, s["mass_out"], s["pos_out"], s["lens_out"]


def _plain_prefix(s):
    k, v, pk, pv = s["k"], s["v"], s["pk"], s["pv"]
    B, H, n, _ = k.shape
    P = pk.shape[1]
    held = torch.arange(n, device=k.device) < s["lens"][:, None, None, None]
    q = s["q"].float().view(B, H, -1, D)
    G = q.shape[2]
    x = torch.empty((B, H, G, P + n), device=k.device)
    shared = q.transpose(0, 1).reshape(H, B * G, D)
    x[..., :P] = torch.matmul(shared, pk.float().transpose(-1, -2)).view(H, B, G, P).transpose(0, 1)
    x[..., P:] = torch.matmul(q, k.float().transpose(-1, -2)).masked_fill_(~held, -math.inf)
    w = _softmax(x.mul_(SCALE))
    front = w[..., :P].transpose(0, 1).reshape(H, B * G, P)
    o = torch.matmul(front, pv.float()).view(H, B, G, D).transpose(0, 1)
    o = o + torch.matmul(w[..., P:], v.float())
    s["out"].copy_(o.reshape(s["out"].shape))
    return s["out"]


PLAIN = {"window": _plain_window, "mass": _plain_mass, "evict": _plain_evict,
         "prefix": _plain_prefix}


def run(s):
    if own:
        return _own(s)
    return PLAIN[s["case"]["op"]](s)


# -- what a pass cannot do without ---------------------------------------------------------------
def _mean_len(case):
    """Mean of lens: whole, or (ragged) uniform in [rows / 2, rows] but for one whole sequence."""
    n, B = case["rows"], case["batch"]
    return n if not case["ragged"] else (n + (B - 1) * 0.75 * n) / B


def work(case):
    B, H, n = case["batch"], case["kv"], _mean_len(case)
    rb = TYPES[case["rows_type"]].itemsize * D * 2                    # a row's key and value
    if case["op"] == "evict":
        R = case["budget"]
        gone = max(0.0, n - R)
        moved = gone * R / n                      # freed slots below the budget, each refilled
        bytes_ = B * H * (8 * n + 8 * min(n, R) + 2 * rb * moved)
        return {"bytes": bytes_, "flops": float(B * H * n)}
    G = case["group"]
    ib = TYPES[case["io"]].itemsize * D * 2                           # a query and its output
    if case["op"] == "window":
        m = case["m"] if not case["ragged"] else (case["m"] + (B - 1) * 0.75 * case["m"]) / B
        p = n - m + np.arange(max(1, int(m)))                         # positions of the tokens
        before = np.maximum(0, p + 1 - case["window"])                # rows that the window left
        seen = np.minimum(p + 1, case["window"]) + np.minimum(case["sinks"], before)
        rows = min(n, m - 1 + case["window"] + case["sinks"])
        return {"bytes": float(B * H * (rows * rb + G * m * ib)),
                "flops": float(B * H * G * 4 * D * seen.sum())}
    if case["op"] == "mass":
        return {"bytes": B * H * (n * (rb + 8) + G * ib), "flops": B * H * G * n * 4.0 * D}
    P = case["prefix"]
    return {"bytes": H * P * rb + B * H * (n * rb + G * ib),
            "flops": B * H * G * (P + n) * 4.0 * D}


# -- the definitions, in 64 bits -----------------------------------------------------------------
def _attend(q, k, v):
    """Weights and outputs of queries [g][128] over rows [n][128] that all are visible."""
    z = (q.double() @ k.double().T) / math.sqrt(D)
    w = torch.softmax(z, dim=-1) if z.shape[-1] else z
    return w, w @ v.double()


def exact(case, seed):
    s = prepare(case, seed)
    B, H, n = case["batch"], case["kv"], case["rows"]
    lens = s["lens"].tolist()
    if case["op"] == "evict":
        return _exact_evict(s, lens)
    G = case["group"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "mass":
        mass = torch.zeros(s["mass"].shape, dtype=torch.float64, device="cuda")
        for b in range(B):
            for h in range(H):
                w, o = _attend(s["q"][b, h * G:(h + 1) * G], s["k"][b, h, :lens[b]],
                               s["v"][b, h, :lens[b]])
                out[b, h * G:(h + 1) * G] = o
                mass[b, h, :lens[b]] = s["mass"][b, h, :lens[b]].double() + w.sum(0)
        return out, mass
    if case["op"] == "prefix":
        for b in range(B):
            for h in range(H):
                k = torch.cat([s["pk"][h], s["k"][b, h, :lens[b]]])
                v = torch.cat([s["pv"][h], s["v"][b, h, :lens[b]]])
                out[b, h * G:(h + 1) * G] = _attend(s["q"][b, h * G:(h + 1) * G], k, v)[1]
        return out
    q_lens = s["q_lens"].tolist()
    for b in range(B):
        for g in range(H * G):
            k, v = s["k"][b, g // G].double(), s["v"][b, g // G].double()
            for lo in range(0, q_lens[b], 1024):
                hi = min(lo + 1024, q_lens[b])
                first, last = lens[b] - q_lens[b] + lo, lens[b] - q_lens[b] + hi - 1
                begin = max(min(case["sinks"], n), first - case["window"] + 1)   # after the sinks
                at = torch.cat([torch.arange(0, min(case["sinks"], last + 1), device="cuda"),
                                torch.arange(begin, last + 1, device="cuda")])
                p = torch.arange(first, last + 1, device="cuda")[:, None]
                z = (s["q"][b, g, lo:hi].double() @ k[at].T) / math.sqrt(D)
                see = (at <= p) & ((at < case["sinks"]) | (p - at < case["window"]))
                z[~see] = -math.inf
                out[b, g, lo:hi] = torch.softmax(z, dim=-1) @ v[at]
    return out


def _exact_evict(s, lens):
    case = s["case"]
    k, v = s["k"].double(), s["v"].double()
    mass, pos = s["mass"].cpu().numpy(), s["pos"].cpu().numpy()
    mass_out, pos_out = np.zeros(mass.shape, np.float64), np.zeros(pos.shape, np.int32)
    R = case["budget"]
    for b, n in enumerate(lens):
        for h in range(case["kv"]):
            a, w = pos[b, h, :n], mass[b, h, :n].astype(np.float64)
            low = ~((a < case["sinks"]) | (a >= a.max() + 1 - case["recent"]))
            chosen = np.lexsort((np.arange(n), -w, low))[:R]           # fixed first, then heavy
            chosen = set(chosen.tolist())
            target = [i for i in range(min(R, n)) if i not in chosen]
            source = sorted(i for i in chosen if i >= R)
            where = np.arange(min(R, n))
            where[target] = source
            mass_out[b, h, :len(where)] = w[where]
            pos_out[b, h, :len(where)] = a[where]
            if target:
                k[b, h, target], v[b, h, target] = k[b, h, source], v[b, h, source]
    return (k, v, torch.from_numpy(mass_out), torch.from_numpy(pos_out),
            torch.tensor([min(n, R) for n in lens], dtype=torch.int32))
