"""The serving operators' cases: what is run, on what inputs, and what one pass of it has to do.

Four operators that stand before and beside the decode step, on one layer's tensors:

  rope    per-head RMS norm of the queries and keys and the rotation by position, in one pass
  append  the same for the step's tokens, the keys and values written into the cache as they are
          made, in 8 bits (e4m3 codes, one power-of-two scale for each row) or in bf16
  read    rows of an 8-bit cache read back: a range of rows, or the rows of selected sets
  tree    attention of a tree of drafted tokens over the cache (one token: the dense decode)

``run`` computes them in plain torch operations, or, where ``own`` is true, by the calls a user
makes of this package.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
E8M0_MIN = 27  # smallest scale byte that is written: 2^-100


# ------------------------------------------------------------------ cases


def listed():
    return [
        # the norms and the rotation of one decode step: four sequences, Qwen3-8B's heads
        dict(name="rope_decode", op="rope", rows=4, hq=32, hkv=8, d=128, dtype="bf16", norm=True,
             rot=128, interleaved=False, far=65536),
        # the same over a prompt's tokens
        dict(name="rope_prompt", op="rope", rows=8192, hq=32, hkv=8, d=128, dtype="bf16", norm=True,
             rot=128, interleaved=False, far=131072),
        # fp32, head_dim 64, an odd number of rows, half of each head rotated in adjacent pairs, no norm
        dict(name="rope_fp32_partial", op="rope", rows=1023, hq=16, hkv=2, d=64, dtype="fp32",
             norm=False, rot=32, interleaved=True, far=655360),
        # one decode step's tokens made and written: four sequences, pages of 64 rows
        dict(name="append_decode", op="append", B=4, T=1, hq=32, hkv=8, d=128, cap=1024, page=64,
             norm=True, rotate=True, with_q=True, ragged=False, e4m3=True),
        # a prompt's tokens made and written, contiguous cache
        dict(name="append_prompt", op="append", B=2, T=4096, hq=32, hkv=8, d=128, cap=4160, page=0,
             norm=True, rotate=True, with_q=True, ragged=False, e4m3=True),
        # keys and values that come ready, ragged counts, pages of 48 rows, head_dim 64
        dict(name="append_ragged", op="append", B=5, T=333, hq=8, hkv=2, d=64, cap=720, page=48,
             norm=False, rotate=False, with_q=False, ragged=True, e4m3=True),
        # a whole 32K cache read back for a step that wants bf16 rows
        dict(name="read_32k", op="read", B=1, hq=32, hkv=8, d=128, cap=32768, page=0, m=32768, sets=0),
        # the rows of per-head sets of 4096 tokens out of a paged 32K cache
        dict(name="read_sets", op="read", B=1, hq=32, hkv=8, d=128, cap=32768, page=64, m=4096, sets=32),
        # one token over a short cache: the smallest call
        dict(name="tree_one_token", op="tree", B=1, T=1, hq=32, hkv=8, d=128, n=4097, page=0,
             ragged=False, e4m3=False),
        # four sequences verifying 16 drafted tokens each over an 8-bit paged cache
        dict(name="tree_verify_b4", op="tree", B=4, T=16, hq=32, hkv=8, d=128, n=65536, page=64,
             ragged=True, e4m3=True),
        # 32 drafted tokens at 128K
        dict(name="tree_128k", op="tree", B=1, T=32, hq=32, hkv=8, d=128, n=131072, page=0,
             ragged=False, e4m3=False),
        # a wide tree, more query rows than one tile of 128
        dict(name="tree_wide", op="tree", B=2, T=64, hq=32, hkv=8, d=128, n=32768, page=16,
             ragged=True, e4m3=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "tree", "tree"])
    hq, hkv = rng.choice([(32, 8), (16, 2), (8, 8), (4, 2), (32, 4), (12, 4), (5, 1)])
    d = rng.choice([64, 128, 128])
    if op == "rope":
        return dict(op=op, rows=_log(rng, 1, 8192), hq=hq, hkv=hkv, d=d, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    norm=rng.random() < 0.7, rot=rng.choice([d, d, d // 2, d // 4]),
                    interleaved=rng.random() < 0.4, far=_log(rng, 16, 655360))
    if op == "append":
        B = _log(rng, 1, 24)
        T = _log(rng, 1, max(1, 8192 // B))
        return dict(op=op, B=B, T=T, hq=hq, hkv=hkv, d=d, cap=T + rng.randint(0, 200),
                    page=rng.choice([0, 16, 48, 64, 256, 7]), norm=rng.random() < 0.6, rotate=rng.random() < 0.7,
                    with_q=rng.random() < 0.6, ragged=rng.random() < 0.5, e4m3=rng.random() < 0.75)
    if op == "read":
        B = _log(rng, 1, 8)
        cap = _log(rng, 8, max(8, 32768 // B))
        sets = rng.choice([0, hkv, hq])
        m = _log(rng, 1, cap if not sets else max(1, min(cap, 4096 // B)))
        return dict(op=op, B=B, hq=hq, hkv=hkv, d=d, cap=cap, page=rng.choice([0, 16, 48, 64, 256]), m=m, sets=sets)
    B = _log(rng, 1, 16)
    T = min(80, _log(rng, 1, 96))
    n = _log(rng, T, max(T, min(131072, int(4.0e6 / (B * max(T, 16)) * 32 / hq))))
    return dict(op=op, B=B, T=T, hq=hq, hkv=hkv, d=d, n=n, page=rng.choice([0, 0, 16, 64, 64, 48, 256, 5]),
                ragged=rng.random() < 0.5, e4m3=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _inv_freq(rot):
    # the usual geometric frequencies, base 500000 as long contexts have it
    j = torch.arange(0, rot, 2, dtype=torch.float64)
    return (500000.0 ** (-j / rot)).to(torch.float32).to(DEV)


def _weights(g, d, dtype):
    return (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dtype)


def _quantised(x):
    """(codes, scale bytes) of bf16 rows: the scale is the smallest power of two that brings the
    row's largest magnitude to 448 or less."""
    amax = x.abs().amax(-1).float().view(torch.int32)
    byte = (amax >> 23) - 8 + ((amax & 0x7FFFFF) > 0x600000).to(torch.int32)
    byte = byte.clamp(E8M0_MIN, 254)
    inv = ((254 - byte) << 23).view(torch.float32)
    return (x.float() * inv[..., None]).to(torch.float8_e4m3fn), byte.to(torch.uint8)


def _cache(g, B, hkv, d, cap, page, e4m3):
    """One layer's cache in the layout a program has it in: contiguous [B][Hkv][rows][d], or pages
    [pages][page_rows][Hkv][d] named by a block table in shuffled order."""
    blocks = -(-cap // page) if page else 0
    shape = (B * blocks + 3, page, hkv, d) if page else (B, hkv, cap, d)
    out = {}
    for name in ("k", "v"):
        x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        # a few strong channels in K, rows of uneven size in V: what makes 8 bits hard
        x.normal_(generator=g)
        if name == "k":
            x *= torch.exp(0.4 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)
        else:
            x *= torch.exp(0.5 * torch.randn((*shape[:-1], 1), generator=g, device=DEV)).to(torch.bfloat16)
        if e4m3:
            codes, byte = _quantised(x)
            out[name] = codes
            if page:  # the scales of a head's rows in a page lie together
                byte = byte.transpose(1, 2).contiguous().transpose(1, 2)
            out[name + "_scale"] = byte.view(torch.float8_e8m0fnu)
        else:
            out[name] = x
            out[name + "_scale"] = None
        del x
    out["block_table"] = None
    if page:
        perm = torch.randperm(B * blocks + 3, generator=g, device=DEV)[: B * blocks]
        out["block_table"] = perm.to(torch.int32).reshape(B, blocks).contiguous()
    out["page"] = page
    return out


def _lengths(rng, B, T, cap, ragged):
    t = rng.integers(0 if B > 1 else 1, T + 1, size=B) if ragged else np.full(B, T)
    lo = max(T, cap // 2)
    n = rng.integers(lo, cap + 1, size=B) if ragged else np.full(B, cap)
    return n, t


def _tree(rng, T):
    """Ancestors (each node among its own) of a random tree of T nodes in order, some from the root."""
    words = -(-T // 64)
    m = []
    for t in range(T):
        parent = int(rng.integers(max(-1, t - 12), t)) if t else -1
        m.append((m[parent] if parent >= 0 else 0) | (1 << t))
    return np.array([[(x >> (64 * w)) & (2**64 - 1) for w in range(words)] for x in m], dtype=np.uint64).view(np.int64)


def prepare(case, seed):
    g, rng = _gen(seed), np.random.default_rng(int(seed))
    c = dict(case)
    s = {"case": c}
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "rope":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        R = c["rows"]
        # the projection's output: queries, keys and values of a token side by side
        qkv = torch.randn((R, (hq + 2 * hkv) * d), generator=g, device=DEV).to(dt)
        s["q"] = qkv[:, : hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d : (hq + hkv) * d].unflatten(1, (hkv, d))
        s["pos"] = torch.randint(0, c["far"], (R,), generator=g, device=DEV).to(torch.int32)
        s["inv_freq"] = _inv_freq(c["rot"])
        s["q_weight"] = _weights(g, d, dt) if c["norm"] else None
        s["k_weight"] = _weights(g, d, dt) if c["norm"] else None
        s["q_out"] = torch.zeros((R, hq, d), dtype=dt, device=DEV)
        s["k_out"] = torch.zeros((R, hkv, d), dtype=dt, device=DEV)
        return s
    B = c["B"]
    if c["op"] == "append":
        T = c["T"]
        s.update(_cache(g, B, hkv, d, c["cap"], c["page"], c["e4m3"]))
        n, t = _lengths(rng, B, T, c["cap"], c["ragged"])
        s["n"] = torch.tensor(n, dtype=torch.int32, device=DEV)
        s["t_len"] = torch.tensor(t, dtype=torch.int32, device=DEV) if c["ragged"] else None
        qkv = torch.randn((B, T, (hq + 2 * hkv) * d), generator=g, device=DEV).to(torch.bfloat16)
        s["q"] = qkv[..., : hq * d].unflatten(2, (hq, d)) if c["with_q"] else None
        s["k_new"] = qkv[..., hq * d : (hq + hkv) * d].unflatten(2, (hkv, d))
        s["v_new"] = qkv[..., (hq + hkv) * d :].unflatten(2, (hkv, d))
        s["inv_freq"] = _inv_freq(d) if c["rotate"] else None
        s["q_weight"] = _weights(g, d, torch.bfloat16) if c["norm"] and c["with_q"] else None
        s["k_weight"] = _weights(g, d, torch.bfloat16) if c["norm"] else None
        s["q_out"] = torch.zeros((B, T, hq, d), dtype=torch.bfloat16, device=DEV) if c["with_q"] else None
        return s
    if c["op"] == "read":
        cap, m, sets = c["cap"], c["m"], c["sets"]
        s.update(_cache(g, B, hkv, d, cap, c["page"], True))
        n = rng.integers(max(1, cap // 2), cap + 1, size=B) if B > 1 else np.full(B, cap)
        s["n"] = torch.tensor(n, dtype=torch.int32, device=DEV)
        s["sets"] = None
        if sets:  # ascending, -1 behind a short element's rows, as the selection writes them
            r = torch.rand((B, sets, cap), generator=g, device=DEV)
            r.masked_fill_(torch.arange(cap, device=DEV) >= s["n"][:, None, None], 2.0)
            v, idx = r.topk(min(m, cap), dim=-1, largest=False)
            idx = torch.where(v < 1.5, idx, cap).sort(-1).values
            s["sets"] = torch.where(idx < cap, idx, -1).to(torch.int32)
        h = sets or hkv
        s["k_out"] = torch.zeros((B, h, m, d), dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.zeros((B, h, m, d), dtype=torch.bfloat16, device=DEV)
        return s
    T, n_max = c["T"], c["n"]
    s.update(_cache(g, B, hkv, d, n_max, c["page"], c["e4m3"]))
    n, t = _lengths(rng, B, T, n_max, c["ragged"])
    s["n"] = torch.tensor(n, dtype=torch.int32, device=DEV)
    s["t_len"] = torch.tensor(t, dtype=torch.int32, device=DEV) if c["ragged"] else None
    s["q"] = torch.randn((B, T, hq, d), generator=g, device=DEV).to(torch.bfloat16)
    s["mask"] = torch.from_numpy(np.stack([_tree(rng, T) for _ in range(B)])).to(DEV)
    s["out"] = torch.zeros((B, T, hq, d), dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------ the plain forms


def _f32_of_byte(byte):
    return (byte.view(torch.uint8).to(torch.int32) << 23).view(torch.float32)


def _normed(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _rotated(x, pos, inv_freq, interleaved):
    """x [..., H, d] fp32 rotated by its position [...]: far positions' angles in 64 bits."""
    if inv_freq is None:
        return x
    half = inv_freq.numel()
    ang = pos.double()[..., None, None] * inv_freq.double()
    cos, sin = ang.cos().float(), ang.sin().float()
    if interleaved:
        a, b = x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half : 2 * half]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., 2 * half :]), -1)


def _row_of(s, b, row):
    """Where rows `row` of elements `b` lie: (page or element, row in it)."""
    if not s["page"]:
        return b, row
    return s["block_table"][b, row // s["page"]].long(), row % s["page"]


def _put(s, name, at, x):
    """Writes x [rows][Hkv][d] fp32 at rows `at` of the cache, in the cache's own type."""
    first, row = at
    cache, scale = s[name], s[name + "_scale"]
    put = (first, row) if s["page"] else (first, slice(None), row)
    if scale is None:
        cache[put] = x.to(torch.bfloat16)
        return
    codes, byte = _quantised(x)
    cache.view(torch.uint8)[put] = codes.view(torch.uint8)
    scale.view(torch.uint8)[put] = byte


def _rows(s, name, rows):
    """Rows 0..rows-1 of every element and head as fp32 [B][Hkv][rows][d]."""
    x, scale = s[name], s[name + "_scale"]
    if scale is None:
        x = x.float()
    else:
        x = x.float() * _f32_of_byte(scale)[..., None]
    if s["page"]:
        x = x[s["block_table"].long()].flatten(1, 2).transpose(1, 2)
    return x[:, :, :rows]


def _plain_rope(s):
    c = s["case"]
    for_q = _rotated(_normed(s["q"], s["q_weight"]), s["pos"], s["inv_freq"], c["interleaved"])
    for_k = _rotated(_normed(s["k"], s["k_weight"]), s["pos"], s["inv_freq"], c["interleaved"])
    s["q_out"].copy_(for_q)
    s["k_out"].copy_(for_k)
    return s["q_out"], s["k_out"]


def _plain_append(s):
    B, T = s["k_new"].shape[:2]
    t_len = s["t_len"] if s["t_len"] is not None else torch.full_like(s["n"], T)
    t = torch.arange(T, device=DEV)
    live = t < t_len[:, None]
    row = (s["n"] - t_len)[:, None] + t
    k = _rotated(_normed(s["k_new"], s["k_weight"]), row, s["inv_freq"], False)
    b, at = live.nonzero(as_tuple=True)
    where = _row_of(s, b, row[b, at].long())
    _put(s, "k", where, k[b, at])
    _put(s, "v", where, s["v_new"].float()[b, at])
    out = {name: s[name] for name in ("k", "v", "k_scale", "v_scale") if s[name] is not None}
    if s["q"] is not None:
        q = _rotated(_normed(s["q"], s["q_weight"]), row, s["inv_freq"], False)
        s["q_out"].copy_(torch.where(live[..., None, None], q.to(torch.bfloat16), s["q_out"]))
        out["q"] = s["q_out"]
    return out


def _plain_read(s):
    c = s["case"]
    for name in ("k", "v"):
        x = _rows(s, name, c["cap"])
        if s["sets"] is None:
            live = (torch.arange(c["m"], device=DEV) < s["n"][:, None])[:, None, :, None]
            got = x[:, :, : c["m"]]
        else:
            idx = s["sets"].long()
            live = (idx >= 0)[..., None]
            x = x.repeat_interleave(c["sets"] // c["hkv"], 1)
            got = x.gather(2, idx.clamp(min=0)[..., None].expand(-1, -1, -1, c["d"]))
        out = s[name + "_out"]
        out.copy_(torch.where(live, got.to(torch.bfloat16), out))
    return s["k_out"], s["v_out"]


def _plain_tree(s):
    c = s["case"]
    B, T, hq, d = s["q"].shape
    hkv, N = c["hkv"], c["n"]
    G = hq // hkv
    t_len = s["t_len"] if s["t_len"] is not None else torch.full_like(s["n"], T)
    k, v = _rows(s, "k", N), _rows(s, "v", N)
    q = s["q"].float().view(B, T, hkv, G, d).transpose(1, 2).reshape(B, hkv, T * G, d)
    x = (q @ k.transpose(2, 3)) * d**-0.5
    # node t sees the rows before the draft, and the drafted rows of its mask
    first = s["n"] - t_len
    node = torch.arange(N, device=DEV) - first[:, None]  # [B][N]
    word = (node.clamp(0, T - 1) // 64)[:, None, :].expand(B, T, N)
    bit = (s["mask"].gather(2, word) >> (node.clamp(0, T - 1) % 64)[:, None, :]) & 1
    seen = (node < 0)[:, None, :] | ((node < t_len[:, None])[:, None, :] & (bit != 0))
    seen = seen[:, None, :, None, :].expand(B, hkv, T, G, N).reshape(B, hkv, T * G, N)
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    v = torch.where((node < t_len[:, None])[:, None, :, None], v, 0.0)
    den = p.sum(-1, keepdim=True)
    o = torch.where(den > 0, (p @ v) / den, 0.0)
    o = o.view(B, hkv, T, G, d).transpose(1, 2).reshape(B, T, hq, d).to(torch.bfloat16)
    live = (torch.arange(T, device=DEV) < t_len[:, None])[..., None, None]
    s["out"].copy_(torch.where(live, o, s["out"]))
    return s["out"]


# ------------------------------------------------------------------ a pass


def _handle(s):
    """The description of the layer's cache that a program keeps beside it."""
    if "cache" not in s:
        from hybrid_head_sparse_b200 import lyc
        s["cache"] = lyc.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["block_table"])
    return s["cache"]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "tree": _plain_tree}[op](s)
    from hybrid_head_sparse_b200 import lyc
    if op == "rope":
        lyc.qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], s["q_out"], s["k_out"],
                         q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"])
        return s["q_out"], s["k_out"]
    if op == "append":
        lyc.cache_append(_handle(s), s["n"], s["k_new"], s["v_new"], t_len=s["t_len"], q=s["q"], q_out=s["q_out"],
                         inv_freq=s["inv_freq"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
        out = {name: s[name] for name in ("k", "v", "k_scale", "v_scale") if s[name] is not None}
        if s["q"] is not None:
            out["q"] = s["q_out"]
        return out
    if op == "read":
        lyc.cache_read(_handle(s), s["n"], s["k_out"], s["v_out"], sets=s["sets"])
        return s["k_out"], s["v_out"]
    lyc.tree_attention(s["q"], _handle(s), s["n"], s["out"], mask=s["mask"], t_len=s["t_len"])
    return s["out"]


def _mean_len(c, cap):
    """The expected rows of an element as prepare() draws them."""
    lo = max(c.get("T", 1), cap // 2)
    return (lo + cap) / 2 if c.get("ragged") else cap


def work(case):
    """Each input read once and each output written once, at the expected lengths of ragged cases."""
    c = case
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "rope":
        es = 2 if c["dtype"] == "bf16" else 4
        x = c["rows"] * (hq + hkv) * d
        return {"bytes": 2 * x * es + 4 * c["rows"], "flops": x * ((4 if c["norm"] else 0) + 3 * c["rot"] / d)}
    if c["op"] == "append":
        share = 0.5 if c["ragged"] else 1.0
        rows = c["B"] * c["T"] * share
        kv = rows * hkv * d
        q = rows * hq * d if c["with_q"] else 0
        held = kv * (1 + 1 / d) if c["e4m3"] else 2 * kv
        per = (4 if c["norm"] else 0) + (3 if c["rotate"] else 0)
        return {"bytes": 2 * q * 2 + 2 * kv * 2 + 2 * held, "flops": (q + kv) * per + 2 * kv * 2}
    if c["op"] == "read":
        n = c["cap"] if c["B"] == 1 else 0.75 * c["cap"]
        rows = c["B"] * (c["sets"] or hkv) * min(c["m"], n)
        idx = 4 * c["B"] * c["sets"] * c["m"]
        # sets of one KV head share its rows: each row is read from the cache once
        distinct = min(rows, c["B"] * hkv * n)
        return {"bytes": 2 * distinct * (d + 1) + 2 * rows * d * 2 + idx, "flops": 2 * rows * d}
    n = _mean_len(c, c["n"])
    T = c["T"] * (0.5 if c["ragged"] else 1.0)
    row = 2 * (d + 1) if c["e4m3"] else 4 * d
    words = -(-c["T"] // 64)
    return {"bytes": c["B"] * (n * hkv * row + 2 * T * hq * d * 2 + 8 * T * words),
            "flops": 4.0 * d * c["B"] * T * hq * n}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_head(x, w, pos, freq, interleaved):
    """x [R][H][d] (any type), pos [R]: norm and rotation as complex numbers, in float64."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    if freq is None:
        return x
    h = freq.numel()
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV), torch.outer(pos.double(), freq.double()))[:, None, :]
    pairs = x[..., : 2 * h].reshape(*x.shape[:-1], h, 2) if interleaved else x[..., : 2 * h].reshape(*x.shape[:-1], 2, h).transpose(-1, -2)
    z = torch.view_as_real(torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * turn)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat((z, x[..., 2 * h :]), -1)


def _exact_codes(x):
    """The e4m3 code values and the scale of float64 rows: nearest of the type's values, ties to even."""
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2((amax / 448.0).clamp(min=2.0**-100)))
    e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where((amax <= 448.0 * torch.exp2(e - 1)) & (e > -100), e - 1, e)
    y = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)
    return torch.round(y / step) * step, torch.exp2(e[..., 0])


def _element(s, name, b, rows):
    """Rows 0..rows-1 of element b as float64 [Hkv][rows][d]."""
    x = s[name].to(torch.float32)
    scale = None if s[name + "_scale"] is None else s[name + "_scale"].view(torch.uint8).double()
    if s["page"]:
        pages = s["block_table"][b].tolist()
        x = torch.cat([x[p] for p in pages])[:rows].transpose(0, 1)
        scale = None if scale is None else torch.cat([scale[p] for p in pages])[:rows].transpose(0, 1)
    else:
        x = x[b][:, :rows]
        scale = None if scale is None else scale[b][:, :rows]
    x = x.double()
    return x if scale is None else x * torch.exp2(scale - 127.0)[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return (_exact_head(s["q"], s["q_weight"], s["pos"], s["inv_freq"], c["interleaved"]),
                _exact_head(s["k"], s["k_weight"], s["pos"], s["inv_freq"], c["interleaved"]))
    n = s["n"].tolist()
    t_len = s["t_len"].tolist() if s.get("t_len") is not None else [c.get("T", 0)] * c["B"]
    if c["op"] == "append":
        out = {}
        for name in ("k", "v"):
            out[name] = s[name].to(torch.float32).double()
            if c["e4m3"]:
                out[name + "_scale"] = torch.exp2(s[name + "_scale"].view(torch.uint8).double() - 127.0)
        if s["q"] is not None:
            out["q"] = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        for b in range(c["B"]):
            cnt = t_len[b]
            if cnt == 0:
                continue
            pos = torch.arange(n[b] - cnt, n[b], device=DEV)
            new = {"k": _exact_head(s["k_new"][b, :cnt], s["k_weight"], pos, s["inv_freq"], False),
                   "v": s["v_new"][b, :cnt].double()}
            if s["q"] is not None:
                out["q"][b, :cnt] = _exact_head(s["q"][b, :cnt], s["q_weight"], pos, s["inv_freq"], False)
            page = pos // c["page"] if c["page"] else pos
            for name in ("k", "v"):
                vals, sc = _exact_codes(new[name]) if c["e4m3"] else (new[name], None)
                if c["page"]:
                    at = (s["block_table"][b].long()[page], pos % c["page"])
                    out[name][at] = vals
                    if sc is not None:
                        out[name + "_scale"][at] = sc
                else:
                    out[name][b, :, pos] = vals.transpose(0, 1)
                    if sc is not None:
                        out[name + "_scale"][b, :, pos] = sc.transpose(0, 1)
        return out
    if c["op"] == "read":
        out = {}
        for name in ("k", "v"):
            o = torch.zeros(s[name + "_out"].shape, dtype=torch.float64, device=DEV)
            for b in range(c["B"]):
                x = _element(s, name, b, c["cap"])
                for h in range(o.shape[1]):
                    if s["sets"] is None:
                        live = min(c["m"], n[b])
                        o[b, h, :live] = x[h, :live]
                    else:
                        idx = s["sets"][b, h]
                        idx = idx[idx >= 0].long()
                        o[b, h, : idx.numel()] = x[h // (c["sets"] // c["hkv"]), idx]
            out[name] = o
        return out["k"], out["v"]
    B, T, hq, d = s["q"].shape
    G = hq // c["hkv"]
    out = torch.zeros((B, T, hq, d), dtype=torch.float64, device=DEV)
    for b in range(B):
        cnt, first = t_len[b], n[b] - t_len[b]
        if cnt == 0:
            continue
        k, v = _element(s, "k", b, n[b]), _element(s, "v", b, n[b])
        words = s["mask"][b].cpu().numpy().view(np.uint64)
        sees = np.array([[(int(words[t, j // 64]) >> (j % 64)) & 1 for j in range(cnt)] for t in range(cnt)], dtype=bool)
        block = torch.ones((cnt, n[b]), dtype=torch.bool, device=DEV)
        block[:, first:] = torch.from_numpy(sees).to(DEV)
        for h in range(hq):
            x = s["q"][b, :cnt, h].double() @ k[h // G].T / math.sqrt(d)
            x = torch.where(block, x, torch.tensor(-math.inf, dtype=torch.float64, device=DEV))
            out[b, :cnt, h] = torch.softmax(x, -1) @ v[h // G]
    return out
