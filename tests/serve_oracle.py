"""The serving operators (norm and rotation, cache append and read, tree
attention) written out in float64 on the host, with the bound that their
arithmetic gives each result.  Test infrastructure: shares no code with the
library.  Unit roundoffs: bf16 2^-8, fp16 2^-11, fp32 2^-24, e4m3 2^-4."""
from __future__ import annotations

import math

import numpy as np
import torch

U32, U16, UB, U8 = 2.0**-24, 2.0**-11, 2.0**-8, 2.0**-4


def norm_rope(x, w, pos, freq, interleaved, eps):
    """x [..., H, d] with pos [...]: (y, slack) in float64.  slack bounds what
    fp32 arithmetic adds before the last rounding: with |a|, |b| the normed pair,
    (|a| + |b|) times 32 roundoffs (the sum of d squares in a tree of at most 13
    additions, half of which reaches rsqrt; rsqrt 4, two products, the turn's
    rounding pi, sincospi 4, the pair's products and sum 4)."""
    x = x.detach().cpu().double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.cpu().double()
    if freq is None:
        return x, x.abs() * 32 * U32
    h = freq.numel()
    ang = pos.cpu().double()[..., None, None] * freq.cpu().double()
    c, s = torch.cos(ang), torch.sin(ang)
    y, m = x.clone(), x.abs().clone()
    for i in range(h):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        a, b = x[..., ia], x[..., ib]
        y[..., ia] = a * c[..., i] - b * s[..., i]
        y[..., ib] = b * c[..., i] + a * s[..., i]
        m[..., ia] = m[..., ib] = a.abs() + b.abs()
    return y, m * 32 * U32


def e4m3_row(x):
    """Definition of the 8-bit row for float64 x [..., d]: (codes' values, scale byte)."""
    x = x.double()
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    e = torch.full_like(amax, -100.0)
    ok = (amax > 0) & ~bad
    e[ok] = torch.ceil(torch.log2(amax[ok] / 448.0))
    e[ok & (amax > 448.0 * torch.exp2(e))] += 1
    e[ok & (amax <= 448.0 * torch.exp2(e - 1))] -= 1
    e = e.clamp(min=-100.0)
    y = x / torch.exp2(e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)
    code = torch.round(y / step) * step
    code[bad] = 0.0
    byte = e + 127
    byte[bad] = 255
    return code, byte.to(torch.int64)


def rows_of(cache, b, count):
    """Rows 0..count-1 of element b of a KvCache as float64 K, V [Hkv][count][d]
    and a mask of the rows whose page exists."""
    k, v, ks, vs, bt = cache.tensors
    out, have = [], torch.ones(count, dtype=torch.bool)
    for x, sc in ((k, ks), (v, vs)):
        x = x.detach().cpu().float().double()
        if sc is not None:
            byte = sc.cpu().view(torch.uint8).double()
            x = x * torch.where(byte == 255, math.nan, torch.exp2(byte - 127))[..., None]
        if bt is None:
            out.append(x[b, :, :count])
        else:
            page_rows = x.shape[1]
            i = torch.arange(count)
            page = bt.cpu()[b].long()[i // page_rows]
            have = (page >= 0) & (page < x.shape[0])
            out.append(x[page.clamp(0, x.shape[0] - 1), i % page_rows].transpose(0, 1))
    return out[0], out[1], have


def sees(mask, b, t, j):
    if mask is None:
        return j <= t
    return bool((int(mask[b, t, j // 64]) >> (j % 64)) & 1)


def tree(q, cache, n, t_len, mask, scale):
    """(out, bound) [B][T][Hq][d] float64; NaN where a query is padding.

    Bound: each probability carries its rounding u and e^delta - 1.  u is bf16's
    for both caches: p(1 + r), |r| <= 2^-8 (8 significant bits, to nearest); the fp16
    of e4m3 rows is within that (2^-11).  delta is what fp32
    does to a logit: d + 8 roundoffs of sum |q k| scale, and four of the logit in
    log2 units (at most 1.5 times it, plus 130 for a scale's exponent); over an e4m3
    cache also what a query's elements lose as fp16 under the row's largest, scaled
    to [1, 2): 8 significant bits end at fp16's last place 2^-24 for elements under
    2^-17, which are off by half of it.  The output has its own rounding."""
    q = q.detach().cpu().double()
    B, T, Hq, d = q.shape
    G = Hq // cache.heads
    out = torch.full(q.shape, math.nan, dtype=torch.float64)
    bound = torch.zeros_like(out)
    m = None if mask is None else mask.cpu().numpy().astype(np.int64).view(np.uint64)
    u = UB
    for b in range(B):
        nb, cnt = int(n[b]), int(t_len[b])
        if cnt <= 0 or nb < cnt:
            continue
        K, V, have = rows_of(cache, b, nb)
        vis = torch.zeros((cnt, nb), dtype=torch.bool)
        vis[:, : nb - cnt] = True
        for t in range(cnt):
            for j in range(cnt):
                vis[t, nb - cnt + j] = sees(m, b, t, j)
        vis &= have
        for h in range(Hq):
            k, v = K[h // G], V[h // G]
            x = q[b, :cnt, h] @ k.nan_to_num().T * scale
            x = torch.where(torch.isnan(k).any(-1), math.nan, x)
            x = torch.where(vis, x, -math.inf)
            top = x.nan_to_num(nan=-math.inf).amax(-1, keepdim=True).clamp(min=-1e300)
            p = torch.exp(x - top)
            p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
            o = torch.zeros((cnt, d), dtype=torch.float64)
            for t in range(cnt):  # only the rows seen: 0 * NaN is not in the definition
                o[t] = p[t, vis[t]] @ v[vis[t]]
            a = p.nan_to_num() @ v.abs().nan_to_num(posinf=0.0)
            mag = (q[b, :cnt, h].abs() @ k.abs().nan_to_num(posinf=0.0).T * scale).amax(-1, keepdim=True)
            lost = 0.0
            if cache.e4m3:
                top_q = torch.exp2(torch.floor(torch.log2(q[b, :cnt, h].abs().amax(-1, keepdim=True).clamp(min=1e-300))))
                small = (q[b, :cnt, h].abs() < 2.0**-17 * top_q).double() * 2.0**-25 * top_q
                lost = (small @ k.abs().nan_to_num(posinf=0.0).T * scale).amax(-1, keepdim=True)
            delta = lost + (d + 8) * U32 * mag + 4 * U32 * (1.5 * mag + (130 if cache.e4m3 else 0)) + 8 * U32
            out[b, :cnt, h] = o
            bound[b, :cnt, h] = a * (u + 2 * torch.expm1(delta)) * (1 + 2 * UB) + UB * o.abs() * (1 + UB)
    return out, bound


def close(got, want, bound, what):
    """Every value within its bound; NaN and infinities in the same places."""
    got = got.detach().cpu().double()
    want, bound = want.double(), bound.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), f"{what}: infinities differ"
    over = ((got - want).abs() - bound)[fin]
    assert over.numel() == 0 or float(over.max()) <= 0.0, \
        f"{what}: {int((over > 0).sum())} of {over.numel()} values out of bound, worst by {float(over.max()):.3g}"
