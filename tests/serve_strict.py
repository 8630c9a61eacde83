"""Tree attention and 8-bit rows in float64, a second time: with the bound that
each cache's own roundings give (fp16 probabilities over e4m3 rows, where
tests/serve_oracle.py allows bf16's to both), and the 8-bit row found by search
over the type's 127 magnitudes.  Runs on the device of its inputs.  Test
infrastructure: shares no code with the library or with the other oracle."""
from __future__ import annotations

import math

import torch

U32, U16, UB = 2.0**-24, 2.0**-11, 2.0**-8
LOST = 2.0**-30  # of a query's largest probability * scale: what fp16 probabilities may be off by


def magnitudes():
    """The e4m3 magnitudes by code: 0 .. 7 times 2^-9, then 1.mmm times 2^-6 .. 2^8."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0**-9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return torch.tensor(out, dtype=torch.float64)


def e4m3_row(x):
    """(codes as bytes, scale byte) of float64 rows x [..., d], by search: the first
    e >= -100 with max|x| <= 448 * 2^e, then the nearest magnitude of each element,
    the one of the even code where two are as near."""
    x = x.double().cpu()
    amax = x.abs().amax(-1)
    edges = 448.0 * torch.exp2(torch.arange(-100, 121, dtype=torch.float64))
    i = torch.searchsorted(edges, amax.nan_to_num(nan=0.0, posinf=0.0))  # the first edge that is not below
    table = magnitudes()
    y = x.abs().nan_to_num(nan=0.0, posinf=0.0) / torch.exp2(i.double() - 100)[..., None]
    hi = torch.searchsorted(table, y).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    over, under = table[hi] - y, y - table[lo]
    code = torch.where((under < over) | ((under == over) & (lo % 2 == 0)), lo, hi)
    code = code + 128 * torch.signbit(x).long()
    bad = ~torch.isfinite(amax)
    byte = torch.where(bad, 255, i + 27)
    return torch.where(bad[..., None], 0, code), byte


def _rows(cache, b, count):
    """Rows of element b: values, |codes| and scales of V's (1 where there are none)
    [Hkv][count](d), and which rows there are."""
    k, v, ks, vs, bt = cache.tensors
    i = torch.arange(count, device=k.device)
    if bt is None:
        at, have = (b, slice(None), i), torch.ones(count, dtype=torch.bool, device=k.device)
    else:
        page = bt[b].long()[i // k.shape[1]]
        have = (page >= 0) & (page < k.shape[0])
        at = (page.clamp(0, k.shape[0] - 1), i % k.shape[1])
    table = torch.cat([magnitudes(), torch.tensor([math.nan], dtype=torch.float64)]).to(k.device)
    out = []
    for x, s in ((k, ks), (v, vs)):
        if s is None:
            val = x[at].double()
            mag, scale = val.abs(), torch.ones(val.shape[:2], dtype=torch.float64, device=k.device)
        else:
            code = x.view(torch.uint8)[at].long()
            byte = s.view(torch.uint8)[at].long()
            scale = torch.where(byte == 255, math.nan, torch.exp2((byte if x is k else byte.clamp(min=27)).double() - 127))
            mag = table[code & 127]
            val = torch.where(code >= 128, -mag, mag) * scale[..., None]
        if bt is not None:
            val, mag, scale = val.transpose(0, 1), mag.transpose(0, 1), scale.transpose(0, 1)
        out.append((val, mag, scale))
    return out[0][0], out[1], have


def tree(q, cache, n, t_len, mask, scale, lost=LOST):
    """(out, bound) [B][T][Hq][d] float64, NaN where a query is padding.

    Bound: a probability p is rounded to p (1 + r), |r| <= 2^-8 (bf16 rows) or 2^-11
    (e4m3); over e4m3 rows, whose p * scale goes to fp16, also by `lost` of the query's
    largest p * scale where that is subnormal.  A logit is off by delta: d + 8
    fp32 roundoffs of sum |q k| scale, four of the logit in log2 units (at most 1.5
    times it, plus 130 for a scale's exponent), and over e4m3 rows by what the query's
    elements below 2^-17 of its largest lose in fp16 (2^-25 of that).  The output is
    rounded to bf16."""
    B, T, Hq, d = q.shape
    G, dev = Hq // cache.heads, q.device
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=dev)
    bound = torch.zeros_like(out)
    u = U16 if cache.e4m3 else UB
    for b in range(B):
        nb, cnt = int(n[b]), int(t_len[b])
        if cnt <= 0 or nb < cnt:
            continue
        K, (V, codes, vscale), have = _rows(cache, b, nb)
        vis = torch.ones((cnt, nb), dtype=torch.bool, device=dev)
        j = torch.arange(cnt, device=dev)
        if mask is None:
            vis[:, nb - cnt:] = j <= j[:, None]
        else:
            vis[:, nb - cnt:] = ((mask[b, :cnt].view(torch.int64)[:, j // 64] >> (j % 64)) & 1).bool()
        vis &= have
        for h in range(Hq):
            g = h // G
            k, v, w, sc = K[g], V[g], codes[g], vscale[g]
            x = q[b, :cnt, h].double()
            z = (x @ k.nan_to_num().T) * scale
            z[:, torch.isnan(k).any(-1)] = math.nan
            z = torch.where(vis, z, -math.inf)
            top = z.nan_to_num(nan=-math.inf).amax(-1, keepdim=True).clamp(min=-1e300)
            p = torch.exp(z - top)
            p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
            # 0 * NaN is not in the definition: finite values by the product, others where seen
            odd = ~torch.isfinite(v)
            o = p @ torch.where(odd, 0.0, v)
            for r in odd.any(-1).nonzero().flatten().tolist():
                o[vis[:, r]] = o[vis[:, r]] + torch.where(odd[r], v[r], 0.0)
            fin = torch.where(odd, 0.0, v).abs()
            p = p.nan_to_num()
            ka = k.abs().nan_to_num(posinf=0.0).T
            mag = torch.where(vis, x.abs() @ ka * scale, 0.0).amax(-1, keepdim=True)
            delta = (d + 8) * U32 * mag + 4 * U32 * (1.5 * mag + (130 if cache.e4m3 else 0)) + 8 * U32
            off = 0.0
            if cache.e4m3:
                big = torch.exp2(torch.floor(torch.log2(x.abs().amax(-1, keepdim=True).clamp(min=1e-300))))
                small = (x.abs() < 2.0**-17 * big).double() * 2.0**-25 * big
                delta = delta + torch.where(vis, small @ ka * scale, 0.0).amax(-1, keepdim=True)
                most = (p * sc.nan_to_num()).amax(-1, keepdim=True)
                off = lost * most * (vis.double() @ torch.where(odd, 0.0, w.nan_to_num()))
            out[b, :cnt, h] = o
            bound[b, :cnt, h] = ((p @ fin) * (u + 2 * torch.expm1(delta)) + off) * (1 + 2 * UB) + UB * o.abs() * (1 + UB)
    return out, bound
