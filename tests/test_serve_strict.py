"""The serving operators' second oracle (tests/serve_strict.py) on the host: the two
oracles agree, the bound takes the arithmetic that it is for and turns away coarser
ones (probabilities in bf16, a tail that is lost)."""
from __future__ import annotations

import math
from types import SimpleNamespace

import pytest
import torch

from tests import serve_oracle as SO
from tests import serve_strict as SS


def cache_of(seed, B, hkv, rows, d, spread):
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        x = torch.randn((B, hkv, rows, d), generator=g) * torch.exp2(spread * torch.randn((B, hkv, rows, 1), generator=g))
        code, byte = SS.e4m3_row(x)
        out.append((code.to(torch.uint8).view(torch.float8_e4m3fn), byte.to(torch.uint8)))
    (k, ks), (v, vs) = out
    v.view(torch.uint8).bitwise_and_(0x7F)  # one sign: roundings do not cancel against each other
    return SimpleNamespace(tensors=(k, v, ks, vs, None), heads=hkv, e4m3=True)


def attend(q, cache, n, to16, lost):
    """The attention with probabilities * scale under their largest rounded by to16 and
    dropped below `lost`; sums as they are."""
    k, v, ks, vs, _ = cache.tensors
    B, T, Hq, d = q.shape
    out = torch.zeros(q.shape, dtype=torch.float64)
    for b in range(B):
        for h in range(Hq):
            g = h // (Hq // cache.heads)
            scale = torch.exp2(vs[b, g, :n].double() - 127)
            K = k[b, g, :n].double() * torch.exp2(ks[b, g, :n].double() - 127)[:, None]
            z = q[b, :, h].double() @ K.T * d**-0.5
            z[:, n - T:] = torch.where(torch.tril(torch.ones(T, T)).bool(), z[:, n - T:], -math.inf)
            p = torch.exp(z - z.amax(-1, keepdim=True))
            w = p * scale
            top = w.amax(-1, keepdim=True)
            w = torch.where(w < lost * top, 0.0, to16(w / top))
            out[b, :, h] = (w @ v[b, g, :n].double()) * top / p.sum(-1, keepdim=True)
    return out.to(torch.bfloat16)


@pytest.mark.parametrize("d,spread", [(64, 0.5), (128, 1.5)])
def test_the_bound_tells_fp16_from_bf16(d, spread):
    n, T = 700, 3
    cache = cache_of(d, 1, 2, n, d, spread)
    q = torch.randn((1, T, 4, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16) * 0.25
    want, bound = SS.tree(q, cache, [n], [T], None, d**-0.5)
    first, loose = SO.tree(q, cache, [n], [T], None, d**-0.5)
    assert torch.allclose(want, first, rtol=1e-12, atol=0)
    SO.close(attend(q, cache, n, lambda x: (x * 2.0**15).half().double() / 2.0**15, 2.0**-30), want, bound, "fp16")
    # one probability each, the worst a rounding to 8 bits can do: inside the first bound, outside this one
    bf16 = attend(q, cache, n, lambda x: x * (1 + 2.0**-8), 0.0)
    SO.close(bf16, want, loose, "bf16")
    with pytest.raises(AssertionError):
        SO.close(bf16, want, bound, "bf16")


def test_the_bound_sees_a_lost_tail():
    n, d = 4096, 64
    cache = cache_of(3, 1, 1, n, d, 0.0)
    k, v, ks, vs, _ = cache.tensors
    k.view(torch.uint8).zero_()
    ks.fill_(127)
    vs.fill_(127)
    k[0, 0, 1:, 0] = torch.tensor(-14.0).to(torch.float8_e4m3fn)
    q = torch.zeros((1, 1, 1, d), dtype=torch.bfloat16)
    q[..., 0] = math.log(2.0) * d**0.5
    want, bound = SS.tree(q, cache, [n], [1], None, d**-0.5)
    SO.close(attend(q, cache, n, lambda x: x, 2.0**-30), want, bound, "kept")
    with pytest.raises(AssertionError):
        SO.close(attend(q, cache, n, lambda x: x, 2.0**-13), want, bound, "lost")


def test_the_two_oracles_of_the_8_bit_row_agree():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((500, 64), generator=g, dtype=torch.float64)
    x *= torch.exp2(torch.randint(-120, 119, (500, 1), generator=g).double())
    x[0], x[1, 3], x[2, 5] = 0.0, math.nan, math.inf
    code, byte = SS.e4m3_row(x)
    value, byte2 = SO.e4m3_row(x)
    assert torch.equal(byte, byte2)
    assert torch.equal(torch.where(code >= 128, -1.0, 1.0) * SS.magnitudes()[code & 127], value)
    # every magnitude is the type's own
    assert torch.equal(SS.magnitudes().float(), torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float())
