"""The serving operators (include/lyc.h, "Serving operators") on a B200 against
float64 (tests/serve_oracle.py), at the sizes, masks and layouts where they can
go wrong, and run together as a program uses them."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from tests import serve_oracle as SO

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lyc():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from hybrid_head_sparse_b200 import lyc as m
    m.load()
    return m


def randn(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def inv_freq(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def random_tree(rng, B, T, empty=()):
    """int64 [B][T][W] ancestor masks; nodes in `empty` see nothing."""
    W = -(-T // 64)
    m = np.zeros((B, T, W), dtype=np.uint64)
    for b in range(B):
        seen = []
        for t in range(T):
            parent = int(rng.integers(-1, t)) if t else -1
            s = (seen[parent] if parent >= 0 else 0) | (1 << t)
            seen.append(s)
            for w in range(W):
                m[b, t, w] = 0 if t in empty else (s >> (64 * w)) & (2**64 - 1)
    return torch.from_numpy(m.view(np.int64)).cuda()


def block_table(rng, B, blocks, extra=2):
    pages = B * blocks + extra
    return i32(rng.permutation(pages)[: B * blocks].reshape(B, blocks).tolist()), pages


def fill(lyc, B, hkv, d, cap, page, e4m3, seed):
    """A cache whose every row holds a value, unused pages and rows NaN (bf16) or
    NaN scales (e4m3)."""
    rng = np.random.default_rng(seed)
    bt, pages = (None, 0) if not page else block_table(rng, B, -(-cap // page))
    cache = lyc.KvCache.empty(B, hkv, d, rows=cap, page_rows=page, num_pages=pages, block_table=bt, e4m3=e4m3)
    k, v, ks, vs, _ = cache.tensors
    for x, s, sd in ((k, ks, seed), (v, vs, seed + 1)):
        val = randn(sd, *x.shape).float() * torch.exp(0.7 * randn(sd + 7, *x.shape[:3], 1).float())
        if e4m3:
            code, byte = SO.e4m3_row(val.cpu())
            x.copy_(code.float().cuda().to(torch.float8_e4m3fn))
            s.view(torch.uint8).copy_(byte.to(torch.uint8).cuda())
        else:
            x.copy_(val.to(BF))
    return cache


def poison_past(cache, n):
    """Rows at and past n[b], and pages no element uses: NaN (bf16) or NaN scales."""
    k, v, ks, vs, bt = cache.tensors
    if bt is None:
        for b, nb in enumerate(n):
            if ks is None:
                k[b, :, nb:] = math.nan
                v[b, :, nb:] = math.nan
            else:
                ks.view(torch.uint8)[b, :, nb:] = 255
                vs.view(torch.uint8)[b, :, nb:] = 255
        return
    page_rows = k.shape[1]
    used = torch.zeros(k.shape[:2], dtype=torch.bool)
    table = bt.cpu()
    for b, nb in enumerate(n):
        for i in range(nb):
            p = int(table[b, i // page_rows])
            if 0 <= p < k.shape[0]:
                used[p, i % page_rows] = True
    free = (~used).cuda()
    if ks is None:
        k[free] = math.nan
        v[free] = math.nan
    else:
        ks.view(torch.uint8)[free] = 255
        vs.view(torch.uint8)[free] = 255


# ------------------------------------------------------------------ norm and rotation


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rows,hq,hkv,d,rot,inter,norm", [
    (1, 32, 8, 128, 128, False, True),
    (7, 5, 1, 128, 128, True, True),
    (130, 16, 2, 64, 64, False, False),
    (33, 3, 3, 64, 32, True, True),
    (19, 8, 4, 128, 48, False, True),
    (5, 4, 2, 64, 16, False, True),
    (3, 1, 1, 128, 0, False, True),
    (1025, 2, 1, 64, 48, True, False),
])
def test_norm_rope(lyc, dtype, rows, hq, hkv, d, rot, inter, norm):
    qkv = randn(rows + d, rows, (hq + 2 * hkv) * d, dtype=dtype)
    q, k = qkv[:, : hq * d].unflatten(1, (hq, d)), qkv[:, hq * d: (hq + hkv) * d].unflatten(1, (hkv, d))
    pos = torch.randint(0, 655360, (rows,), device="cuda", dtype=torch.int32)
    pos[0] = 655359
    freq = inv_freq(rot) if rot else None
    wq, wk = (1 + randn(3, d, scale=0.2).float()).to(dtype), (1 + randn(4, d, scale=0.2).float()).to(dtype)
    qo = torch.full((rows, hq, d), math.nan, dtype=dtype, device="cuda")
    ko = torch.full((rows, hkv, d), math.nan, dtype=dtype, device="cuda")
    lyc.qk_norm_rope(q, k, pos, freq, qo, ko, wq if norm else None, wk if norm else None, eps=1e-5, interleaved=inter)
    u = SO.UB if dtype == BF else SO.U32
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        y, slack = SO.norm_rope(x, w if norm else None, pos, freq, inter, 1e-5)
        SO.close(got, y, y.abs() * u + slack * (1 + u), "norm and rotation")


def test_norm_rope_in_place_padding_strides_and_one_side(lyc):
    """In place; rows of negative position left alone; outputs in another order;
    only k; zero rows; a row of zeros, of NaN and of infinities."""
    rows, hq, hkv, d = 9, 4, 2, 128
    q, k = randn(1, rows, hq, d), randn(2, rows, hkv, d)
    q[3] = 0
    q[4, 1, 5] = math.nan
    k[5, 0, 7] = math.inf
    pos = i32([5, -1, 0, 9, 2, 3, 1000, -7, 8])
    w, freq = randn(3, d), inv_freq(d)
    want_q, sq = SO.norm_rope(q, w, pos, freq, False, 1e-6)
    want_k, sk = SO.norm_rope(k, w, pos, freq, False, 1e-6)
    q0, k0 = q.clone(), k.clone()
    out_t = torch.full((hkv, rows, d), 7.0, dtype=BF, device="cuda")  # heads outermost
    lyc.qk_norm_rope(q, k, pos, freq, q, out_t.transpose(0, 1), w, w)
    live = [0, 2, 3, 6, 8]
    SO.close(q[live], want_q[live], (want_q.abs() * SO.UB + 2 * sq)[live], "in place")
    assert torch.equal(q[[1, 7]], q0[[1, 7]])
    assert torch.equal(out_t.transpose(0, 1)[[1, 7]], torch.full((2, hkv, d), 7.0, dtype=BF, device="cuda"))
    SO.close(out_t.transpose(0, 1)[live], want_k[live], (want_k.abs() * SO.UB + 2 * sk)[live], "strided output")
    assert torch.isnan(q[4, 1]).all() and torch.isfinite(q[4, 0].float()).all()  # a NaN stays in its head
    assert not torch.isfinite(out_t[0, 5].float()).all() and torch.isfinite(out_t[1, 5].float()).all()
    ko = torch.zeros_like(k)
    lyc.qk_norm_rope(None, k, pos, freq, None, ko, None, w)
    SO.close(ko[live], want_k[live], (want_k.abs() * SO.UB + 2 * sk)[live], "only k")
    assert torch.equal(k, k0)
    lyc.qk_norm_rope(q[:0], k[:0], pos[:0], freq, q[:0], k[:0], w, w)


# ------------------------------------------------------------------ append and read


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("B,T,hq,hkv,d,cap,page,norm,rot,inter", [
    (1, 1, 4, 2, 128, 1, 0, True, 128, False),
    (3, 5, 8, 2, 64, 40, 0, True, 64, True),
    (2, 17, 5, 1, 128, 100, 7, False, 128, False),
    (4, 33, 4, 4, 64, 64, 16, True, 32, False),
    (2, 130, 2, 2, 128, 300, 64, True, 0, False),
    (2, 3, 2, 2, 64, 9, 1, False, 0, False),
])
def test_append_then_read(lyc, e4m3, B, T, hq, hkv, d, cap, page, norm, rot, inter):
    rng = np.random.default_rng(T)
    cache = fill(lyc, B, hkv, d, cap, page, e4m3, seed=T)
    before = [x.clone() if x is None else x.view(torch.uint8 if e4m3 else torch.int16).clone()
              for x in cache.tensors[:2]]
    cnt = [T] + [int(rng.integers(0, T + 1)) for _ in range(B - 1)]
    real_cap = cap if not page else -(-cap // page) * page
    n = [int(rng.integers(c, real_cap + 1)) for c in cnt]
    n[0] = real_cap  # up to the very last row
    qkv = randn(T + 1, B, T, (hq + 2 * hkv) * d)
    q = qkv[..., : hq * d].unflatten(2, (hq, d))
    k = qkv[..., hq * d: (hq + hkv) * d].unflatten(2, (hkv, d))
    v = qkv[..., (hq + hkv) * d:].unflatten(2, (hkv, d))
    w = (1 + randn(9, d, scale=0.2).float()).to(BF) if norm else None
    freq = inv_freq(rot) if rot else None
    qo = torch.full((B, T, hq, d), 3.0, dtype=BF, device="cuda")
    st = status_word()
    lyc.cache_append(cache, i32(n), k, v, t_len=i32(cnt), q=q, q_out=qo, inv_freq=freq, q_weight=w, k_weight=w,
                     eps=1e-6, interleaved=inter, status=st)
    assert int(st) == 0
    pos = torch.tensor(n)[:, None] - torch.tensor(cnt)[:, None] + torch.arange(T)
    want_q, sq = SO.norm_rope(q, w, pos, freq, inter, 1e-6)
    want_k, sk = SO.norm_rope(k, w, pos, freq, inter, 1e-6)
    m = max(n)
    ko = torch.full((B, hkv, m, d), 5.0, dtype=torch.float32, device="cuda")
    vo = ko.clone()
    lyc.cache_read(cache, i32(n), ko, vo, status=st)
    assert int(st) == 0
    written = torch.zeros(cache.tensors[0].shape[:3], dtype=torch.bool)  # rows of the storage
    for b in range(B):
        c, first = cnt[b], n[b] - cnt[b]
        SO.close(qo[b, :c], want_q[b, :c], (want_q.abs() * SO.UB + 2 * sq)[b, :c], "q")
        assert bool((qo[b, c:] == 3.0).all())
        assert bool((ko[b, :, n[b]:] == 5.0).all()) and bool((vo[b, :, n[b]:] == 5.0).all())
        got_k, got_v = ko[b, :, first:n[b]].transpose(0, 1), vo[b, :, first:n[b]].transpose(0, 1)
        if e4m3:
            code, byte = SO.e4m3_row(v[b, :c].cpu())
            exact = code * torch.exp2(byte.double() - 127)[..., None]
            assert torch.equal(got_v.cpu().double(), exact)  # bf16 values: the definition to the bit
            _, kb = SO.e4m3_row(want_k[b, :c])
            # half a step of the code (2^-4 of it, 2^-10 units below the normal codes); a
            # scale next to its border may come out a factor of two larger
            tol = want_k[b, :c].abs() * SO.U8 + 2.0**-9 * torch.exp2(kb.double() - 127)[..., None] + 2 * sk[b, :c]
        else:
            assert torch.equal(got_v, v[b, :c].float())
            tol = want_k[b, :c].abs() * SO.UB + 2 * sk[b, :c]
        SO.close(got_k, want_k[b, :c], tol, "k")
        bt = cache.tensors[4]
        for i in range(first, n[b]):
            if bt is None:
                written[b, :, i] = True
            else:
                written[int(bt[b, i // page]), i % page] = True
    # nothing else was touched
    for x, old in zip(cache.tensors[:2], before):
        now = x.view(old.dtype)
        assert torch.equal(now[~written.cuda()], old[~written.cuda()])
    # the same rows by sets, every KV head's twice, bf16, -1 between
    H = 2 * hkv
    sets = torch.full((B, H, 11), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        if n[b]:
            sets[b, :, ::2] = torch.randint(0, n[b], (H, 6), device="cuda", dtype=torch.int32)
    so, sv = torch.full((B, H, 11, d), 9.0, dtype=BF, device="cuda"), torch.full((B, H, 11, d), 9.0, dtype=BF, device="cuda")
    lyc.cache_read(cache, i32(n), so, sv, sets=sets, status=st)
    assert int(st) == 0
    for b in range(B):
        for h in range(H):
            for i in range(11):
                r = int(sets[b, h, i])
                want = torch.full((d,), 9.0) if r < 0 else ko[b, h // 2, r].cpu()
                assert torch.equal(so[b, h, i].float().cpu(), want.to(BF).float())
                want = torch.full((d,), 9.0) if r < 0 else vo[b, h // 2, r].cpu()
                assert torch.equal(sv[b, h, i].float().cpu(), want.to(BF).float())


def test_quantised_rows_at_the_edges(lyc):
    """Zero rows, subnormals, the scale's border 1.75 * 2^k and its neighbours,
    the largest bf16, NaN and infinities; every code value comes back as itself."""
    d = 128
    rows = [torch.zeros(d), torch.full((d,), 2.0**-133), torch.full((d,), 3.3895e38)]
    for k in (-90, -9, 0, 8, 60):
        for f in (1.75, 1.7421875, 1.7578125, 1.0, 1.9921875):
            r = torch.zeros(d)
            r[3], r[77] = f * 2.0**k, -f * 2.0**k / 3
            rows.append(r)
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    codes = codes[torch.isfinite(codes)]
    for part in (codes[:127], codes[127:]):
        r = torch.zeros(d)
        r[: len(part)] = part
        r[127] = 448.0  # keeps the scale at one
        rows.append(r)
    for bad in (math.nan, math.inf, -math.inf):
        r = torch.ones(d)
        r[d - 1] = bad
        rows.append(r)
    x = torch.stack(rows).to(BF).cuda()[None, :, None]  # [1][T][1][d]
    T = x.shape[1]
    cache = lyc.KvCache.empty(1, 1, d, rows=T)
    lyc.cache_append(cache, i32([T]), x, x)
    code, byte = SO.e4m3_row(x[0, :, 0].cpu())
    for t, s in ((cache.tensors[0], cache.tensors[2]), (cache.tensors[1], cache.tensors[3])):
        assert torch.equal(s.view(torch.uint8)[0, 0].cpu().long(), byte)
        assert torch.equal(t[0, 0].float().cpu().double(), code)
    ko, vo = torch.zeros((1, 1, T, d), device="cuda"), torch.zeros((1, 1, T, d), device="cuda")
    lyc.cache_read(cache, i32([T]), ko, vo)
    assert torch.equal(torch.isnan(ko).all(-1)[0, 0].cpu(), byte == 255)
    fin = byte != 255
    # in fp32, whose range ends below 2^128: 1.9922 * 2^127 has code 256 at scale 2^120
    want = (code * torch.exp2(byte.double() - 127)[:, None])[fin].float()
    assert torch.equal(ko[0, 0][fin.cuda()].cpu(), want)
    assert torch.equal(ko.nan_to_num(), vo.nan_to_num())


def test_append_and_read_refuse_on_the_device(lyc):
    """Lengths, pages and indices out of range: skipped and reported, the other
    elements as they should be."""
    B, T, hkv, d, page = 4, 3, 2, 64, 4
    rng = np.random.default_rng(0)
    cache = fill(lyc, B, hkv, d, 12, page, True, seed=5)
    bt = cache.tensors[4]
    bt[2, 1] = cache.tensors[0].shape[0]  # past the pool
    bt[3, 0] = -1
    before = cache.tensors[0].view(torch.uint8).clone()
    k = randn(1, B, T, hkv, d)
    st = status_word()
    # element 0: more rows than the cache; 1: t_len past n; 2: rows 2, 3 fit and 4 is on the bad page; 3: rows 4..6 fit
    lyc.cache_append(cache, i32([13, 2, 5, 7]), k, k, t_len=i32([3, 3, 3, 3]), status=st)
    assert int(st) == lyc.LYC_OP_BAD_LENGTH | lyc.LYC_OP_BAD_PAGE
    changed = (cache.tensors[0].view(torch.uint8) != before).any(-1).any(-1)
    expect = torch.zeros_like(changed)
    expect[int(bt[2, 0]), 2:4] = True
    expect[int(bt[3, 1]), 0:3] = True
    assert torch.equal(changed, expect)
    st.zero_()
    out = [torch.full((B, hkv, 6, d), 2.0, dtype=BF, device="cuda") for _ in range(2)]
    lyc.cache_read(cache, i32([6, 0, 6, 6]), *out, status=st)
    assert int(st) == lyc.LYC_OP_BAD_PAGE
    kept = (out[0] == 2.0).all(-1).all(1).cpu()
    assert kept.tolist() == [[False] * 6, [True] * 6, [False] * 4 + [True] * 2, [True] * 4 + [False] * 2]
    st.zero_()
    sets = i32([[[0, -1, 6, 5]] * hkv, [[0, -1, -1, -1]] * hkv, [[3, 2, -2, 1]] * hkv, [[5, 4, 5, 2**30]] * hkv])
    out = [torch.full((B, hkv, 4, d), 2.0, dtype=BF, device="cuda") for _ in range(2)]
    lyc.cache_read(cache, i32([6, -1, 6, 6]), *out, sets=sets, status=st)
    assert int(st) == lyc.LYC_OP_BAD_INDEX | lyc.LYC_OP_BAD_LENGTH
    kept = (out[1] == 2.0).all(-1).all(1).cpu()
    assert kept.tolist() == [[False, True, True, False], [True] * 4, [False, False, True, False],
                             [False, False, False, True]]


def test_append_position_argument_and_first(lyc):
    """Nodes of a tree share depths: positions apart from the rows; a read that
    starts past the front."""
    T, d = 6, 128
    cache = lyc.KvCache.empty(1, 1, d, rows=32, e4m3=False)
    k, v = randn(1, 1, T, 1, d), randn(2, 1, T, 1, d)
    pos, freq = i32([[10, 11, 11, 12, 12, 12]]), inv_freq(d)
    lyc.cache_append(cache, i32([20]), k, v, pos=pos, inv_freq=freq)
    want, slack = SO.norm_rope(k, None, pos, freq, False, 1e-6)
    ko, vo = torch.zeros((1, 1, 9, d), dtype=BF, device="cuda"), torch.zeros((1, 1, 9, d), dtype=BF, device="cuda")
    lyc.cache_read(cache, i32([20]), ko, vo, first=14)
    SO.close(ko[0, 0, :6], want[0, :, 0], (want.abs() * SO.UB + 2 * slack)[0, :, 0], "k at its depth")
    assert torch.equal(vo[0, 0, :6], v[0, :, 0]) and not vo[0, 0, 6:].any()


# ------------------------------------------------------------------ tree attention


def run_tree(lyc, cache, q, n, t_len=None, mask=None, scale=None, out=None, **kw):
    B, T = q.shape[:2]
    if out is None:
        out = torch.full(q.shape, 1234.0, dtype=BF, device="cuda")
    st = status_word()
    lyc.tree_attention(q, cache, i32(n), out, mask=mask, t_len=None if t_len is None else i32(t_len), scale=scale,
                       status=st, **kw)
    return out, int(st)


def check_tree(lyc, cache, q, n, t_len=None, mask=None, scale=None, what="", status=0):
    B, T = q.shape[:2]
    out, st = run_tree(lyc, cache, q, n, t_len, mask, scale)
    assert st == status
    cnt = [T] * B if t_len is None else t_len
    want, bound = SO.tree(q, cache, n, cnt, mask, q.shape[3]**-0.5 if scale is None else scale)
    for b in range(B):
        c = max(0, cnt[b])
        SO.close(out[b, :c], want[b, :c], bound[b, :c], f"{what} element {b}")
        assert bool((out[b, c:] == 1234.0).all()), "padding was written"
    return out


LENGTHS = [1, 15, 16, 17, 63, 64, 127, 128, 129, 255, 256, 257, 511, 513, 1000, 2049]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_one_token_every_length(lyc, e4m3, d):
    """T = 1 over lengths at and beside every tile edge, one element each; what
    lies past an element's rows is NaN."""
    n = LENGTHS
    cache = fill(lyc, len(n), 2, d, max(n), 0, e4m3, seed=d)
    poison_past(cache, n)
    check_tree(lyc, cache, randn(1, len(n), 1, 8, d), n, what="one token")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,page", [
    (2, 4, 2, 128, 0), (3, 5, 1, 64, 5), (16, 8, 2, 128, 64), (17, 16, 2, 64, 16), (5, 16, 1, 128, 48),
    (63, 4, 4, 128, 1), (64, 8, 2, 128, 16), (65, 2, 1, 64, 128), (130, 4, 2, 128, 0), (256, 2, 2, 64, 64),
    (12, 32, 8, 128, 64), (33, 12, 3, 128, 256), (20, 8, 2, 128, 8), (40, 4, 1, 128, 24), (256, 8, 2, 128, 192),
    (48, 6, 6, 128, 0), (9, 64, 1, 128, 0), (9, 64, 1, 128, 12),
])
def test_tree_shapes(lyc, e4m3, T, hq, hkv, d, page):
    """Trees of every size over ragged lengths: n = t (no prefix), drafts across
    tile and page edges, elements without queries and without rows."""
    rng = np.random.default_rng(T * 1000 + hq)
    n = [T, T + 1, T + 100, 400, 700, 0, T + 300]
    t_len = [T, max(1, T // 2), T, max(0, T - 1), 1, 0, 0]
    n = [max(a, c) for a, c in zip(n, t_len)]
    cache = fill(lyc, len(n), hkv, d, max(n), page, e4m3, seed=T)
    poison_past(cache, n)
    q = randn(T, len(n), T, hq, d)
    mask = random_tree(rng, len(n), T, empty=(T - 1,) if T > 2 else ())
    check_tree(lyc, cache, q, n, t_len, mask, what="tree")
    check_tree(lyc, cache, q, n, t_len, None, what="chain")
    check_tree(lyc, cache, q[:, :, :hkv], n, None if min(n) >= T else t_len, mask, scale=0.3, what="one head a group")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [8, 16, 60])
def test_tree_long_and_split(lyc, e4m3, T):
    """One element cut over many CTAs beside short ones; the same call twice is
    the same to the bit; a peaked softmax whose tail matters."""
    cache = fill(lyc, 4, 2, 128, 20000, 64, e4m3, seed=3)
    n, t_len = [20000, T, 5000, 1], [T, min(3, T), T - 1, 1]
    poison_past(cache, n)
    q = randn(5, 4, T, 8, 128, scale=2.0)
    mask = random_tree(np.random.default_rng(1), 4, T)
    a = check_tree(lyc, cache, q, n, t_len, mask, what="long")
    b, _ = run_tree(lyc, cache, q, n, t_len, mask)
    assert torch.equal(a, b)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,hq", [(5, 2), (40, 8)])
def test_tree_rows_not_seen_do_not_matter(lyc, e4m3, T, hq):
    """NaN and infinities in drafted rows that a node does not see leave it alone,
    and reach the nodes that do see them."""
    d, n = 128, [T + 250, T]
    rng = np.random.default_rng(T)
    cache = fill(lyc, 2, 1, d, max(n), 0, e4m3, seed=8)
    poison_past(cache, n)
    mask = random_tree(rng, 2, T)
    q = randn(3, 2, T, hq, d)
    k, v, ks, vs, _ = cache.tensors
    for b in range(2):
        first = n[b] - T
        if e4m3:
            vs.view(torch.uint8)[b, 0, first + 2] = 255
            ks.view(torch.uint8)[b, 0, first + 3] = 255
        else:
            v[b, 0, first + 2, 5] = math.nan
            v[b, 0, first + 2, 64] = math.inf
            v[b, 0, first + 4] = -math.inf
            k[b, 0, first + 3, 0] = math.nan
    out = check_tree(lyc, cache, q, n, None, mask, what="unseen rows")
    assert torch.isnan(out.float()).any() and torch.isfinite(out.float()).any()


def test_tree_without_anything_to_see(lyc):
    """No prefix and an empty mask: zeros.  Elements of no rows: untouched."""
    cache = fill(lyc, 3, 2, 64, 40, 0, False, seed=2)
    q = randn(1, 3, 4, 4, 64)
    mask = torch.zeros((3, 4, 1), dtype=torch.int64, device="cuda")
    mask[0, 1, 0] = 0b0110
    mask[:, :, 0] |= -16  # bits at and past t_len are not looked at
    out, st = run_tree(lyc, cache, q, [4, 30, 0], [4, 4, 0], mask)
    assert st == 0
    assert not out[0, [0, 2, 3]].any() and out[0, 1].any() and bool((out[2] == 1234.0).all())
    check_tree(lyc, cache, q, [4, 30, 0], [4, 4, 0], mask)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page,hq", [(20, 4), (20, 16), (8, 16), (16, 32)])
def test_tree_bad_pages_and_lengths(lyc, e4m3, page, hq):
    """Lengths that do not fit leave an element out; rows on pages outside the
    pool are not seen; both are reported."""
    cap = 300 // page * page
    cache = fill(lyc, 6, 2, 128, cap, page, e4m3, seed=4)
    poison_past(cache, [min(290, cap), 0, 0, 0, 0, 0])
    bt = cache.tensors[4]
    bt[0, 3] = -5
    bt[0, 286 // page] = 2**31 - 1  # holds drafted rows
    q = randn(1, 6, 7, hq, 128)
    n, t_len = [min(290, cap), 301, 5, -1, 100, 50], [7, 7, 6, 0, 8, -1]
    out, st = run_tree(lyc, cache, q, n, t_len)
    assert st == lyc.LYC_OP_BAD_LENGTH | lyc.LYC_OP_BAD_PAGE
    assert bool((out[1:] == 1234.0).all())
    w, bd = SO.tree(q[:1], cache, n[:1], [7], None, 128**-0.5)
    SO.close(out[:1], w, bd, "rows on bad pages")


@pytest.mark.parametrize("T", [8, 70])
def test_tree_query_values(lyc, T):
    """Queries of extreme size, zero, NaN and infinity, over both caches."""
    for e4m3 in (False, True):
        cache = fill(lyc, 1, 1, 128, 200, 0, e4m3, seed=6)
        q = randn(2, 1, T, 1, 128)
        q[0, 0] = 0
        q[0, 1] *= 2.0**-120
        q[0, 2] *= 2.0**20
        q[0, 3, 0, 5] = math.nan
        q[0, 4, 0, 7] = math.inf
        q[0, 5, 0, 1:] *= 2.0**-12  # one large element beside small ones
        out, _ = run_tree(lyc, cache, q, [200])
        assert torch.isnan(out[0, 3]).all() and torch.isnan(out[0, 4]).all()
        ok = [0, 1, 2, 5, 6, 7]
        want, bound = SO.tree(q.nan_to_num(), cache, [200], [T], None, 128**-0.5)
        # a logit of 2^20 has an absolute error beyond the softmax: hardest row only finite
        assert torch.isfinite(out[0, ok].float()).all()
        for t in (0, 1, 5, 6, 7):
            SO.close(out[0, t], want[0, t], bound[0, t], f"query {t}")


@pytest.mark.parametrize("T", [6, 24])
def test_tree_strides_streams_graphs(lyc, T):
    """Queries inside a projection's output, heads-first outputs, another stream, a
    captured call replayed at other lengths, and two captured calls at once."""
    B, hq, hkv, d, cap = 2, 8, 2, 128, 3000
    cache = fill(lyc, B, hkv, d, cap, 0, True, seed=9)
    qkv = randn(4, B, T, (hq + 4) * d)
    q = qkv[..., 2 * d: (2 + hq) * d].unflatten(2, (hq, d))
    out_t = torch.full((B, hq, T, d), 1234.0, dtype=BF, device="cuda")
    ref, _ = run_tree(lyc, cache, q, [3000, 27])
    run_tree(lyc, cache, q, [3000, 27], out=out_t.transpose(1, 2))
    assert torch.equal(out_t.transpose(1, 2), ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out_s = torch.zeros_like(ref)
    n = i32([3000, 27])
    lyc.tree_attention(q, cache, n, out_s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out_s, ref)
    # two graphs, each with its own workspace, replayed on two streams at once
    lens = [i32([3000, 27]), i32([100, 2999])]
    outs = [torch.zeros_like(ref) for _ in range(2)]
    graphs = []
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lyc.tree_attention(q, cache, lens[i], outs[i])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for lengths in ([[3000, 27], [100, 2999]], [[T + 1, T], [1500, 1000]], [[128, 129], [T, T]]):
        for i in range(2):
            lens[i].copy_(i32(lengths[i]))
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            want, _ = run_tree(lyc, cache, q, lengths[i])
            assert torch.equal(outs[i], want), (lengths, i)


def test_offsets_past_32_bits(lyc):
    """A pool of more than 2^31 elements: pages at its end."""
    d, page_rows, hkv = 128, 256, 8
    pages = (1 << 31) // (page_rows * hkv * d) + 40
    pool = torch.empty((2, pages, page_rows, hkv, d), dtype=BF, device="cuda")
    bt = i32([[pages - 1, 0, pages - 2, 5]])
    for p in bt[0].tolist():
        pool[:, p] = randn(p, 2, page_rows, hkv, d)
    cache = lyc.KvCache(pool[0], pool[1], block_table=bt)
    k, v = randn(1, 1, 3, hkv, d), randn(2, 1, 3, hkv, d)
    lyc.cache_append(cache, i32([700]), k, v)
    assert torch.equal(pool[0, pages - 2, 185:188], k[0]) and torch.equal(pool[1, pages - 2, 185:188], v[0])
    ko, vo = torch.zeros((1, hkv, 4, d), dtype=BF, device="cuda"), torch.zeros((1, hkv, 4, d), dtype=BF, device="cuda")
    lyc.cache_read(cache, i32([700]), ko, vo, first=697)
    assert torch.equal(ko[0, :, :3].transpose(0, 1), k[0])
    small = lyc.KvCache(pool[0][bt[0].long()].contiguous(), pool[1][bt[0].long()].contiguous(), block_table=i32([[0, 1, 2, 3]]))
    q = randn(3, 1, 3, 16, d)
    a, _ = run_tree(lyc, cache, q, [700])
    b, _ = run_tree(lyc, small, q, [700])
    assert torch.equal(a, b)
    check_tree(lyc, small, q, [700])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,hq,cap,page", [
    (3, 4, 90, 0), (12, 8, 90, 16), (12, 8, 400, 16), (60, 8, 300, 0), (33, 2, 520, 8),
])
def test_tree_many_elements(lyc, e4m3, T, hq, cap, page):
    """More elements than a warp has lanes, most of them short: several whole
    groups a CTA, caches of one tile, blocks of few rows beside full ones."""
    B, hkv = 41, 2
    rng = np.random.default_rng(cap + T)
    cap = -(-cap // page) * page if page else cap
    t_len = [int(x) for x in rng.integers(0, T + 1, B)]
    n = [int(rng.integers(c, cap + 1)) for c in t_len]
    t_len[7], n[7], t_len[40], n[40] = T, cap, T, T
    cache = fill(lyc, B, hkv, 128, cap, page, e4m3, seed=cap)
    poison_past(cache, n)
    q = randn(T, B, T, hq, 128)
    mask = random_tree(rng, B, T)
    check_tree(lyc, cache, q, n, t_len, mask, what="many")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,hq,hkv,B", [(1, 4, 2, 300), (12, 4, 1, 300), (3, 2, 2, 90)])
def test_tree_large_batches(lyc, e4m3, T, hq, hkv, B):
    """Far more groups than CTAs, a few of them cut over several: lengths of zero to
    200, and some of thousands at the ends and edges of the windows of 32 elements."""
    rng = np.random.default_rng(B + T)
    page, cap = 16, 6000
    t_len = [int(x) for x in rng.integers(0, T + 1, B)]
    n = [int(rng.integers(c, 200)) for c in t_len]
    for b, x in ((0, 5000), (31, 6000), (32, 3000), (33, 1), (64, 4096), (B - 1, 5999)):
        t_len[b], n[b] = min(T, x), x
    pages = [-(-x // page) for x in n]
    table = torch.zeros((B, cap // page), dtype=torch.int32)
    order, at = rng.permutation(sum(pages)), 0
    for b in range(B):
        table[b, : pages[b]] = torch.from_numpy(order[at: at + pages[b]].astype(np.int32))
        at += pages[b]
    proto = fill(lyc, 1, hkv, 128, sum(pages) * page, page, e4m3, seed=B)
    k, v, ks, vs, _ = proto.tensors
    cache = lyc.KvCache(k, v, ks, vs, block_table=table.cuda())
    check_tree(lyc, cache, randn(T, B, T, hq, 128), n, t_len, random_tree(rng, B, T), what="large batch")


@pytest.mark.parametrize("T,page", [(3, 0), (3, 16), (20, 0), (20, 16)])
def test_tree_scales_of_every_size(lyc, T, page):
    """Scales far from 1 in K and V: V's to 2^23 apart over few query rows (fp16
    probabilities times scales hold 2^30), to 2^120 over many."""
    cap, n = 320, [310, 131]
    cache = fill(lyc, 2, 1, 128, cap, page, True, seed=12)
    k, v, ks, vs, _ = cache.tensors
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    # codes of 1 .. 7 times 2^-9 with a scale of 2^9 or 2^10: keys of ordinary size
    small = torch.randint(1, 8, k.shape, generator=g, device="cuda", dtype=torch.uint8)
    sign = torch.randint(0, 2, k.shape, generator=g, device="cuda", dtype=torch.uint8) << 7
    k.view(torch.uint8).copy_(small | sign)
    ks.view(torch.uint8).copy_(torch.randint(136, 138, ks.shape, generator=g, device="cuda", dtype=torch.uint8))
    v.view(torch.uint8).copy_(small.flip(0) + 0x30 | sign)  # no zeros: 1.0 .. 1.875 / 2
    choice = torch.tensor([127, 134, 135, 150] if T * 4 <= 32 else [30, 127, 135, 150], dtype=torch.uint8, device="cuda")
    vs.view(torch.uint8).copy_(choice[torch.randint(0, 4, vs.shape, generator=g, device="cuda")])
    q = randn(7, 2, T, 4, 128, scale=0.3)
    check_tree(lyc, cache, q, n, None, None, what="scales")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,hq,page", [(6, 2, 0), (12, 4, 16), (40, 4, 0), (130, 1, 16)])
def test_tree_rows_that_nobody_wrote(lyc, e4m3, T, hq, page):
    """Drafted rows that no node sees hold any bytes at all (codes and scales of every
    value, or bf16 bits): the outputs are those over rows of zeros, to the bit, except
    that with many query rows over an e4m3 cache the scales of a tile's rows choose
    between two ways to scale its products, each within the bound."""
    n, cap = [T + 333, T, T + 120], T + 352 - T % 16
    rng = np.random.default_rng(T)
    mask = random_tree(rng, 3, T)
    dead = [t for t in range(T) if t % 3 == 1]
    words = mask.cpu().numpy().view(np.uint64)
    for t in dead:
        words[:, :, t // 64] &= np.uint64(2**64 - 1 - (1 << (t % 64)))
    mask = torch.from_numpy(words.view(np.int64)).cuda()
    cache = fill(lyc, 3, 1, 128, cap, page, e4m3, seed=T)
    poison_past(cache, n)
    k, v, ks, vs, bt = cache.tensors
    q = randn(9, 3, T, hq, 128)
    for kind in range(4):  # zeros, any bytes, the largest scales and codes, NaN codes
        for x in (k, v, ks, vs):
            if x is None:
                continue
            b8 = x.view(torch.uint8)
            for b in range(3):
                for t in dead:
                    row = n[b] - T + t
                    at = (b, 0, row) if bt is None else (int(bt[b, row // page]), row % page, 0)
                    if kind == 1:
                        b8[at] = torch.randint(0, 256, b8[at].shape, device="cuda", dtype=torch.uint8)
                    else:
                        b8[at] = (0, 0, 254, 127)[kind]
        if kind == 0:
            zeros = check_tree(lyc, cache, q, n, None, mask, what="zeros")
            want, bound = SO.tree(q, cache, n, [T] * 3, mask, 128**-0.5)
        out, st = run_tree(lyc, cache, q, n, None, mask)
        assert st == 0
        SO.close(out, want, bound, f"kind {kind}")
        if not (e4m3 and T * hq > 32):
            assert torch.equal(out, zeros), kind


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [4, 20])
def test_tree_cache_orders(lyc, e4m3, T):
    """The same rows in other orders and with padding between them: rows before
    heads, pages with heads outermost, scales of a page row by row and unaligned,
    one prefix shared by all elements."""
    B, hkv, d, cap, page = 3, 2, 128, 400, 16
    n = [400, 77, T]
    q = randn(5, B, T, 8, d)
    mask = random_tree(np.random.default_rng(T), B, T)
    base = fill(lyc, B, hkv, d, cap, 0, e4m3, seed=21)
    k, v, ks, vs, _ = base.tensors
    want = check_tree(lyc, base, q, n, None, mask, what="plain")
    es, by = (torch.uint8, torch.uint8) if e4m3 else (BF, None)

    def wide(x, shape, perm):
        """x copied into a tensor of order `perm` whose rows are 16 elements longer"""
        x = x.view(es) if e4m3 else x
        y = torch.zeros([shape[p] for p in perm] + [d + 16], dtype=es, device="cuda")
        y = y.permute([perm.index(i) for i in range(3)] + [3])[..., :d]
        y.copy_(x)
        return y.view(k.dtype) if e4m3 else y

    def apart(s, perm, pad):
        if s is None:
            return None
        s = s.view(torch.uint8)
        y = torch.zeros([s.shape[p] for p in perm[:2]] + [s.shape[perm[2]] + pad], dtype=torch.uint8, device="cuda")
        y = y[..., 1: s.shape[perm[2]] + 1].permute([perm.index(i) for i in range(3)])  # starts at an odd byte
        y.copy_(s)
        return y

    for perm in ([0, 2, 1], [2, 1, 0], [1, 0, 2]):
        c = lyc.KvCache(wide(k, k.shape, perm), wide(v, v.shape, perm), apart(ks, perm, 5), apart(vs, perm, 5))
        out, st = run_tree(lyc, c, q, n, None, mask)
        assert st == 0 and torch.equal(out, want), perm
    # pages
    rng = np.random.default_rng(2)
    bt, pages = block_table(rng, B, cap // page)
    idx = bt.long().flatten()

    def paged(x, shape):
        y = torch.zeros((pages, page, hkv) + shape, dtype=x.dtype, device="cuda")
        y[idx] = x.transpose(1, 2).unflatten(1, (cap // page, page)).flatten(0, 1)
        return y

    def as_bytes(x):
        return x.view(torch.uint8) if e4m3 else x

    pk, pv = (paged(as_bytes(x), (d,)) for x in (k, v))
    ps = [paged(s.view(torch.uint8), ()) if e4m3 else None for s in (ks, vs)]
    for perm in ([0, 1, 2], [0, 2, 1], [2, 0, 1], [1, 2, 0]):
        c = lyc.KvCache(wide(pk, pk.shape, perm), wide(pv, pv.shape, perm), apart(ps[0], perm, 3), apart(ps[1], perm, 3),
                        block_table=bt)
        out, st = run_tree(lyc, c, q, n, None, mask)
        assert st == 0 and torch.equal(out, want), perm
    # every element reads element 0's rows
    one = [None if x is None else as_bytes(x)[:1].expand(x.shape) for x in (k, v)]
    two = [None if s is None else s.view(torch.uint8)[:1].expand(s.shape) for s in (ks, vs)]
    c = lyc.KvCache(one[0].view(k.dtype) if e4m3 else one[0], one[1].view(k.dtype) if e4m3 else one[1], *two)
    check_tree(lyc, c, q, n, None, mask, what="shared prefix")


@pytest.mark.parametrize("e4m3", [False, True])
def test_tree_pages_too_small_for_a_tile(lyc, e4m3):
    """Pages of 4 and 6 rows under many query rows: blocks of 32 rows of the kernel
    that looks up every row."""
    for page in (4, 6):
        n = [150, 40]
        cache = fill(lyc, 2, 1, 128, 156, page, e4m3, seed=page)
        poison_past(cache, n)
        check_tree(lyc, cache, randn(3, 2, 17, 4, 128), n, None, random_tree(np.random.default_rng(1), 2, 17), what="small pages")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [2, 24])
def test_tree_two_calls_at_once(lyc, e4m3, T):
    """Two eager calls on two streams over one cache, each with a workspace of its
    own that held anything, and one that is too small or is not aligned."""
    cache = fill(lyc, 2, 2, 128, 6000, 64, e4m3, seed=30)
    qs = [randn(i, 2, T, 8, 128) for i in range(2)]
    lens = [[6000, 500], [900, 5999]]
    want = [run_tree(lyc, cache, qs[i], lens[i])[0] for i in range(2)]
    need = lyc.tree_workspace_bytes(cache, T, 8)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.zeros_like(want[0]) for _ in range(2)]
    ns = [i32(x) for x in lens]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            lyc.tree_attention(qs[i], cache, ns[i], outs[i], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want[i])
    for bad in (ws[0][: need - 1], ws[0].new_empty(need + 16)[8: need + 8]):
        with pytest.raises(lyc.LycError):
            lyc.tree_attention(qs[0], cache, ns[0], outs[0], workspace=bad)


def test_captured_step_follows_its_lengths(lyc):
    """Norm, append, attention and read captured once; replayed with lengths,
    positions and tokens changed on the device, it does each step's work."""
    B, hq, hkv, d = 2, 8, 2, 128
    bt, pages = block_table(np.random.default_rng(3), B, 12)
    make = lambda: lyc.KvCache.empty(B, hkv, d, page_rows=16, num_pages=pages, block_table=bt)  # noqa: E731
    a, b = make(), make()
    freq, w = inv_freq(d), (1 + randn(1, d, scale=0.1).float()).to(BF)
    q, k, v = randn(2, B, 1, hq, d), randn(3, B, 1, hkv, d), randn(4, B, 1, hkv, d)
    n, pos = i32([1, 1]), i32([0, 0])
    qo, out, kn = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k[:, 0])
    ko = torch.zeros((B, hkv, 8, d), dtype=torch.float32, device="cuda")
    vo = torch.zeros_like(ko)

    def step(cache, qo, out, kn, ko, vo):
        lyc.qk_norm_rope(None, k[:, 0], pos, freq, None, kn, k_weight=w)
        lyc.cache_append(cache, n, k, v, q=q, q_out=qo, inv_freq=freq, q_weight=w, k_weight=w)
        lyc.tree_attention(qo, cache, n, out)
        lyc.cache_read(cache, n, ko, vo)

    step(a, qo, out, kn, ko, vo)  # outside a capture first
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a, qo, out, kn, ko, vo)
    mine = [torch.empty_like(qo), torch.empty_like(out), torch.empty_like(kn), torch.zeros_like(ko), torch.zeros_like(vo)]
    step(b, *mine)
    for i in range(1, 150):
        q.copy_(randn(100 + i, *q.shape))
        k.copy_(randn(300 + i, *k.shape))
        n.copy_(i32([i + 1, i // 2 + 1]))
        pos.copy_(n - 1)
        g.replay()
        step(b, *mine)
        if i % 37 == 0 or i == 149:
            torch.cuda.synchronize()
            for x, y in zip((qo, out, kn, ko, vo), mine):
                assert torch.equal(x, y), i
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.tensors[:4], b.tensors[:4]))


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_norm_rope_many_heads_and_rows(lyc, dtype):
    """More than 256 rows of heads that are many times and no multiple of what a
    block takes at once, in place."""
    rows, hq, hkv, d = 300, 41, 11, 128
    q, k = randn(1, rows, hq, d, dtype=dtype), randn(2, rows, hkv, d, dtype=dtype)
    pos = torch.arange(rows, device="cuda", dtype=torch.int32) * 977
    freq, w = inv_freq(64), (1 + randn(3, d, scale=0.2).float()).to(dtype)
    qo, ko = q.clone(), k.clone()
    lyc.qk_norm_rope(qo, ko, pos, freq, qo, ko, w, w, interleaved=False)
    u = SO.UB if dtype == BF else SO.U32
    for got, x in ((qo, q), (ko, k)):
        y, slack = SO.norm_rope(x, w, pos, freq, False, 1e-6)
        SO.close(got, y, y.abs() * u + slack * (1 + u), "many heads")


def test_append_many_tokens(lyc):
    """A prompt of more than 256 tokens of many heads: the bytes that the same
    tokens give one at a time."""
    B, T, hq, hkv, d = 1, 300, 20, 9, 64
    freq, w = inv_freq(d), (1 + randn(1, d, scale=0.1).float()).to(BF)
    q, k, v = randn(2, B, T, hq, d), randn(3, B, T, hkv, d), randn(4, B, T, hkv, d)
    a, b = (lyc.KvCache.empty(B, hkv, d, rows=310) for _ in range(2))
    qa, qb = torch.empty_like(q), torch.empty_like(q)
    lyc.cache_append(a, i32([T]), k, v, q=q, q_out=qa, inv_freq=freq, q_weight=w, k_weight=w)
    for t in range(T):
        s = slice(t, t + 1)
        lyc.cache_append(b, i32([t + 1]), k[:, s], v[:, s], q=q[:, s], q_out=qb[:, s], inv_freq=freq, q_weight=w, k_weight=w)
    assert torch.equal(qa, qb)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.tensors[:4], b.tensors[:4]))


def test_wrappers_refuse_what_does_not_fit(lyc):
    """Wrong types, shapes, orders and devices are refused before anything runs."""
    cache = lyc.KvCache.empty(2, 2, 64, rows=32)
    q, k = randn(1, 2, 3, 4, 64), randn(2, 2, 3, 2, 64)
    n, out = i32([5, 5]), torch.empty((2, 3, 4, 64), dtype=BF, device="cuda")
    bad = [
        lambda: lyc.tree_attention(q.float(), cache, n, out),
        lambda: lyc.tree_attention(q[:1], cache, n, out),
        lambda: lyc.tree_attention(q.transpose(2, 3).contiguous().transpose(2, 3), cache, n, out),
        lambda: lyc.tree_attention(q, cache, n.long(), out),
        lambda: lyc.tree_attention(q, cache, n.cpu(), out),
        lambda: lyc.tree_attention(q, cache, n[:1], out),
        lambda: lyc.tree_attention(q, cache, n, out, mask=torch.zeros((2, 3), dtype=torch.int64, device="cuda")),
        lambda: lyc.tree_attention(q, cache, n, out[..., :32]),
        lambda: lyc.tree_attention(q, cache, n, out, status=torch.zeros(1, device="cuda")),
        lambda: lyc.tree_attention(randn(1, 2, 257, 4, 64), cache, n, torch.empty((2, 257, 4, 64), dtype=BF, device="cuda")),
        lambda: lyc.cache_append(cache, n, k, k.float()),
        lambda: lyc.cache_append(cache, n, k[:, :, :1], k[:, :, :1]),
        lambda: lyc.cache_append(cache, n, k, k, q=q),
        lambda: lyc.cache_append(cache, n, k, k, inv_freq=inv_freq(64).double()),
        lambda: lyc.cache_read(cache, n, k.transpose(1, 2).half(), k.transpose(1, 2)),
        lambda: lyc.cache_read(cache, n, k, k),
        lambda: lyc.qk_norm_rope(q[0], k[0], None, inv_freq(64), q[0], k[0]),
        lambda: lyc.qk_norm_rope(q[0], k[0].float(), i32([0, 1, 2]), inv_freq(64), q[0], k[0]),
        lambda: lyc.qk_norm_rope(q[0], None, i32([0, 1]), inv_freq(64), q[0], None),
        lambda: lyc.KvCache(cache.tensors[0], cache.tensors[1]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(lyc.LycError):
            call()
            pytest.fail(f"call {i} was taken")


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("e4m3", [True, False])
def test_a_drafting_program(lyc, e4m3):
    """A prompt, then rounds of drafting: append the drafted nodes at their depths,
    verify them, keep a path, go on from there; at the end the cache read back
    feeds the decode step, whose all-retrieval layer is the one-token attention."""
    B, hq, hkv, d, page = 2, 8, 2, 128, 16
    rng = np.random.default_rng(0)
    bt, pages = block_table(rng, B, 20)
    cache = lyc.KvCache.empty(B, hkv, d, page_rows=page, num_pages=pages, block_table=bt, e4m3=e4m3)
    freq, w = inv_freq(d), (1 + randn(1, d, scale=0.1).float()).to(BF)
    lens = [150, 93]
    T0 = max(lens)
    k, v = randn(2, B, T0, hkv, d), randn(3, B, T0, hkv, d)
    lyc.cache_append(cache, i32(lens), k, v, t_len=i32(lens), inv_freq=freq, k_weight=w)
    for step in range(4):
        T = 7
        mask = random_tree(rng, B, T)
        depth = torch.tensor([[bin(int(mask[b, t, 0])).count("1") - 1 for t in range(T)] for b in range(B)])
        pos = (torch.tensor(lens)[:, None] + depth).to(torch.int32).cuda()
        n = [x + T for x in lens]
        q = randn(10 + step, B, T, hq, d)
        k, v = randn(20 + step, B, T, hkv, d), randn(30 + step, B, T, hkv, d)
        qo, out = torch.empty_like(q), torch.empty_like(q)
        st = status_word()
        lyc.cache_append(cache, i32(n), k, v, q=q, q_out=qo, pos=pos, inv_freq=freq, q_weight=w, k_weight=w, status=st)
        lyc.tree_attention(qo, cache, i32(n), out, mask=mask, status=st)
        assert int(st) == 0
        wq, sq = SO.norm_rope(q, w, pos, freq, False, 1e-6)
        SO.close(qo, wq, wq.abs() * SO.UB + 2 * sq, "q of the draft")
        want, bound = SO.tree(qo, cache, n, [T] * B, mask, d**-0.5)
        SO.close(out, want, bound, f"verification {step}")
        lens = [x + 1 + step % 2 for x in lens]  # a chain of one or two nodes is kept
    n = max(lens)
    K = torch.zeros((1, B, hkv, n, d), dtype=BF, device="cuda")
    V = torch.zeros_like(K)
    lyc.cache_read(cache, i32(lens), K[0], V[0])
    q = randn(77, B, 1, hq, d)
    out = torch.empty_like(q)
    lyc.tree_attention(q, cache, i32(lens), out)
    ctx = lyc.Lyc(1, B, hq, hkv, d, n, 8)
    o, S = torch.zeros((1, B, hq, d), device="cuda"), torch.zeros((B, hq, 8), dtype=torch.int32, device="cuda")
    ctx.decode_step_batch(q.transpose(0, 1).contiguous(), K, V, lens, np.ones((1, hq), np.uint8), 8, o, S)
    assert ctx.sync_status() == 0
    ctx.close()
    want, bound = SO.tree(q, cache, lens, [1] * B, None, d**-0.5)
    SO.close(out, want, bound, "one token")
    # both sides round their probabilities to bf16 at most: twice the bound, and the step's fp32 sums
    SO.close(o[0][:, None], want, 2 * bound + 2 * SO.UB * want.abs().max(), "the decode step on the rows read back")
    # the rows of the step's sets, gathered: the sparse head's rows
    so = torch.zeros((B, hq, 8, d), dtype=BF, device="cuda")
    sv = torch.zeros_like(so)
    lyc.cache_read(cache, i32(lens), so, sv, sets=S)
    for b in range(B):
        for h in range(hq):
            assert torch.equal(so[b, h], K[0, b, h // (hq // hkv)][S[b, h].long()])
