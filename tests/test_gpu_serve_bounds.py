"""The serving operators on a B200 where their arithmetic is at its limits: the
bounds of each cache's own roundings (tests/serve_strict.py), probabilities and
scales that lie far apart, states merged within a block, and bytes of the cache
that a call may not touch."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from tests import serve_strict as SS
from tests.serve_oracle import close
from tests.test_gpu_serve_ops import BF, check_tree, fill, i32, poison_past, randn, random_tree, run_tree, status_word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lyc():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from hybrid_head_sparse_b200 import lyc as m
    m.load()
    return m


def strict(lyc, cache, q, n, t_len=None, mask=None, scale=None, what="", lost=SS.LOST):
    B, T = q.shape[:2]
    out, st = run_tree(lyc, cache, q, n, t_len, mask, scale)
    assert st == 0
    cnt = [T] * B if t_len is None else t_len
    want, bound = SS.tree(q, cache, n, cnt, mask, q.shape[3]**-0.5 if scale is None else scale, lost)
    for b in range(B):
        close(out[b, :cnt[b]], want[b, :cnt[b]].cpu(), bound[b, :cnt[b]].cpu(), f"{what} element {b}")
        assert bool((out[b, cnt[b]:] == 1234.0).all()), "padding was written"
    return out


def plain_scales(cache):
    for s in cache.tensors[2:4]:
        s.view(torch.uint8).fill_(127)


def e4m3(x):
    return torch.tensor(x, device="cuda").to(torch.float8_e4m3fn)


# ------------------------------------------------------------------ probabilities


def shared_by(lyc, one, B):
    """B elements that all read the one element of `one`: a block then has many of its
    tiles, where a single element's are dealt to all blocks."""
    k, v, ks, vs, _ = (None if x is None else x.view(torch.uint8) for x in one.tensors)
    wide = [x.expand(B, *x.shape[1:]) for x in (k, v, ks, vs)]
    return lyc.KvCache(*(x.view(torch.float8_e4m3fn) for x in wide[:2]), *wide[2:])


def check_shared(lyc, one, q, n, mask, what):
    """q of one element, asked for by 150 of them, with q . k as the natural logarithm
    of 2^(q . k)."""
    B = 150
    wide = None if mask is None else mask.expand(B, -1, -1).contiguous()
    out, st = run_tree(lyc, shared_by(lyc, one, B), q.expand(B, -1, -1, -1), [n] * B, None, wide, scale=math.log(2.0))
    assert st == 0
    want, bound = SS.tree(q, one, [n], [q.shape[1]], mask, math.log(2.0))
    for b in range(B):
        close(out[b], want[0].cpu(), bound[0].cpu(), f"{what} element {b}")


def one_hot(T):
    q = torch.zeros((1, T, 1, 128), dtype=BF, device="cuda")
    q[..., 0] = 1.0
    return q


@pytest.mark.parametrize("spread", [5, 6, 7, 14, 15])
@pytest.mark.parametrize("T,unseen", [(20, False), (40, False), (40, True), (100, False), (100, True)])
def test_a_tail_beside_a_larger_scale(lyc, T, spread, unseen):
    """65536 rows, each 2^-18 of the top one's probability, are a fifth of the sum; in
    the top row's tile a row that hardly counts (2^-60), or that no node sees, has a V
    scale 2^spread larger.  What it does to the probabilities' range costs nothing."""
    N, d = 65536 + (64 if unseen else 0), 128
    n = N + T
    cache = lyc.KvCache.empty(1, 1, d, rows=n)
    plain_scales(cache)
    k, v, _, vs, _ = cache.tensors
    k[0, 0, :, 0] = e4m3(-18.0)
    v.copy_(e4m3(1.5).expand(v.shape))
    v[0, 0, :, 1::2] = e4m3(-1.25)
    vs.view(torch.uint8).fill_(127 - spread)
    mask = torch.zeros((1, T, -(-T // 64)), dtype=torch.int64, device="cuda")
    top, odd = (N - 1, N + 3) if unseen else (70, 3)
    if not unseen:  # every node sees itself
        for t in range(T):
            mask[0, t, t // 64] = 1 << (t % 64) if t % 64 < 63 else -(1 << 63)
    k[0, 0, top, 0] = e4m3(0.0)
    v[0, 0, top] = e4m3(1.0)
    k[0, 0, odd, 0] = e4m3(-60.0)
    vs.view(torch.uint8)[0, 0, odd] = 127
    check_shared(lyc, cache, one_hot(T), n, mask, "tail")


@pytest.mark.parametrize("T,hq,hkv,d,page,n", [
    (1, 8, 2, 128, 0, 5000), (1, 8, 2, 64, 16, 5000), (4, 16, 2, 128, 48, 3000), (24, 2, 2, 64, 5, 700),
    (40, 4, 4, 128, 0, 9000), (20, 8, 2, 128, 16, 3000), (64, 8, 2, 128, 7, 1000), (130, 2, 1, 128, 64, 2500),
    (70, 8, 4, 64, 0, 900),
])
def test_e4m3_probabilities_are_fp16(lyc, T, hq, hkv, d, page, n):
    """Both kernels over an 8-bit cache, its rows' scales up to 2^8 apart, within
    fp16's rounding: bf16 probabilities, eight times as coarse, would not be."""
    B = 3
    lens = [n, max(T, n // 3), T]
    cnt = [T, max(1, T - 1), T]
    cache = fill(lyc, B, hkv, d, n, page, True, seed=T + d)
    poison_past(cache, lens)
    q = randn(T, B, T, hq, d)
    mask = random_tree(np.random.default_rng(T), B, T, empty=(T - 1,) if T > 4 else ())
    strict(lyc, cache, q, lens, cnt, mask, what="tree")
    strict(lyc, cache, q, lens, cnt, None, what="chain")
    # all the rows of V one sign, all of one size: what the bound is for
    for x in cache.tensors[1:2]:
        b = x.view(torch.uint8)
        b &= 0x7F
    strict(lyc, cache, q * 0.125, lens, cnt, None, what="one sign")


# ------------------------------------------------------------------ sums


@pytest.mark.parametrize("T,hq", [(1, 4), (3, 8), (40, 2), (70, 2)])
def test_rows_of_the_smallest_scales(lyc, T, hq):
    """Rows that are counted but were never written (zero codes, scale byte 0) are
    rows of zeros of their own tiles and blocks, beside written ones: they count in
    the sum."""
    d, rows = 128, 20000
    cache = fill(lyc, 2, 1, d, rows, 0, True, seed=40)
    for x in cache.tensors[:4]:
        b = x.view(torch.uint8)
        b[0, :, :15000] = 0
        b[1, :, 400:] = 0
    strict(lyc, cache, randn(1, 2, T, hq, d), [rows, rows], None, None, what="unwritten")


@pytest.mark.parametrize("step", [4, 8])
@pytest.mark.parametrize("T", [1, 40, 70])
def test_long_runs_of_zero_values(lyc, T, step):
    """A quarter of a million V rows of zeros (scale 2^-100) in one block, their logits
    as far above the first ones as the running maximum does not move for: the sum
    stays finite, and the one row of ones has its share."""
    rows = 1 << 18
    one = lyc.KvCache.empty(1, 1, 128, rows=rows + T)
    plain_scales(one)
    k, v, _, vs, _ = one.tensors
    vs.view(torch.uint8).fill_(27)
    k[0, 0, :, 0] = e4m3(-16.0)
    k[0, 0, 4096:, 0] = e4m3(-16.0 + step)
    k[0, 0, rows - 1, 0] = e4m3(0.0)
    v[0, 0, rows - 1] = e4m3(256.0)
    vs.view(torch.uint8)[0, 0, rows - 1] = 119
    check_shared(lyc, one, one_hot(T), rows + T, None, "zeros")


# ------------------------------------------------------------------ states merged within a block


def whole_groups(n, hkv, blocks, sms=148, tile=128):
    """By CTA, the tiles of each group that its run holds whole (the runs are equal
    shares of all tiles)."""
    spans, total = [], 0
    for nb in n:
        for _ in range(hkv * blocks):
            t = -(-nb // tile)
            spans.append((total, total + t))
            total += t
    grid = min(sms, total)
    share, more = divmod(total, grid)
    runs = [c * share + min(c, more) for c in range(grid + 1)]
    return [[b - a for a, b in spans if runs[c] <= a and b <= runs[c + 1]] for c in range(grid)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,hq", [(12, 32), (16, 32), (40, 8)])
def test_long_whole_groups_of_few_rows(lyc, e4m3, T, hq):
    """Blocks of 33 to 64 query rows whose whole group, 16 tiles or more, is one CTA's:
    its query rows lie in the lanes twice, and the copies are merged there.  Short
    groups, with one copy, and cut ones come between.  A drafted V row holds a NaN (an
    infinity beside it, over bf16 rows) that some nodes see."""
    B, hkv, d, page, pool = 40, 8, 128, 16, 600
    rng = np.random.default_rng(T + e4m3)
    n = [int(rng.integers(2048, 4000)) if b % 3 else int(rng.integers(T + 20, 1900)) for b in range(B)]
    n[4] = n[5] = 2048
    groups = whole_groups(n, hkv, 1, torch.cuda.get_device_properties(0).multi_processor_count)
    merged = [[t >= 16 for t in g] for g in groups]
    assert sum(map(sum, merged)) > 50 and any(any(m) and not all(m) for m in merged)
    proto = fill(lyc, 1, hkv, d, (pool + 5 * B) * page, page, e4m3, seed=T)
    k, v, ks, vs, _ = proto.tensors
    table = rng.integers(0, pool, (B, 4000 // page + 1))
    for b in range(B):  # the drafted rows' pages are the element's own
        last = (n[b] - 1) // page
        for i in range(5):
            if last - i >= 0:
                table[b, last - i] = pool + 5 * b + i
    cache = lyc.KvCache(k, v, ks, vs, block_table=i32(table.tolist()))
    for b in range(0, B, 2):
        row = n[b] - T + 3
        at = (int(table[b, row // page]), row % page)
        if e4m3:
            vs.view(torch.uint8)[at[0], at[1], b % hkv] = 255
        else:
            v[at[0], at[1], b % hkv, 5] = math.nan
            v[at[0], at[1], b % hkv, 70] = math.inf
    mask = random_tree(rng, B, T)
    q = randn(T, B, T, hq, d)
    out = strict(lyc, cache, q, n, None, mask, what="whole groups")
    assert torch.isnan(out.float()).any() and torch.isfinite(out.float()).any()
    again, _ = run_tree(lyc, cache, q, n, None, mask)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,n", [(1, 40, 40, 64, 3000), (1, 100, 50, 128, 5000), (2, 96, 96, 64, 900),
                                          (160, 64, 8, 128, 1200), (128, 64, 8, 128, 700), (3, 149, 149, 64, 600)])
def test_one_element_of_many_groups(lyc, e4m3, T, hq, hkv, d, n):
    """One element whose groups do not divide the blocks evenly: runs cut across
    groups, or whole blocks for each."""
    cache = fill(lyc, 1, hkv, d, n, 0, e4m3, seed=hkv)
    q = randn(T, 1, T, hq, d)
    mask = random_tree(np.random.default_rng(T), 1, T)
    out = strict(lyc, cache, q, [n], None, mask, what="one element")
    again, _ = run_tree(lyc, cache, q, [n], None, mask)
    assert torch.equal(out, again)


# ------------------------------------------------------------------ bytes of the cache


@pytest.mark.parametrize("page", [0, 7, 16, 64])
def test_append_writes_its_rows_and_no_other_byte(lyc, page):
    """Codes and scales of K and of V against the definition by search, and every other
    byte of the four tensors as it was, around rows written at ragged lengths; then
    the same where elements and pages are refused."""
    B, T, hkv, d, cap = 4, 9, 3, 128, 130
    rng = np.random.default_rng(page)
    cache = fill(lyc, B, hkv, d, cap, page, True, seed=50 + page)
    tensors = [x.view(torch.uint8) for x in cache.tensors[:4]]
    bt = cache.tensors[4]
    for refuse in (False, True):
        before = [x.clone() for x in tensors]
        cnt = [T, 0, 4, 1]
        n = [cap, 77, 4, 65]
        bad = set()
        if refuse:
            n[0] = 3  # fewer rows than tokens
            bad.add(0)
            if page:
                bt[3, 64 // page] = 10**6
                bad.add(3)
        k, v = randn(60 + refuse, B, T, hkv, d), randn(61 + refuse, B, T, hkv, d, scale=1e-3)
        st = status_word()
        lyc.cache_append(cache, i32(n), k, v, t_len=i32(cnt), status=st)
        assert (int(st) != 0) == refuse
        want = [x.clone() for x in before]
        for b in range(B):
            if b in bad:
                continue
            for t in range(cnt[b]):
                row = n[b] - cnt[b] + t
                for i, x in ((0, k), (1, v)):
                    code, byte = SS.e4m3_row(x[b, t].cpu())
                    at = (b, slice(None), row) if bt is None else (int(bt[b, row // page]), row % page)
                    want[i][at] = code.to(torch.uint8).cuda()
                    want[2 + i][at] = byte.to(torch.uint8).cuda()
        for name, x, w in zip(("k", "v", "k_scale", "v_scale"), tensors, want):
            assert torch.equal(x, w), name


# ------------------------------------------------------------------ errors


def test_a_refused_device_leaves_no_error_behind(lyc):
    """A device that is not there is refused with its code, the current device stays,
    and the program's next CUDA calls do not meet the error."""
    cache = fill(lyc, 1, 1, 64, 40, 0, False, seed=1)
    q = randn(2, 1, 2, 2, 64)
    out, _ = run_tree(lyc, cache, q, [40])
    a = lyc.lyc_layer_cache.from_buffer_copy(cache.desc)
    a.device = torch.cuda.device_count() + 7
    assert lyc.lyc_tree_workspace_bytes(a, 2, 2) == 0 and lyc.lyc_operator_status() == lyc.LYC_ERR_CUDA
    n, ko = i32([40]), torch.zeros((1, 1, 4, 64), dtype=BF, device="cuda")
    args = lyc.lyc_read_args(ko.data_ptr(), ko.data_ptr(), 256, 256, 64, n.data_ptr(), None, 0, 4, 1, lyc.LYC_BF16, None)
    assert lyc.lyc_cache_read(a, args, None) == lyc.LYC_ERR_CUDA
    assert torch.cuda.current_device() == 0
    again, _ = run_tree(lyc, cache, q, [40])
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    # an entry point that asks for the last error after its launch
    qs, k = randn(3, 1, 2, 64), randn(4, 1, 1, 1, 40, 64)
    kv = lyc.lyc_kv_cache(k.data_ptr(), k.data_ptr(), 40, 0, *k.stride()[1:4])
    S = torch.arange(8, device="cuda", dtype=torch.int32).expand(1, 2, 8).contiguous()
    o = torch.empty((1, 2, 64), device="cuda")
    assert lyc.lyc_cache_read(a, args, None) == lyc.LYC_ERR_CUDA
    assert lyc.lyc_sparse_attention_noalloc(qs.data_ptr(), kv, 1, 2, 1, 64, S.data_ptr(), 8, o.data_ptr(), None,
                                            torch.cuda.current_stream().cuda_stream) == lyc.LYC_OK
    torch.cuda.synchronize()


def test_numbers_that_do_not_fit_are_refused(lyc):
    """An eps or a scale past fp32, a first row past 64 bits, what is no number: refused
    as other wrong arguments are."""
    cache = fill(lyc, 1, 1, 64, 40, 0, True, seed=1)
    q, k, n, ko = randn(2, 1, 2, 2, 64), randn(3, 1, 2, 1, 64), i32([40]), torch.zeros((1, 1, 4, 64), dtype=BF, device="cuda")
    out, v = torch.zeros_like(q), ko.clone()
    bad = [lambda: lyc.qk_norm_rope(q[0], None, None, None, out[0], None, eps=1e39),
           lambda: lyc.cache_append(cache, n, k, k, eps=1e39),
           lambda: lyc.cache_append(cache, n, k, k, eps="small"),
           lambda: lyc.cache_read(cache, n, ko, v, first=1 << 64),
           lambda: lyc.cache_read(cache, n, ko, v, first=0.5),
           lambda: lyc.tree_attention(q, cache, n, out, scale=1e39)]
    for i, call in enumerate(bad):
        with pytest.raises(lyc.LycError) as e:
            call()
        assert e.value.code == lyc.LYC_ERR_INVALID_ARG, i
    assert not out.any() and not ko.any()
