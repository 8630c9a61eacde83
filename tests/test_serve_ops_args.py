"""The serving operators' refusals, on the host alone: every bad argument is
turned away before anything is enqueued, with a code and a reason (no GPU
needed: the pointers are never followed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lyc():
    from hybrid_head_sparse_b200 import build as B
    B.build()
    from hybrid_head_sparse_b200 import lyc as m
    m.load()
    return m


P = 1 << 20  # an aligned address that nothing reads


def cache(lyc, **kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, s_batch=4096 * 256, s_head=4096 * 128, s_token=128, ss_batch=8192,
             ss_head=4096, ss_token=1, rows=4096, type=lyc.LYC_CACHE_E4M3, batch=2, num_kv_heads=2, head_dim=128)
    d.update(kw)
    return lyc.lyc_layer_cache(**d)


def paged(lyc, **kw):
    return cache(lyc, **{**dict(block_table=P, page_rows=16, max_blocks=8, num_pages=40, s_page=16 * 256, s_token=256,
                                s_head=128, ss_page=32, ss_head=16, rows=0), **kw})


def rope(lyc, **kw):
    d = dict(q=P, k=P, q_out=P, k_out=P, q_row=1024, q_head=128, k_row=256, k_head=128, qo_row=1024, qo_head=128,
             ko_row=256, ko_head=128, pos=P, inv_freq=P, rows=4, num_q_heads=8, num_kv_heads=2, head_dim=128,
             rot_dim=128, eps=1e-6)
    d.update(kw)
    return lyc.lyc_rope_args(**d)


def append(lyc, **kw):
    d = dict(k=P, v=P, k_batch=1024, k_token=256, k_head=128, v_batch=1024, v_token=256, v_head=128, n=P, T=4, eps=1e-6)
    d.update(kw)
    return lyc.lyc_append_args(**d)


def read(lyc, **kw):
    d = dict(k_out=P, v_out=P, o_batch=4096, o_head=2048, o_row=128, n=P, m=16, num_heads=2)
    d.update(kw)
    return lyc.lyc_read_args(**d)


def tree(lyc, **kw):
    d = dict(q=P, out=P, q_batch=4096, q_token=1024, q_head=128, o_batch=4096, o_token=1024, o_head=128, n=P, T=4,
             num_q_heads=8, scale=0.1, workspace=P, workspace_bytes=1 << 40)
    d.update(kw)
    return lyc.lyc_tree_args(**d)


CACHES = [
    (dict(k=None), -1), (dict(v=P + 8), -1), (dict(k_scale=None), -1), (dict(type=2), -1),
    (dict(type=0), -1), (dict(head_dim=96), -2), (dict(batch=0), -1), (dict(num_kv_heads=0), -1),
    (dict(rows=0), -1), (dict(rows=(1 << 30) + 1), -1), (dict(s_token=120), -1), (dict(s_token=136), -1),
    (dict(s_token=-128), -1), (dict(s_head=64), -1), (dict(s_batch=8), -1), (dict(ss_token=-1), -1),
]
PAGED = [
    (dict(page_rows=0), -1), (dict(max_blocks=0), -1), (dict(num_pages=0), -1), (dict(s_page=100), -1),
    (dict(page_rows=1 << 20, max_blocks=1 << 11), -1), (dict(num_pages=1 << 31), -1),
]


def calls(lyc, c):
    yield "append", lyc.lyc_cache_append(c, append(lyc), None)
    yield "read", lyc.lyc_cache_read(c, read(lyc), None)
    yield "tree", lyc.lyc_tree_attention(c, tree(lyc), None)


@pytest.mark.parametrize("kw,code", CACHES)
def test_bad_caches(lyc, kw, code):
    for name, rc in calls(lyc, cache(lyc, **kw)):
        assert rc == code, (name, lyc.lyc_operator_error())
        assert lyc.lyc_operator_error()
    assert lyc.lyc_tree_workspace_bytes(cache(lyc, **kw), 1, 8) == 0


@pytest.mark.parametrize("kw,code", PAGED)
def test_bad_paged_caches(lyc, kw, code):
    for name, rc in calls(lyc, paged(lyc, **kw)):
        assert rc == code, (name, lyc.lyc_operator_error())


def test_a_cache_that_is_written_needs_rows_of_its_own(lyc):
    for kw in (dict(s_batch=0), dict(ss_token=0), dict(ss_head=0)):
        assert lyc.lyc_cache_append(cache(lyc, **kw), append(lyc), None) == -1
    shared = cache(lyc, s_batch=0)  # one prefix read by every element is fine to read
    assert lyc.lyc_cache_read(shared, read(lyc, m=0), None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(q=None, k=None), -1), (dict(q_out=None), -1), (dict(k_out=P + 2), -1), (dict(q_weight=P + 4), -1),
    (dict(dtype=2), -1), (dict(head_dim=80), -2), (dict(rows=-1), -1), (dict(rot_dim=24), -1), (dict(rot_dim=144), -1),
    (dict(rot_dim=-16), -1), (dict(inv_freq=None), -1), (dict(pos=None), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(q_head=132), -1), (dict(qo_row=64), -1), (dict(k_row=-256), -1),
    (dict(num_q_heads=0), -1), (dict(num_kv_heads=0), -1),
])
def test_bad_rope(lyc, kw, code):
    assert lyc.lyc_qk_norm_rope(rope(lyc, **kw), None) == code, lyc.lyc_operator_error()


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(n=None), dict(T=0), dict(T=1 << 30), dict(v=P + 8), dict(k_token=100), dict(v_head=-128),
    dict(rot_dim=8), dict(rot_dim=128), dict(q=P), dict(q_out=P), dict(q_weight=P), dict(eps=float("inf")),
    dict(q=P, q_out=P, num_q_heads=0), dict(q=P, q_out=P, num_q_heads=8, qo_batch=4096, qo_token=8, qo_head=128),
])
def test_bad_append(lyc, kw):
    assert lyc.lyc_cache_append(cache(lyc), append(lyc, **kw), None) == -1
    assert lyc.lyc_operator_error()


@pytest.mark.parametrize("kw", [
    dict(k_out=None), dict(n=None), dict(v_out=P + 4), dict(m=-1), dict(first=-1), dict(num_heads=3), dict(num_heads=4),
    dict(num_heads=0, sets=P), dict(num_heads=5, sets=P), dict(sets=P, first=1), dict(o_row=100), dict(o_head=0), dict(dtype=3),
])
def test_bad_read(lyc, kw):
    assert lyc.lyc_cache_read(cache(lyc), read(lyc, **kw), None) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(out=P + 8), -1), (dict(n=None), -1), (dict(T=0), -2), (dict(T=257), -2),
    (dict(num_q_heads=7), -1), (dict(num_q_heads=0), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(q_head=100), -1), (dict(o_token=0), -1),
])
def test_bad_tree(lyc, kw, code):
    assert lyc.lyc_tree_attention(cache(lyc), tree(lyc, **kw), None) == code, lyc.lyc_operator_error()


def test_null_structs_and_nothing_to_do(lyc):
    lib = lyc.load()
    assert lib.lyc_qk_norm_rope(None, None) == -1
    assert lib.lyc_cache_append(None, ctypes.byref(append(lyc)), None) == -1
    assert lib.lyc_cache_append(cache(lyc), None, None) == -1
    assert lib.lyc_cache_read(cache(lyc), None, None) == -1
    assert lib.lyc_tree_attention(cache(lyc), None, None) == -1
    assert lib.lyc_tree_attention(None, ctypes.byref(tree(lyc)), None) == -1
    # no rows: nothing is enqueued, and no device is needed
    assert lyc.lyc_qk_norm_rope(rope(lyc, rows=0), None) == 0
    assert lyc.lyc_cache_read(cache(lyc), read(lyc, m=0), None) == 0


def test_mirrors_follow_the_header(lyc, tmp_path):
    """Sizes and offsets of the ctypes structs against the C compiler's."""
    import os
    import subprocess
    names = ["lyc_layer_cache", "lyc_rope_args", "lyc_append_args", "lyc_read_args", "lyc_tree_args"]
    lines = []
    for n in names:
        lines.append(f'printf("{n} . %zu\\n", sizeof({n}));')
        lines += [f'printf("{n} {f} %zu\\n", offsetof({n}, {f}));' for f, _ in getattr(lyc, n)._fields_]
    src = tmp_path / "sizes.c"
    src.write_text('#include "lyc.h"\n#include <stdio.h>\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0;\n}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "sizes")], check=True)
    for line in subprocess.run([str(tmp_path / "sizes")], capture_output=True, text=True, check=True).stdout.splitlines():
        n, f, value = line.split()
        cls = getattr(lyc, n)
        assert int(value) == (ctypes.sizeof(cls) if f == "." else getattr(cls, f).offset), (n, f)


def test_wrapper_refuses_tensors_off_the_gpu(lyc):
    import torch
    k = torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(lyc.LycError) as e:
        lyc.KvCache(k, k)
    assert e.value.code == lyc.LYC_ERR_INVALID_ARG
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(lyc.LycError):
        lyc.qk_norm_rope(q, None, torch.zeros(2, dtype=torch.int32), torch.ones(32), q, None)


def test_pages_and_scales_that_are_written_lie_apart(lyc):
    for kw in (dict(s_page=0), dict(s_page=64), dict(ss_page=0)):
        assert lyc.lyc_cache_append(paged(lyc, **kw), append(lyc), None) == -1
        assert "of its own" in lyc.lyc_operator_error() or "of their own" in lyc.lyc_operator_error()
    assert lyc.lyc_cache_append(cache(lyc, ss_batch=0), append(lyc), None) == -1
    assert lyc.lyc_cache_read(paged(lyc, s_page=0, ss_page=0), read(lyc, m=0), None) == 0
