"""More of the serving operators' refusals, on the host alone: codes that reach the
caller, and addresses that the device could not read (no GPU needed: the pointers
are never followed)."""
from types import SimpleNamespace

import pytest

from tests.test_serve_ops_args import P, append, cache, calls, lyc, paged, read, rope, tree  # noqa: F401


def test_workspace_refusals_keep_their_code(lyc):  # noqa: F811
    handle = SimpleNamespace(desc=cache(lyc), _workspace={})
    for T, hq, code in ((257, 8, lyc.LYC_ERR_UNSUPPORTED), (0, 8, lyc.LYC_ERR_UNSUPPORTED), (4, 7, lyc.LYC_ERR_INVALID_ARG)):
        with pytest.raises(lyc.LycError) as e:
            lyc.tree_workspace_bytes(handle, T, hq)
        assert e.value.code == code == lyc.lyc_operator_status()
    handle.desc = cache(lyc, device=1 << 20)
    with pytest.raises(lyc.LycError) as e:
        lyc.tree_workspace_bytes(handle, 4, 8)
    assert e.value.code == lyc.LYC_ERR_CUDA
    assert not handle._workspace


def test_words_that_are_not_aligned(lyc):  # noqa: F811
    """Lengths, positions, tables, sets, masks and the status word are read and written
    whole: an address that is not their elements' is refused."""
    odd = P + 2
    for kw in (dict(pos=odd), dict(inv_freq=odd)):
        assert lyc.lyc_qk_norm_rope(rope(lyc, **kw), None) == -1
        assert "aligned" in lyc.lyc_operator_error()
    for kw in (dict(n=odd), dict(t_len=odd), dict(pos=odd), dict(inv_freq=odd, rot_dim=16), dict(status=odd)):
        assert lyc.lyc_cache_append(cache(lyc), append(lyc, **kw), None) == -1
        assert "aligned" in lyc.lyc_operator_error()
    for kw in (dict(n=odd), dict(sets=odd), dict(status=odd)):
        assert lyc.lyc_cache_read(cache(lyc), read(lyc, **kw), None) == -1
        assert "aligned" in lyc.lyc_operator_error()
    for kw in (dict(n=odd), dict(t_len=odd), dict(mask=P + 4), dict(status=odd)):
        assert lyc.lyc_tree_attention(cache(lyc), tree(lyc, **kw), None) == -1
        assert "aligned" in lyc.lyc_operator_error()
    for name, rc in calls(lyc, paged(lyc, block_table=odd)):
        assert rc == -1 and "aligned" in lyc.lyc_operator_error(), name
    assert lyc.lyc_tree_workspace_bytes(paged(lyc, block_table=odd), 4, 8) == 0
    # no rotation: pos and inv_freq are not read, whatever they are
    assert lyc.lyc_qk_norm_rope(rope(lyc, rot_dim=0, pos=odd, inv_freq=odd, rows=0), None) == 0
