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
