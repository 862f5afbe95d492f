"""The paged cache's names and refusals that need no GPU."""
import os
import subprocess
import sys

import pytest


@pytest.mark.parametrize("how", ["blocked", "absent", "broken"])
def test_a_star_import_needs_no_torch(tmp_path, how):
    """Without torch the package's host plan works, and a star import takes what there is."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    (tmp_path / "torch").mkdir()
    (tmp_path / "torch" / "__init__.py").write_text("raise ImportError('not this one')\n")
    start = {"blocked": "import sys; sys.modules['torch'] = None",
             "absent": "import sys, importlib.abc\n"
                       "class F(importlib.abc.MetaPathFinder):\n"
                       "    def find_spec(self, name, path, target=None):\n"
                       "        if name.split('.')[0] == 'torch': raise ModuleNotFoundError(name, name=name)\n"
                       "sys.meta_path.insert(0, F())",
             "broken": f"import sys; sys.path.insert(0, {str(tmp_path)!r})"}[how]
    code = start + """
from context_parallelism_fcp_gb300 import *
assert Plan and FcpError and MASK_FULL == 0 and callable(block_attn_fwd)
assert 'PagedCache' not in globals()
import context_parallelism_fcp_gb300 as fcp
assert 'PagedCache' not in fcp.__all__ and 'Plan' in fcp.__all__
try:
    fcp.PagedCache
except ImportError:
    print('fine')
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


def test_a_star_import_takes_the_cache(fcp):
    names = {}
    exec("from context_parallelism_fcp_gb300 import *", names)
    assert names["PagedCache"] is fcp.PagedCache and names["Plan"] is fcp.Plan
    assert set(fcp.__all__) <= set(dir(fcp))


@pytest.mark.parametrize("shape", [(2, 0, 16, 64), (0, 0, 16, 64)])
def test_a_cache_without_heads_is_refused(fcp, shape):
    import torch

    pages = torch.zeros(shape, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="KV head"):
        fcp.PagedCache.wrap(pages, pages.clone())
    with pytest.raises(ValueError, match="KV head"):
        fcp.PagedCache(shape[0], shape[2], shape[1], shape[3], device="cpu")
