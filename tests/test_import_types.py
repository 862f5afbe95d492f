"""The package's paged cache with a torch that lacks the type of two 4-bit codes: everything else of it is there."""
import subprocess
import sys

CODE = """
import torch
del torch.float4_e2m1fn_x2
import context_parallelism_fcp_gb300 as fcp
from context_parallelism_fcp_gb300 import paged
assert {fcp.PagedCache, fcp.PagePool, fcp.Rotary} and callable(fcp.rotary_write)
assert set(paged._DTYPES) == {torch.bfloat16, torch.float8_e4m3fn}
for dtype in (None, torch.float32):
    try:
        fcp.PagedCache(4, 16, 2, 64, dtype=dtype, device="cpu")
    except TypeError as e:
        assert "dtype must be" in str(e)
    else:
        raise AssertionError("no such cache")
for dtype in (torch.bfloat16, torch.float8_e4m3fn):
    try:
        fcp.PagedCache(4, 16, 2, 64, dtype=dtype, device="cpu")
    except ValueError as e:
        assert "CUDA" in str(e)  # as ever on the CPU: nothing of the missing type stood in the way
    else:
        raise AssertionError("a cache on the CPU")
try:
    fcp.PagedCache.wrap(torch.zeros(4, 2, 16, 64), None)
except TypeError as e:
    assert "bfloat16" in str(e)
print("fine")
"""


def test_without_the_4_bit_type(fcp):
    import os

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", CODE], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip().endswith("fine"), run.stderr[-2000:]
