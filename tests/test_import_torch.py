"""The binding under a torch that lacks the 4-bit types: it loads, and every other call is as it was.

CPU only, in a process of its own."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in ("float4_e2m1fn_x2", "float8_e8m0fnu"):
    if hasattr(torch, name):
        delattr(torch, name)
import draft_selection_amd as ds
for dt, code in ((torch.bfloat16, 1), (torch.float8_e4m3fn, 2)):
    k = torch.zeros((3, 16, 2, 64), dtype=torch.uint8).to(dt)
    packed, shape = ds._cache(k.device, k, k)
    assert shape == (1, 3, 16, 2, 64) and ds.CacheArgs.from_buffer_copy(packed).dt == code
    assert ds.tree_attn_workspace_bytes(2, 9, 32, 8, 128, dt, 1 << 20) > 0
    assert ds._moving(k, k, k) == (None, None)
for dt in (torch.float16, torch.uint8):
    k = torch.zeros((3, 16, 2, 64), dtype=dt)
    try:
        ds._cache(k.device, k, k)
    except TypeError:
        continue
    raise SystemExit("taken: %s" % dt)
print("as before")
"""


def test_a_torch_without_the_types_of_four_bits():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as before" in r.stdout, r.stdout + r.stderr
