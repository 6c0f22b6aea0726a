"""GPU tests that the first call of a process may be a captured one."""

import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import os, sys
sys.path.insert(0, os.path.join(os.getcwd(), "tests"))
import torch
import dequant_gemm_int4_b200 as q4
from cache_checks import made_cache, made_table
path, op = int(sys.argv[1]), sys.argv[2]
table, pages = made_table([300, 70], 16)
packed, scales, zeros = made_cache(pages, 16, 2, 64, 64, True)
q = torch.randn((8, 4, 64), device="cuda").bfloat16()
lens = torch.tensor([300, 70], dtype=torch.int32, device="cuda")
slots = torch.arange(8, device="cuda")
k = torch.randn((8, 2, 64), device="cuda").bfloat16()
def call():
    if op == "write":
        q4.int4_cache_write(k, k, packed, scales, slots, 64, zeros=zeros)
    if op != "attend":
        return q4.int4_cache_read(packed, scales, slots, 64, 64, zeros=zeros)
    return q4.int4_cache_attention(q, packed, scales, table, lens, 64, zeros=zeros, return_lse=True, path=path)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = call()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, call()))
assert q4.device_status() == q4.OK
"""


@pytest.mark.parametrize("path, op", [(1, "attend"), (2, "attend"), (3, "attend"), (0, "read"), (0, "write")])
def test_the_first_call_is_captured(path, op):
    run = subprocess.run([sys.executable, "-c", CODE, str(path), op], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr[-2000:]
