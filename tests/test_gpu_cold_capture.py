"""The first calls of a process may be captured ones: nothing is left for a warm-up."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import torch
from quantized_expert_ffn_gemv_gb300 import attention, sampling
torch.manual_seed(0)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
T, D = {T}, {D}
cache = attention.KvCache(8, 64, 2, D, {bits})
batch = attention.KvBatch(i32([[3, 1, 0, 5]]), i32([200]), i32([0, T]), T, T)
table = attention.rope_table(256, 64, 1e4)
q, k, v = (torch.randn(T, n, D, device="cuda").{dtype}() for n in (4, 2, 2))
z, u = torch.randn(3, 40000, device="cuda"), torch.rand(3, device="cuda")
cache.data.fill_(128 if {bits} == 8 else 0x88)
out = []

def run():
    r = cache.append_norm_rope(q, k, v, batch, table)
    out[:] = [r, cache.attend(r, batch), *cache.read(batch, dtype=q.dtype), *sampling.sample(z, u)]

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
first = [x.clone() for x in out]
run()
cache.check()
assert all(torch.equal(a, b) for a, b in zip(first, out))
"""


@pytest.mark.parametrize("T,D,bits,dtype", [(1, 128, 8, "bfloat16"), (90, 128, 4, "half"), (30, 256, 4, "bfloat16")])
def test_first_call_captured(T, D, bits, dtype):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE.format(T=T, D=D, bits=bits, dtype=dtype)], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
