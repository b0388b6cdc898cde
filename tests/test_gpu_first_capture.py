"""The serving operators' first call in a process may be one that a graph captures."""

import os
import subprocess
import sys

import pytest
import torch

import gpu_util as gu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
import torch
import block_sparse_attention_key_b200 as qsa

i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
rnd = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)
n, hq, hkv, cap, page = 50, 8, 2, 128, 16
dims = qsa.make_dims(1, hq, hkv, cap)
t = [torch.zeros((cap // page, hkv, page, w), dtype=torch.uint8, device="cuda") for w in (64, 8, 64, 8)]
table, ref = torch.full((1, cap // page), -1, dtype=torch.int32, device="cuda"), i32([0] * (cap // page))
cache, pools = qsa.kv4_cache(*t, table, page, cap // page), qsa.page_pools(t, page, cap // page)
q, k, v, out = rnd(n, hq, 128), rnd(n, hkv, 128), rnd(n, hkv, 128), torch.zeros((n, hq, 128), dtype=torch.bfloat16, device="cuda")
q1, out1, seq, pos = rnd(1, hq, 128), torch.zeros((1, hq, 128), dtype=torch.bfloat16, device="cuda"), i32([0]), i32([n - 1])
sel, cnt = torch.full((1, 512), -1, dtype=torch.int32, device="cuda"), i32([12])
sel[0, :12] = torch.arange(12)
cu, before, after, live = i32([0, n]), i32([0]), i32([n]), i32([0])
ws = torch.zeros(qsa.qsa_pages_workspace_bytes(dims, page, cap // page), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
calls = dict(
    prompt=lambda: qsa.qsa_prompt_attn(dims, q, k, v, cu, n, out, ws),
    update=lambda: qsa.qsa_pages_update(dims, pools, table, ref, before, after, ws),
    append=lambda: qsa.qsa_kv4_append(dims, cache, k, v, cu, before, n, ws),
    attend=lambda: qsa.qsa_sparse_attn_kv4(dims, cache, q1, seq, pos, sel, cnt, 1, out1, ws),
    compact=lambda: qsa.qsa_pages_compact(dims, pools, table, ref, live, ws))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
    for name in sys.argv[1].split(","):
        calls[name]()
graph.replay()
torch.cuda.synchronize()
got = out.clone(), out1.clone(), table.clone(), live.clone()
table.fill_(-1), ref.fill_(0), live.fill_(0), out.fill_(0), out1.fill_(0), [x.fill_(0) for x in t]
for name in sys.argv[1].split(","):
    calls[name]()
assert qsa.qsa_read_device_status(ws) == 0
for a, b in zip(got, (out, out1, table, live)):
    assert torch.equal(a, b)
print("replayed")
"""


@pytest.mark.parametrize("calls", ["prompt", "update,append,attend,compact"])
def test_the_first_call_of_a_process_is_captured(calls):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    gu.ensure_built()
    r = subprocess.run([sys.executable, "-c", CODE, calls], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "replayed" in r.stdout, r.stderr[-2000:]
