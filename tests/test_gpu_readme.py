"""The README's serving example, run as it is printed: prompts, then a decode step whose
selections are those of all complete blocks, the prompt's and the new ones among them."""

import os
import re

import pytest
import torch

import block_sparse_attention_key_b200 as qsa

import gpu_util as gu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    gu.ensure_built()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_the_paged_4_bit_example_selects_among_every_complete_block():
    text = open(os.path.join(ROOT, "README.md")).read()
    block = re.search(r"```python\n(import torch.*?)```", text, re.S).group(1)
    setup, prompts, decode = re.split(r"^(?=# prompts|# decode)", block, flags=re.M)
    # one sequence per slot: 2,603 tokens (its 651st block is completed by the decode step), 5, and an ended one
    batch, hq, hkv, cap, page, n_pages = 3, 8, 2, 4096, 64, 100
    g = torch.Generator(device="cuda").manual_seed(40)
    rnd = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    lens, n_tok = [2603, 5, 70], 2678
    # a block's score is its rank: 32 x (its tokens' first dim) + the second, exact in bf16 and fp32
    idx_k = torch.zeros((batch, cap, 64), dtype=torch.bfloat16, device="cuda")
    rank = torch.randperm(cap // 4, generator=g, device="cuda").repeat_interleave(4)
    idx_k[:, :, 0], idx_k[:, :, 1] = rank // 32, rank % 32
    q_idx = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    q_idx[:, 0, 0], q_idx[:, 0, 1] = 32, 1
    name = dict(batch=batch, n_q_heads=hq, n_kv_heads=hkv, kv_capacity=cap, page=page, n_pages=n_pages)
    exec(setup, name)
    dims = name["dims"]
    ws = gu.new_workspace(max(qsa.qsa_pages_workspace_bytes(dims, page, n_pages),
                              qsa.qsa_workspace_bytes(dims, batch, cap // 4, qsa.QSA_MODE_DECODE)))
    name.update(q=rnd(n_tok, hq, 128), k=rnd(n_tok, hkv, 128), v=rnd(n_tok, hkv, 128), cu_len=_i32([0, 2603, 2608, 2678]),
                n_tok=n_tok, out=torch.empty((n_tok, hq, 128), dtype=torch.bfloat16, device="cuda"), workspace=ws,
                len_before=_i32([0, 0, 0]), len_after=_i32(lens), idx_k=idx_k, longest=2603,
                pooled=torch.zeros((batch, cap // 4, 64), dtype=torch.bfloat16, device="cuda"))
    exec(prompts, name)
    assert torch.isfinite(name["out"]).all()
    # the third request ended, the second is forked into its slot; all three append one token
    name.update(ended=_i32([2]), n=1, src=_i32([1]), dst=_i32([2]), m=1, len_before=_i32([2603, 5, 5]),
                len_after=_i32([2604, 6, 6]), k1=rnd(3, hkv, 128), v1=rnd(3, hkv, 128), cu_one=_i32([0, 1, 2, 3]),
                q_idx=q_idx[[0, 0, 1]].contiguous(), w=torch.ones((3, 4), device="cuda"), q_seq=_i32([0, 1, 2]),
                q_pos=_i32([2603, 5, 5]), max_blocks=cap // 4, q1=rnd(3, hq, 128),
                sel_idx=torch.empty((3, 512), dtype=torch.int32, device="cuda"), sel_cnt=_i32([0, 0, 0]),
                out1=torch.empty((3, hq, 128), dtype=torch.bfloat16, device="cuda"))
    name["pooled"][2] = name["pooled"][1]
    exec(decode, name)
    assert qsa.qsa_read_device_status(ws) == 0
    best = rank[::4][:651].topk(512).indices.sort().values
    assert name["sel_cnt"].tolist() == [512, 1, 1]
    assert torch.equal(name["sel_idx"][0].long(), best)
    assert name["sel_idx"][1, 0] == 0 and name["sel_idx"][2, 0] == 0
    assert torch.isfinite(name["out1"]).all()
    # one page of the fork is shared no more: each has its own token behind the common five
    assert name["table"][1, 0] != name["table"][2, 0] and not torch.equal(name["out1"][1], name["out1"][2])
