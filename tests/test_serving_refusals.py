"""Argument checks of the serving operators: host only, nothing is launched."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def qsa():
    from block_sparse_attention_key_b200 import build, qsa
    build.build()
    qsa.load()
    if torch.cuda.is_available():
        pytest.skip("uses fabricated addresses: host-only test")
    return qsa


def _dims(qsa, **kw):
    base = dict(batch=4, n_q_heads=32, n_kv_heads=4, kv_capacity=4096)
    base.update(kw)
    return qsa.make_dims(**base)


def test_prompt_refusals(qsa):
    lib = qsa.load()
    d = _dims(qsa)
    good = dict(q=16, k=16, v=16, q_ld=4096, k_ld=512, v_ld=512, cu_len=16, n_tok=100, out=16)

    def call(dims=d, ws=None, **kw):
        a = qsa.qsa_prompt_args(**{**good, **kw})
        return lib.qsa_prompt_attn(ctypes.byref(dims), ctypes.byref(a), ws, None)

    for kw in (dict(q=None), dict(k=8), dict(v=None), dict(cu_len=None), dict(out=24), dict(n_tok=-1), dict(q_ld=4095),
               dict(q_ld=4088), dict(k_ld=504), dict(v_ld=516), dict(ws=8), dict(dims=_dims(qsa, n_q_heads=30))):
        assert call(**kw) == qsa.QSA_ERR_INVALID_ARG, kw
    assert lib.qsa_prompt_attn(ctypes.byref(d), None, None, None) == qsa.QSA_ERR_INVALID_ARG
    for kw in (dict(n_tok=(1 << 30) + 1), dict(dims=_dims(qsa, n_q_heads=33 * 4)), dict(dims=_dims(qsa, head_dim=64)),
               dict(k_ld=1 << 38)):
        assert call(**kw) == qsa.QSA_ERR_UNSUPPORTED, kw
    assert call(n_tok=0, q=None, out=None) == qsa.QSA_OK


def test_prompt_binding_checks_types_shapes_and_strides(qsa):
    d = _dims(qsa, n_q_heads=2, n_kv_heads=1, batch=1)
    bf = torch.bfloat16
    q, k, cu = torch.zeros(5, 2, 128, dtype=bf), torch.zeros(5, 1, 128, dtype=bf), torch.zeros(2, dtype=torch.int32)
    for bad in (dict(q=q.float()), dict(k=k[:4]), dict(q=q[:, :1])):
        a = {**dict(q=q, k=k, v=k), **bad}
        with pytest.raises(ValueError, match="expected"):
            qsa.qsa_prompt_attn(d, a["q"], a["k"], a["v"], cu, 5, q)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.qsa_prompt_attn(d, q, k, k, cu, 5, q)


def test_tensors_of_another_device_are_refused(qsa, monkeypatch):
    class Far:
        is_cuda = True
        device = torch.device("cuda", 1)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        qsa._here(None, Far())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    qsa._here(None, Far())
