"""Argument checks of the serving operators: host only, nothing is launched."""

import ctypes
import os

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


class _On:
    """A CPU tensor that says it lies on a CUDA device."""

    def __init__(self, t, dev=0):
        self.t, self.dev = t, dev

    def get_device(self):
        return self.dev

    def view(self, *a):
        return _On(self.t.view(*a), self.dev)

    def __getattr__(self, name):
        return getattr(self.t, name)


def _on(*s, dtype=torch.int32, dev=0):
    return _On(torch.zeros(s, dtype=dtype), dev)


@pytest.fixture
def device0(qsa, monkeypatch):
    monkeypatch.setattr(qsa, "_current_device", lambda: 0)


def test_prompt_binding_checks_types_shapes_strides_and_devices(qsa, device0):
    d = _dims(qsa, n_q_heads=2, n_kv_heads=2, batch=1)
    bf = torch.bfloat16
    good = dict(q=_on(5, 2, 128, dtype=bf), k=_on(5, 2, 128, dtype=bf), v=_on(5, 2, 128, dtype=bf), cu=_on(2),
                out=_on(5, 2, 128, dtype=bf))

    def call(**kw):
        a = {**good, **kw}
        qsa.qsa_prompt_attn(d, a["q"], a["k"], a["v"], a["cu"], 5, a["out"], a.get("ws"))

    for bad in (dict(q=_on(5, 2, 128)), dict(k=_on(4, 2, 128, dtype=bf)), dict(v=_on(5, 1, 128, dtype=bf)), dict(cu=_on(3)),
                dict(out=_on(5, 2, 64, dtype=bf))):
        with pytest.raises(ValueError, match="expected"):
            call(**bad)
    apart = _On(torch.zeros(5, 128, 2, dtype=bf).transpose(1, 2))
    with pytest.raises(ValueError, match="heads of a token"):
        call(k=apart)
    with pytest.raises(ValueError, match="contiguous"):
        call(out=apart)
    with pytest.raises(ValueError, match="CUDA"):
        call(q=good["q"].t)
    for name in good:
        x = good[name]
        with pytest.raises(ValueError, match="current device"):
            call(**{name: _On(x.t, 1)})
    with pytest.raises(ValueError, match="current device"):
        call(ws=_on(256, dtype=torch.uint8, dev=1))


def _cache(qsa, **kw):
    base = dict(k_codes=16, k_scales=32, v_codes=48, v_scales=64, page_table=None, page_tokens=0, n_pages=0)
    return qsa.qsa_kv4_cache(**{**base, **kw})


def test_kv4_append_refusals(qsa):
    lib = qsa.load()
    d = _dims(qsa)
    good = dict(k=16, k_ld=512, v=16, v_ld=512, cu=16, before=16, n=5)

    def call(dims=d, cache=None, ws=None, **kw):
        a = {**good, **kw}
        return lib.qsa_kv4_append(ctypes.byref(dims), ctypes.byref(cache or _cache(qsa)), a["k"], a["k_ld"], a["v"],
                                  a["v_ld"], a["cu"], a["before"], a["n"], ws, None)

    for kw in (dict(k=None), dict(v=8), dict(cu=None), dict(before=4), dict(n=-1), dict(k_ld=504), dict(v_ld=515), dict(ws=8),
               dict(cache=_cache(qsa, k_codes=None)), dict(cache=_cache(qsa, v_scales=24)),
               dict(cache=_cache(qsa, page_table=16, page_tokens=6, n_pages=4)),
               dict(cache=_cache(qsa, page_table=16, page_tokens=16, n_pages=0)),
               dict(cache=_cache(qsa, page_table=16, page_tokens=4096 * 2, n_pages=4))):
        assert call(**kw) == qsa.QSA_ERR_INVALID_ARG, kw
    assert lib.qsa_kv4_append(ctypes.byref(d), None, 16, 512, 16, 512, 16, 16, 1, None, None) == qsa.QSA_ERR_INVALID_ARG
    assert call(dims=_dims(qsa, n_q_heads=1 << 20, n_kv_heads=1 << 20), k_ld=1 << 27, v_ld=1 << 27,
                n=1 << 20) == qsa.QSA_ERR_UNSUPPORTED
    assert call(n=0, k=None) == qsa.QSA_OK


def test_kv4_attention_refusals(qsa):
    lib = qsa.load()
    d = _dims(qsa)
    good = dict(q=16, q_seq=16, q_pos=16, sel_idx=16, sel_cnt=16, n_q=4, group_q=1, out=16)

    def call(dims=d, cache=None, ws=None, **kw):
        a = qsa.qsa_attn_args(**{**good, **kw})
        return lib.qsa_sparse_attn_kv4(ctypes.byref(dims), ctypes.byref(cache or _cache(qsa)), ctypes.byref(a), ws, None)

    for kw in (dict(q=None), dict(q_seq=4), dict(q_pos=None), dict(sel_idx=8), dict(sel_cnt=None), dict(out=None),
               dict(n_q=-1), dict(group_q=0), dict(group_q=3), dict(k_cache=16), dict(v_cache=16), dict(page_table=16),
               dict(page_tokens=16), dict(n_pages=1), dict(ws=24), dict(cache=_cache(qsa, k_scales=None)),
               dict(cache=_cache(qsa, page_table=16, page_tokens=16, n_pages=-1))):
        assert call(**kw) == qsa.QSA_ERR_INVALID_ARG, kw
    assert lib.qsa_sparse_attn_kv4(ctypes.byref(d), ctypes.byref(_cache(qsa)), None, None, None) == qsa.QSA_ERR_INVALID_ARG
    for kw in (dict(n_q=65536), dict(n_q=8, group_q=8), dict(dims=_dims(qsa, n_q_heads=65536, n_kv_heads=65536)),
               dict(dims=_dims(qsa, batch=1024, kv_capacity=1 << 20)),
               dict(cache=_cache(qsa, page_table=16, page_tokens=4096, n_pages=1 << 18))):
        assert call(**kw) == qsa.QSA_ERR_UNSUPPORTED, kw
    assert call(n_q=0, q=None) == qsa.QSA_OK


def test_kv4_binding_checks_the_cache(qsa, device0):
    u8 = lambda *s: _on(*s, dtype=torch.uint8)  # noqa: E731
    small = dict(n_q_heads=4, n_kv_heads=2, kv_capacity=64)
    c = qsa.kv4_cache(u8(4, 2, 64, 64), u8(4, 2, 64, 8), u8(4, 2, 64, 64), _on(4, 2, 64, 8, dtype=torch.float8_e4m3fn))
    qsa._fits(_dims(qsa, **small), c, 0)
    for kw in (dict(batch=5), dict(n_q_heads=1, n_kv_heads=1), dict(kv_capacity=128)):
        with pytest.raises(ValueError, match="dims give"):
            qsa._fits(_dims(qsa, **{**small, **kw}), c, 0)
    with pytest.raises(ValueError, match="current device"):
        qsa._fits(_dims(qsa, **small), c, 1)
    table = _on(4, 4)
    pages = (u8(9, 2, 16, 64), u8(9, 2, 16, 8), u8(9, 2, 16, 64), u8(9, 2, 16, 8))
    p = qsa.kv4_cache(*pages, table, 16, 9)
    qsa._fits(_dims(qsa, **small), p, 0)
    with pytest.raises(ValueError, match="dims give"):
        qsa._fits(_dims(qsa, **{**small, "kv_capacity": 80}), p, 0)
    for bad in ((pages[0], pages[1], pages[2], u8(4, 2, 16, 8), table, 16, 9), (_on(9, 2, 16, 64), *pages[1:], table, 16, 9),
                (*pages, _on(4, 4, dtype=torch.int64), 16, 9), (*pages, _on(16), 16, 9), (*pages, table, 16, 8),
                (*pages, table, 32, 9)):
        with pytest.raises(ValueError, match="expected"):
            qsa.kv4_cache(*bad)
    with pytest.raises(ValueError, match="current device"):
        qsa.kv4_cache(*pages, _on(4, 4, dev=1), 16, 9)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.kv4_cache(*(x.t for x in pages), table, 16, 9)
    # the calls: every array's type and size
    d, bf = _dims(qsa, **small), torch.bfloat16
    rows = dict(q=_on(6, 4, 128, dtype=bf), q_seq=_on(6), q_pos=_on(6), sel_idx=_on(3, 512), sel_cnt=_on(3), n_q=6,
                out=_on(6, 4, 128, dtype=bf), group_q=2)
    for bad in (dict(q=_on(6, 2, 128, dtype=bf)), dict(q_seq=_on(5)), dict(q_pos=_on(6, dtype=torch.int64)),
                dict(sel_idx=_on(6, 512)), dict(sel_cnt=_on(6)), dict(out=_on(6, 4, 128))):
        with pytest.raises(ValueError, match="expected"):
            qsa.qsa_sparse_attn_kv4(d, p, **{**rows, **bad})
    tok = dict(k=_on(5, 2, 128, dtype=bf), v=_on(5, 2, 128, dtype=bf), cu_len=_on(5), len_before=_on(4), n_tok=5)
    for bad in (dict(k=_on(5, 4, 128, dtype=bf)), dict(v=_on(6, 2, 128, dtype=bf)), dict(cu_len=_on(4)), dict(len_before=_on(5))):
        with pytest.raises(ValueError, match="expected"):
            qsa.qsa_kv4_append(d, p, **{**tok, **bad})


def test_kv4_plans_fit_the_hardware(qsa):
    """Launch shapes of the 4-bit attention: every tile of the longest list has a split, no split is
    empty, merge buffers and stages fit 227 KB (an independent restatement of the layout)."""
    import itertools
    import math
    for rows, bs, pairs in itertools.product((1, 8, 9, 16, 17, 32), (1, 2, 4, 8, 16), (1, 2, 3, 7, 9, 16, 37, 64, 100, 147, 148, 149, 296, 297, 5000)):
        rp = 8 if rows <= 8 else 16 if rows <= 16 else 32
        d = qsa.make_dims(1, rows, 1, 65536, block_size=bs)
        info = qsa.qsa_attn_plan_info()
        assert qsa.load().qsa_attn_kv4_plan(ctypes.byref(d), pairs, 1, ctypes.byref(info)) == qsa.QSA_OK
        per_tile = 32 // bs
        tiles = math.ceil(514 / per_tile)
        assert 1 <= info.n_split <= 8 and info.rows == rows and info.ctas == pairs * info.n_split
        assert info.n_split == 1 or info.ctas <= 148
        own = math.ceil(tiles / info.n_split)
        assert (info.n_split - 1) * own < tiles            # the last split has a tile
        assert own * per_tile <= 576                       # items of a split fit their list
        warps = info.threads // 32
        assert info.n_stages % warps == 0 and 1 <= info.n_stages // warps
        area = max(info.n_stages * 4608, warps * rp * 130 * 4)   # rings, then partials
        assert info.smem_bytes >= rp * 256 + area + info.n_stages * 128 + 576 * 8 + 256
        assert info.smem_bytes + 1024 <= 227 * 1024


def test_pages_refusals(qsa):
    lib = qsa.load()
    d = _dims(qsa)

    def pools(n=1, pool=16, size=64, page_tokens=16, n_pages=100):
        p = qsa.qsa_page_pools(n, page_tokens, n_pages)
        p.pool[0], p.page_bytes[0] = pool, size
        return p

    need = qsa.qsa_pages_workspace_bytes(d, 16, 100)
    assert need > 0
    good = dict(table=16, ref=16, free=16, n_free=1, src=16, dst=16, n_fork=1, before=16, after=16, ws=16, n=need, live=16)

    def update(dims=d, p=None, **kw):
        a = {**good, **kw}
        return lib.qsa_pages_update(ctypes.byref(dims), ctypes.byref(p or pools()), a["table"], a["ref"], a["free"],
                                    a["n_free"], a["src"], a["dst"], a["n_fork"], a["before"], a["after"], a["ws"],
                                    a["n"], None)

    def compact(dims=d, p=None, **kw):
        a = {**good, **kw}
        return lib.qsa_pages_compact(ctypes.byref(dims), ctypes.byref(p or pools()), a["table"], a["ref"], a["live"],
                                     a["ws"], a["n"], None)

    both = (dict(table=None), dict(ref=8), dict(ws=None), dict(p=pools(n=-1)), dict(p=pools(n=129)), dict(p=pools(pool=None)),
            dict(p=pools(pool=8)), dict(p=pools(size=0)), dict(p=pools(size=40)), dict(p=pools(page_tokens=6)),
            dict(p=pools(page_tokens=0)), dict(p=pools(n_pages=0)), dict(dims=_dims(qsa, batch=0)))
    for kw in both:
        assert update(**kw) == compact(**kw) == qsa.QSA_ERR_INVALID_ARG, kw
    for kw in (dict(n_free=-1), dict(n_fork=-1), dict(free=None), dict(src=None), dict(dst=4), dict(before=None), dict(after=8)):
        assert update(**kw) == qsa.QSA_ERR_INVALID_ARG, kw
    assert compact(live=None) == qsa.QSA_ERR_INVALID_ARG
    assert update(n=need - 1) == compact(n=need - 1) == qsa.QSA_ERR_WORKSPACE_TOO_SMALL
    for kw in (dict(p=pools(n_pages=(1 << 30) + 1)), dict(p=pools(size=(1 << 31) + 16)),
               dict(dims=_dims(qsa, batch=65535, kv_capacity=1 << 20))):
        assert update(**kw) == compact(**kw) == qsa.QSA_ERR_UNSUPPORTED, kw
    # counters run up to a stride past the last entry: 2^30 entries are the most
    wide = _dims(qsa, batch=32, kv_capacity=(1 << 30) // 32 * 16)
    assert update(dims=wide, n=0) == compact(dims=wide, n=0) == qsa.QSA_ERR_WORKSPACE_TOO_SMALL
    wider = _dims(qsa, batch=33, kv_capacity=(1 << 30) // 32 * 16)
    assert update(dims=wider) == compact(dims=wider) == qsa.QSA_ERR_UNSUPPORTED
    entries = d.kv_capacity // 16
    assert update(n_free=(1 << 30) // entries + 1) == update(n_fork=(1 << 30) // entries + 1) == qsa.QSA_ERR_UNSUPPORTED
    for bad in ((d, 16, 0), (d, 5, 10), (_dims(qsa, top_k=0), 16, 10), (_dims(qsa, batch=65535, kv_capacity=1 << 20), 16, 10)):
        assert qsa.qsa_pages_workspace_bytes(*bad) == 0


def test_pages_binding_checks(qsa, device0):
    d = _dims(qsa)
    p = qsa.page_pools([_on(7, 4, 16, 128, dtype=torch.bfloat16), _on(7, 4, 16, 8, dtype=torch.uint8)], 16, 7)
    assert list(p.page_bytes[:2]) == [4 * 16 * 256, 4 * 16 * 8] and p.n_pools == 2
    with pytest.raises(ValueError, match="pages expected"):
        qsa.page_pools([_on(6, 16)], 16, 7)
    with pytest.raises(ValueError, match="at most"):
        qsa.page_pools([_on(7, 16)] * 129, 16, 7)
    table, ref, n4, ws = _on(4, 256), _on(7), _on(4), _on(16, dtype=torch.uint8)
    for bad in (dict(table=_on(4, 255)), dict(ref=_on(8)), dict(before=_on(5)), dict(after=_on(4, dtype=torch.int64)),
                dict(n_free=1), dict(n_fork=5, src=n4, dst=n4), dict(n_fork=4, src=n4, dst=_on(4, dtype=torch.int64))):
        a = {**dict(table=table, ref=ref, before=n4, after=n4, n_free=0, src=None, dst=None, n_fork=0), **bad}
        with pytest.raises(ValueError, match="expected"):
            qsa.qsa_pages_update(d, p, a["table"], a["ref"], a["before"], a["after"], ws, n_free=a["n_free"],
                                 fork_src=a["src"], fork_dst=a["dst"], n_fork=a["n_fork"])
    with pytest.raises(ValueError, match="n_live"):
        qsa.qsa_pages_compact(d, p, table, ref, _on(2), ws)
    with pytest.raises(ValueError, match="workspace"):
        qsa.qsa_pages_compact(d, p, table, ref, _on(1), None)
    with pytest.raises(ValueError, match="workspace"):
        qsa.qsa_pages_update(d, p, table, ref, n4, n4, None)
    with pytest.raises(ValueError, match="one page"):
        qsa.page_pools([_on(0, 16)], 16, 0)
    with pytest.raises(ValueError, match="current device"):
        qsa.qsa_pages_compact(d, p, table, _on(7, dev=1), _on(1), ws)


def test_package_import_leaves_torch_alone():
    """The binding's calls by pointer need no torch; it is imported with the first call that takes tensors."""
    import subprocess
    import sys
    code = "import sys, block_sparse_attention_key_b200; sys.exit('torch' in sys.modules)"
    assert subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__)))).returncode == 0


def test_page_pools_refuses_pages_without_tokens_and_pools_without_pages(qsa, device0):
    for page_tokens in (0, -16):
        with pytest.raises(ValueError, match="at least one"):
            qsa.page_pools([_on(7, 16)], page_tokens, 7)
    with pytest.raises(ValueError, match="pages expected"):
        qsa.page_pools([_on()], 16, 7)


def test_a_workspace_holds_at_least_the_status_word(qsa, device0):
    d = _dims(qsa, n_q_heads=1, n_kv_heads=1, batch=1)
    rows = _on(5, 1, 128, dtype=torch.bfloat16)
    for n in (0, 3):
        with pytest.raises(ValueError, match="status word"):
            qsa.qsa_prompt_attn(d, rows, rows, rows, _on(2), 5, rows, _on(n, dtype=torch.uint8))
    p = qsa.page_pools([_on(7, 16)], 16, 7)
    with pytest.raises(ValueError, match="status word"):
        qsa.qsa_pages_compact(_dims(qsa), p, _on(4, 256), _on(7), _on(1), _on(0, dtype=torch.uint8))
