"""Thin ctypes binding of libqsa.so (the C ABI in include/qsa.h).

Argument marshalling only: every step runs in the CUDA library.  Tensors are
torch CUDA tensors (device memory and streams come from PyTorch); their
data_ptr() values and the current stream's handle are passed straight through.
There is no CPU fallback: if the library or a GPU is missing, calls raise.
"""

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqsa.so")

QSA_SEL_CAP = 512

QSA_OK = 0
QSA_ERR_INVALID_ARG = -1
QSA_ERR_WORKSPACE_TOO_SMALL = -2
QSA_ERR_UNSUPPORTED = -3
QSA_ERR_CUDA = -4

QSA_DEV_BAD_SEQ = 0x1
QSA_DEV_BAD_POS = 0x2
QSA_DEV_BLOCKS_OVER = 0x4
QSA_DEV_BAD_LEN = 0x8
QSA_DEV_BAD_SEL = 0x10
QSA_DEV_TOO_MANY_NEW = 0x20
QSA_DEV_TIMEOUT = 0x40
QSA_DEV_BAD_PAGE = 0x80

QSA_MODE_DECODE = 0
QSA_MODE_PREFILL = 1
QSA_MODE_MIXED = 2

EXPORTED = (
    "qsa_workspace_bytes", "qsa_workspace_init", "qsa_read_device_status", "qsa_status_string",
    "qsa_pool_block_keys", "qsa_index_scores", "qsa_topk_blocks", "qsa_sparse_attn", "qsa_forward",
    "qsa_sparse_attn_noalloc", "qsa_sparse_attn_ex", "qsa_select_blocks",
    "qsa_cp_workspace_bytes", "qsa_cp_select_keys", "qsa_cp_merge_keys", "qsa_cp_attn_partial", "qsa_cp_combine",
    "qsa_attn_plan", "qsa_prompt_attn", "qsa_kv4_append", "qsa_sparse_attn_kv4",
    "qsa_attn_kv4_plan", "qsa_pages_workspace_bytes", "qsa_pages_update", "qsa_pages_compact",
)

CP_PART_ROW = 132  # floats per (query, head) partial of a context shard


class QsaError(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__(f"{fn} failed: {msg} ({code})")
        self.code = code


class qsa_dims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("n_idx_heads", ctypes.c_int32), ("idx_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32), ("top_k", ctypes.c_int32), ("kv_capacity", ctypes.c_int64),
        ("softmax_scale", ctypes.c_float),
    ]


class qsa_forward_args(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("idx_k", ctypes.c_void_p), ("pooled", ctypes.c_void_p), ("q_idx", ctypes.c_void_p),
        ("w", ctypes.c_void_p), ("len_before", ctypes.c_void_p), ("len_after", ctypes.c_void_p),
        ("q_seq", ctypes.c_void_p), ("q_pos", ctypes.c_void_p), ("n_q", ctypes.c_int32),
        ("max_new_tokens", ctypes.c_int32), ("max_blocks", ctypes.c_int64), ("mode", ctypes.c_int32),
        ("sel_idx", ctypes.c_void_p), ("sel_cnt", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("group_q", ctypes.c_int32), ("page_table", ctypes.c_void_p), ("page_tokens", ctypes.c_int32),
        ("n_pages", ctypes.c_int64), ("n_decode", ctypes.c_int32),
    ]


class qsa_attn_args(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("q_seq", ctypes.c_void_p), ("q_pos", ctypes.c_void_p), ("sel_idx", ctypes.c_void_p),
        ("sel_cnt", ctypes.c_void_p), ("n_q", ctypes.c_int32), ("group_q", ctypes.c_int32),
        ("page_table", ctypes.c_void_p), ("page_tokens", ctypes.c_int32), ("n_pages", ctypes.c_int64),
        ("out", ctypes.c_void_p),
    ]


class qsa_attn_plan_info(ctypes.Structure):
    _fields_ = [
        ("n_split", ctypes.c_int32), ("n_stages", ctypes.c_int32), ("threads", ctypes.c_int32),
        ("smem_bytes", ctypes.c_int32), ("ctas", ctypes.c_int64), ("cluster_merge", ctypes.c_int32),
        ("rows", ctypes.c_int32),
    ]


class qsa_prompt_args(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_ld", ctypes.c_int64),
        ("k_ld", ctypes.c_int64), ("v_ld", ctypes.c_int64), ("cu_len", ctypes.c_void_p), ("n_tok", ctypes.c_int32),
        ("out", ctypes.c_void_p),
    ]


class qsa_kv4_cache(ctypes.Structure):
    _fields_ = [
        ("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("page_tokens", ctypes.c_int32),
        ("n_pages", ctypes.c_int64),
    ]


QSA_MAX_POOLS = 128


class qsa_page_pools(ctypes.Structure):
    _fields_ = [
        ("n_pools", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("n_pages", ctypes.c_int64),
        ("pool", ctypes.c_void_p * QSA_MAX_POOLS), ("page_bytes", ctypes.c_int64 * QSA_MAX_POOLS),
    ]


_lib = None


def load(path=LIB_PATH):
    """Load libqsa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libqsa.so not built at {path}: run `python -m block_sparse_attention_key_b200.build`")
    L = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    D = ctypes.POINTER(qsa_dims)
    L.qsa_workspace_bytes.argtypes = [D, I32, I64, I32]
    L.qsa_workspace_bytes.restype = SZ
    L.qsa_workspace_init.argtypes = [P, SZ, P]
    L.qsa_read_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), P]
    L.qsa_status_string.argtypes = [ctypes.c_int]
    L.qsa_status_string.restype = ctypes.c_char_p
    L.qsa_pool_block_keys.argtypes = [D, P, P, P, P, I32, P, P]
    L.qsa_index_scores.argtypes = [D, P, P, P, P, P, I32, I64, P, I64, P, P]
    L.qsa_topk_blocks.argtypes = [D, P, I64, P, I32, I64, P, P, P, SZ, P]
    L.qsa_sparse_attn.argtypes = [D, P, P, P, P, P, P, P, I32, P, P, SZ, P]
    L.qsa_forward.argtypes = [D, ctypes.POINTER(qsa_forward_args), P, SZ, P]
    L.qsa_sparse_attn_noalloc.argtypes = [D, P, P, P, P, P, P, P, I32, P, P]
    L.qsa_sparse_attn_ex.argtypes = [D, ctypes.POINTER(qsa_attn_args), P, SZ, P]
    L.qsa_select_blocks.argtypes = [D, P, P, P, P, P, I32, I64, I32, P, P, P, SZ, P]
    L.qsa_cp_workspace_bytes.argtypes = [D, I32]
    L.qsa_cp_workspace_bytes.restype = SZ
    L.qsa_cp_select_keys.argtypes = [D, P, P, P, P, P, I32, I64, P, P, P, SZ, P]
    L.qsa_cp_merge_keys.argtypes = [D, I32, P, P, I32, I64, P, P, P, P, P]
    L.qsa_cp_attn_partial.argtypes = [D, P, P, P, P, P, I32, I64, P, P, P, P, SZ, P]
    L.qsa_cp_combine.argtypes = [D, I32, P, I32, P, P]
    L.qsa_attn_plan.argtypes = [D, I32, I32, ctypes.POINTER(qsa_attn_plan_info)]
    L.qsa_prompt_attn.argtypes = [D, ctypes.POINTER(qsa_prompt_args), P, P]
    C = ctypes.POINTER(qsa_kv4_cache)
    L.qsa_kv4_append.argtypes = [D, C, P, I64, P, I64, P, P, I32, P, P]
    L.qsa_attn_kv4_plan.argtypes = [D, I32, I32, ctypes.POINTER(qsa_attn_plan_info)]
    L.qsa_sparse_attn_kv4.argtypes = [D, C, ctypes.POINTER(qsa_attn_args), P, P]
    PP = ctypes.POINTER(qsa_page_pools)
    L.qsa_pages_workspace_bytes.argtypes = [D, I32, I64]
    L.qsa_pages_workspace_bytes.restype = SZ
    L.qsa_pages_update.argtypes = [D, PP, P, P, P, I32, P, P, I32, P, P, P, SZ, P]
    L.qsa_pages_compact.argtypes = [D, PP, P, P, P, P, SZ, P]
    for name in EXPORTED:
        if name not in ("qsa_workspace_bytes", "qsa_status_string", "qsa_cp_workspace_bytes",
                        "qsa_pages_workspace_bytes"):
            getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def make_dims(batch, n_q_heads, n_kv_heads, kv_capacity, head_dim=128, n_idx_heads=4, idx_dim=64,
              block_size=4, top_k=512, softmax_scale=0.0):
    return qsa_dims(batch, n_q_heads, n_kv_heads, head_dim, n_idx_heads, idx_dim, block_size, top_k,
                    kv_capacity, softmax_scale)


def status_string(code):
    return load().qsa_status_string(code).decode()


def _check(fn, rc):
    if rc != QSA_OK:
        raise QsaError(fn, rc, status_string(rc))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("libqsa takes CUDA tensors only (no CPU path)")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch

    return torch.cuda.current_stream().cuda_stream


# ---------------------------------------------------------------- entry points (same names as the C ABI)

def qsa_workspace_bytes(dims, n_q, max_blocks, mode):
    return int(load().qsa_workspace_bytes(ctypes.byref(dims), n_q, max_blocks, mode))


def qsa_workspace_init(workspace, stream=None):
    _check("qsa_workspace_init", load().qsa_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                                           _stream(stream)))


def qsa_read_device_status(workspace, stream=None):
    flags = ctypes.c_uint32(0)
    _check("qsa_read_device_status", load().qsa_read_device_status(_ptr(workspace), ctypes.byref(flags),
                                                                   _stream(stream)))
    return flags.value


def qsa_pool_block_keys(dims, idx_k, pooled, len_before, len_after, max_new_tokens, workspace=None, stream=None):
    _check("qsa_pool_block_keys", load().qsa_pool_block_keys(
        ctypes.byref(dims), _ptr(idx_k), _ptr(pooled), _ptr(len_before), _ptr(len_after), max_new_tokens,
        _ptr(workspace), _stream(stream)))


def qsa_index_scores(dims, q_idx, w, pooled, q_seq, q_pos, n_q, max_blocks, scores, ld_scores,
                     workspace=None, stream=None):
    _check("qsa_index_scores", load().qsa_index_scores(
        ctypes.byref(dims), _ptr(q_idx), _ptr(w), _ptr(pooled), _ptr(q_seq), _ptr(q_pos), n_q, max_blocks,
        _ptr(scores), ld_scores, _ptr(workspace), _stream(stream)))


def qsa_topk_blocks(dims, scores, ld_scores, q_pos, n_q, max_blocks, sel_idx, sel_cnt, workspace, stream=None):
    _check("qsa_topk_blocks", load().qsa_topk_blocks(
        ctypes.byref(dims), _ptr(scores), ld_scores, _ptr(q_pos), n_q, max_blocks, _ptr(sel_idx), _ptr(sel_cnt),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def qsa_select_blocks(dims, q_idx, w, pooled, q_seq, q_pos, n_q, max_blocks, mode, sel_idx, sel_cnt, workspace,
                      stream=None):
    _check("qsa_select_blocks", load().qsa_select_blocks(
        ctypes.byref(dims), _ptr(q_idx), _ptr(w), _ptr(pooled), _ptr(q_seq), _ptr(q_pos), n_q, max_blocks, mode,
        _ptr(sel_idx), _ptr(sel_cnt), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def qsa_sparse_attn(dims, q, k_cache, v_cache, q_seq, q_pos, sel_idx, sel_cnt, n_q, out, workspace, stream=None):
    _check("qsa_sparse_attn", load().qsa_sparse_attn(
        ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(q_seq), _ptr(q_pos), _ptr(sel_idx),
        _ptr(sel_cnt), n_q, _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def qsa_sparse_attn_noalloc(dims, q, k_cache, v_cache, q_seq, q_pos, sel_idx, sel_cnt, n_q, out, stream=None):
    """qsa_sparse_attn for callers that cannot allocate: scratch comes from a fixed
    16 MiB array inside the library (see include/qsa.h)."""
    _check("qsa_sparse_attn_noalloc", load().qsa_sparse_attn_noalloc(
        ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(q_seq), _ptr(q_pos), _ptr(sel_idx),
        _ptr(sel_cnt), n_q, _ptr(out), _stream(stream)))


def qsa_sparse_attn_ex(dims, *, q, k_cache, v_cache, q_seq, q_pos, sel_idx, sel_cnt, n_q, out, workspace,
                       group_q=1, page_table=None, page_tokens=0, n_pages=0, stream=None):
    args = qsa_attn_args(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(q_seq), _ptr(q_pos), _ptr(sel_idx),
                         _ptr(sel_cnt), n_q, group_q, _ptr(page_table), page_tokens, n_pages, _ptr(out))
    _check("qsa_sparse_attn_ex", load().qsa_sparse_attn_ex(ctypes.byref(dims), ctypes.byref(args), _ptr(workspace),
                                                           workspace.numel() * workspace.element_size(),
                                                           _stream(stream)))


def qsa_attn_plan(dims, n_q, group_q=1):
    """The attention launch for n_q queries in groups of group_q (host arithmetic only):
    a dict of splits, stages, threads, shared memory, CTAs, cluster merge and rows."""
    info = qsa_attn_plan_info()
    _check("qsa_attn_plan", load().qsa_attn_plan(ctypes.byref(dims), n_q, group_q, ctypes.byref(info)))
    return {name: getattr(info, name) for name, _ in qsa_attn_plan_info._fields_}


def qsa_forward(dims, *, q, k_cache, v_cache, idx_k, pooled, q_idx, w, len_before, len_after, q_seq, q_pos,
                n_q, max_new_tokens, max_blocks, mode, out, workspace, sel_idx=None, sel_cnt=None, group_q=0,
                page_table=None, page_tokens=0, n_pages=0, n_decode=0, stream=None):
    args = qsa_forward_args(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(idx_k), _ptr(pooled), _ptr(q_idx),
                            _ptr(w), _ptr(len_before), _ptr(len_after), _ptr(q_seq), _ptr(q_pos), n_q,
                            max_new_tokens, max_blocks, mode, _ptr(sel_idx), _ptr(sel_cnt), _ptr(out), group_q,
                            _ptr(page_table), page_tokens, n_pages, n_decode)
    _check("qsa_forward", load().qsa_forward(ctypes.byref(dims), ctypes.byref(args), _ptr(workspace),
                                             workspace.numel() * workspace.element_size(), _stream(stream)))


# ---------------------------------------------------------------- checked arguments of the serving operators

# torch is imported with the first of these calls, as it is by _stream above
_BF16 = _I32 = _U8 = _E4M3 = None


def _bind_types():
    global _BF16, _I32, _U8, _E4M3
    import torch

    _BF16, _I32, _U8, _E4M3 = torch.bfloat16, torch.int32, torch.uint8, torch.float8_e4m3fn


# the calls behind torch.cuda.current_device() and current_stream(), without their wrappers' few
# microseconds (a decode step's kernels take not many more); only used beside CUDA tensors
def _current_device():
    global _current_device
    from torch._C import _cuda_getDevice as _current_device
    return _current_device()


def _current_stream(dev):
    global _current_stream
    from torch._C import _cuda_getCurrentRawStream as _current_stream
    return _current_stream(dev)


def _stream_on(stream, dev):
    if stream is None:
        return _current_stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _device_of(t):
    """Device index of a call's first tensor.  Launches go to the current device, so it has to be that."""
    if _BF16 is None:
        _bind_types()
    dev = t.get_device()
    if dev < 0:
        raise ValueError("libqsa takes CUDA tensors only (no CPU path)")
    if dev != _current_device():
        raise ValueError(f"tensor on cuda:{dev}, but the current device is cuda:{_current_device()}")
    return dev


def _arg(name, t, dtype, shape, dev):
    """Pointer of a dense tensor of this type, shape (the C ABI sees neither) and device."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: {dtype} {shape} expected, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: tensor on {t.device}, but the current device is cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous")
    return t.data_ptr()


def _rows_arg(name, t, n_tok, heads, dev):
    """Pointer and token stride of bf16 [n_tok][heads][128], heads dense, tokens at any stride."""
    if t.dtype is not _BF16 or t.shape != (n_tok, heads, 128):
        raise ValueError(f"{name}: torch.bfloat16 {(n_tok, heads, 128)} expected, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: tensor on {t.device}, but the current device is cuda:{dev}")
    tok, head, one = t.stride()
    if n_tok and (one != 1 or (heads > 1 and head != 128)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), tok if n_tok > 1 else heads * 128


def _workspace_arg(workspace, dev):
    """Pointer of an optional workspace."""
    if workspace is None:
        return None
    if workspace.get_device() != dev:
        raise ValueError(f"workspace: tensor on {workspace.device}, but the current device is cuda:{dev}")
    if not workspace.is_contiguous():
        raise ValueError("workspace: tensors must be contiguous")
    if workspace.nbytes < 4:
        raise ValueError("workspace: at least the 4 bytes of the status word expected")
    return workspace.data_ptr()


# ---------------------------------------------------------------- whole prompts

def qsa_prompt_attn(dims, q, k, v, cu_len, n_tok, out, workspace=None, stream=None):
    """Causal attention over packed whole prompts.  q, k, v: bf16 [n_tok][heads][128], also as
    slices of a fused projection; cu_len: i32 [batch + 1]; out: bf16 [n_tok][n_q_heads][128]."""
    dev, hq, hkv = _device_of(q), dims.n_q_heads, dims.n_kv_heads
    qp, q_ld = _rows_arg("q", q, n_tok, hq, dev)
    kp, k_ld = _rows_arg("k", k, n_tok, hkv, dev)
    vp, v_ld = _rows_arg("v", v, n_tok, hkv, dev)
    args = qsa_prompt_args(qp, kp, vp, q_ld, k_ld, v_ld, _arg("cu_len", cu_len, _I32, (dims.batch + 1,), dev),
                           n_tok, _arg("out", out, _BF16, (n_tok, hq, 128), dev))
    rc = (_lib or load()).qsa_prompt_attn(dims, args, _workspace_arg(workspace, dev), _stream_on(stream, dev))
    if rc:
        _check("qsa_prompt_attn", rc)


# ---------------------------------------------------------------- caches in 4 bits

def kv4_cache(k_codes, k_scales, v_codes, v_scales, page_table=None, page_tokens=0, n_pages=0):
    """The handle of a 4-bit cache: u8 codes [..., 64] and scales [..., 8] over the leading sizes
    [batch][n_kv_heads][kv_capacity], or [n_pages][n_kv_heads][page_tokens] with a page table
    (i32 [batch][kv_capacity / page_tokens]).  It keeps the tensors alive; make it once."""
    lead = tuple(k_codes.shape[:-1])
    if len(lead) != 3:
        raise ValueError("codes: [batch or pages][n_kv_heads][tokens][64] expected")
    if _U8 is None:
        _bind_types()
    dev = k_codes.get_device()
    if dev < 0:
        raise ValueError("libqsa takes CUDA tensors only (no CPU path)")
    p = [_arg(name, t.view(_U8) if t.dtype is _E4M3 else t, _U8, (*lead, n), dev)
         for name, t, n in (("k_codes", k_codes, 64), ("k_scales", k_scales, 8), ("v_codes", v_codes, 64),
                            ("v_scales", v_scales, 8))]
    table = None
    if page_table is None:
        sizes = lead
    else:
        if page_table.dim() != 2:
            raise ValueError("page_table: i32 [batch][kv_capacity / page_tokens] expected")
        table = _arg("page_table", page_table, _I32, tuple(page_table.shape), dev)
        if lead[0] != n_pages or lead[2] != page_tokens:
            raise ValueError(f"pools of {n_pages} pages of {page_tokens} tokens expected, got {lead}")
        sizes = (page_table.shape[0], lead[1], page_table.shape[1] * page_tokens)
    cache = qsa_kv4_cache(*p, table, page_tokens, n_pages)
    cache.sizes = sizes           # batch, KV heads, capacity: what dims have to say
    cache.device = dev
    cache.tensors = (k_codes, k_scales, v_codes, v_scales, page_table)
    return cache


def _fits(dims, cache, dev):
    if cache.sizes != (dims.batch, dims.n_kv_heads, dims.kv_capacity):
        raise ValueError(f"cache of {cache.sizes}, but dims give {(dims.batch, dims.n_kv_heads, dims.kv_capacity)}")
    if cache.device != dev:
        raise ValueError(f"cache on cuda:{cache.device}, but the current device is cuda:{dev}")


def qsa_kv4_append(dims, cache, k, v, cu_len, len_before, n_tok, workspace=None, stream=None):
    """Round packed K/V rows (bf16 [n_tok][n_kv_heads][128], also slices of a projection) to 4 bits
    into `cache` (kv4_cache): tokens [cu_len[s], cu_len[s+1]) at len_before[s] on."""
    dev, batch, hkv = _device_of(k), dims.batch, dims.n_kv_heads
    _fits(dims, cache, dev)
    kp, k_ld = _rows_arg("k", k, n_tok, hkv, dev)
    vp, v_ld = _rows_arg("v", v, n_tok, hkv, dev)
    rc = (_lib or load()).qsa_kv4_append(
        dims, cache, kp, k_ld, vp, v_ld, _arg("cu_len", cu_len, _I32, (batch + 1,), dev),
        _arg("len_before", len_before, _I32, (batch,), dev), n_tok, _workspace_arg(workspace, dev), _stream_on(stream, dev))
    if rc:
        _check("qsa_kv4_append", rc)


def qsa_attn_kv4_plan(dims, n_q, group_q=1):
    """qsa_sparse_attn_kv4's launch for n_q queries in groups of group_q (see qsa_attn_plan)."""
    info = qsa_attn_plan_info()
    _check("qsa_attn_kv4_plan", load().qsa_attn_kv4_plan(ctypes.byref(dims), n_q, group_q, ctypes.byref(info)))
    return {name: getattr(info, name) for name, _ in qsa_attn_plan_info._fields_}


def qsa_sparse_attn_kv4(dims, cache, q, q_seq, q_pos, sel_idx, sel_cnt, n_q, out, workspace=None, group_q=1,
                        stream=None):
    """qsa_sparse_attn_ex over a 4-bit cache (kv4_cache); needs no workspace but for its status."""
    dev, rows = _device_of(q), (n_q, dims.n_q_heads, 128)
    _fits(dims, cache, dev)
    groups, i32 = n_q // group_q if group_q > 1 else n_q, _I32
    args = qsa_attn_args(_arg("q", q, _BF16, rows, dev), None, None, _arg("q_seq", q_seq, i32, (n_q,), dev),
                         _arg("q_pos", q_pos, i32, (n_q,), dev),
                         _arg("sel_idx", sel_idx, i32, (groups, QSA_SEL_CAP), dev),
                         _arg("sel_cnt", sel_cnt, i32, (groups,), dev), n_q, group_q, None, 0, 0,
                         _arg("out", out, _BF16, rows, dev))
    rc = (_lib or load()).qsa_sparse_attn_kv4(dims, cache, args, _workspace_arg(workspace, dev), _stream_on(stream, dev))
    if rc:
        _check("qsa_sparse_attn_kv4", rc)


# ---------------------------------------------------------------- pages of a paged cache

def page_pools(pools, page_tokens, n_pages):
    """The handle of the pools that share one page table: tensors whose first size is n_pages, of any
    type (K and V, or codes and scales, of every layer).  It keeps them alive; make it once."""
    if len(pools) > QSA_MAX_POOLS:
        raise ValueError(f"at most {QSA_MAX_POOLS} pools")
    if n_pages < 1 or page_tokens < 1:
        raise ValueError("at least one page of at least one token expected")
    p = qsa_page_pools(len(pools), page_tokens, n_pages)
    for i, t in enumerate(pools):
        if t.dim() < 1 or t.shape[0] != n_pages:
            raise ValueError(f"pool {i}: {n_pages} pages expected, got {tuple(t.shape)}")
        p.pool[i] = _arg(f"pool {i}", t, t.dtype, tuple(t.shape), pools[0].get_device())
        p.page_bytes[i] = t.numel() // n_pages * t.element_size()
    p.device = pools[0].get_device() if pools else None
    p.tensors = tuple(pools)
    return p


def qsa_pages_workspace_bytes(dims, page_tokens, n_pages):
    return int(load().qsa_pages_workspace_bytes(ctypes.byref(dims), page_tokens, n_pages))


def _page_state(dims, pools, page_table, page_ref, dev):
    if pools.device is not None and pools.device != dev:
        raise ValueError(f"pools on cuda:{pools.device}, but the current device is cuda:{dev}")
    return (_arg("page_table", page_table, _I32, (dims.batch, dims.kv_capacity // pools.page_tokens), dev),
            _arg("page_ref", page_ref, _I32, (pools.n_pages,), dev))


def _scratch_arg(workspace, dev):
    """Pointer and bytes of a workspace that the call needs."""
    if workspace is None:
        raise ValueError("workspace: a tensor of qsa_pages_workspace_bytes expected")
    return _workspace_arg(workspace, dev), workspace.nbytes


def _list_arg(name, t, n, dev):
    """Pointer of the first n of a list of sequences."""
    if n <= 0:
        return None
    if t is None or t.dim() != 1 or t.numel() < n:
        raise ValueError(f"{name}: {n} int32 values expected")
    return _arg(name, t, _I32, t.shape, dev)


def qsa_pages_update(dims, pools, page_table, page_ref, len_before, len_after, workspace, free_seq=None, n_free=0,
                     fork_src=None, fork_dst=None, n_fork=0, stream=None):
    """A scheduler's step on a paged cache (page_pools): free sequences, fork others, then make every
    page of positions [len_before, len_after) the sequence's own, copying what was shared."""
    dev, i32, batch = _device_of(page_table), _I32, (dims.batch,)
    table, ref = _page_state(dims, pools, page_table, page_ref, dev)
    rc = (_lib or load()).qsa_pages_update(
        dims, pools, table, ref, _list_arg("free_seq", free_seq, n_free, dev), n_free,
        _list_arg("fork_src", fork_src, n_fork, dev), _list_arg("fork_dst", fork_dst, n_fork, dev), n_fork,
        _arg("len_before", len_before, i32, batch, dev), _arg("len_after", len_after, i32, batch, dev),
        *_scratch_arg(workspace, dev), _stream_on(stream, dev))
    if rc:
        _check("qsa_pages_update", rc)


def qsa_pages_compact(dims, pools, page_table, page_ref, n_live, workspace, stream=None):
    """Move the live pages of every pool to the ids [0, n_live) (n_live: i32 [1], written)."""
    dev = _device_of(page_table)
    table, ref = _page_state(dims, pools, page_table, page_ref, dev)
    rc = (_lib or load()).qsa_pages_compact(dims, pools, table, ref, _arg("n_live", n_live, _I32, (1,), dev),
                                  *_scratch_arg(workspace, dev), _stream_on(stream, dev))
    if rc:
        _check("qsa_pages_compact", rc)


# ---------------------------------------------------------------- context parallelism (see include/qsa.h)

def qsa_cp_workspace_bytes(shard_dims, n_q):
    return int(load().qsa_cp_workspace_bytes(ctypes.byref(shard_dims), n_q))


def qsa_cp_select_keys(shard_dims, q_idx, w, pooled_shard, q_seq, q_pos, n_q, blk_lo, keys, key_cnt, workspace,
                       stream=None):
    _check("qsa_cp_select_keys", load().qsa_cp_select_keys(
        ctypes.byref(shard_dims), _ptr(q_idx), _ptr(w), _ptr(pooled_shard), _ptr(q_seq), _ptr(q_pos), n_q, blk_lo,
        _ptr(keys), _ptr(key_cnt), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def qsa_cp_merge_keys(shard_dims, n_ranks, keys_all, cnt_all, n_q, blk_lo, sel_local, cnt_local, sel_global=None,
                      cnt_global=None, stream=None):
    _check("qsa_cp_merge_keys", load().qsa_cp_merge_keys(
        ctypes.byref(shard_dims), n_ranks, _ptr(keys_all), _ptr(cnt_all), n_q, blk_lo, _ptr(sel_local),
        _ptr(cnt_local), _ptr(sel_global), _ptr(cnt_global), _stream(stream)))


def qsa_cp_attn_partial(shard_dims, q, k_shard, v_shard, q_seq, q_pos, n_q, blk_lo, sel_local, cnt_local, part,
                        workspace, stream=None):
    _check("qsa_cp_attn_partial", load().qsa_cp_attn_partial(
        ctypes.byref(shard_dims), _ptr(q), _ptr(k_shard), _ptr(v_shard), _ptr(q_seq), _ptr(q_pos), n_q, blk_lo,
        _ptr(sel_local), _ptr(cnt_local), _ptr(part), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def qsa_cp_combine(dims, n_ranks, parts_all, n_q, out, stream=None):
    _check("qsa_cp_combine", load().qsa_cp_combine(ctypes.byref(dims), n_ranks, _ptr(parts_all), n_q, _ptr(out),
                                                   _stream(stream)))
