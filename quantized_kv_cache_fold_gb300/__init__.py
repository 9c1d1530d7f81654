"""Rotated 4-bit KV-cache decode path for GB300 (sm_103a): Python binding of libkvq.so.

The functions here carry the C-ABI names of include/kvq.h and only marshal arguments:
torch tensors (device memory) and numpy arrays (host memory) become raw pointers, every
computation runs in the CUDA kernels of libkvq.so. A non-zero kvq_status raises KvqError.
There is no CPU fallback: importing fails loudly when the library is missing.
"""

from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvq.so")

HEAD_DIM = 128
PAGE_SIZE = 64
MAX_SEQS = 1024
MAX_TREE = 64
MAX_CACHES = 64
F32, BF16, F16 = 0, 1, 2
DEVERR_PAGE, DEVERR_POS, DEVERR_NONFINITE, DEVERR_RANGE, DEVERR_TIMEOUT = 0x1, 0x2, 0x4, 0x8, 0x10
DEVERR_POOL = 0x20


class KvqError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


INT4_BLOCK_BYTES = 8704  # one (page, KV head): K codes 4096, V codes 4096, K meta 256, V meta 256
FP8_BLOCK_BYTES = 16384  # 64 ring slots of one head: K 8192, V 8192


class Int4Cache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("num_seqs", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class Fp8Ring(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_seqs", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run `python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, f32, u64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint64, ctypes.c_size_t
    L.kvq_status_string.restype = ctypes.c_char_p
    L.kvq_status_string.argtypes = [i32]
    L.kvq_build_rotation.restype = i32
    L.kvq_build_rotation.argtypes = [u64, i32, vp, vp]
    L.kvq_fold_qk.restype = i32
    L.kvq_fold_qk.argtypes = [vp, vp, vp, i32, vp, vp]
    L.kvq_fold_qk_fwht.restype = i32
    L.kvq_fold_qk_fwht.argtypes = [vp, vp, vp, i32, vp, vp]
    for name in ("kvq_rotate_quant_append", "kvq_rotate_quant_append_fwht"):
        getattr(L, name).restype = i32
        getattr(L, name).argtypes = [ctypes.POINTER(Int4Cache), vp, vp, vp, i32, i32, vp, vp, f32, vp, vp]
    L.kvq_decode_workspace_bytes.restype = sz
    L.kvq_decode_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.kvq_fp8_swa_plan.restype = i32
    L.kvq_fp8_swa_plan.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(ctypes.c_int32)]
    for name in ("kvq_decode_attn_int4", "kvq_decode_attn_int4_fwht"):
        getattr(L, name).restype = i32
        getattr(L, name).argtypes = [ctypes.POINTER(Int4Cache), vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, f32,
                                     f32, vp, vp, sz, vp, vp, vp]
    L.kvq_fp8_append.restype = i32
    L.kvq_fp8_append.argtypes = [ctypes.POINTER(Fp8Ring), vp, vp, i32, i32, vp, vp, f32, f32, vp, vp]
    L.kvq_decode_attn_int4_noalloc.restype = i32
    L.kvq_decode_attn_int4_noalloc.argtypes = [ctypes.POINTER(Int4Cache), vp, vp, vp, i32, i32, i32, i32, vp, vp, vp,
                                               f32, f32, vp, vp, vp, vp]
    L.kvq_set_stage_wait_limit_ns.restype = i32
    L.kvq_set_stage_wait_limit_ns.argtypes = [u64]
    L.kvq_decode_attn_fp8_swa.restype = i32
    L.kvq_decode_attn_fp8_swa.argtypes = [ctypes.POINTER(Fp8Ring), vp, i32, i32, i32, i32, vp, i32, vp, vp, f32,
                                          f32, f32, vp, vp, sz, vp, vp]
    i64 = ctypes.c_int64
    for name in ("kvq_prompt_workspace_bytes", "kvq_tree_workspace_bytes"):
        getattr(L, name).restype = sz
        getattr(L, name).argtypes = [i32, i32, i32, i32]
    L.kvq_prompt_attn.restype = i32
    L.kvq_prompt_attn.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, ctypes.POINTER(i64), vp, i32, f32, vp, vp, sz,
                                  vp, vp]
    for name in ("kvq_tree_attn_int4", "kvq_tree_attn_int4_fwht"):
        getattr(L, name).restype = i32
        getattr(L, name).argtypes = [ctypes.POINTER(Int4Cache), vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, f32,
                                     f32, vp, i32, vp, sz, vp, vp]
    L.kvq_tree_attn_fp8_swa.restype = i32
    L.kvq_tree_attn_fp8_swa.argtypes = [ctypes.POINTER(Fp8Ring), vp, i32, i32, i32, i32, vp, vp, i32, vp, vp, f32,
                                        f32, f32, vp, i32, vp, sz, vp, vp]
    L.kvq_tree_commit_int4.restype = i32
    L.kvq_tree_commit_int4.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    L.kvq_tree_commit_fp8.restype = i32
    L.kvq_tree_commit_fp8.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    for name in ("kvq_pages_alloc", "kvq_pages_free"):
        getattr(L, name).restype = i32
        getattr(L, name).argtypes = [vp, i32, vp, i32, i32, i32, vp, vp, vp, vp, vp]
    L.kvq_pages_fork.restype = i32
    L.kvq_pages_fork.argtypes = [vp, i32, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    L.kvq_pages_compact.restype = i32
    L.kvq_pages_compact.argtypes = [vp, i32, vp, i32, i32, vp, vp, vp, vp, vp]
    L.kvq_pages_copy.restype = i32
    L.kvq_pages_copy.argtypes = [vp, i32, i32, vp, vp, vp, vp, vp]
    return L


lib = _load()


def _ptr(x):
    """Device/host address of a torch tensor, numpy array, raw int or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if isinstance(x, np.ndarray):
        return x.ctypes.data
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, status):
    if status != 0:
        raise KvqError(fn, status)


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def status_string(status: int) -> str:
    return lib.kvq_status_string(int(status)).decode()


# ---------------------------------------------------------------- host-side steps

def kvq_build_rotation(seed: int, head_dim: int = HEAD_DIM):
    """R = H diag(s)/sqrt(128) as float32[128,128] and the signs s as int8[128] (numpy)."""
    R = np.empty((head_dim, head_dim), np.float32)
    s = np.empty(head_dim, np.int8)
    _check("kvq_build_rotation", lib.kvq_build_rotation(seed & (2**64 - 1), head_dim, s.ctypes.data, R.ctypes.data))
    return R, s


def kvq_fold_qk(R, g_q, g_k):
    """(M_q, M_k) = (R diag(g_q g_k), R) as float32[128,128] numpy arrays."""
    R = np.ascontiguousarray(R, np.float32)
    g_q = np.ascontiguousarray(g_q, np.float32)
    g_k = np.ascontiguousarray(g_k, np.float32)
    n = R.shape[0]
    Mq = np.empty((n, n), np.float32)
    Mk = np.empty((n, n), np.float32)
    _check("kvq_fold_qk", lib.kvq_fold_qk(R.ctypes.data, g_q.ctypes.data, g_k.ctypes.data, n, Mq.ctypes.data,
                                          Mk.ctypes.data))
    return Mq, Mk


# ---------------------------------------------------------------- cache descriptors

def int4_cache(pages, block_table) -> Int4Cache:
    """Descriptor over caller-owned device tensors: pages uint8 [num_pages, num_kv_heads, 8704]
    and block_table int32 [num_seqs, max_pages_per_seq] (see kvq.h for the block layout)."""
    num_seqs, max_pages = block_table.shape
    num_pages, num_kv_heads, nbytes = pages.shape
    assert nbytes == INT4_BLOCK_BYTES
    return Int4Cache(_ptr(pages), _ptr(block_table), num_seqs, max_pages, num_pages, num_kv_heads, PAGE_SIZE,
                     HEAD_DIM)


def fp8_ring(data) -> Fp8Ring:
    """data uint8 [num_seqs, num_kv_heads, capacity/64, 16384]."""
    num_seqs, num_kv, nblk, nbytes = data.shape
    assert nbytes == FP8_BLOCK_BYTES
    return Fp8Ring(_ptr(data), num_seqs, num_kv, nblk * PAGE_SIZE, HEAD_DIM)


def alloc_int4_cache(num_pages: int, num_kv_heads: int, block_table, device="cuda"):
    """Device tensors for an int4 cache (plumbing only: torch allocates, kernels fill)."""
    import torch
    pages = torch.zeros((num_pages, num_kv_heads, INT4_BLOCK_BYTES), dtype=torch.uint8, device=device)
    bt = block_table.to(device=device, dtype=torch.int32).contiguous()
    return {"pages": pages, "block_table": bt}, int4_cache(pages, bt)


def alloc_fp8_ring(num_seqs: int, num_kv_heads: int, capacity: int, device="cuda"):
    import torch
    assert capacity % PAGE_SIZE == 0
    data = torch.zeros((num_seqs, num_kv_heads, capacity // PAGE_SIZE, FP8_BLOCK_BYTES), dtype=torch.uint8,
                       device=device)
    return {"data": data}, fp8_ring(data)


# ---------------------------------------------------------------- device calls

def kvq_fold_qk_fwht(s, g_q, g_k):
    """(w_q, w_k) = (s g_q g_k, s) as float32[128] numpy arrays: the multipliers of the FWHT prologue."""
    s = np.ascontiguousarray(s, np.int8)
    g_q = np.ascontiguousarray(g_q, np.float32)
    g_k = np.ascontiguousarray(g_k, np.float32)
    n = s.shape[0]
    wq = np.empty(n, np.float32)
    wk = np.empty(n, np.float32)
    _check("kvq_fold_qk_fwht", lib.kvq_fold_qk_fwht(s.ctypes.data, g_q.ctypes.data, g_k.ctypes.data, n,
                                                    wq.ctypes.data, wk.ctypes.data))
    return wq, wk


def kvq_rotate_quant_append(cache: Int4Cache, Mk, k, v, seq_ids, positions, dev_err, eps: float = 1e-6,
                            stream=None, fwht: bool = False):
    """fwht=False: Mk is the 128x128 matrix; fwht=True: Mk is the multiplier vector w_k."""
    T = k.shape[0]
    name = "kvq_rotate_quant_append_fwht" if fwht else "kvq_rotate_quant_append"
    _check(name, getattr(lib, name)(ctypes.byref(cache), _ptr(Mk), _ptr(k), _ptr(v), _dtype_code(k), T,
                                    _ptr(seq_ids), _ptr(positions), eps, _ptr(dev_err), _stream(stream)))


def kvq_decode_workspace_bytes(B: int, S: int, num_q_heads: int, num_kv_heads: int) -> int:
    return int(lib.kvq_decode_workspace_bytes(B, S, num_q_heads, num_kv_heads))


def kvq_fp8_swa_plan(capacity: int, B: int, S: int, num_q_heads: int, num_kv_heads: int) -> tuple:
    """(CTAs per pair or 0 for the split-K path, streams per CTA, stages, units per stream)."""
    out = (ctypes.c_int32 * 4)()
    _check("kvq_fp8_swa_plan", lib.kvq_fp8_swa_plan(capacity, B, S, num_q_heads, num_kv_heads, out))
    return tuple(int(x) for x in out)


def kvq_decode_attn_int4(cache: Int4Cache, Mq, Mk, q, ctx_len, out, workspace, dev_err, k_new=None, v_new=None,
                         sm_scale: float = HEAD_DIM ** -0.5, eps: float = 1e-6, q_rot_out=None, stream=None,
                         fwht: bool = False):
    """fwht=False: Mq, Mk are the folded matrices; fwht=True: the multiplier vectors w_q, w_k."""
    B, S, Hq, _ = q.shape
    ws_bytes = workspace.numel() * workspace.element_size()
    name = "kvq_decode_attn_int4_fwht" if fwht else "kvq_decode_attn_int4"
    _check(name, getattr(lib, name)(ctypes.byref(cache), _ptr(Mq), _ptr(Mk), _ptr(q), _dtype_code(q), B, S, Hq,
                                    _ptr(ctx_len), _ptr(k_new), _ptr(v_new), sm_scale, eps, _ptr(out),
                                    _ptr(workspace), ws_bytes, _ptr(q_rot_out), _ptr(dev_err), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 16 << 20
ERR_SCRATCH_TOO_SMALL = 4


def kvq_decode_attn_int4_noalloc(cache: Int4Cache, Mq, Mk, q, ctx_len, out, dev_err, k_new=None, v_new=None,
                                 sm_scale: float = HEAD_DIM ** -0.5, eps: float = 1e-6, q_rot_out=None, stream=None):
    """kvq_decode_attn_int4 without a caller workspace: for callers that cannot allocate device
    memory while decoding. Uses the library's fixed scratch (NOALLOC_SCRATCH_BYTES per device);
    calls that overlap on the GPU race on it. The first call on a device must precede any
    stream capture."""
    B, S, Hq, _ = q.shape
    _check("kvq_decode_attn_int4_noalloc",
           lib.kvq_decode_attn_int4_noalloc(ctypes.byref(cache), _ptr(Mq), _ptr(Mk), _ptr(q), _dtype_code(q), B, S,
                                            Hq, _ptr(ctx_len), _ptr(k_new), _ptr(v_new), sm_scale, eps, _ptr(out),
                                            _ptr(q_rot_out), _ptr(dev_err), _stream(stream)))


STAGE_WAIT_DEFAULT_NS = 2_000_000_000


def kvq_set_stage_wait_limit_ns(ns: int):
    """Test hook: the split-K attention kernel's stage-wait limit for later launches (default 2 s)."""
    _check("kvq_set_stage_wait_limit_ns", lib.kvq_set_stage_wait_limit_ns(int(ns)))


def kvq_fp8_append(ring: Fp8Ring, k, v, seq_ids, positions, k_scale: float, v_scale: float, dev_err, stream=None):
    T = k.shape[0]
    _check("kvq_fp8_append",
           lib.kvq_fp8_append(ctypes.byref(ring), _ptr(k), _ptr(v), _dtype_code(k), T, _ptr(seq_ids),
                              _ptr(positions), k_scale, v_scale, _ptr(dev_err), _stream(stream)))


def kvq_decode_attn_fp8_swa(ring: Fp8Ring, q, pos0, window: int, k_scale: float, v_scale: float, out, workspace,
                            dev_err, k_new=None, v_new=None, sm_scale: float = HEAD_DIM ** -0.5, stream=None):
    B, S, Hq, _ = q.shape
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("kvq_decode_attn_fp8_swa",
           lib.kvq_decode_attn_fp8_swa(ctypes.byref(ring), _ptr(q), _dtype_code(q), B, S, Hq, _ptr(pos0), window,
                                       _ptr(k_new), _ptr(v_new), k_scale, v_scale, sm_scale, _ptr(out),
                                       _ptr(workspace), ws_bytes, _ptr(dev_err), _stream(stream)))


def alloc_workspace(B: int, S: int, num_q_heads: int, num_kv_heads: int, device="cuda"):
    import torch
    n = kvq_decode_workspace_bytes(B, S, num_q_heads, num_kv_heads)
    if n == 0:
        raise KvqError("kvq_decode_workspace_bytes", 2)
    return torch.empty(n, dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- around decoding: prompt, tree, pages
#
# These calls take a few microseconds on the GPU for small batches, so their checks are written to cost
# little on the host: one comparison chain per tensor, the raw stream handle, addresses passed as they are.

_th = None  # torch, imported by the first call


def _torch():
    global _th
    if _th is None:
        import torch
        _th = torch
    return _th


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _dev(t, name):
    """The device that the call's tensors have to be on: that of `t`, a device tensor (_here asks that it is the current one)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a device tensor")
    return dev


def _is(t, dtype, shape, name, dev):
    """Address of `t`, a contiguous tensor of this type and shape on device `dev`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous tensor of {dtype} and shape {tuple(shape)} on cuda:{dev}, got "
                     f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _err(t, dev):
    """Address of the device error word."""
    if t.dtype is _th.int32 and t.get_device() == dev and t.numel():
        return t.data_ptr()
    raise ValueError(f"dev_err must be int32 on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _here(dev, stream):
    """The raw stream of a call on device `dev`, which has to be the current one (kvq.h)."""
    c = _th._C
    if dev != c._cuda_getDevice():
        raise ValueError(f"tensors on cuda:{dev}, but cuda:{c._cuda_getDevice()} is the current device")
    if stream is None:
        return c._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _bytes(workspace, dev):
    if workspace.get_device() == dev and workspace.is_contiguous():
        return workspace.numel() * workspace.element_size()
    raise ValueError(f"the workspace must be a contiguous tensor on cuda:{dev}")


def kvq_prompt_workspace_bytes(T: int, B: int, num_q_heads: int, num_kv_heads: int) -> int:
    return int(lib.kvq_prompt_workspace_bytes(T, B, num_q_heads, num_kv_heads))


def alloc_prompt_workspace(T: int, B: int, num_q_heads: int, num_kv_heads: int, device="cuda"):
    n = kvq_prompt_workspace_bytes(T, B, num_q_heads, num_kv_heads)
    if n == 0:
        raise KvqError("kvq_prompt_workspace_bytes", 2)
    torch = _torch()
    return torch.empty(n, dtype=torch.uint8, device=device)


def kvq_prompt_attn(q, k, v, cu_seqlens, out, workspace, dev_err, window: int = 0,
                    sm_scale: float = HEAD_DIM ** -0.5, stream=None):
    """Causal attention over packed prompts. q, out [T, Hq, 128], k, v [T, Hkv, 128] (bf16 or fp16; any
    token and head strides that are multiples of 8, such as views of one projection's output),
    cu_seqlens int32[B + 1]; window <= 0: none."""
    torch = _torch()
    dtype = q.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError(f"unsupported dtype {dtype}")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if not (D == HEAD_DIM and out.shape == q.shape and k.shape == v.shape == (T, Hkv, D)):
        raise ValueError(f"shapes: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}, out {tuple(out.shape)}")
    if not (k.dtype is v.dtype is out.dtype is dtype and q.is_cuda and
            q.get_device() == k.get_device() == v.get_device() == out.get_device()):
        raise ValueError("q, k, v and out must be tensors of one dtype on one device")
    B, dev = cu_seqlens.shape[0] - 1, q.get_device()
    cu = _is(cu_seqlens, torch.int32, (B + 1,), "cu_seqlens", dev)
    sq, sk, sv, so = q.stride(), k.stride(), v.stride(), out.stride()
    if not sq[2] == sk[2] == sv[2] == so[2] == 1:
        raise ValueError("the rows of q, k, v and out must be contiguous")
    if T > 1 and Hq > 1 and Hkv > 1:
        strides = _Strides(sq[0], sq[1], sk[0], sk[1], sv[0], sv[1], so[0], so[1])
    else:  # of an extent of one the stride does not matter: the packed one
        strides = _Strides(*(x for st, h in ((sq, Hq), (sk, Hkv), (sv, Hkv), (so, Hq))
                             for x in (st[0] if T > 1 else max(1, h) * D, st[1] if h > 1 else D)))
    status = lib.kvq_prompt_attn(q.data_ptr(), k.data_ptr(), v.data_ptr(), BF16 if dtype is torch.bfloat16 else F16, T,
                                 B, Hq, Hkv, strides, cu, window, sm_scale, out.data_ptr(), workspace.data_ptr(),
                                 _bytes(workspace, dev), _err(dev_err, dev), _here(dev, stream))
    if status:
        raise KvqError("kvq_prompt_attn", status)


_Strides = ctypes.c_int64 * 8


def kvq_tree_workspace_bytes(B: int, N: int, num_q_heads: int, num_kv_heads: int) -> int:
    return int(lib.kvq_tree_workspace_bytes(B, N, num_q_heads, num_kv_heads))


def alloc_tree_workspace(B: int, N: int, num_q_heads: int, num_kv_heads: int, device="cuda"):
    n = kvq_tree_workspace_bytes(B, N, num_q_heads, num_kv_heads)
    if n == 0:
        raise KvqError("kvq_tree_workspace_bytes", 2)
    torch = _torch()
    return torch.empty(n, dtype=torch.uint8, device=device)


def _tree_args(q, ctx_len, tree_mask, out, k_new, v_new, Hkv):
    """(device, B, N, Hq, dtype code, addresses of ctx_len, mask, k_new, v_new, out's dtype code)."""
    torch = _torch()
    B, N, Hq, D = q.shape
    if not (q.dtype is torch.bfloat16 or q.dtype is torch.float32) or D != HEAD_DIM or not (q.is_cuda and q.is_contiguous()):
        raise ValueError(f"q must be a contiguous device tensor [B, N, Hq, 128] of fp32 or bf16, got {q.dtype} {tuple(q.shape)}")
    if not (out.dtype is torch.bfloat16 or out.dtype is torch.float32):
        raise ValueError(f"out must be fp32 or bf16, got {out.dtype}")
    dev = q.get_device()
    _is(out, out.dtype, q.shape, "out", dev)
    if k_new is not None:
        _is(k_new, q.dtype, (B, N, Hkv, D), "k_new", dev)
    if v_new is not None:
        _is(v_new, q.dtype, (B, N, Hkv, D), "v_new", dev)
    mask = _is(tree_mask, torch.uint64 if tree_mask.dtype is torch.uint64 else torch.int64, (B, N), "tree_mask", dev)
    return (dev, B, N, Hq, BF16 if q.dtype is torch.bfloat16 else F32, _is(ctx_len, torch.int32, (B,), "ctx_len", dev), mask,
            None if k_new is None else k_new.data_ptr(), None if v_new is None else v_new.data_ptr(),
            BF16 if out.dtype is torch.bfloat16 else F32)


def kvq_tree_attn_int4(cache: Int4Cache, Mq, Mk, q, ctx_len, tree_mask, out, workspace, dev_err, k_new=None,
                       v_new=None, sm_scale: float = HEAD_DIM ** -0.5, eps: float = 1e-6, stream=None,
                       fwht: bool = False):
    """Attention of N drafted tokens per sequence over the int4 cache: q [B, N, Hq, 128] (fp32 or bf16),
    tree_mask int64 [B, N] (bit j: attends to drafted token j), out fp32 or bf16. fwht as in
    kvq_decode_attn_int4."""
    dev, B, N, Hq, dt, ctx, mask, kn, vn, odt = _tree_args(q, ctx_len, tree_mask, out, k_new, v_new, cache.num_kv_heads)
    fn = lib.kvq_tree_attn_int4_fwht if fwht else lib.kvq_tree_attn_int4
    fold = (HEAD_DIM,) if fwht else (HEAD_DIM, HEAD_DIM)
    status = fn(ctypes.byref(cache), _is(Mq, _th.float32, fold, "Mq", dev), None if Mk is None else _is(Mk, _th.float32, fold, "Mk", dev),
                q.data_ptr(), dt, B, N, Hq, ctx,
                mask, kn, vn, sm_scale, eps, out.data_ptr(), odt, workspace.data_ptr(), _bytes(workspace, dev),
                _err(dev_err, dev), _here(dev, stream))
    if status:
        raise KvqError("kvq_tree_attn_int4_fwht" if fwht else "kvq_tree_attn_int4", status)


def kvq_tree_attn_fp8_swa(ring: Fp8Ring, q, pos0, tree_mask, window: int, k_scale: float, v_scale: float, out,
                          workspace, dev_err, k_new=None, v_new=None, sm_scale: float = HEAD_DIM ** -0.5,
                          stream=None):
    """kvq_tree_attn_int4 over the e4m3 ring of a sliding-window layer (q used as given)."""
    dev, B, N, Hq, dt, ctx, mask, kn, vn, odt = _tree_args(q, pos0, tree_mask, out, k_new, v_new, ring.num_kv_heads)
    status = lib.kvq_tree_attn_fp8_swa(ctypes.byref(ring), q.data_ptr(), dt, B, N, Hq, ctx, mask, window, kn, vn, k_scale,
                                       v_scale, sm_scale, out.data_ptr(), odt, workspace.data_ptr(), _bytes(workspace, dev),
                                       _err(dev_err, dev), _here(dev, stream))
    if status:
        raise KvqError("kvq_tree_attn_fp8_swa", status)


def _layers(layers, kind):
    """The layers' descriptors, all of one kind, one behind the other (each a ctypes structure: its bytes)."""
    if list(map(type, layers)).count(kind) != len(layers):
        raise TypeError(f"the layers must be {kind.__name__}, got {sorted(t.__name__ for t in set(map(type, layers)))}")
    return b"".join(layers)


def _tree_commit(name, kind, layers, ctx_len, path, n_accept, dev_err, ctx_out, stream):
    i32, descriptors = _torch().int32, _layers(layers, kind)
    (B, N), dev = path.shape, _dev(path, "path")
    status = getattr(lib, name)(descriptors, len(layers), B, N, _is(ctx_len, i32, (B,), "ctx_len", dev),
                                _is(path, i32, (B, N), "path", dev), _is(n_accept, i32, (B,), "n_accept", dev),
                                None if ctx_out is None else _is(ctx_out, i32, (B,), "ctx_out", dev), _err(dev_err, dev),
                                _here(dev, stream))
    if status:
        raise KvqError(name, status)


def kvq_tree_commit_int4(caches, ctx_len, path, n_accept, dev_err, ctx_out=None, stream=None):
    """Moves the accepted tokens path[b, :n_accept[b]] of each tree right behind the context in every
    one of the layers `caches` (a list of Int4Cache); ctx_out receives the new context lengths."""
    _tree_commit("kvq_tree_commit_int4", Int4Cache, caches, ctx_len, path, n_accept, dev_err, ctx_out, stream)


def kvq_tree_commit_fp8(rings, pos0, path, n_accept, dev_err, ctx_out=None, stream=None):
    """kvq_tree_commit_int4 for sliding-window layers (a list of Fp8Ring)."""
    _tree_commit("kvq_tree_commit_fp8", Fp8Ring, rings, pos0, path, n_accept, dev_err, ctx_out, stream)


def _pool(page_refs, block_table):
    i32 = _torch().int32
    S, M = block_table.shape
    n, dev = page_refs.shape[0], _dev(page_refs, "page_refs")
    return dev, _is(page_refs, i32, (n,), "page_refs", dev), n, _is(block_table, i32, (S, M), "block_table", dev), S, M


def kvq_pages_alloc(page_refs, block_table, seq_ids, len_old, len_new, dev_err, stream=None):
    """Gives sequences seq_ids the pages to grow from len_old to len_new tokens (lowest free first)."""
    (dev, *pool), i32, n = _pool(page_refs, block_table), _th.int32, seq_ids.shape[0]
    status = lib.kvq_pages_alloc(*pool, n, _is(seq_ids, i32, (n,), "seq_ids", dev), _is(len_old, i32, (n,), "len_old", dev),
                                 _is(len_new, i32, (n,), "len_new", dev), _err(dev_err, dev), _here(dev, stream))
    if status:
        raise KvqError("kvq_pages_alloc", status)


def kvq_pages_fork(page_refs, block_table, parents, children, lens, copy_src, copy_dst, dev_err, stream=None):
    """Children share their parents' full pages of the first lens tokens and get a page of their own
    for a partly filled last one: kvq_pages_copy(caches, copy_src, copy_dst) then fills it."""
    (dev, *pool), i32, n = _pool(page_refs, block_table), _th.int32, parents.shape[0]
    status = lib.kvq_pages_fork(*pool, n, _is(parents, i32, (n,), "parents", dev), _is(children, i32, (n,), "children", dev),
                                _is(lens, i32, (n,), "lens", dev), _is(copy_src, i32, (n,), "copy_src", dev),
                                _is(copy_dst, i32, (n,), "copy_dst", dev), _err(dev_err, dev), _here(dev, stream))
    if status:
        raise KvqError("kvq_pages_fork", status)


def kvq_pages_free(page_refs, block_table, seq_ids, len_old, len_new, dev_err, stream=None):
    """Gives back the pages of sequences seq_ids behind len_new tokens."""
    (dev, *pool), i32, n = _pool(page_refs, block_table), _th.int32, seq_ids.shape[0]
    status = lib.kvq_pages_free(*pool, n, _is(seq_ids, i32, (n,), "seq_ids", dev), _is(len_old, i32, (n,), "len_old", dev),
                                _is(len_new, i32, (n,), "len_new", dev), _err(dev_err, dev), _here(dev, stream))
    if status:
        raise KvqError("kvq_pages_free", status)


def kvq_pages_compact(page_refs, block_table, copy_src, copy_dst, n_moves, dev_err, stream=None):
    """Renames the pages in use to the front of the pool; kvq_pages_copy(caches, copy_src, copy_dst,
    count=n_moves) then moves them. copy_src, copy_dst: int32, at least num_pages // 2 entries."""
    (dev, *pool), i32 = _pool(page_refs, block_table), _th.int32
    src, dst = _is(copy_src, i32, copy_src.shape, "copy_src", dev), _is(copy_dst, i32, copy_dst.shape, "copy_dst", dev)
    _need(min(copy_src.numel(), copy_dst.numel()) >= page_refs.shape[0] // 2,
          "copy_src and copy_dst must hold num_pages // 2 entries")
    status = lib.kvq_pages_compact(*pool, src, dst, _is(n_moves, i32, (1,), "n_moves", dev), _err(dev_err, dev),
                                   _here(dev, stream))
    if status:
        raise KvqError("kvq_pages_compact", status)


def kvq_pages_copy(caches, src, dst, dev_err, count=None, stream=None):
    """Copies page src[i] to page dst[i] in every one of the layers `caches` (pairs with -1 are passed
    over), for i < n or i < count (a device int32 tensor of one entry)."""
    i32, descriptors = _torch().int32, _layers(caches, Int4Cache)
    n, dev = src.shape[0], _dev(src, "src")
    status = lib.kvq_pages_copy(descriptors, len(caches), n, _is(src, i32, (n,), "src", dev), _is(dst, i32, (n,), "dst", dev),
                                None if count is None else _is(count, i32, (1,), "count", dev), _err(dev_err, dev),
                                _here(dev, stream))
    if status:
        raise KvqError("kvq_pages_copy", status)
