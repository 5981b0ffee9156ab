"""GB300 multi-token-prediction (MTP) speculative decoding step.

Thin Python binding of ``libmtp.so`` (C ABI declared in ``include/mtp.h``):
argument marshalling only.  Every step of the drafter head, the flush, the
sampling transforms, the verify and the rollback runs in the library's CUDA
kernels; there is no Python or CPU fallback.  Tensors are passed as torch
device tensors (PyTorch supplies device memory and streams only).
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmtp.so")

MTP_DTYPE_F32 = 0
MTP_DTYPE_BF16 = 1

STATUS = {
    0: "MTP_OK", 1: "MTP_ERR_UNSUPPORTED_ARCH", 2: "MTP_ERR_MISSING_TENSOR", 3: "MTP_ERR_DUP_TENSOR",
    4: "MTP_ERR_UNKNOWN_TENSOR", 5: "MTP_ERR_SHAPE", 6: "MTP_ERR_CONFIG_BOUNDS", 7: "MTP_ERR_NOT_BOUND",
    8: "MTP_ERR_KV_CAPACITY", 9: "MTP_ERR_BAD_ARG", 10: "MTP_ERR_NONFINITE", 11: "MTP_ERR_TIMEOUT",
    12: "MTP_ERR_CUDA", 13: "MTP_ERR_LAYOUT",
}

# Every symbol include/mtp.h declares.
EXPORTS = (
    "mtp_default_block_size", "mtp_status_str", "mtp_load", "mtp_free", "mtp_get_lengths",
    "mtp_set_lengths", "mtp_device_status", "mtp_flush", "mtp_draft", "spec_verify_workspace_bytes",
    "spec_verify", "kv_rollback", "mtp_profile_enable", "mtp_profile_kinds", "mtp_profile_kind_name",
    "mtp_profile_read", "mtp_kernel_launches", "spec_verify_noalloc",
    "mtp_depth_ctl_create", "mtp_depth_ctl_free", "mtp_depth_ctl_next", "mtp_depth_ctl_observe",
    "mtp_depth_ctl_state", "mtp_set_draft_head", "mtp_test_verify_stall",
    "kv_q4_row_bytes", "kv_page_plan", "kv_q4_append", "kv_q4_read", "kv_q4_attend_workspace_bytes",
    "kv_q4_attend", "spec_logprobs_workspace_bytes", "spec_logprobs",
    "mtp_rope_init", "kv_q4_append_rope", "kv_tree_plan", "kv_q4_attend_tree", "kv_q4_tree_commit",
    "kv_attend_prompt_workspace_bytes", "kv_attend_prompt",
)


class MTPError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}")


class Config(ctypes.Structure):
    _fields_ = [("architecture", ctypes.c_char_p), ("hidden", ctypes.c_int32), ("n_q", ctypes.c_int32),
                ("n_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("mtp_layers", ctypes.c_int32), ("max_rows", ctypes.c_int32),
                ("kv_capacity", ctypes.c_int32), ("max_depth", ctypes.c_int32), ("eps", ctypes.c_float),
                ("rope_theta", ctypes.c_float), ("dtype", ctypes.c_int32)]


class Tensor(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("data", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("ndim", ctypes.c_int32), ("shape", ctypes.c_int64 * 2)]


class Sampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("rep_penalty", ctypes.c_float), ("top_p", ctypes.c_float),
                ("min_p", ctypes.c_float), ("top_k", ctypes.c_int32), ("flags", ctypes.c_int32)]


class KV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("len", ctypes.c_void_p)]


class Q4Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
                ("v_exp", ctypes.c_void_p), ("n_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page", ctypes.c_int32), ("n_pages", ctypes.c_int32)]


MTP_TREE_MAX, MTP_MAX_CACHES, MTP_ROPE_MAX = 128, 64, 128


class Rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("turn", ctypes.c_uint64 * MTP_ROPE_MAX)]


_lib = None


def lib():
    """The loaded C library; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libmtp.so is not built at {LIB_PATH}; run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        L.mtp_default_block_size.argtypes = [ctypes.POINTER(Config)]
        L.mtp_default_block_size.restype = i32
        L.mtp_status_str.argtypes = [ctypes.c_int]
        L.mtp_status_str.restype = ctypes.c_char_p
        L.mtp_load.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Tensor), i32, vp, vp, KV, vp, vp,
                               ctypes.POINTER(vp)]
        L.mtp_free.argtypes = [vp]
        L.mtp_get_lengths.argtypes = [vp, vp]
        L.mtp_set_lengths.argtypes = [vp, vp, vp]
        L.mtp_device_status.argtypes = [vp]
        L.mtp_device_status.restype = vp
        L.mtp_flush.argtypes = [vp, vp, i32, vp, i32, vp, vp, i32]
        L.mtp_draft.argtypes = [vp, vp, i32, i32, vp, i32, vp, vp, i32, ctypes.POINTER(Sampling), vp, i32,
                                vp, vp, vp, vp, vp]
        L.spec_verify_workspace_bytes.argtypes = [i32, i32, i32]
        L.spec_verify_workspace_bytes.restype = sz
        L.spec_verify.argtypes = [vp, i32, i32, i32, vp, vp, vp, ctypes.POINTER(Sampling), vp, i32, vp, vp,
                                  vp, vp, vp, vp, vp]
        L.spec_verify_noalloc.argtypes = [vp, i32, i32, i32, vp, vp, vp, ctypes.POINTER(Sampling), vp, i32,
                                          vp, vp, vp, vp, vp, vp]
        L.mtp_test_verify_stall.argtypes = [i32, i32]
        L.kv_rollback.argtypes = [vp, vp, i32, vp, vp, i32, i32]
        L.mtp_profile_enable.argtypes = [vp, i32]
        L.mtp_profile_kinds.restype = i32
        L.mtp_profile_kind_name.argtypes = [i32]
        L.mtp_profile_kind_name.restype = ctypes.c_char_p
        L.mtp_profile_read.argtypes = [vp, vp, vp]
        L.mtp_kernel_launches.restype = ctypes.c_int64
        i64, cache = ctypes.c_int64, ctypes.POINTER(Q4Cache)
        L.kv_q4_row_bytes.argtypes = [i32]
        L.kv_q4_row_bytes.restype = sz
        L.kv_page_plan.argtypes = [vp, i32, i32, i32, i32, i32] + [vp] * 10
        L.kv_q4_append.argtypes = [vp, cache, i32, vp, i64, i64, vp, i64, i64, i32, vp, vp]
        L.kv_q4_read.argtypes = [vp, cache, i32, vp, vp, vp, i32, vp]
        L.kv_q4_attend_workspace_bytes.argtypes = [cache, i32, i32, i32]
        L.kv_q4_attend_workspace_bytes.restype = sz
        L.kv_q4_attend.argtypes = [vp, cache, i32, i32, i32, vp, i64, i64, i32, vp, i32, vp, vp, i32,
                                   ctypes.c_float, i32, vp, vp, vp, vp]
        L.spec_logprobs_workspace_bytes.argtypes = [i32, i32, i32]
        L.spec_logprobs_workspace_bytes.restype = sz
        L.spec_logprobs.argtypes = [vp, i32, i32, vp, i64, i32, vp, i32] + [vp] * 7
        f32 = ctypes.c_float
        L.mtp_rope_init.argtypes = [i32, ctypes.c_double, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(Rope)]
        L.kv_q4_append_rope.argtypes = [vp, cache, i32, i32, vp, i64, i64, vp, i64, i64, vp, i64, i64, i32, vp, vp, f32,
                                        ctypes.POINTER(Rope), vp, vp, vp, vp, vp]
        L.kv_tree_plan.argtypes = [vp, i32, i32, vp, vp, vp, i32, vp, vp, vp]
        L.kv_q4_attend_tree.argtypes = [vp, cache, i32, i32, i32, vp, i64, i64, i32, vp, i32, vp, vp, vp, vp, i32, f32, i32,
                                        vp, vp, vp, vp]
        L.kv_q4_tree_commit.argtypes = [vp, cache, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, i32] + [vp] * 5
        L.kv_attend_prompt_workspace_bytes.argtypes = [i32, i32]
        L.kv_attend_prompt_workspace_bytes.restype = sz
        L.kv_attend_prompt.argtypes = [vp, i32, i32, i32, i32, i32, vp, i64, i64, vp, i64, i64, vp, i64, i64, i32, vp, i32,
                                       f32, i32, vp, vp, vp, vp]
        for name in ("mtp_load", "mtp_free", "mtp_get_lengths", "mtp_set_lengths", "mtp_flush", "mtp_draft",
                     "spec_verify", "spec_verify_noalloc", "kv_rollback", "mtp_profile_enable",
                     "mtp_profile_read", "mtp_test_verify_stall", "kv_page_plan", "kv_q4_append", "kv_q4_read",
                     "kv_q4_attend", "spec_logprobs", "mtp_rope_init", "kv_q4_append_rope", "kv_tree_plan",
                     "kv_q4_attend_tree", "kv_q4_tree_commit", "kv_attend_prompt"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc: int, where: str):
    if rc != 0:
        raise MTPError(rc, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = None


def _stream(stream):
    """The cudaStream_t of a torch stream, an integer, or the current stream (None)."""
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if _raw_stream is None:
        import torch
        # the current stream's handle without a Stream object around it (3 us on a Grace core), where torch has it
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = torch.cuda.current_device
        _raw_stream = (lambda: raw(device())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


_BF16 = None


def _dtype_code(t) -> int:
    global _BF16
    if _BF16 is None:
        import torch
        _BF16 = torch.bfloat16
    return MTP_DTYPE_BF16 if t.dtype is _BF16 else MTP_DTYPE_F32


def _i32_array(values):
    """Host int32 array for a C pointer argument (a list/tuple or a numpy array)."""
    if isinstance(values, np.ndarray):
        values = values.astype(np.int32, copy=False).ravel().tolist()
    return (ctypes.c_int32 * len(values))(*values)


MTP_SAMPLE_ARGMAX_DRAFT = 1


def sampling_array(params) -> ctypes.Array:
    """params: list of dicts (temperature, rep_penalty, top_k, top_p, min_p,
    argmax_draft) or tuples (temperature, rep_penalty, top_k, top_p, min_p)."""
    arr = (Sampling * len(params))()
    for i, p in enumerate(params):
        flags = 0
        if isinstance(p, dict):
            flags = MTP_SAMPLE_ARGMAX_DRAFT if p.get("argmax_draft", False) else 0
            p = (p.get("temperature", 0.0), p.get("rep_penalty", 1.0), p.get("top_k", 0),
                 p.get("top_p", 1.0), p.get("min_p", 0.0))
        t, r, k, tp, mp = p
        arr[i] = Sampling(float(t), float(r), float(tp), float(mp), int(k), flags)
    return arr


def make_config(shape, max_rows: int, kv_capacity: int, max_depth: int,
                architecture: str = "qwen3_5_mtp") -> Config:
    return Config(architecture.encode(), shape.hidden, shape.n_q, shape.n_kv, shape.head_dim, shape.inter,
                  shape.vocab, 1, max_rows, kv_capacity, max_depth, shape.eps, shape.rope_theta,
                  MTP_DTYPE_BF16 if shape.dtype == "bf16" else MTP_DTYPE_F32)


def mtp_default_block_size(cfg: Config) -> int:
    return lib().mtp_default_block_size(ctypes.byref(cfg))


def mtp_status_str(code: int) -> str:
    return lib().mtp_status_str(code).decode()


class Handle:
    """An mtp_t plus the ctypes objects that must outlive it."""

    def __init__(self, ptr, cfg, keep):
        self.ptr = ptr
        self.cfg = cfg
        self._keep = keep

    def close(self):
        if self.ptr:
            lib().mtp_free(self.ptr)
            self.ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def mtp_load(cfg: Config, tensors: dict, embed, lm_head, kv_k, kv_v, kv_len, lengths=None,
             stream=None) -> Handle:
    """tensors: name -> torch device tensor (names as in the checkpoint)."""
    names = list(tensors)
    arr = (Tensor * len(names))()
    keep = [cfg]
    for i, n in enumerate(names):
        t = tensors[n]
        b = n.encode()
        keep.append(b)
        shp = (ctypes.c_int64 * 2)(*(list(t.shape) + [0, 0])[:2])
        arr[i] = Tensor(b, _ptr(t), _dtype_code(t), t.dim(), shp)
    keep.append(arr)
    kv = KV(_ptr(kv_k), _ptr(kv_v), _ptr(kv_len))
    hl = None
    if lengths is not None:
        hl = np.ascontiguousarray(lengths, dtype=np.int32)
        keep.append(hl)
    out = ctypes.c_void_p()
    rc = lib().mtp_load(ctypes.byref(cfg), arr, len(names), _ptr(embed), _ptr(lm_head), kv,
                        hl.ctypes.data if hl is not None else None, _stream(stream), ctypes.byref(out))
    _check(rc, "mtp_load")
    return Handle(out.value, cfg, keep)


def mtp_get_lengths(h: Handle) -> np.ndarray:
    out = np.zeros(h.cfg.max_rows, np.int32)
    _check(lib().mtp_get_lengths(h.ptr, out.ctypes.data), "mtp_get_lengths")
    return out


def mtp_set_lengths(h: Handle, lengths, stream=None):
    _check(lib().mtp_set_lengths(h.ptr, _stream(stream), _i32_array(lengths)), "mtp_set_lengths")


def mtp_device_status(h: Handle) -> int:
    return lib().mtp_device_status(h.ptr)


def mtp_flush(h: Handle, pairs, tok, hid, stream=None):
    """pairs: host int list [rows]; tok [rows, pmax] int32; hid [rows, pmax, H]."""
    hp = np.ascontiguousarray(pairs, dtype=np.int32)
    rc = lib().mtp_flush(h.ptr, _stream(stream), len(hp), hp.ctypes.data, tok.shape[1], _ptr(tok), _ptr(hid),
                         _dtype_code(hid))
    _check(rc, "mtp_flush")


def mtp_draft(h: Handle, depth: int, pairs, tok, hid, params, draft, hist=None, u=None, q=None, logits=None,
              hidden=None, stream=None):
    # (on the host path between two rounds: argument marshalling kept lean)
    hp = _i32_array(pairs)
    sp = params if isinstance(params, ctypes.Array) else sampling_array(params)
    hist_w = 0 if hist is None else hist.shape[1]
    rc = lib().mtp_draft(h.ptr, stream if type(stream) is int else _stream(stream), len(hp), depth, hp,
                         tok.shape[1], _ptr(tok), _ptr(hid), _dtype_code(hid), sp, _ptr(hist), hist_w, _ptr(u),
                         _ptr(draft), _ptr(q), _ptr(logits), _ptr(hidden))
    _check(rc, "mtp_draft")


def spec_verify_workspace_bytes(rows: int, depth: int, vocab: int) -> int:
    return lib().spec_verify_workspace_bytes(rows, depth, vocab)


def spec_verify(logits, draft, params, u, n_acc, out_tok, workspace, q=None, hist=None, stats=None,
                h_out=None, status=None, stream=None):
    """logits [rows, depth+1, V] f32; draft [rows, depth] i32; u [rows, depth+1] f32;
    status: optional device int32 word (OR of 1 << MTP_ERR_* seen on the device)."""
    rows, dp1, V = logits.shape
    sp = params if isinstance(params, ctypes.Array) else sampling_array(params)
    hist_w = 0 if hist is None else hist.shape[1]
    rc = lib().spec_verify(_stream(stream), rows, dp1 - 1, V, _ptr(logits), _ptr(draft), _ptr(q), sp,
                           _ptr(hist), hist_w, _ptr(u), _ptr(n_acc), _ptr(out_tok), _ptr(stats), _ptr(h_out),
                           _ptr(status), _ptr(workspace))
    _check(rc, "spec_verify")


def spec_verify_noalloc(logits, draft, params, u, n_acc, out_tok, q=None, hist=None, stats=None, h_out=None,
                        status=None, stream=None):
    """spec_verify with the library's fixed scratch instead of a workspace
    (for callers that cannot allocate device memory)."""
    rows, dp1, V = logits.shape
    sp = params if isinstance(params, ctypes.Array) else sampling_array(params)
    hist_w = 0 if hist is None else hist.shape[1]
    rc = lib().spec_verify_noalloc(_stream(stream), rows, dp1 - 1, V, _ptr(logits), _ptr(draft), _ptr(q), sp,
                                   _ptr(hist), hist_w, _ptr(u), _ptr(n_acc), _ptr(out_tok), _ptr(stats),
                                   _ptr(h_out), _ptr(status))
    _check(rc, "spec_verify_noalloc")


def mtp_test_verify_stall(stage: int, wait_polls: int) -> None:
    """Test hook: the next streaming-path spec_verify leaves ring stage
    `stage` unfilled and gives each wait `wait_polls` polls (its waits run out
    and it reports MTP_ERR_TIMEOUT)."""
    _check(lib().mtp_test_verify_stall(int(stage), int(wait_polls)), "mtp_test_verify_stall")


def kv_rollback(h: Handle, rows: int, depth: int, n_acc=None, target_len=None, zero_tail: bool = False,
                stream=None):
    rc = lib().kv_rollback(h.ptr, _stream(stream), rows, _ptr(n_acc), _ptr(target_len), depth,
                           1 if zero_tail else 0)
    _check(rc, "kv_rollback")


def _want(ok: bool, where: str):
    """Checks that the C side cannot make (shapes, element types): a bad argument like its own."""
    if not ok:
        raise MTPError(9, where)


_torch = None


def _t():
    """torch, imported with the first call that needs it."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _whole(where: str, *tensors, n=None):
    """Contiguous int32 tensors (None passes), of n elements if n is given."""
    i32 = _t().int32
    for t in tensors:
        if t is not None and (t.dtype is not i32 or not t.is_contiguous() or (n is not None and t.numel() != n)):
            raise MTPError(9, where)


def kv_q4_row_bytes(head_dim: int) -> int:
    return lib().kv_q4_row_bytes(head_dim)


class PagedCache:
    """A kv_q4_cache and the tensors it points to."""

    def __init__(self, c, keep):
        self.c = c
        self.ref = ctypes.byref(c)
        self.n_kv, self.head_dim = c.n_kv, c.head_dim  # (a field of the structure costs 0.1 us a read)
        self._keep = keep


def kv_q4_cache(k, v, k_exp=None, v_exp=None) -> PagedCache:
    """k, v: uint8 [n_pages, n_kv, page, kv_q4_row_bytes(head_dim)]; k_exp, v_exp: int32 [n_kv] exponents."""
    n_pages, n_kv, page, row = k.shape
    _want(k.shape == v.shape and k.element_size() == v.element_size() == 1 and k.is_contiguous()
          and v.is_contiguous() and row in (36, 72, 144), "kv_q4_cache")
    _whole("kv_q4_cache", k_exp, v_exp, n=n_kv)
    return PagedCache(Q4Cache(_ptr(k), _ptr(v), _ptr(k_exp), _ptr(v_exp), n_kv, row * 16 // 9, page, n_pages),
                      (k, v, k_exp, v_exp))


def kv_page_plan(cover, keep, new, table, free, cover_out, start, slot, pos, page: int, status=None, stream=None):
    """cover, keep, new, cover_out [rows]; table [rows, max_pages]; free [n_pages]; start [rows + 1];
    slot, pos [max_tokens]; all int32. See kv_page_plan in include/mtp.h."""
    rows, max_pages = table.shape
    _whole("kv_page_plan", cover, keep, new, cover_out, n=rows)
    _whole("kv_page_plan", table, free, start, slot, pos)
    _want(start.numel() == rows + 1 and slot.numel() == pos.numel(), "kv_page_plan")
    rc = lib().kv_page_plan(_stream(stream), rows, page, max_pages, free.numel(), slot.numel(), _ptr(cover),
                            _ptr(keep), _ptr(new), _ptr(table), _ptr(free), _ptr(cover_out), _ptr(start), _ptr(slot),
                            _ptr(pos), _ptr(status))
    _check(rc, "kv_page_plan")


def _dtype_q4(where: str, *tensors) -> int:
    """The dtype code of tensors of one type, fp32 or bf16."""
    torch, dt = _t(), tensors[0].dtype
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise MTPError(9, where)
    for t in tensors:
        if t.dtype is not dt:
            raise MTPError(9, where)
    return MTP_DTYPE_BF16 if dt is torch.bfloat16 else MTP_DTYPE_F32


def kv_q4_append(cache: PagedCache, k, v, slot, status=None, stream=None):
    """k, v: [tokens, n_kv, head_dim], fp32 or bf16, the last dimension contiguous; slot [tokens] int32."""
    shape = (slot.numel(), cache.n_kv, cache.head_dim)
    _want(k.shape == shape and v.shape == shape and k.stride(2) == 1 and v.stride(2) == 1, "kv_q4_append")
    _whole("kv_q4_append", slot)
    rc = lib().kv_q4_append(_stream(stream), cache.ref, shape[0], _ptr(k), k.stride(0), k.stride(1), _ptr(v), v.stride(0),
                            v.stride(1), _dtype_q4("kv_q4_append", k, v), _ptr(slot), _ptr(status))
    _check(rc, "kv_q4_append")


def kv_q4_read(cache: PagedCache, slot, k, v, status=None, stream=None):
    """slot [tokens] int32; k, v: [tokens, n_kv, head_dim] out, contiguous, fp32 or bf16."""
    shape = (slot.numel(), cache.n_kv, cache.head_dim)
    _want(k.shape == shape and v.shape == shape and k.is_contiguous() and v.is_contiguous(), "kv_q4_read")
    _whole("kv_q4_read", slot)
    rc = lib().kv_q4_read(_stream(stream), cache.ref, shape[0], _ptr(slot), _ptr(k), _ptr(v),
                          _dtype_q4("kv_q4_read", k, v), _ptr(status))
    _check(rc, "kv_q4_read")


def _device() -> int:
    """The current device's index, -1 before torch has set CUDA up (the library then looks at the first device)."""
    cuda = _t().cuda
    return cuda.current_device() if cuda.is_initialized() else -1


# Workspace sizes depend on the call's sizes and the current device's SM count, and are asked for by every call that
# checks its workspace.
@functools.lru_cache(maxsize=1024)
def _attend_bytes(device: int, n_kv: int, head_dim: int, n_q: int, max_q: int, dt: int) -> int:
    c = Q4Cache(None, None, None, None, n_kv, head_dim, 16, 1)
    return lib().kv_q4_attend_workspace_bytes(ctypes.byref(c), n_q, max_q, dt)


@functools.lru_cache(maxsize=1024)
def _logprobs_bytes(device: int, n: int, vocab: int, top: int) -> int:
    return lib().spec_logprobs_workspace_bytes(n, vocab, top)


@functools.lru_cache(maxsize=1024)
def _prompt_bytes(tokens: int, rows: int) -> int:
    return lib().kv_attend_prompt_workspace_bytes(tokens, rows)


def kv_q4_attend_workspace_bytes(cache: PagedCache, n_q: int, max_q: int, dtype) -> int:
    """dtype: the queries' torch dtype."""
    return _attend_bytes(_device(), cache.n_kv, cache.head_dim, n_q, max_q,
                         MTP_DTYPE_BF16 if dtype is _t().bfloat16 else MTP_DTYPE_F32)


def kv_q4_attend(cache: PagedCache, q, table, start, length, out, workspace, max_q: int, scale: float, window: int = 0,
                 lse=None, status=None, stream=None):
    """q: [tokens, n_q, head_dim], fp32 or bf16, the last dimension contiguous; table [rows, max_pages], start [rows + 1],
    length [rows] int32; out [tokens, n_q, head_dim]; lse [tokens, n_q] float; workspace:
    kv_q4_attend_workspace_bytes(cache, n_q, max_q, q.dtype) bytes."""
    tokens, n_q, dh = q.shape
    rows, max_pages = table.shape
    _want(dh == cache.head_dim and q.stride(2) == 1 and out.shape == q.shape and out.is_contiguous()
          and (lse is None or (lse.dtype is _t().float32 and lse.numel() == tokens * n_q and lse.is_contiguous())),
          "kv_q4_attend")
    _whole("kv_q4_attend", table, start, length)
    _want(start.numel() == rows + 1 and length.numel() == rows, "kv_q4_attend")
    dt = _dtype_q4("kv_q4_attend", q, out)
    _want(workspace.nbytes >= _attend_bytes(_device(), cache.n_kv, dh, n_q, max_q, dt), "kv_q4_attend")
    rc = lib().kv_q4_attend(_stream(stream), cache.ref, rows, n_q, tokens, _ptr(q), q.stride(0), q.stride(1), dt,
                            _ptr(table), max_pages, _ptr(start), _ptr(length), max_q, scale, window, _ptr(out), _ptr(lse),
                            _ptr(status), _ptr(workspace))
    _check(rc, "kv_q4_attend")


def spec_logprobs_workspace_bytes(n: int, vocab: int, top: int) -> int:
    return lib().spec_logprobs_workspace_bytes(n, vocab, top)


def spec_logprobs(logits, tok, logprob, workspace, rank=None, entropy=None, top_id=None, top_lp=None, status=None,
                  stream=None):
    """logits [n, V] fp32 or bf16, rows contiguous; tok [n] int32; logprob [n] float out; optional outputs rank [n]
    int32, entropy [n] float, top_id [n, top] int32 and top_lp [n, top] float; workspace:
    spec_logprobs_workspace_bytes(n, V, top) bytes."""
    n, V = logits.shape
    top = 0 if top_id is None else top_id.shape[1]
    _whole("spec_logprobs", tok, rank, n=n)
    _whole("spec_logprobs", top_id, n=n * top)
    f32 = _t().float32
    for t, size in ((logprob, n), (entropy, n), (top_lp, n * top)):
        if t is not None and (t.dtype is not f32 or not t.is_contiguous() or t.numel() != size):
            raise MTPError(9, "spec_logprobs")
    _want(logits.stride(1) == 1 and (top_id is None) == (top_lp is None)
          and workspace.nbytes >= _logprobs_bytes(_device(), n, V, top), "spec_logprobs")
    rc = lib().spec_logprobs(_stream(stream), n, V, _ptr(logits), logits.stride(0), _dtype_q4("spec_logprobs", logits),
                             _ptr(tok), top, _ptr(logprob), _ptr(rank), _ptr(entropy), _ptr(top_id), _ptr(top_lp),
                             _ptr(status), _ptr(workspace))
    _check(rc, "spec_logprobs")


def mtp_rope(rot_dim: int, theta: float = 10000.0, freq=None) -> Rope:
    """Frequencies of a rotation over the first rot_dim dimensions: theta^(-2i/rot_dim) radians a position, or freq[i]."""
    out = Rope()
    f = None
    if freq is not None:
        _want(len(freq) == rot_dim // 2, "mtp_rope_init")
        f = (ctypes.c_double * max(len(freq), 1))(*[float(x) for x in freq])
    _check(lib().mtp_rope_init(int(rot_dim), float(theta), f, ctypes.byref(out)), "mtp_rope_init")
    return out


def _f32(where: str, *tensors, n):
    """Contiguous float32 tensors of n elements (None passes)."""
    f32 = _t().float32
    for t in tensors:
        if t is not None and (t.dtype is not f32 or not t.is_contiguous() or t.numel() != n):
            raise MTPError(9, where)


def kv_q4_append_rope(cache: PagedCache, q, k, v, rope: Rope, pos, slot, q_out, k_out=None, q_norm=None, k_norm=None,
                      eps: float = 1e-6, status=None, stream=None):
    """q [tokens, n_q, head_dim], k, v [tokens, n_kv, head_dim], fp32 or bf16, the last dimension contiguous; pos, slot
    [tokens] int32; q_out, k_out: contiguous like q and k (k_out optional); q_norm, k_norm [head_dim] float (None: no norm);
    rope: mtp_rope(...). See kv_q4_append_rope in include/mtp.h."""
    tokens, n_q, dh = q.shape
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    shape = (tokens, cache.n_kv, cache.head_dim)
    _want(k.shape == shape and v.shape == shape and dh == cache.head_dim and qs[2] == 1 and ks[2] == 1
          and vs[2] == 1 and q_out.shape == q.shape and q_out.is_contiguous()
          and (k_out is None or (k_out.shape == shape and k_out.is_contiguous())), "kv_q4_append_rope")
    _whole("kv_q4_append_rope", pos, slot, n=tokens)
    _f32("kv_q4_append_rope", q_norm, k_norm, n=dh)
    dt = _dtype_q4("kv_q4_append_rope", q, k, v, q_out) if k_out is None else _dtype_q4("kv_q4_append_rope", q, k, v, q_out, k_out)
    rc = lib().kv_q4_append_rope(_stream(stream), cache.ref, tokens, n_q, q.data_ptr(), qs[0], qs[1], k.data_ptr(),
                                 ks[0], ks[1], v.data_ptr(), vs[0], vs[1], dt, _ptr(q_norm), _ptr(k_norm),
                                 eps, ctypes.byref(rope), _ptr(pos), _ptr(slot), q_out.data_ptr(), _ptr(k_out),
                                 _ptr(status))
    _check(rc, "kv_q4_append_rope")


def kv_tree_plan(parent, start, length, pos, mask, window: int = 0, status=None, stream=None):
    """parent, pos [tokens], start [rows + 1], length [rows], mask [tokens, MTP_TREE_MAX / 32], all int32. See kv_tree_plan
    in include/mtp.h."""
    tokens, rows = parent.numel(), length.numel()
    _whole("kv_tree_plan", parent, pos, n=tokens)
    _whole("kv_tree_plan", mask, n=tokens * (MTP_TREE_MAX // 32))
    _whole("kv_tree_plan", start, n=rows + 1)
    _whole("kv_tree_plan", length)
    rc = lib().kv_tree_plan(_stream(stream), rows, tokens, parent.data_ptr(), _ptr(start), length.data_ptr(), window, _ptr(pos),
                            _ptr(mask), _ptr(status))
    _check(rc, "kv_tree_plan")


def kv_q4_attend_tree(cache: PagedCache, q, table, start, length, mask, out, workspace, max_q: int, scale: float,
                      window: int = 0, pos=None, lse=None, status=None, stream=None):
    """kv_q4_attend for trees: mask [tokens, MTP_TREE_MAX / 32] and pos [tokens] (with a window) int32, kv_tree_plan's;
    the other arguments as there."""
    tokens, n_q, dh = q.shape
    qs = q.stride()
    rows, max_pages = table.shape
    _want(dh == cache.head_dim and qs[2] == 1 and out.shape == q.shape and out.is_contiguous(), "kv_q4_attend_tree")
    _f32("kv_q4_attend_tree", lse, n=tokens * n_q)
    _whole("kv_q4_attend_tree", table)
    _whole("kv_q4_attend_tree", start, n=rows + 1)
    _whole("kv_q4_attend_tree", length, n=rows)
    _whole("kv_q4_attend_tree", mask, n=tokens * (MTP_TREE_MAX // 32))
    _whole("kv_q4_attend_tree", pos, n=tokens)
    dt = _dtype_q4("kv_q4_attend_tree", q, out)
    _want(workspace.nbytes >= _attend_bytes(_device(), cache.n_kv, dh, n_q, max_q, dt), "kv_q4_attend_tree")
    rc = lib().kv_q4_attend_tree(_stream(stream), cache.ref, rows, n_q, tokens, q.data_ptr(), qs[0], qs[1], dt,
                                 table.data_ptr(), max_pages, _ptr(start), _ptr(length), _ptr(mask), _ptr(pos), max_q, scale,
                                 window, out.data_ptr(), _ptr(lse), _ptr(status), workspace.data_ptr())
    _check(rc, "kv_q4_attend_tree")


class PagedCaches:
    """The layers of one kv_q4_tree_commit: an array of kv_q4_cache and the tensors it points to."""

    def __init__(self, caches):
        self.n = len(caches)
        self.c = (Q4Cache * max(self.n, 1))(*[x.c for x in caches])
        self._keep = list(caches)


def kv_q4_caches(caches) -> PagedCaches:
    """caches: the layers' PagedCache objects, of one shape, at most MTP_MAX_CACHES."""
    return PagedCaches(caches)


def kv_q4_tree_commit(caches: PagedCaches, table, start, length, parent, tok, choice, n_acc, out_tok, keep, path=None,
                      status=None, stream=None):
    """table [rows, max_pages], start [rows + 1], length, n_acc, keep [rows], parent, tok, choice [tokens], out_tok and
    path [rows, max_path], all int32. See kv_q4_tree_commit in include/mtp.h."""
    rows, max_path = out_tok.shape
    tokens, max_pages = parent.numel(), 1 if table is None else table.shape[1]
    _want(table is None or table.shape[0] == rows, "kv_q4_tree_commit")
    _whole("kv_q4_tree_commit", table, out_tok)
    _whole("kv_q4_tree_commit", start, n=rows + 1)
    _whole("kv_q4_tree_commit", length, n_acc, keep, n=rows)
    _whole("kv_q4_tree_commit", parent, tok, choice, n=tokens)
    _whole("kv_q4_tree_commit", path, n=rows * max_path)
    rc = lib().kv_q4_tree_commit(_stream(stream), caches.c, caches.n, rows, tokens, _ptr(table), max_pages, _ptr(start),
                                 _ptr(length), parent.data_ptr(), _ptr(tok), _ptr(choice), max_path, _ptr(n_acc),
                                 out_tok.data_ptr(), _ptr(keep), _ptr(path), _ptr(status))
    _check(rc, "kv_q4_tree_commit")


def kv_attend_prompt_workspace_bytes(tokens: int, rows: int) -> int:
    return lib().kv_attend_prompt_workspace_bytes(tokens, rows)


def kv_attend_prompt(q, k, v, start, out, workspace, max_len: int, scale: float, window: int = 0, lse=None, status=None,
                     stream=None):
    """q [tokens, n_q, head_dim], k, v [tokens, n_kv, head_dim], fp32 or bf16, the last dimension contiguous, 16-byte aligned
    rows; start [rows + 1] int32; out like q, contiguous; lse [tokens, n_q] float; workspace:
    kv_attend_prompt_workspace_bytes(tokens, rows) bytes. See kv_attend_prompt in include/mtp.h."""
    tokens, n_q, dh = q.shape
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    rows, n_kv = start.numel() - 1, k.shape[1]
    _want(k.shape == (tokens, n_kv, dh) and v.shape == k.shape and qs[2] == 1 and ks[2] == 1 and vs[2] == 1
          and out.shape == q.shape and out.is_contiguous(), "kv_attend_prompt")
    _f32("kv_attend_prompt", lse, n=tokens * n_q)
    _whole("kv_attend_prompt", start)
    dt = _dtype_q4("kv_attend_prompt", q, k, v, out)
    _want(workspace.nbytes >= _prompt_bytes(tokens, rows), "kv_attend_prompt")
    rc = lib().kv_attend_prompt(_stream(stream), rows, n_q, n_kv, dh, tokens, q.data_ptr(), qs[0], qs[1], k.data_ptr(),
                                ks[0], ks[1], v.data_ptr(), vs[0], vs[1], dt, start.data_ptr(), max_len, scale,
                                window, out.data_ptr(), _ptr(lse), _ptr(status), workspace.data_ptr())
    _check(rc, "kv_attend_prompt")


PROFILE_KINDS = ("fc", "qkv", "qkv_post", "attention", "o_proj", "gate_up", "down", "lm_head", "sample",
                 "flush_fc", "flush_kv", "rollback")


def mtp_profile_enable(h: Handle, kinds=True):
    """kinds: True (all), False (off), or an iterable of kind names."""
    if kinds is True:
        mask = -1
    elif not kinds:
        mask = 0
    else:
        mask = 0
        for k in kinds:
            mask |= 1 << PROFILE_KINDS.index(k)
    _check(lib().mtp_profile_enable(h.ptr, mask), "mtp_profile_enable")


def mtp_profile_read(h: Handle) -> dict:
    n = lib().mtp_profile_kinds()
    ms = np.zeros(n, np.float32)
    cnt = np.zeros(n, np.int32)
    _check(lib().mtp_profile_read(h.ptr, ms.ctypes.data, cnt.ctypes.data), "mtp_profile_read")
    return {lib().mtp_profile_kind_name(i).decode(): (float(ms[i]), int(cnt[i])) for i in range(n)}


def mtp_kernel_launches() -> int:
    return int(lib().mtp_kernel_launches())


MTP_HEAD_BF16, MTP_HEAD_FP8 = 0, 1


def mtp_set_draft_head(h: Handle, fmt: int, stream=None) -> None:
    """MTP_HEAD_FP8: the drafter reads an e4m3 copy of the tied head (per-row
    scales); MTP_HEAD_BF16: the borrowed head itself."""
    L = lib()
    L.mtp_set_draft_head.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32]
    _check(L.mtp_set_draft_head(h.ptr, _stream(stream), int(fmt)), "mtp_set_draft_head")


class DepthController:
    """Draft-depth controller (host-side, in libmtp): next() is the depth to
    draft this round, observe(depth, n_acc, seconds) feeds back the round run."""

    def __init__(self, max_depth: int):
        L = lib()
        L.mtp_depth_ctl_create.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_void_p)]
        L.mtp_depth_ctl_next.argtypes = [ctypes.c_void_p]
        L.mtp_depth_ctl_next.restype = ctypes.c_int32
        L.mtp_depth_ctl_observe.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_double]
        L.mtp_depth_ctl_state.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
        L.mtp_depth_ctl_free.argtypes = [ctypes.c_void_p]
        self.max_depth = max_depth
        self.ptr = ctypes.c_void_p()
        _check(L.mtp_depth_ctl_create(max_depth, ctypes.byref(self.ptr)), "mtp_depth_ctl_create")

    def next(self) -> int:
        return int(lib().mtp_depth_ctl_next(self.ptr))

    def observe(self, depth: int, n_acc: int, seconds: float) -> None:
        _check(lib().mtp_depth_ctl_observe(self.ptr, depth, n_acc, float(seconds)), "mtp_depth_ctl_observe")

    def state(self):
        a = np.zeros(max(self.max_depth, 1), np.float64)
        c = np.zeros(self.max_depth + 1, np.float64)
        iv = ctypes.c_int32(0)
        _check(lib().mtp_depth_ctl_state(self.ptr, a.ctypes.data, c.ctypes.data, ctypes.byref(iv)),
               "mtp_depth_ctl_state")
        return a[: self.max_depth], c, int(iv.value)

    def close(self):
        if self.ptr:
            lib().mtp_depth_ctl_free(self.ptr)
            self.ptr = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
