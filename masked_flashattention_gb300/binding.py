"""Thin ctypes binding of libcm.so, with the same names as the C ABI (include/cm.h).

Argument marshalling only: every step of the hot path runs in the library's CUDA kernels.
PyTorch supplies device memory (tensor data pointers) and streams; nothing here computes a
descriptor or an attention value, and there is no fallback when the library is missing.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcm.so")

CM_OK = 0
CM_ERR_PARSE = -1
CM_ERR_INVALID_ARG = -2
CM_ERR_UNSUPPORTED = -3
CM_ERR_CUDA = -4
CM_ERR_TIMEOUT = -5
CM_ERR_DEVICE_CHECK = -6
CM_ERR_DESC_MISMATCH = -7

TILE = 128


class CMError(RuntimeError):
    def __init__(self, code: int, what: str, detail: str = ""):
        self.code = code
        msg = f"{what}: {cm_error_string(code)} ({code})"
        super().__init__(msg + (f": {detail}" if detail else ""))


class cm_meta(ctypes.Structure):
    _fields_ = [("seg", ctypes.c_void_p), ("nseg", ctypes.c_void_p), ("nseg_max", ctypes.c_int32)]


class cm_descriptor(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("S", ctypes.c_int32), ("tile", ctypes.c_int32),
                ("ni_f", ctypes.c_int32), ("ni_b", ctypes.c_int32), ("form", ctypes.c_int32),
                ("itab_f", ctypes.c_void_p), ("bm_f", ctypes.c_void_p),
                ("itab_b", ctypes.c_void_p), ("bm_b", ctypes.c_void_p),
                ("sched_f", ctypes.c_void_p), ("sched_b", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class cm_kv_cache(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("H_kv", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("k_page_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("summary", ctypes.c_void_p), ("summary_scale", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class cm_kv_seqs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("page_table", ctypes.c_void_p), ("lens", ctypes.c_void_p)]


class cm_kv_pages(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("B", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("page_table", ctypes.c_void_p), ("free_pages", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


_Strides3 = ctypes.c_int64 * 3


class cm_kv_new(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
                ("k_stride", _Strides3), ("v_stride", _Strides3), ("q_stride", _Strides3),
                ("q_out_stride", _Strides3), ("k_out_stride", _Strides3),
                ("cu_new", ctypes.c_void_p), ("n_new", ctypes.c_void_p),
                ("n_tokens", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("H_q", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("rope_len", ctypes.c_int32),
                ("rope", ctypes.c_void_p), ("new_lens", ctypes.c_void_p), ("granted", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built (there is no other code path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "masked_flashattention_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.cm_compile_spec.argtypes = [ctypes.c_char_p, ctypes.POINTER(vp), ctypes.c_char_p, sz]
        L.cm_spec_free.argtypes = [vp]
        L.cm_spec_free.restype = None
        L.cm_spec_num_intervals.argtypes = [vp, ctypes.POINTER(i32)]
        L.cm_spec_describe.argtypes = [vp, ctypes.c_char_p, sz, ctypes.POINTER(sz)]
        L.cm_spec_kernel_source.argtypes = [vp, ctypes.c_char_p, sz, ctypes.POINTER(sz)]
        L.cm_spec_kernel_status.argtypes = [vp, i32, ctypes.c_char_p, sz]
        L.cm_descriptor_kernel_source.argtypes = [vp, vp, ctypes.c_char_p, sz, ctypes.POINTER(sz)]
        L.cm_descriptor_kernel_status.argtypes = [vp, vp, i32, ctypes.c_char_p, sz]
        L.cm_set_preprocess_mode.argtypes = [i32]
        L.cm_set_interval_check.argtypes = [i32]
        L.cm_descriptor_sizes.argtypes = [vp, vp, i32, i32, i32, i32, ctypes.POINTER(sz)]
        L.cm_build_descriptor.argtypes = [vp, vp, ctypes.POINTER(cm_meta), i32, i32,
                                          ctypes.POINTER(cm_descriptor), vp]
        L.cm_attn_fwd.argtypes = [ctypes.POINTER(cm_descriptor), vp, vp, vp, vp, vp,
                                  i32, i32, i32, i32, ctypes.c_float, vp]
        L.cm_attn_bwd_workspace_size.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
        L.cm_attn_bwd.argtypes = [ctypes.POINTER(cm_descriptor), vp, vp, vp, vp, vp, vp, vp, vp,
                                  vp, vp, sz, i32, i32, i32, i32, ctypes.c_float, vp]
        L.cm_attn_bwd_prologue.argtypes = [vp, vp, vp, vp, sz, i32, i32, i32, i32, vp]
        L.cm_attn_bwd_dkdv.argtypes = [ctypes.POINTER(cm_descriptor), vp, vp, vp, vp, vp, vp, vp,
                                       sz, i32, i32, i32, i32, ctypes.c_float, vp]
        L.cm_attn_bwd_dq.argtypes = [ctypes.POINTER(cm_descriptor), vp, vp, vp, vp, vp, vp, vp,
                                     vp, sz, i32, i32, i32, i32, ctypes.c_float, vp]
        L.cm_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
        L.cm_attn_bwd_noalloc.argtypes = [ctypes.POINTER(cm_descriptor), vp, vp, vp, vp, vp, vp,
                                          vp, vp, vp, i32, i32, i32, i32, ctypes.c_float, vp]
        L.cm_get_status.argtypes = [ctypes.POINTER(cm_descriptor), vp]
        cache_p, seqs_p = ctypes.POINTER(cm_kv_cache), ctypes.POINTER(cm_kv_seqs)
        i64_p, size_p = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(sz)
        L.cm_kv_append.argtypes = [cache_p, seqs_p, ctypes.POINTER(cm_kv_new), vp]
        L.cm_attn_decode_workspace_size.argtypes = [i32, i32, i32, i32, size_p]
        L.cm_attn_decode.argtypes = [cache_p, seqs_p, ctypes.POINTER(cm_descriptor), vp, vp, i32,
                                     vp, i64_p, vp, i64_p, vp, i32, ctypes.c_float, vp, sz, vp]
        L.cm_attn_decode_window.argtypes = [cache_p, seqs_p, i32, i32, vp, i64_p, vp, i64_p, vp, i32,
                                            ctypes.c_float, vp, sz, vp]
        L.cm_select_pages_workspace_size.argtypes = [i32, i32, i32, size_p]
        L.cm_select_pages.argtypes = [cache_p, seqs_p, vp, i64_p, i32, i32, i32, vp, vp, i32,
                                      vp, sz, vp]
        L.cm_kv_status.argtypes = [cache_p, vp]
        pages_p = ctypes.POINTER(cm_kv_pages)
        L.cm_kv_reserve.argtypes = [pages_p, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp]
        L.cm_kv_release.argtypes = [pages_p, vp, vp, vp, vp, vp]
        L.cm_kv_pages_status.argtypes = [pages_p, vp]
        L.cm_error_string.argtypes = [i32]
        L.cm_error_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def cm_error_string(code: int) -> str:
    try:
        return lib().cm_error_string(code).decode()
    except RuntimeError:
        return f"error {code}"


def _check(rc: int, what: str, detail: str = "") -> None:
    if rc != CM_OK:
        raise CMError(rc, what, detail)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ------------------------------------------------------------------------------------------------
# compiler
# ------------------------------------------------------------------------------------------------
class Spec:
    """Owns a compiled MaskSpec (host memory inside the library)."""

    def __init__(self, handle: int, text: str):
        self.handle = ctypes.c_void_p(handle)
        self.text = text

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None and self.handle.value:
            _lib.cm_spec_free(self.handle)
            self.handle = ctypes.c_void_p(0)


def cm_compile_spec(text: str) -> Spec:
    out = ctypes.c_void_p()
    err = ctypes.create_string_buffer(512)
    rc = lib().cm_compile_spec(text.encode(), ctypes.byref(out), err, 512)
    _check(rc, "cm_compile_spec", err.value.decode())
    return Spec(out.value, text)


def cm_spec_num_intervals(spec: Spec) -> int:
    n = ctypes.c_int()
    _check(lib().cm_spec_num_intervals(spec.handle, ctypes.byref(n)), "cm_spec_num_intervals")
    return n.value


def cm_spec_describe(spec: Spec) -> str:
    need = ctypes.c_size_t()
    _check(lib().cm_spec_describe(spec.handle, None, 0, ctypes.byref(need)), "cm_spec_describe")
    buf = ctypes.create_string_buffer(need.value)
    _check(lib().cm_spec_describe(spec.handle, buf, need.value, None), "cm_spec_describe")
    return buf.value.decode()


def cm_spec_kernel_source(spec: Spec) -> str:
    """CUDA C++ source of the spec's mask-specific preprocess kernel."""
    need = ctypes.c_size_t()
    _check(lib().cm_spec_kernel_source(spec.handle, None, 0, ctypes.byref(need)),
           "cm_spec_kernel_source")
    buf = ctypes.create_string_buffer(need.value)
    _check(lib().cm_spec_kernel_source(spec.handle, buf, need.value, None), "cm_spec_kernel_source")
    return buf.value.decode()


def cm_descriptor_kernel_source(fwd: Spec, bwd: Spec) -> str:
    """CUDA C++ source of the mask-specific preprocess kernel of a (forward, backward) pair."""
    need = ctypes.c_size_t()
    _check(lib().cm_descriptor_kernel_source(fwd.handle, bwd.handle, None, 0, ctypes.byref(need)),
           "cm_descriptor_kernel_source")
    buf = ctypes.create_string_buffer(need.value)
    _check(lib().cm_descriptor_kernel_source(fwd.handle, bwd.handle, buf, need.value, None),
           "cm_descriptor_kernel_source")
    return buf.value.decode()


def cm_descriptor_kernel_status(fwd: Spec, bwd: Spec, load: bool = True) -> tuple[int, str]:
    """(code, log) of the pair's generated kernel: compiled (load=False, host only) or compiled
    and loaded on the current GPU (load=True), as cm_build_descriptor does on first use."""
    buf = ctypes.create_string_buffer(1 << 16)
    rc = lib().cm_descriptor_kernel_status(fwd.handle, bwd.handle, 1 if load else 0, buf, len(buf))
    return rc, buf.value.decode(errors="replace")


def cm_spec_kernel_status(spec: Spec, load: bool = True) -> tuple[int, str]:
    """(code, log): CM_OK when the spec's generated preprocess kernel compiles (load=False, host
    only) or compiles and loads on the current GPU (load=True); otherwise the code and the reason."""
    buf = ctypes.create_string_buffer(1 << 16)
    rc = lib().cm_spec_kernel_status(spec.handle, 1 if load else 0, buf, len(buf))
    return rc, buf.value.decode(errors="replace")


CM_PREPROCESS_GENERATED = 0
CM_PREPROCESS_GENERIC = 1


def cm_set_preprocess_mode(mode: int) -> None:
    """Process-wide choice of descriptor kernels: generated per spec (default) or generic."""
    _check(lib().cm_set_preprocess_mode(mode), "cm_set_preprocess_mode")


CM_CHECK_UNSIGNED = 0
CM_CHECK_TWO_COMPARE = 1
CM_CHECK_RANGE_MASK = 3

CM_FORM_VISIBLE = 0
CM_FORM_MASKED = 1


def cm_set_interval_check(mode: int) -> None:
    """Process-wide form of the attention kernels' partial-tile check: per-row range masks
    (default), or per score the unsigned test or two comparisons (the paper's section 4.4
    forms)."""
    _check(lib().cm_set_interval_check(mode), "cm_set_interval_check")


def cm_descriptor_sizes(fwd: Spec, bwd: Spec, B: int, S: int, tile: int = TILE,
                        form: int = CM_FORM_VISIBLE) -> list[int]:
    sizes = (ctypes.c_size_t * 7)()
    _check(lib().cm_descriptor_sizes(fwd.handle, bwd.handle, B, S, tile, form, sizes),
           "cm_descriptor_sizes")
    return list(sizes)


# ------------------------------------------------------------------------------------------------
# descriptor
# ------------------------------------------------------------------------------------------------
class Descriptor:
    """Device buffers of an Execution Descriptor, allocated with torch on ``device``.  ``form``:
    CM_FORM_VISIBLE (visible intervals per row) or CM_FORM_MASKED (the masked runs)."""

    def __init__(self, fwd: Spec, bwd: Spec, B: int, S: int, device="cuda",
                 form: int = CM_FORM_VISIBLE):
        sizes = cm_descriptor_sizes(fwd, bwd, B, S, form=form)
        self.fwd, self.bwd, self.B, self.S, self.form = fwd, bwd, B, S, form
        self.ni_f = cm_spec_num_intervals(fwd) + form
        self.ni_b = cm_spec_num_intervals(bwd) + form
        self.NT = S // TILE
        self.W = (self.NT + 15) // 16
        self.itab_f = torch.empty(sizes[0] // 4, dtype=torch.int32, device=device)
        self.bm_f = torch.empty(sizes[1] // 4, dtype=torch.int32, device=device)
        self.itab_b = torch.empty(sizes[2] // 4, dtype=torch.int32, device=device)
        self.bm_b = torch.empty(sizes[3] // 4, dtype=torch.int32, device=device)
        self.sched_f = torch.empty(sizes[4] // 4, dtype=torch.int32, device=device)
        self.sched_b = torch.empty(sizes[5] // 4, dtype=torch.int32, device=device)
        self.status = torch.zeros((sizes[6] + 3) // 4, dtype=torch.int32, device=device)
        self.c = cm_descriptor(B, S, TILE, self.ni_f, self.ni_b, form,
                               self.itab_f.data_ptr(), self.bm_f.data_ptr(),
                               self.itab_b.data_ptr(), self.bm_b.data_ptr(),
                               self.sched_f.data_ptr(), self.sched_b.data_ptr(),
                               self.status.data_ptr())

    def nbytes(self) -> int:
        return sum(t.numel() * 4 for t in (self.itab_f, self.bm_f, self.itab_b, self.bm_b,
                                           self.sched_f, self.sched_b, self.status))

    # host views for checking
    def interval_table_fwd(self):
        return self.itab_f.view(self.B, self.ni_f, self.S, 2).cpu().numpy()

    def interval_table_bwd(self):
        return self.itab_b.view(self.B, self.ni_b, self.S, 2).cpu().numpy()

    def bitmap_fwd(self):
        return self.bm_f.view(self.B, self.NT, self.W).cpu().numpy().view("uint32")

    def bitmap_bwd(self):
        return self.bm_b.view(self.B, self.NT, self.W).cpu().numpy().view("uint32")


def cm_build_descriptor(fwd: Spec, bwd: Spec, seg: torch.Tensor, nseg: torch.Tensor,
                        desc: Descriptor, stream=None) -> None:
    """seg: device int32 [B, nseg_max + 1]; nseg: device int32 [B]."""
    for t in (seg, nseg):
        if not (t.is_cuda and t.dtype == torch.int32 and t.is_contiguous()):
            raise ValueError("metadata must be contiguous int32 CUDA tensors")
    meta = cm_meta(seg.data_ptr(), nseg.data_ptr(), seg.shape[1] - 1)
    _check(lib().cm_build_descriptor(fwd.handle, bwd.handle, ctypes.byref(meta), desc.B, desc.S,
                                     ctypes.byref(desc.c), _stream(stream)),
           "cm_build_descriptor")


def cm_get_status(desc: Descriptor, stream=None) -> int:
    return lib().cm_get_status(ctypes.byref(desc.c), _stream(stream))


# ------------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------------
def _bhsd(t: torch.Tensor, name: str):
    if not (t.is_cuda and t.dtype == torch.bfloat16 and t.dim() == 4 and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor [B, H, S, d]")
    return t.shape


def cm_attn_fwd(desc: Descriptor, q, k, v, o, lse, scale: float | None = None,
                stream=None) -> None:
    B, H, S, d = _bhsd(q, "q")
    for t, n in ((k, "k"), (v, "v"), (o, "o")):
        if _bhsd(t, n) != (B, H, S, d):
            raise ValueError(f"{n} shape mismatch")
    if not (lse.is_cuda and lse.dtype == torch.float32 and lse.shape == (B, H, S)):
        raise ValueError("lse must be fp32 CUDA [B, H, S]")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    _check(lib().cm_attn_fwd(ctypes.byref(desc.c), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                             o.data_ptr(), lse.data_ptr(), B, H, S, d, scale, _stream(stream)),
           "cm_attn_fwd")


def cm_attn_bwd_workspace_size(B: int, H: int, S: int, d: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().cm_attn_bwd_workspace_size(B, H, S, d, ctypes.byref(n)),
           "cm_attn_bwd_workspace_size")
    return n.value


def cm_attn_bwd(desc: Descriptor, q, k, v, o, lse, d_o, dq, dk, dv, workspace: torch.Tensor,
                scale: float | None = None, stream=None) -> None:
    B, H, S, d = _bhsd(q, "q")
    for t, n in ((k, "k"), (v, "v"), (o, "o"), (d_o, "dO"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        if _bhsd(t, n) != (B, H, S, d):
            raise ValueError(f"{n} shape mismatch")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().cm_attn_bwd(ctypes.byref(desc.c), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                             o.data_ptr(), lse.data_ptr(), d_o.data_ptr(), dq.data_ptr(),
                             dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), nbytes,
                             B, H, S, d, scale, _stream(stream)),
           "cm_attn_bwd")


def _bwd_shapes(q, others):
    B, H, S, d = _bhsd(q, "q")
    for t, n in others:
        if _bhsd(t, n) != (B, H, S, d):
            raise ValueError(f"{n} shape mismatch")
    return B, H, S, d


def cm_attn_bwd_prologue(o, lse, d_o, workspace: torch.Tensor, stream=None) -> None:
    """Per-row -D and -LSE * log2(e) of every row into the workspace, for callers that run
    cm_attn_bwd_dkdv without cm_attn_bwd_dq (cm_attn_bwd itself does not use it)."""
    B, H, S, d = _bwd_shapes(o, ((d_o, "dO"),))
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().cm_attn_bwd_prologue(o.data_ptr(), lse.data_ptr(), d_o.data_ptr(),
                                      workspace.data_ptr(), nbytes, B, H, S, d, _stream(stream)),
           "cm_attn_bwd_prologue")


def cm_attn_bwd_dkdv(desc: Descriptor, q, k, v, d_o, dk, dv, workspace: torch.Tensor,
                     scale: float | None = None, stream=None) -> None:
    """Second stage of cm_attn_bwd: dK and dV along key tiles (backward descriptor); reads the
    per-row constants that cm_attn_bwd_dq (or cm_attn_bwd_prologue) wrote into the workspace."""
    B, H, S, d = _bwd_shapes(q, ((k, "k"), (v, "v"), (d_o, "dO"), (dk, "dk"), (dv, "dv")))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().cm_attn_bwd_dkdv(ctypes.byref(desc.c), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                  d_o.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                  workspace.data_ptr(), nbytes, B, H, S, d, scale, _stream(stream)),
           "cm_attn_bwd_dkdv")


def cm_attn_bwd_dq(desc: Descriptor, q, k, v, o, lse, d_o, dq, workspace: torch.Tensor,
                   scale: float | None = None, stream=None) -> None:
    """First stage of cm_attn_bwd: dQ along query tiles (forward descriptor); also writes the
    workspace's per-row constants (-D and -LSE*log2e) that cm_attn_bwd_dkdv reads."""
    B, H, S, d = _bwd_shapes(q, ((k, "k"), (v, "v"), (o, "O"), (d_o, "dO"), (dq, "dq")))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().cm_attn_bwd_dq(ctypes.byref(desc.c), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                o.data_ptr(), lse.data_ptr(), d_o.data_ptr(), dq.data_ptr(),
                                workspace.data_ptr(), nbytes, B, H, S, d, scale, _stream(stream)),
           "cm_attn_bwd_dq")


def cm_set_wait_limit_ns(ns: int) -> None:
    """Process-wide limit of the attention kernels' bounded waits (0 = the 2 s default).  A
    diagnostic hook: a tiny limit makes ordinary waits expire and exercises the time-out path."""
    _check(lib().cm_set_wait_limit_ns(int(ns)), "cm_set_wait_limit_ns")


def cm_attn_bwd_noalloc(desc: Descriptor, q, k, v, o, lse, d_o, dq, dk, dv,
                        scale: float | None = None, stream=None) -> None:
    """cm_attn_bwd without a workspace, for callers that cannot allocate device memory.

    The library's fixed scratch array (CM_NOALLOC_SCRATCH_BYTES per GPU) stands in for the
    workspace; see include/cm.h for its limit and for the rule that overlapping calls race."""
    B, H, S, d = _bhsd(q, "q")
    for t, n in ((k, "k"), (v, "v"), (o, "o"), (d_o, "dO"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        if _bhsd(t, n) != (B, H, S, d):
            raise ValueError(f"{n} shape mismatch")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    _check(lib().cm_attn_bwd_noalloc(ctypes.byref(desc.c), q.data_ptr(), k.data_ptr(),
                                     v.data_ptr(), o.data_ptr(), lse.data_ptr(), d_o.data_ptr(),
                                     dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, S, d,
                                     scale, _stream(stream)),
           "cm_attn_bwd_noalloc")


NOALLOC_SCRATCH_BYTES = 32 << 20


# ------------------------------------------------------------------------------------------------
# convenience: one call for each pass, allocating outputs with torch
# ------------------------------------------------------------------------------------------------
def attention_forward(desc: Descriptor, q, k, v, scale=None, stream=None):
    B, H, S, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty(B, H, S, dtype=torch.float32, device=q.device)
    cm_attn_fwd(desc, q, k, v, o, lse, scale, stream)
    return o, lse


def attention_backward(desc: Descriptor, q, k, v, o, lse, d_o, scale=None, stream=None,
                       workspace=None):
    B, H, S, d = q.shape
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = torch.empty(cm_attn_bwd_workspace_size(B, H, S, d), dtype=torch.uint8,
                                device=q.device)
    cm_attn_bwd(desc, q, k, v, o, lse, d_o, dq, dk, dv, workspace, scale, stream)
    return dq, dk, dv


# ------------------------------------------------------------------------------------------------
# serving: a paged key-value cache
# ------------------------------------------------------------------------------------------------
CM_KV_BF16 = 0
CM_KV_E4M3 = 1
CM_KV_E4M3_BLOCK = 2
CM_KV_INT8_BLOCK = 3
KV_BLOCK = 16  # tokens that share a scale in a block type


def _pool(t: torch.Tensor, name: str):
    if not (t.is_cuda and t.dim() == 4 and t.dtype in (torch.bfloat16, torch.float8_e4m3fn, torch.int8)):
        raise ValueError(f"{name} must be a bf16, float8_e4m3fn or int8 CUDA tensor "
                         "[num_pages, H_kv, page_size, d]")
    n, H, P, d = t.shape
    if t[:1].is_contiguous() and (n == 1 or t.stride(0) >= H * P * d):
        return t.shape, (t.stride(0) if n > 1 else H * P * d)
    raise ValueError(f"{name}: every page must be contiguous, and pages must not overlap")


class KVCache:
    """A paged key-value cache over the caller's tensors (cm_kv_cache): k, v
    [num_pages, H_kv, page_size, d], bf16, float8_e4m3fn or int8; the 8-bit types take k_scale and v_scale,
    fp32 [num_pages, H_kv, page_size / 16] (a power of two for each block of 16 tokens and head, which
    cm_kv_append chooses), or for e4m3 fp32 [H_kv] (fixed by the caller).  Pages may lie apart (a view such as kv[:, 0] of a [num_pages, 2, H_kv, page_size, d]
    tensor).  summary (int8 [num_pages, H_kv, 2, d]) with summary_scale (fp32 [num_pages, H_kv])
    holds the page summaries that cm_select_pages reads."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale=None, v_scale=None, summary=None,
                 summary_scale=None):
        shape, k_stride = _pool(k, "k")
        v_shape, v_stride = _pool(v, "v")
        if v_shape != shape or v.dtype != k.dtype or v.device != k.device:
            raise ValueError("v must have the shape, type and device of k")
        n, H, P, d = shape
        self.device, self.index = k.device, k.get_device()
        bits8 = k.dtype != torch.bfloat16
        blocks = k.dtype == torch.int8 or (bits8 and k_scale is not None and k_scale.dim() == 3)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if (t is not None) != bits8:
                raise ValueError("an 8-bit cache takes k_scale and v_scale, a bf16 cache neither")
            if bits8:
                _kv_tensor(t, name, torch.float32, (n, H, P // KV_BLOCK) if blocks else (H,), self.index)
        dtype = (CM_KV_BF16 if not bits8 else CM_KV_E4M3 if not blocks
                 else CM_KV_INT8_BLOCK if k.dtype == torch.int8 else CM_KV_E4M3_BLOCK)
        if (summary is None) != (summary_scale is None):
            raise ValueError("summary and summary_scale come together")
        if summary is not None:
            _kv_tensor(summary, "summary", torch.int8, (n, H, 2, d), self.index)
            _kv_tensor(summary_scale, "summary_scale", torch.float32, (n, H), self.index)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.summary, self.summary_scale = summary, summary_scale
        self.num_pages, self.H_kv, self.page_size, self.d = n, H, P, d
        self.scale = 1.0 / math.sqrt(d)  # of scores, where a call names none
        self.status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self.c = cm_kv_cache(n, P, H, d, dtype, k_stride, v_stride,
                             k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale),
                             _ptr(summary), _ptr(summary_scale), self.status.data_ptr())
        self._address = ctypes.addressof(self.c)

    @classmethod
    def alloc(cls, num_pages: int, H_kv: int, page_size: int, d: int, dtype=torch.bfloat16,
              device="cuda", k_scale=None, v_scale=None, summaries: bool = False,
              block_scales: bool = False) -> "KVCache":
        """A cache in new memory (not initialised: what no token was written to is never used).  int8, and e4m3 with
        block_scales, come with scales of their own."""
        k, v = (torch.empty(num_pages, H_kv, page_size, d, dtype=dtype, device=device)
                for _ in range(2))
        if block_scales or dtype == torch.int8:
            if k_scale is not None or v_scale is not None:
                raise ValueError("block scales are the cache's own")
            k_scale, v_scale = (torch.empty(num_pages, H_kv, page_size // KV_BLOCK, device=device) for _ in range(2))
        more = {}
        if summaries:
            more = {"summary": torch.empty(num_pages, H_kv, 2, d, dtype=torch.int8, device=device),
                    "summary_scale": torch.empty(num_pages, H_kv, device=device)}
        return cls(k, v, k_scale, v_scale, **more)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _kv_tensor(t, name, dtype, shape, device: int):
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{device}")


# These calls are a few microseconds of GPU work each, so they are written to be quick: one device number
# instead of device objects, shapes and strides read once, structs packed in one go, and function
# objects of their own that take them as bytes.
_I32 = torch.int32
_SEQS = struct.Struct("2i2P")      # cm_kv_seqs, field by field
_NEW = struct.Struct("5P15q2P6i3P")  # cm_kv_new
_TWO = struct.Struct("2q")
assert _SEQS.size == ctypes.sizeof(cm_kv_seqs) and _NEW.size == ctypes.sizeof(cm_kv_new)
_calls = None


def _serving():
    """(cm_kv_append, cm_attn_decode, cm_select_pages, cm_attn_decode_window, cm_kv_reserve, cm_kv_release)
    with every pointer as an address or bytes."""
    global _calls
    if _calls is None:
        L, vp, i32, sz = lib(), ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t

        def call(name, *args):
            return ctypes.CFUNCTYPE(i32, *args)((name, L))

        _calls = (call("cm_kv_append", vp, vp, vp, vp),
                  call("cm_attn_decode", vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, i32,
                       ctypes.c_float, vp, sz, vp),
                  call("cm_select_pages", vp, vp, vp, vp, i32, i32, i32, vp, vp, i32, vp, sz, vp),
                  call("cm_attn_decode_window", vp, vp, i32, i32, vp, vp, vp, vp, vp, i32,
                       ctypes.c_float, vp, sz, vp),
                  call("cm_kv_reserve", vp, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp),
                  call("cm_kv_release", vp, vp, vp, vp, vp, vp))
    return _calls


def _kv_stream(cache, stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(cache.index)
    return _stream(stream)


def _on_current_device(cache):
    if cache.index != torch._C._cuda_getDevice():
        what = "pool" if isinstance(cache, KVPages) else "cache"
        raise ValueError(f"the {what} is on {cache.device}, which is not the current device")


def _kv_seqs(cache: KVCache, page_table, lens):
    """B and the packed cm_kv_seqs."""
    dev, shape = cache.index, page_table.shape
    _on_current_device(cache)
    if not (len(shape) == 2 and page_table.dtype is _I32 and page_table.get_device() == dev
            and page_table.is_contiguous()):
        raise ValueError("page_table must be a contiguous int32 tensor [B, max_pages] on "
                         f"{cache.device}")
    B, n = shape
    if not (lens.dtype is _I32 and lens.shape == (B,) and lens.get_device() == dev
            and lens.is_contiguous()):
        raise ValueError(f"lens must be a contiguous int32 tensor [{B}] on {cache.device}")
    return B, _SEQS.pack(B, n, page_table.data_ptr(), lens.data_ptr())


def _tokens(t, name, cache: KVCache, packed: bool):
    """Shape and strides {sequence, head, token} of new tokens: packed [n, H, d] or padded
    [B, H, T, d].  The stride of an axis with one entry is 0: any will do."""
    shape, s = t.shape, t.stride()
    if not (t.dtype is torch.bfloat16 and t.get_device() == cache.index
            and len(s) == (3 if packed else 4) and shape[-1] == cache.d and s[-1] == 1):
        raise ValueError(f"{name} must be a bf16 tensor " +
                         ("[n, H, d]" if packed else "[B, H, T, d]") +
                         f" on {cache.device} with d = {cache.d} contiguous")
    if 1 in shape:
        s = [x if n > 1 else 0 for n, x in zip(shape, s)]
    return shape, (0, s[1], s[0]) if packed else s[:3]


_NONE3 = (0, 0, 0)


def _addr(t):
    return 0 if t is None else t.data_ptr()


def cm_kv_append(cache: KVCache, page_table, lens, k, v, q=None, q_out=None, k_out=None, rope=None,
                 interleaved: bool = False, cu_new=None, n_new=None, max_new: int | None = None,
                 new_lens=None, stream=None, granted=None) -> None:
    """Store the new tokens' keys and values behind the lens[b] tokens that each sequence holds,
    rotating keys (and queries, into q_out) to their positions.  With cu_new (int32 [B + 1]) the
    tokens are packed, k, v [n, H_kv, d] and q [n, H_q, d]; without it they are padded, [B, H, T, d],
    and n_new (int32 [B]) says how many of T each sequence has (all of them where it is not given).
    max_new: the most tokens of any sequence (default: as many as the tensors hold).  rope: fp32
    [positions, rot_dim / 2, 2] of cosines and sines.  new_lens (int32 [B]) receives the new
    lengths.  granted (int32 [B], packed tokens): of each sequence's tokens only the first so many, as reserve_pages
    says; padded tokens take it as n_new."""
    B, seqs = _kv_seqs(cache, page_table, lens)
    dev, packed = cache.index, cu_new is not None
    shape, ks = _tokens(k, "k", cache, packed)
    v_shape, vs = _tokens(v, "v", cache, packed)
    if shape[1] != cache.H_kv or v_shape != shape or not (packed or shape[0] == B):
        raise ValueError("k and v must have the cache's heads, one shape and one row a sequence")
    n = shape[0] if packed else shape[2]
    qs = qos = kos = _NONE3
    H_q = rope_len = rot_dim = 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    if q is not None:
        q_shape, qs = _tokens(q, "q", cache, packed)
        o_shape, qos = _tokens(q_out, "q_out", cache, packed)
        H_q = q_shape[1]
        if q_shape != o_shape or q_shape[0] != shape[0] or q_shape[2:] != shape[2:]:
            raise ValueError("q and q_out must have one shape, with the tokens of k")
    if k_out is not None:
        o_shape, kos = _tokens(k_out, "k_out", cache, packed)
        if o_shape != shape:
            raise ValueError("k_out must have the shape of k")
    if packed:
        if n_new is not None:
            raise ValueError("n_new is for padded tokens, cu_new for packed ones")
        _kv_tensor(cu_new, "cu_new", torch.int32, (B + 1,), dev)
    elif n_new is not None:
        _kv_tensor(n_new, "n_new", torch.int32, (B,), dev)
    if granted is not None:
        if not packed:
            raise ValueError("granted is for packed tokens; padded ones take it as n_new")
        _kv_tensor(granted, "granted", torch.int32, (B,), dev)
    if rope is not None:
        rope_len, half, two = rope.shape
        if two != 2:
            raise ValueError("rope must be [positions, rot_dim / 2, 2]")
        _kv_tensor(rope, "rope", torch.float32, (rope_len, half, 2), dev)
        rot_dim = 2 * half
    if new_lens is not None:
        _kv_tensor(new_lens, "new_lens", torch.int32, (B,), dev)
    tok = _NEW.pack(
        k.data_ptr(), v.data_ptr(), _addr(q), _addr(q_out), _addr(k_out), *ks, *vs, *qs, *qos, *kos,
        _addr(cu_new), _addr(n_new), n, n if max_new is None else max_new, H_q, rot_dim,
        interleaved, rope_len, _addr(rope), _addr(new_lens), _addr(granted))
    rc = _serving()[0](cache._address, seqs, tok, _kv_stream(cache, stream))
    if rc != CM_OK:
        raise CMError(rc, "cm_kv_append")


def cm_attn_decode_workspace_size(B: int, H_q: int, H_kv: int, d: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().cm_attn_decode_workspace_size(B, H_q, H_kv, d, ctypes.byref(n)),
           "cm_attn_decode_workspace_size")
    return n.value


def _one_token(t, name, cache: KVCache, B: int):
    shape, s = t.shape, t.stride()
    if not (t.dtype is torch.bfloat16 and len(s) == 3 and t.get_device() == cache.index
            and shape[0] == B and shape[2] == cache.d and s[2] == 1):
        raise ValueError(f"{name} must be a bf16 tensor [B, H_q, d] on {cache.device} with d = "
                         f"{cache.d} contiguous")
    return _TWO.pack(s[0] if B > 1 else 0, s[1] if shape[1] > 1 else 0)


def _workspace(w, cache: KVCache):
    if not (w.get_device() == cache.index and w.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {cache.device}")


def cm_attn_decode(cache: KVCache, page_table, lens, q, o, lse, workspace: torch.Tensor,
                   desc: Descriptor | None = None, sel=None, nsel=None,
                   scale: float | None = None, stream=None, window: int | None = None,
                   sinks: int = 0) -> None:
    """Attention of the last of each sequence's lens[b] tokens over the cache: q, o bf16
    [B, H_q, d]; lse fp32 [B, H_q] or None.  desc: the mask, whose row lens[b] - 1 the token sees by;
    or sel (int32 [B, H_kv, n]) with nsel (int32 [B, H_kv]): the pages to attend to; or window, with
    sinks: the token sees the last `window` tokens, itself among them, and the first `sinks`
    (cm_attn_decode_window)."""
    B, seqs = _kv_seqs(cache, page_table, lens)
    dev, H = cache.index, q.shape[1]
    qs, os = _one_token(q, "q", cache, B), _one_token(o, "o", cache, B)
    if o.shape[1] != H:
        raise ValueError("o shape mismatch")
    if lse is not None:
        _kv_tensor(lse, "lse", torch.float32, (B, H), dev)
    sel_max = 0
    if (sel is None) != (nsel is None):
        raise ValueError("sel and nsel come together")
    if sel is not None:
        sel_max = sel.shape[-1]
        _kv_tensor(sel, "sel", torch.int32, (B, cache.H_kv, sel_max), dev)
        _kv_tensor(nsel, "nsel", torch.int32, (B, cache.H_kv), dev)
    _workspace(workspace, cache)
    if desc is not None and desc.itab_f.get_device() != dev:
        raise ValueError(f"desc must be on {cache.device}")
    scale = cache.scale if scale is None else scale
    if window is not None:
        if desc is not None or sel is not None:
            raise ValueError("a window comes without desc and without sel")
        if not (-1 << 31 <= window < 1 << 31 and -1 << 31 <= sinks < 1 << 31):  # ctypes would take them modulo 2^32
            raise ValueError("window and sinks must be at least 0 and below 2^31")
        rc = _serving()[3](cache._address, seqs, window, sinks, q.data_ptr(), qs, o.data_ptr(), os,
                           _ptr(lse), H, scale, workspace.data_ptr(), workspace.nbytes,
                           _kv_stream(cache, stream))
        if rc != CM_OK:
            raise CMError(rc, "cm_attn_decode_window")
        return
    if sinks:
        raise ValueError("sinks come with a window")
    rc = _serving()[1](cache._address, seqs, None if desc is None else ctypes.addressof(desc.c),
                       _ptr(sel), _ptr(nsel), sel_max, q.data_ptr(), qs, o.data_ptr(), os,
                       _ptr(lse), H, scale, workspace.data_ptr(), workspace.nbytes,
                       _kv_stream(cache, stream))
    if rc != CM_OK:
        raise CMError(rc, "cm_attn_decode")


def cm_select_pages_workspace_size(B: int, H_kv: int, max_pages: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().cm_select_pages_workspace_size(B, H_kv, max_pages, ctypes.byref(n)),
           "cm_select_pages_workspace_size")
    return n.value


def cm_select_pages(cache: KVCache, page_table, lens, q, sel, nsel, workspace: torch.Tensor,
                    keep_first: int = 0, keep_last: int = 0, stream=None) -> None:
    """The sel.shape[2] pages of each sequence and key-value head whose summaries promise the largest
    scores for the new token's queries q (bf16 [B, H_q, d]), the first keep_first and last keep_last
    pages always among them: sel int32 [B, H_kv, n] in ascending order, -1 behind the last, and
    their number nsel int32 [B, H_kv]."""
    B, seqs = _kv_seqs(cache, page_table, lens)
    if cache.summary is None:
        raise ValueError("the cache has no page summaries")
    if not (sel.dim() == 3 and sel.shape[2] > 0):
        raise ValueError("sel must be [B, H_kv, n]")
    _kv_tensor(sel, "sel", torch.int32, (B, cache.H_kv, sel.shape[2]), cache.index)
    _kv_tensor(nsel, "nsel", torch.int32, (B, cache.H_kv), cache.index)
    _workspace(workspace, cache)
    qs = _one_token(q, "q", cache, B)
    rc = _serving()[2](cache._address, seqs, q.data_ptr(), qs, q.shape[1], keep_first, keep_last,
                       sel.data_ptr(), nsel.data_ptr(), sel.shape[2], workspace.data_ptr(),
                       workspace.nbytes, _kv_stream(cache, stream))
    if rc != CM_OK:
        raise CMError(rc, "cm_select_pages")


def cm_kv_status(cache: KVCache, stream=None) -> int:
    """The first device error since the last call (CM_OK where there was none); zeroes it."""
    _on_current_device(cache)  # another device's stream would not wait for the work that is asked about
    return lib().cm_kv_status(ctypes.byref(cache.c), _kv_stream(cache, stream))


class KVPages:
    """The pages of a pool and their tables (cm_kv_pages) over the caller's tensors: page_table int32
    [B, max_pages], free_pages int32 [num_pages].  window (None or 0: none) and sinks as in cm_attn_decode; the attributes
    are what that takes, None and 0 where the pool has no window.  state and
    spare, int32 [B + 1, 2], are what reserve_pages and release_pages go on from and write to; alloc makes
    them, the low-level calls take their own."""

    def __init__(self, page_table: torch.Tensor, free_pages: torch.Tensor, page_size: int,
                 window: int | None = None, sinks: int = 0, state=None):
        if not (page_table.is_cuda and page_table.dim() == 2 and free_pages.dim() == 1):
            raise ValueError("page_table must be a CUDA tensor [B, max_pages], free_pages [num_pages]")
        self.device, self.index = page_table.device, page_table.get_device()
        self.B, self.max_pages = page_table.shape
        _kv_tensor(page_table, "page_table", _I32, page_table.shape, self.index)
        _kv_tensor(free_pages, "free_pages", _I32, free_pages.shape, self.index)
        window = 0 if window is None else window
        if not (0 <= window < 1 << 31 and 0 <= sinks < 1 << 31):
            raise ValueError("window and sinks must be at least 0 and below 2^31")
        self.page_table, self.free_pages = page_table, free_pages
        self.page_size, self.window, self.sinks = page_size, window or None, sinks if window else 0
        self.num_pages = free_pages.shape[0]
        if not all(0 <= x < 1 << 31 for x in (self.num_pages, page_size, self.B, self.max_pages)):
            raise ValueError("pages, page_size and sequences must be below 2^31")
        self.state = self.spare = None
        if state is not None:
            _kv_tensor(state, "state", _I32, (self.B + 1, 2), self.index)
            self.state, self.spare = state, torch.empty_like(state)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._rows, self._state_shape = torch.Size((self.B,)), torch.Size((self.B + 1, 2))
        self.c = cm_kv_pages(self.num_pages, page_size, self.B, self.max_pages, window, sinks,
                             page_table.data_ptr(), free_pages.data_ptr(), self.status.data_ptr())
        self._address = ctypes.addressof(self.c)

    @classmethod
    def alloc(cls, num_pages: int, B: int, max_pages: int, page_size: int, window: int | None = None,
              sinks: int = 0, device="cuda") -> "KVPages":
        """A pool whose pages are all free, and tables (-1 throughout) of B sequences that own none."""
        state = torch.zeros(B + 1, 2, dtype=torch.int32, device=device)
        state[B, 0] = num_pages
        return cls(torch.full((B, max_pages), -1, dtype=torch.int32, device=device),
                   torch.arange(num_pages, dtype=torch.int32, device=device), page_size, window, sinks, state)


def _pages_state(pages: KVPages, state, new_state, lens):
    dev, shape, rows = pages.index, pages._state_shape, pages._rows
    if (state.dtype is _I32 and new_state.dtype is _I32 and lens.dtype is _I32 and state.shape == shape
            and new_state.shape == shape and lens.shape == rows
            and dev == torch._C._cuda_getDevice() == state.get_device() == new_state.get_device() == lens.get_device()
            and state.is_contiguous() and new_state.is_contiguous() and lens.is_contiguous()):
        return
    _on_current_device(pages)  # one of these says what is wrong
    _kv_tensor(state, "state", _I32, shape, dev)
    _kv_tensor(new_state, "new_state", _I32, shape, dev)
    _kv_tensor(lens, "lens", _I32, rows, dev)


def cm_kv_reserve(pages: KVPages, state, new_state, lens, n_tokens: int, max_new: int | None = None,
                  cu_new=None, n_new=None, granted=None, slots=None, stream=None) -> None:
    """Pages out of the pool for the tokens that each sequence is about to append behind its lens[b]: packed ones
    (cu_new int32 [B + 1]; n_tokens of all sequences) or padded ones (n_new int32 [B] of n_tokens each, all of
    them where it is not given).  max_new: the most tokens of any sequence (default n_tokens).  granted
    (int32 [B]): the tokens that may be appended, all of a sequence's or 0; cm_kv_append takes it as granted beside cu_new,
    or as n_new for padded tokens.  slots (int64 [n_tokens], padded [B,
    n_tokens]): page * page_size + row of every token, -1 where none was granted.  state and new_state: int32
    [B + 1, 2]."""
    _pages_state(pages, state, new_state, lens)
    dev, B = pages.index, pages.B
    if cu_new is not None:
        _kv_tensor(cu_new, "cu_new", _I32, (B + 1,), dev)
    if n_new is not None:
        _kv_tensor(n_new, "n_new", _I32, pages._rows, dev)
    if granted is not None:
        _kv_tensor(granted, "granted", _I32, pages._rows, dev)
    if slots is not None:
        _kv_tensor(slots, "slots", torch.int64, (B, n_tokens) if cu_new is None else (n_tokens,), dev)
    if not (0 <= n_tokens < 1 << 31 and (max_new is None or 0 <= max_new < 1 << 31)):
        raise ValueError("n_tokens and max_new must be at least 0 and below 2^31")
    rc = _serving()[4](pages._address, state.data_ptr(), new_state.data_ptr(), lens.data_ptr(), _ptr(cu_new),
                       _ptr(n_new), n_tokens, n_tokens if max_new is None else max_new, _ptr(granted),
                       _ptr(slots) if n_tokens else None, _kv_stream(pages, stream))
    if rc != CM_OK:
        raise CMError(rc, "cm_kv_reserve")


def cm_kv_release(pages: KVPages, state, new_state, lens, done=None, stream=None) -> None:
    """Pages back into the pool: all of the sequences with done[b] != 0 (int32 [B]), and of the others those that
    lie behind the pool's window.  state and new_state: int32 [B + 1, 2]."""
    _pages_state(pages, state, new_state, lens)
    if done is not None:
        _kv_tensor(done, "done", _I32, pages._rows, pages.index)
    rc = _serving()[5](pages._address, state.data_ptr(), new_state.data_ptr(), lens.data_ptr(), _ptr(done),
                       _kv_stream(pages, stream))
    if rc != CM_OK:
        raise CMError(rc, "cm_kv_release")


def cm_kv_pages_status(pages: KVPages, stream=None) -> int:
    """The first device error since the last call (CM_OK where there was none); zeroes it."""
    _on_current_device(pages)
    return lib().cm_kv_pages_status(ctypes.byref(pages.c), _kv_stream(pages, stream))


def _for_stream(stream, make):
    """make()'s tensors for work on `stream`: new ones from its memory, where nothing that the current
    stream still does can write, and all kept from reuse until both streams have done with them."""
    if stream is None:
        return make()
    if not hasattr(stream, "cuda_stream"):  # ExternalStream(0) would be a new stream of torch's own
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        made = make()
    for t in made:
        t.record_stream(here)
        t.record_stream(stream)
    return made


def decode_attention(cache: KVCache, page_table, lens, q, desc=None, sel=None, nsel=None,
                     scale=None, stream=None, workspace=None, window=None, sinks=0):
    """cm_attn_decode into new tensors: (o, lse)."""
    B, H, d = q.shape

    def make():
        w = workspace
        if w is None:
            w = torch.empty(cm_attn_decode_workspace_size(B, H, cache.H_kv, d), dtype=torch.uint8,
                            device=q.device)
        return (torch.empty(B, H, d, dtype=q.dtype, device=q.device),
                torch.empty(B, H, dtype=torch.float32, device=q.device), w)

    o, lse, workspace = _for_stream(stream, make)
    cm_attn_decode(cache, page_table, lens, q, o, lse, workspace, desc, sel, nsel, scale, stream, window,
                   sinks)
    return o, lse


def select_pages(cache: KVCache, page_table, lens, q, n: int, keep_first: int = 0,
                 keep_last: int = 0, stream=None, workspace=None):
    """cm_select_pages of n pages into new tensors: (sel, nsel)."""
    B = q.shape[0]

    def make():
        w = workspace
        if w is None:
            w = torch.empty(cm_select_pages_workspace_size(B, cache.H_kv, page_table.shape[1]),
                            dtype=torch.uint8, device=q.device)
        return (torch.empty(B, cache.H_kv, n, dtype=torch.int32, device=q.device),
                torch.empty(B, cache.H_kv, dtype=torch.int32, device=q.device), w)

    sel, nsel, workspace = _for_stream(stream, make)
    cm_select_pages(cache, page_table, lens, q, sel, nsel, workspace, keep_first, keep_last, stream)
    return sel, nsel


def _turn(pages: KVPages) -> None:
    pages.state, pages.spare = pages.spare, pages.state


def reserve_pages(pages: KVPages, lens, n_tokens: int, max_new: int | None = None, cu_new=None, n_new=None,
                  slots: bool = False, stream=None):
    """cm_kv_reserve from the pool's own state, with results in new tensors: granted, or (granted, slots).  The state turns
    to the other of its two buffers; a captured graph should hold as many reserve_pages as release_pages, so
    that every replay goes on where the one before ended."""
    if pages.state is None:
        raise ValueError("the pool was made without a state")
    shape = (pages.B, n_tokens) if cu_new is None else (n_tokens,)

    def make():
        made = (torch.empty(pages.B, dtype=torch.int32, device=pages.device),)
        return made + ((torch.full(shape, -1, dtype=torch.int64, device=pages.device),) if slots else ())

    made = _for_stream(stream, make)
    cm_kv_reserve(pages, pages.state, pages.spare, lens, n_tokens, max_new, cu_new, n_new, made[0],
                  made[1] if slots else None, stream)
    _turn(pages)
    return made if slots else made[0]


def release_pages(pages: KVPages, lens, done=None, stream=None) -> None:
    """cm_kv_release from the pool's own state (see reserve_pages)."""
    if pages.state is None:
        raise ValueError("the pool was made without a state")
    cm_kv_release(pages, pages.state, pages.spare, lens, done, stream)
    _turn(pages)
