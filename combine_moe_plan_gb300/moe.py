"""ctypes binding of libmoe (include/moe.h).

Argument marshalling only: torch tensors supply device pointers and the
current stream; every step of the path runs in libmoe's CUDA kernels.  The
library must have been built (``__graft_entry__.build()`` or
``python -m combine_moe_plan_gb300.build``); if it is missing, loading raises
``LibraryMissing`` -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libmoe.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "moe.h")

MOE_OK, MOE_ERR_STATE = 0, -9
STATUS = {0: "MOE_OK", -1: "MOE_ERR_NULL", -2: "MOE_ERR_SIZE", -3: "MOE_ERR_ALIGN", -4: "MOE_ERR_BUF",
          -5: "MOE_ERR_WORKSPACE", -6: "MOE_ERR_CUDA", -7: "MOE_ERR_DEVICE", -8: "MOE_ERR_REPLICA",
          -9: "MOE_ERR_STATE"}
DEVERR_REPLICA, DEVERR_DUPLICATE, DEVERR_SLOT, DEVERR_WINDOW, DEVERR_STALL = 0x1, 0x2, 0x4, 0x8, 0x10
SCORES = {"softmax": 0, "sigmoid": 1}


class LibraryMissing(ImportError):
    pass


class MoeError(RuntimeError):
    def __init__(self, fn, rc, msg):
        super().__init__(f"{fn}: {STATUS.get(rc, rc)} ({msg})")
        self.rc = rc


class Desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T_max", "H", "E", "P", "k", "group", "n_sets")]


class View(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("codes", "scales", "ex_out", "topk_e", "phys", "gates", "slot",
                                              "src_token", "src_k", "counts", "offsets", "error_word")] + \
               [("rows", ctypes.c_int32), ("scale_stride", ctypes.c_int32)]


class Router(ctypes.Structure):
    """The scored router of ``Pool.plan_routed`` (moe_router in include/moe.h):
    ``score`` "sigmoid" or "softmax"; ``topk_group`` of ``n_group`` expert groups
    are kept by the sum of their ``group_top`` best choices; gates are
    renormalised over the k chosen scores if ``renorm`` and multiplied by
    ``scale``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("score", "n_group", "topk_group", "group_top", "renorm")] + \
               [("scale", ctypes.c_float)]

    def __init__(self, score="sigmoid", n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0):
        if score not in SCORES:
            raise ValueError(f"score must be one of {sorted(SCORES)}")
        super().__init__(SCORES[score], n_group, topk_group, group_top, int(bool(renorm)), scale)


class ExpertWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("P", "H", "I")] + \
               [(n, ctypes.c_void_p) for n in ("w13", "s13", "w2", "s2", "error_word")]


_lib = None
_lib_path = LIB_PATH


def use_library(path: str) -> None:
    """Choose which build of the library this process loads (e.g. the trace
    build, libmoe_trace.so).  Must be called before the first call into it."""
    global _lib_path
    if _lib is not None and path != _lib_path:
        raise RuntimeError(f"{_lib_path} is already loaded in this process")
    _lib_path = path


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_lib_path):
        raise LibraryMissing(f"{_lib_path} is not built; run combine_moe_plan_gb300.build.build()")
    L = ctypes.CDLL(_lib_path)
    vp, i32, pp = ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER
    sig = {
        "moe_pool_bytes": [pp(Desc), pp(ctypes.c_size_t)],
        "moe_pool_init": [pp(Desc), vp, ctypes.c_size_t, pp(vp)],
        "moe_pool_destroy": [vp],
        "moe_pool_view": [vp, ctypes.c_int, pp(View)],
        "moe_pool_clear_error": [vp, vp],
        "moe_pool_check": [vp, vp, pp(i32)],
        "moe_pool_launches": [vp, pp(ctypes.c_uint64)],
        "moe_replica_check": [vp, vp, i32, i32],
        "moe_plan": [vp, vp, i32, vp, vp, ctypes.c_int, vp],
        "moe_plan_routed": [vp, pp(Router), vp, vp, i32, vp, vp, ctypes.c_int, vp],
        "moe_dispatch_f8": [vp, vp, i32, ctypes.c_int, vp],
        "moe_experts_up": [pp(ExpertWeights), vp, vp, i32, vp, i32, vp, vp, i32, vp],
        "moe_experts_down": [pp(ExpertWeights), vp, vp, i32, vp, i32, vp, vp],
        "moe_dispatch": [vp, vp, i32, ctypes.c_int, vp],
        "moe_dispatch_after_plan": [vp, vp, i32, ctypes.c_int, vp],
        "moe_plan_dispatch": [vp, vp, i32, vp, vp, vp, ctypes.c_int, vp],
        "moe_identity_experts": [vp, i32, ctypes.c_int, vp],
        "moe_combine": [vp, vp, vp, i32, ctypes.c_int, vp],
        "moe_step_host": [vp, vp, vp, vp, vp, i32, vp, vp, ctypes.c_int, vp],
        "moe_plan_static": [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    L.moe_status_str.argtypes = [ctypes.c_int]
    L.moe_status_str.restype = ctypes.c_char_p
    _lib = L
    return L


def header_functions(path: str = HEADER) -> list[str]:
    """Names of every function a header (default include/moe.h) declares."""
    src = open(path).read()
    return re.findall(r"MOE_API\s+[\w\s\*]+?\b(moe_\w+)\s*\(", src)


def _call(name, *args):
    rc = getattr(_lib or lib(), name)(*args)
    if rc != MOE_OK:
        raise MoeError(name, rc, lib().moe_status_str(rc).decode())
    return rc


# The pair torch.cuda.current_stream() itself reads (a torch without CUDA has neither).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    """The stream's handle; without one the current stream's, read without
    building a torch Stream (2.8 us of a call that takes 2.5 us itself)."""
    if stream is None:
        return _raw_stream(_device())
    return stream.cuda_stream


def pool_bytes(T_max, H, E, P, k, n_sets=2) -> int:
    d = Desc(T_max, H, E, P, k, 128, n_sets)
    n = ctypes.c_size_t()
    _call("moe_pool_bytes", ctypes.byref(d), ctypes.byref(n))
    return n.value


def replica_check(rep_off, rep_ids, E, P) -> int:
    """Host check of a CSR replica map (numpy or CPU tensors); returns the status."""
    import numpy as np
    off = np.ascontiguousarray(rep_off, np.int32)
    ids = np.ascontiguousarray(rep_ids, np.int32)
    return lib().moe_replica_check(off.ctypes.data_as(ctypes.c_void_p), ids.ctypes.data_as(ctypes.c_void_p),
                                   E, P)


class Pool:
    """A static dispatch/combine buffer pool over one device workspace.

    The workspace is one torch uint8 tensor of ``pool_bytes`` bytes; views
    into it (codes, scales, ex_out, plan metadata) are exposed as tensors."""

    def __init__(self, T_max, H, E, P, k, n_sets=2, device="cuda", stream=None):
        self.desc = Desc(T_max, H, E, P, k, 128, n_sets)
        self.T_max, self.H, self.E, self.P, self.k, self.n_sets = T_max, H, E, P, k, n_sets
        self.nbytes = pool_bytes(T_max, H, E, P, k, n_sets)
        self.workspace = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        h = ctypes.c_void_p()
        _call("moe_pool_init", ctypes.byref(self.desc), _ptr(self.workspace), self.nbytes, ctypes.byref(h))
        self.handle = h
        self._views = {}
        self._f8_tokens = [None] * n_sets  # tokens of each set's last dispatch, if that was in E4M3
        _call("moe_pool_clear_error", self.handle, _stream(stream))

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.moe_pool_destroy(h)
            self.handle = None

    # -- views ---------------------------------------------------------------
    def view(self, buf=0) -> dict:
        v = View()
        _call("moe_pool_view", self.handle, buf, ctypes.byref(v))
        base = self.workspace.data_ptr()
        R, H, T, k, P = v.rows, self.H, self.T_max, self.k, self.P

        def t(addr, dtype, shape):
            n = 1
            for s in shape:
                n *= s
            nb = n * torch.empty((), dtype=dtype).element_size()
            off = addr - base
            return self.workspace[off:off + nb].view(dtype).view(*shape)

        return {
            "codes": t(v.codes, torch.int8, (R, H)),
            "codes_f8": t(v.codes, torch.float8_e4m3fn, (R, H)),  # the same bytes after dispatch_f8
            "scales": t(v.scales, torch.float32, (R, v.scale_stride)),
            "ex_out": t(v.ex_out, torch.bfloat16, (R, H)),
            "topk_e": t(v.topk_e, torch.int32, (T, k)),
            "phys": t(v.phys, torch.int32, (T, k)),
            "gates": t(v.gates, torch.float32, (T, k)),
            "slot": t(v.slot, torch.int32, (T, k)),
            "src_token": t(v.src_token, torch.int32, (R,)),
            "src_k": t(v.src_k, torch.int32, (R,)),
            "counts": t(v.counts, torch.int32, (P,)),
            "offsets": t(v.offsets, torch.int32, (P + 1,)),
            "error_word": t(v.error_word, torch.int32, (1,)),
        }

    # -- calls ---------------------------------------------------------------
    def plan(self, logits, rep_off=None, rep_ids=None, buf=0, stream=None):
        T = logits.shape[0]
        _call("moe_plan", self.handle, _ptr(logits), T, _ptr(rep_off), _ptr(rep_ids), buf, _stream(stream))
        return T

    def plan_routed(self, logits, router, bias=None, rep_off=None, rep_ids=None, buf=0, stream=None):
        """moe_plan_routed: the plan with a scored router (a ``Router``);
        ``bias`` fp32 [E] is added to the scores for the choice only.  Every
        tensor is contiguous and on the GPU: ``logits`` fp32 [T, E], ``rep_off``
        int32 [E + 1], ``rep_ids`` int32 [P]; others are refused (ValueError)."""
        T = logits.shape[0]
        _dense("logits", logits, torch.float32, (T, self.E))
        if bias is not None:
            _dense("bias", bias, torch.float32, (self.E,))
        if rep_off is not None:
            _dense("rep_off", rep_off, torch.int32, (self.E + 1,))
        if rep_ids is not None:
            _dense("rep_ids", rep_ids, torch.int32, (self.P,))
        _call("moe_plan_routed", self.handle, ctypes.byref(router), _ptr(logits), _ptr(bias), T, _ptr(rep_off),
              _ptr(rep_ids), buf, _stream(stream))
        return T

    def dispatch_f8(self, x, buf=0, stream=None):
        """moe_dispatch_f8: dispatch with E4M3 codes (view()["codes_f8"]); ``x``
        bf16 [T, H], contiguous, on the GPU."""
        _dense("x", x, torch.bfloat16, (x.shape[0], self.H))
        _call("moe_dispatch_f8", self.handle, _ptr(x), x.shape[0], buf, _stream(stream))
        self._f8_tokens[buf] = x.shape[0]

    def experts(self, experts, T, h, h_scales, buf=0, stream=None):
        """The set's rows (after ``dispatch_f8``) through ``experts``: their
        gated product into ``h`` / ``h_scales`` (``Experts.inner(rows)``), then
        their down projection into the set's ex_out, ready for ``combine``.
        Refused (MOE_ERR_STATE) unless the set's last dispatch was ``dispatch_f8``
        with T tokens: INT8 rows would be read as E4M3."""
        if buf not in self._views:  # a set's buffers never move
            self._views[buf] = self.view(buf)
        if self._f8_tokens[buf] != T:
            raise MoeError("Pool.experts", MOE_ERR_STATE, lib().moe_status_str(MOE_ERR_STATE).decode())
        v, n = self._views[buf], T * self.k
        experts.up(v["codes_f8"], v["scales"], v["offsets"], h, h_scales, rows=n, stream=stream)
        experts.down(h, h_scales, v["offsets"], v["ex_out"], rows=n, stream=stream)

    def dispatch(self, x, buf=0, stream=None, after_plan=False):
        """moe_dispatch; with ``after_plan`` moe_dispatch_after_plan, which
        reads x before waiting for the kernel just before it: only right after
        this set's plan on the same stream, with x written before that plan."""
        fn = "moe_dispatch_after_plan" if after_plan else "moe_dispatch"
        _call(fn, self.handle, _ptr(x), x.shape[0], buf, _stream(stream))
        self._f8_tokens[buf] = None

    def plan_dispatch(self, logits, x, rep_off=None, rep_ids=None, buf=0, stream=None):
        """moe_plan_dispatch: plan and dispatch as one call; the dispatch
        reads x while the plan runs, which the call makes safe."""
        T = logits.shape[0]
        if x.shape[0] != T:
            raise ValueError("logits and x must have the same number of tokens")
        _call("moe_plan_dispatch", self.handle, _ptr(logits), T, _ptr(rep_off), _ptr(rep_ids), _ptr(x), buf,
              _stream(stream))
        self._f8_tokens[buf] = None
        return T

    def identity_experts(self, T, buf=0, stream=None):
        _call("moe_identity_experts", self.handle, T, buf, _stream(stream))

    def combine(self, T, y=None, ex_out=None, buf=0, stream=None):
        if y is None:
            y = torch.empty((T, self.H), dtype=torch.bfloat16, device=self.workspace.device)
        _call("moe_combine", self.handle, _ptr(ex_out), _ptr(y), T, buf, _stream(stream))
        return y

    def step_host(self, h_logits, h_x, h_y, h_ex_out=None, rep_off=None, rep_ids=None, buf=0, stream=None):
        """Whole layer from host tensors (pinned for asynchronous copies)."""
        _call("moe_step_host", self.handle, _ptr(h_logits), _ptr(h_x), _ptr(h_ex_out), _ptr(h_y),
              h_x.shape[0], _ptr(rep_off), _ptr(rep_ids), buf, _stream(stream))
        self._f8_tokens[buf] = None

    def clear_error(self, stream=None):
        _call("moe_pool_clear_error", self.handle, _stream(stream))

    def check(self, stream=None) -> int:
        """Synchronize and return the device error word (0 = clean)."""
        w = ctypes.c_int32()
        rc = lib().moe_pool_check(self.handle, _stream(stream), ctypes.byref(w))
        if rc not in (MOE_OK, -7):
            raise MoeError("moe_pool_check", rc, lib().moe_status_str(rc).decode())
        return w.value

    def launches(self) -> int:
        n = ctypes.c_uint64()
        _call("moe_pool_launches", self.handle, ctypes.byref(n))
        return n.value


def plan_static(logits, k, P=None, rep_off=None, rep_ids=None, out=None, stream=None) -> dict:
    """moe_plan_static: routing metadata into caller-owned tensors, with no
    device allocation inside the library (its scratch is a fixed 4 MiB array
    in the library's device image).  ``out`` may hold preallocated tensors
    (topk_e, gates, phys, counts, offsets, slot, src_token, src_k,
    error_word); missing ones are allocated here by torch, outside the call."""
    T, E = logits.shape
    P = E if P is None else P
    dev = logits.device
    shapes = {"topk_e": ((T, k), torch.int32), "gates": ((T, k), torch.float32), "phys": ((T, k), torch.int32),
              "counts": ((P,), torch.int32), "offsets": ((P + 1,), torch.int32), "slot": ((T, k), torch.int32),
              "src_token": ((T * k,), torch.int32), "src_k": ((T * k,), torch.int32),
              "error_word": ((1,), torch.int32)}
    out = dict(out or {})
    for name, (shape, dtype) in shapes.items():
        if name not in out:
            out[name] = (torch.zeros if name == "error_word" else torch.empty)(shape, dtype=dtype, device=dev)
    _call("moe_plan_static", _ptr(logits), T, E, P, k, _ptr(rep_off), _ptr(rep_ids),
          *[_ptr(out[n]) for n in ("topk_e", "gates", "phys", "counts", "offsets", "slot", "src_token", "src_k",
                                    "error_word")], _stream(stream))
    return out


class Experts:
    """The weights of P gated feed-forward experts, E4M3 with one fp32 scale
    per 128 x 128 block, and their products over expert windows (moe_experts_up,
    moe_experts_down).

    w13 [P, 2 I, H] (gate rows, then up rows) with s13 [P, 2 I / 128, H / 128],
    w2 [P, H, I] with s2 [P, H / 128, I / 128]; either pair may be left out, and
    with it its product.  ``check()`` returns the device error word."""

    def __init__(self, w13=None, s13=None, w2=None, s2=None):
        if (w13 is None) != (s13 is None) or (w2 is None) != (s2 is None) or (w13 is None and w2 is None):
            raise ValueError("give w13 and s13, w2 and s2, or both pairs")
        if (w13 if w13 is not None else w2).dim() != 3:
            raise ValueError("weights have three dimensions: experts, outputs, inputs")
        if w13 is not None:
            self.P, self.I, self.H = w13.shape[0], w13.shape[1] // 2, w13.shape[2]
        else:
            self.P, self.H, self.I = w2.shape
        P, H, I = self.P, self.H, self.I
        if w13 is not None:
            _block_scaled("w13", w13, s13, P, 2 * I, H)
        if w2 is not None:
            _block_scaled("w2", w2, s2, P, H, I)
        _all_on_gpu(*(t for t in (w13, s13, w2, s2) if t is not None))
        self.w13, self.s13, self.w2, self.s2 = w13, s13, w2, s2
        device = (w13 if w13 is not None else w2).device
        self.error_word = torch.zeros(1, dtype=torch.int32, device=device)
        torch.cuda.current_stream(device).synchronize()  # zero before any stream's kernels may set it
        self.weights = ExpertWeights(P, H, I, *[_ptr(t) for t in (w13, s13, w2, s2, self.error_word)])
        self._ref = ctypes.byref(self.weights)

    def inner(self, rows):
        """Buffers for ``rows`` rows between the two products: E4M3 [rows, I]
        and fp32 scales [rows, I / 128 rounded up to 4], neither filled: a fill
        would be of the current stream, and could run after a product of another."""
        dev = self.error_word.device
        return (torch.empty((rows, self.I), dtype=torch.float8_e4m3fn, device=dev),
                torch.empty((rows, (self.I // 128 + 3) // 4 * 4), dtype=torch.float32, device=dev))

    def up(self, codes, scales, offsets, h, h_scales, rows=None, stream=None):
        """h, h_scales = quantised silu(rows gate^T) * (rows up^T) per window;
        the windows lie in the first ``rows`` rows (None: all of ``codes``)."""
        rows = codes.shape[0] if rows is None else rows
        _tensor("codes", codes, torch.float8_e4m3fn, rows, self.H)
        stride = _tensor("scales", scales, torch.float32, rows)
        self._offsets(offsets)
        _tensor("h", h, torch.float8_e4m3fn, rows, self.I)
        h_stride = _tensor("h_scales", h_scales, torch.float32, rows)
        _all_on_gpu(codes, scales, offsets, h, h_scales)
        _call("moe_experts_up", self._ref, codes.data_ptr(), scales.data_ptr(), stride, offsets.data_ptr(),
              rows, h.data_ptr(), h_scales.data_ptr(), h_stride, _stream(stream))
        return h, h_scales

    def down(self, h, h_scales, offsets, out, rows=None, stream=None):
        """out = bf16(h w2^T) per window; ``rows`` as in ``up``."""
        rows = h.shape[0] if rows is None else rows
        _tensor("h", h, torch.float8_e4m3fn, rows, self.I)
        stride = _tensor("h_scales", h_scales, torch.float32, rows)
        self._offsets(offsets)
        _tensor("out", out, torch.bfloat16, rows, self.H)
        _all_on_gpu(h, h_scales, offsets, out)
        _call("moe_experts_down", self._ref, h.data_ptr(), h_scales.data_ptr(), stride,
              offsets.data_ptr(), rows, out.data_ptr(), _stream(stream))
        return out

    def _offsets(self, offsets):
        if offsets.dtype != torch.int32 or offsets.shape != (self.P + 1,) or not offsets.is_contiguous():
            raise ValueError(f"offsets: want a contiguous int32 tensor of {self.P + 1} values")

    def check(self, stream=None) -> int:
        """Wait for ``stream`` and return the device error word (0 = clean)."""
        (stream or torch.cuda.current_stream()).synchronize()
        return int(self.error_word.item())


def _on_gpu(t):
    return t.is_cuda


def _all_on_gpu(*tensors):
    for t in tensors:
        if not _on_gpu(t):
            raise ValueError(f"want every tensor on the GPU, got a {t.dtype} {tuple(t.shape)} on {t.device}")


def _dense(name, t, dtype, shape):
    """A contiguous tensor of this type and shape on the GPU: what the library
    reads from a bare pointer."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or not _on_gpu(t):
        raise ValueError(f"{name}: want a contiguous {dtype} tensor {tuple(shape)} on the GPU, got "
                         f"{'' if t.is_contiguous() else 'a strided '}{t.dtype} {tuple(t.shape)} on {t.device}")


def _tensor(name, t, dtype, rows, width=None):
    """A dense two-dimensional tensor of this type, with at least ``rows`` rows
    of ``width`` elements (None: any); returns its width."""
    shape = t.shape
    if t.dtype != dtype or len(shape) != 2 or shape[0] < rows or (width is not None and shape[1] != width) or \
            not t.is_contiguous():
        raise ValueError(f"{name}: want a contiguous {dtype} tensor of at least {rows} rows of "
                         f"{'any width' if width is None else width}, got {t.dtype} {tuple(shape)}")
    return shape[1]


def _block_scaled(name, w, s, P, n, k):
    """E4M3 weights [P, n, k] and their fp32 scales per 128 x 128 block."""
    if w.dtype != torch.float8_e4m3fn or w.shape != (P, n, k) or not w.is_contiguous() or n % 128 or k % 128:
        raise ValueError(f"{name}: want contiguous float8_e4m3fn [{P}, {n}, {k}], multiples of 128, got {w.dtype} "
                         f"{tuple(w.shape)}")
    if s.dtype != torch.float32 or s.shape != (P, n // 128, k // 128) or not s.is_contiguous():
        raise ValueError(f"s{name[1:]}: want contiguous float32 [{P}, {n // 128}, {k // 128}], got {s.dtype} "
                         f"{tuple(s.shape)}")
