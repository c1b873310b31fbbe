"""Thin ctypes binding of librf.so (declared in include/rf.h).

Argument marshalling only: each function checks that its torch tensors are
CUDA, contiguous and of the right dtype, passes their data pointers, sizes
and the current CUDA stream to the C entry point of the same name, and turns
a non-OK status into ``RFError``. Every step of the computation runs in the
library's kernels; nothing here computes, and there is no CPU fallback -- if
the library is missing, every call raises.

The calls of a serving loop (from ``kv_append_paged`` on) go through a native module (csrc/serving_binding.cpp), which
does the same checks without Python's time for them; arguments that it does not
accept come back here for the error that names them.
"""

import ctypes
import importlib.machinery
import importlib.util
import math
import os

import torch

from . import build as _build

RF_OK, RF_ERR_INVALID, RF_ERR_UNSUPPORTED, RF_ERR_CUDA, RF_ERR_TIMEOUT = range(5)
RF_F32, RF_BF16 = 0, 1
RF_KERNEL_BLOCKWISE, RF_KERNEL_ROWWISE = 0, 1
_STATUS_NAMES = {0: "RF_OK", 1: "RF_ERR_INVALID", 2: "RF_ERR_UNSUPPORTED", 3: "RF_ERR_CUDA",
                 4: "RF_ERR_TIMEOUT"}
TILE = 128


class RFError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s: %s" % (_STATUS_NAMES.get(status, status), message))
        self.status = status


class RFBlockMask(ctypes.Structure):
    _fields_ = [("tile_q", ctypes.c_int), ("tile_k", ctypes.c_int), ("nqt", ctypes.c_int),
                ("nkt", ctypes.c_int), ("row_ptr", ctypes.c_void_p), ("col_idx", ctypes.c_void_p),
                ("per_head", ctypes.c_int), ("tile_bits", ctypes.c_void_p),
                ("bits", ctypes.c_void_p), ("cta_order", ctypes.c_void_p)]


class RFKvPool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + \
        [("%s_%s_stride" % (c, d), ctypes.c_int64) for c in "kv"
         for d in ("layer", "page", "token", "head")] + \
        [(n, ctypes.c_int) for n in ("layers", "num_pages", "page", "Hkv", "d", "dt")]


_LIB = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t

# name: (restype, argtypes) -- mirrors include/rf.h
SIGNATURES = {
    "rf_softmax_rows": (_I, [_P, _P, _I64, _I64, _I, _P]),
    "rf_attn_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I,
                         ctypes.POINTER(RFBlockMask), _I, _P]),
    "rf_attn_decode_splitk": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _I,
                                   _P]),
    "rf_attn_decode_splitk_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _I,
                                           _P]),
    "rf_attn_fwd_host": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I,
                              ctypes.POINTER(RFBlockMask), _I, _P, _SZ, _P]),
    "rf_attn_fwd_host_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "rf_decode_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "rf_splitk_merge": (_I, [_P, _P, _P, _P, _I64, _I, _I, _I, _P]),
    "rf_attn_decode_partials": (_I, [_P, _P, _P, _P, ctypes.c_size_t, _I, _I, _I, _I, _I, _F,
                                     _I, _I, _P]),
    "rf_splitk_merge_strided": (_I, [_P, _P, _P, _P, _I64, _I, _I, _I64, _I64, _I64, _I64, _I,
                                     _P]),
    "rf_blockmask_build": (_I, [_P, _I, _I, _I, _P, _P, _I64, _P]),
    "rf_blockmask_build_elements": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _I64, _P, _P]),
    "rf_blockmask_counts": (_I, [ctypes.POINTER(RFBlockMask), _I, _I, _I, _I, _I, _P, _P]),
    "rf_blockmask_cta_order_len": (_I64, [_I, _I, _I]),
    "rf_blockmask_cta_order": (_I, [ctypes.POINTER(RFBlockMask), _I, _I, _I, _P, _I64, _P]),
    "rf_attn_fwd_rowwise": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I,
                                 ctypes.POINTER(RFBlockMask), _I, _P]),
    "rf_attn_choose_kernel": (_I, [_I, _I, _I, _I, _I, _I64, _I64, _I64, _I]),
    "rf_attn_estimate_us": (_I, [_I, _I, _I, _I, _I, _I64, _I64, _I64, _I,
                                 ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]),
    "rf_moe_route": (_I, [_P, _I64, _I, _I, _I, _P, _P, _P, _I, _P]),
    "rf_row_moments": (_I, [_P, _I64, _I64, _F, _P, _P, _P, _I, _P]),
    "rf_moment_of_inertia": (_I, [_P, _P, _I64, _I64, _P, _P, _P, _P]),
    "rf_rowquant_e4m3": (_I, [_P, _I64, _I64, _P, _P, _I, _P]),
    "rf_mla_decode_workspace_bytes": (_SZ, [_I, _I]),
    "rf_mla_decode": (_I, [_P, _P, _P, _P, _I, _I, _F, _I, _P, _SZ, _P]),
    "rf_paged_slots": (_I, [_P, _P, _P, _I64, _I, _I, _I, _I, _I, _P, _P, _P]),
    "rf_kv_append_paged": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I64,
                                _I64, _I64, _I, _I, _I, _I, _I, _I, _P, _P, _P, _I, _I, _I, _P,
                                _P, _F, _I, _P]),
    "rf_paged_plan_bytes": (_SZ, [_I]),
    "rf_paged_plan": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _SZ, _P]),
    "rf_attn_paged_workspace_bytes": (_SZ, [_I]),
    "rf_attn_paged": (_I, [_P, _I64, _P, _I64, _I64, _I64, _P, _I64, _I64, _I64, _I, _I, _P, _I64,
                           _I, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P, _SZ, _I, _P]),
    "rf_attn_paged_tree": (_I, [_P, _I64, _P, _I64, _I64, _I64, _P, _I64, _I64, _I64, _I, _I, _P,
                                _I64, _I, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P, _SZ, _P, _I, _I,
                                _P]),
    "rf_tree_mask": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "rf_tree_accept": (_I, [_P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P]),
    "rf_sample_rows": (_I, [_P, _I64, _P, _P, _P, _P, _P, _I, _I, _P, _P, _I, _P]),
    "rf_kv_compact_paged": (_I, [ctypes.POINTER(RFKvPool), _P, _I64, _I, _I, _P, _I, _P, _P, _P,
                                 _P]),
    "rf_kv_copy_pages": (_I, [ctypes.POINTER(RFKvPool), _P, _P, _I, _P]),
    "rf_pages_fork": (_I, [_P, _I64, _P, _I, _P, _I, _P, _I64, _P, _P, _I, _I, _I, _P]),
    "rf_pages_grow": (_I, [_P, _I64, _P, _P, _I, _P, _I, _I, _I, _P, _P, _P, _P]),
    "rf_pages_release": (_I, [_P, _I64, _P, _P, _I, _P, _I, _I, _I, _P]),
    "rf_draft_verify_workspace_bytes": (_SZ, [_I, _I]),
    "rf_draft_verify": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _SZ, _I, _P]),
    "rf_fp8_gemm": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "rf_debug_set_visited": (_I, [_P, _I64]),
    "rf_debug_inject_fault": (_I, [_I]),
    "rf_device_status": (_I, [_P, ctypes.POINTER(_I)]),
    "rf_last_error": (ctypes.c_char_p, []),
    "rf_version": (_I, []),
}


def library_path():
    return _build.LIB_PATH


def lib():
    """The loaded librf.so; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                "librf.so is not built (%s); run `python -m online_softmax_attention_rf_gb300.build`"
                % path)
        L = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _check(status):
    if status != RF_OK:
        raise RFError(status, lib().rf_last_error().decode(errors="replace"))


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _dt(t):
    if t.dtype == torch.float32:
        return RF_F32
    if t.dtype == torch.bfloat16:
        return RF_BF16
    raise TypeError("unsupported dtype %s (float32 or bfloat16)" % t.dtype)


def _cuda(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


class BlockMask:
    """Block-sparse 128 x 128 tile lists resident on the device.

    ``row_ptr`` int32 [nheads*nqt + 1] and ``col_idx`` int32 [capacity];
    ``per_head`` is 1 when each (batch, head) has its own lists. With the
    two-level form, ``tile_bits`` int32 (parallel to ``col_idx``, -1 = full
    tile) and ``bits`` uint64 viewed as int64 [partial tiles, 256].
    ``cta_orders`` caches the tensor-core kernel's work order
    (rf_blockmask_cta_order) per (B, H, Sq).
    """

    def __init__(self, row_ptr, col_idx, nqt, nkt, per_head, tile_bits=None, bits=None):
        self.row_ptr, self.col_idx = row_ptr, col_idx
        self.nqt, self.nkt, self.per_head = nqt, nkt, per_head
        self.tile_bits, self.bits = tile_bits, bits
        self.cta_orders = {}

    def as_struct(self, order=None):
        return RFBlockMask(TILE, TILE, self.nqt, self.nkt, self.row_ptr.data_ptr(),
                           self.col_idx.data_ptr(), self.per_head,
                           self.tile_bits.data_ptr() if self.tile_bits is not None else None,
                           self.bits.data_ptr() if self.bits is not None else None,
                           order.data_ptr() if order is not None else None)

    def cta_order(self, B, H, Sq):
        """rf_blockmask_cta_order for an attention of B x H heads and Sq queries:
        computed on the current stream the first time, then cached (the
        kernel reads one entry per CTA)."""
        key = (B, H, Sq)
        if key not in self.cta_orders:
            n = int(lib().rf_blockmask_cta_order_len(B, H, Sq))
            order = torch.empty(max(1, n), dtype=torch.int32, device=self.row_ptr.device)
            bm = self.as_struct()
            _check(lib().rf_blockmask_cta_order(ctypes.byref(bm), B, H, Sq, _ptr(order), n,
                                                _stream()))
            self.cta_orders[key] = order
        return self.cta_orders[key]

    @classmethod
    def from_dense_elements(cls, elem_mask, device="cuda"):
        """Two-level lists (outer tiles + inner 8x8 bitmaps) from a bool/uint8
        element mask [Sq, Sk] (shared) or [nheads, Sq, Sk] (per head), built
        on the device (rf_blockmask_build_elements; a first pass counts the
        partial tiles to size the bitmaps)."""
        em = torch.as_tensor(elem_mask)
        per_head = 1 if em.dim() == 3 else 0
        if em.dim() == 2:
            em = em.unsqueeze(0)
        nheads, Sq, Sk = em.shape
        dense = em.to(device=device, dtype=torch.uint8).contiguous()
        nqt, nkt = -(-Sq // TILE), -(-Sk // TILE)
        row_ptr = torch.empty(nheads * nqt + 1, dtype=torch.int32, device=device)
        col_idx = torch.empty(nheads * nqt * nkt, dtype=torch.int32, device=device)
        tile_bits = torch.empty(nheads * nqt * nkt, dtype=torch.int32, device=device)
        n_partial = torch.zeros(1, dtype=torch.int32, device=device)
        blockmask_build_elements(dense, row_ptr, col_idx, tile_bits, None, n_partial)
        bits = torch.empty((max(1, int(n_partial.item())), 256), dtype=torch.int64, device=device)
        blockmask_build_elements(dense, row_ptr, col_idx, tile_bits, bits, n_partial)
        return cls(row_ptr, col_idx, nqt, nkt, per_head, tile_bits, bits)

    @classmethod
    def from_dense(cls, tile_mask, device="cuda"):
        """Build the lists on the device from a bool/uint8 mask [nqt, nkt] or
        [nheads, nqt, nkt] (rf_blockmask_build)."""
        tm = torch.as_tensor(tile_mask)
        per_head = 1 if tm.dim() == 3 else 0
        if tm.dim() == 2:
            tm = tm.unsqueeze(0)
        nheads, nqt, nkt = tm.shape
        dense = tm.to(device=device, dtype=torch.uint8).contiguous()
        row_ptr = torch.empty(nheads * nqt + 1, dtype=torch.int32, device=device)
        col_idx = torch.empty(max(1, nheads * nqt * nkt), dtype=torch.int32, device=device)
        blockmask_build(dense, row_ptr, col_idx)
        return cls(row_ptr, col_idx, nqt, nkt, per_head)


def blockmask_build(dense_u8, row_ptr, col_idx):
    """rf_blockmask_build on [nheads, nqt, nkt] uint8 -> row_ptr, col_idx (in place)."""
    _cuda(dense_u8, row_ptr, col_idx)
    nheads, nqt, nkt = dense_u8.shape
    _check(lib().rf_blockmask_build(_ptr(dense_u8), nheads, nqt, nkt, _ptr(row_ptr),
                                    _ptr(col_idx), col_idx.numel(), _stream()))


def blockmask_build_elements(dense_u8, row_ptr, col_idx, tile_bits, bits, n_partial=None):
    """rf_blockmask_build_elements on [nheads, Sq, Sk] uint8 (in place); ``bits``
    None builds the lists only (and counts the partial tiles into n_partial)."""
    _cuda(dense_u8, row_ptr, col_idx, tile_bits, bits, n_partial)
    nheads, Sq, Sk = dense_u8.shape
    cap = 0 if bits is None else bits.shape[0]
    _check(lib().rf_blockmask_build_elements(_ptr(dense_u8), nheads, Sq, Sk, _ptr(row_ptr),
                                             _ptr(col_idx), _ptr(tile_bits), _ptr(bits), cap,
                                             _ptr(n_partial), _stream()))


def softmax_rows(x, out=None):
    """rf_softmax_rows: softmax over the last dim of a 2-D float32/bf16 tensor."""
    _cuda(x)
    if x.dim() != 2:
        raise ValueError("x must be [rows, cols]")
    y = torch.empty_like(x) if out is None else out
    _cuda(y)
    _check(lib().rf_softmax_rows(_ptr(x), _ptr(y), x.shape[0], x.shape[1], _dt(x), _stream()))
    return y


def moe_route(logits, k, renorm=False, with_lse=True):
    """rf_moe_route: logits [T, E] -> (idx int32 [T, k], w float32 [T, k], lse or None)."""
    _cuda(logits)
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    idx = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    w = torch.empty(T, k, dtype=torch.float32, device=logits.device)
    lse = torch.empty(T, dtype=torch.float32, device=logits.device) if with_lse else None
    _check(lib().rf_moe_route(_ptr(logits), T, E, int(k), 1 if renorm else 0, _ptr(idx), _ptr(w),
                              _ptr(lse), _dt(logits), _stream()))
    return idx, w, lse


def row_moments(x, eps=1e-5, normalize=True, out=None):
    """rf_row_moments: x [rows, cols] -> (mean, var, y or None), mean/var float32."""
    _cuda(x)
    if x.dim() != 2:
        raise ValueError("x must be [rows, cols]")
    rows = x.shape[0]
    mean = torch.empty(rows, dtype=torch.float32, device=x.device)
    var = torch.empty(rows, dtype=torch.float32, device=x.device)
    y = None
    if normalize:
        y = torch.empty_like(x) if out is None else out
        _cuda(y)
        if y.shape != x.shape or y.dtype != x.dtype:
            raise ValueError("out must match x")
    _check(lib().rf_row_moments(_ptr(x), rows, x.shape[1], float(eps), _ptr(mean), _ptr(var),
                                _ptr(y), _dt(x), _stream()))
    return mean, var, y


def moment_of_inertia(points, masses=None):
    """rf_moment_of_inertia: points [sets, n, 3] float32 (+ masses [sets, n])
    -> (total mass [sets], centre [sets, 3], inertia [sets])."""
    _cuda(points, masses)
    if points.dim() != 3 or points.shape[2] != 3 or points.dtype != torch.float32:
        raise ValueError("points must be float32 [sets, n, 3]")
    sets, n = points.shape[0], points.shape[1]
    if masses is not None and (masses.shape != (sets, n) or masses.dtype != torch.float32):
        raise ValueError("masses must be float32 [sets, n]")
    total = torch.empty(sets, dtype=torch.float32, device=points.device)
    centre = torch.empty(sets, 3, dtype=torch.float32, device=points.device)
    inertia = torch.empty(sets, dtype=torch.float32, device=points.device)
    _check(lib().rf_moment_of_inertia(_ptr(points), _ptr(masses), sets, n, _ptr(total),
                                      _ptr(centre), _ptr(inertia), _stream()))
    return total, centre, inertia


def rowquant_e4m3(x):
    """rf_rowquant_e4m3: x [rows, K] float32/bf16 -> (codes uint8 [rows, K],
    scale float32 [rows])."""
    _cuda(x)
    if x.dim() != 2:
        raise ValueError("x must be [rows, K]")
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    sc = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    _check(lib().rf_rowquant_e4m3(_ptr(x), x.shape[0], x.shape[1], _ptr(q), _ptr(sc), _dt(x),
                                  _stream()))
    return q, sc


def fp8_gemm(a, sa, w, sw, out=None):
    """rf_fp8_gemm: codes a [M, K], w [N, K] (uint8), scales sa [M], sw [N]
    -> C bf16 [M, N]."""
    _cuda(a, sa, w, sw)
    M, K = a.shape
    N = w.shape[0]
    if w.shape[1] != K or a.dtype != torch.uint8 or w.dtype != torch.uint8:
        raise ValueError("a [M, K] and w [N, K] must be uint8 codes")
    c = torch.empty(M, N, dtype=torch.bfloat16, device=a.device) if out is None else out
    _cuda(c)
    _check(lib().rf_fp8_gemm(_ptr(a), _ptr(sa), _ptr(w), _ptr(sw), _ptr(c), M, N, K, _stream()))
    return c


def mla_decode(q, kv, nsplit, scale, workspace=None, out=None, lse=None):
    """rf_mla_decode: q [B, 128, 576], kv [B, Sk, 576] bf16 -> (o [B, 128, 512]
    bf16, lse [B, 128] float32)."""
    _cuda(q, kv)
    B, Sk = kv.shape[0], kv.shape[1]
    if q.shape != (B, 128, 576) or kv.shape[2] != 576:
        raise ValueError("q must be [B, 128, 576] and kv [B, Sk, 576]")
    o = torch.empty(B, 128, 512, dtype=torch.bfloat16, device=q.device) if out is None else out
    if lse is None:
        lse = torch.empty(B, 128, dtype=torch.float32, device=q.device)
    nbytes = int(lib().rf_mla_decode_workspace_bytes(B, nsplit))
    ws = torch.empty(max(1, nbytes // 4), dtype=torch.float32, device=q.device) \
        if workspace is None else workspace
    _cuda(o, lse, ws)
    _check(lib().rf_mla_decode(_ptr(q), _ptr(kv), _ptr(o), _ptr(lse), B, Sk, float(scale),
                               int(nsplit), _ptr(ws), ws.numel() * ws.element_size(), _stream()))
    return o, lse


def attn_fwd(q, k, v, scale=None, causal=False, blockmask=None, out=None, lse=None,
             with_lse=True, kernel="block"):
    """rf_attn_fwd (kernel "block"), rf_attn_fwd_rowwise ("row"), or the one
    rf_attn_choose_kernel picks ("auto"): q [B,H,Sq,d], k/v [B,Hkv,Sk,d] ->
    (o, lse or None)."""
    _cuda(q, k, v)
    B, H, Sq, d = q.shape
    Hkv, Sk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if kernel == "auto":
        counts = selector_counts(B, H, Sq, Sk, causal, blockmask, q.device)
        kernel = "row" if choose_kernel(B, H, Sq, Sk, d, *counts, device=q.device) == \
            RF_KERNEL_ROWWISE else "block"
    if kernel not in ("block", "row"):
        raise ValueError("kernel must be 'block', 'row' or 'auto'")
    o = torch.empty_like(q) if out is None else out
    if lse is None and with_lse:
        lse = torch.empty(B, H, Sq, dtype=torch.float32, device=q.device)
    _cuda(o, lse)
    bm = None
    if blockmask is not None:
        # the tensor-core kernel takes its work in the mask's order (long
        # items first); the other kernels ignore the field
        order = blockmask.cta_order(B, H, Sq) if kernel == "block" and Sq > 0 else None
        bm = ctypes.byref(blockmask.as_struct(order))
    fn = lib().rf_attn_fwd if kernel == "block" else lib().rf_attn_fwd_rowwise
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, Sq, Sk, d, float(scale),
              1 if causal else 0, bm, _dt(q), _stream()))
    return o, lse


def attn_fwd_rowwise(q, k, v, scale=None, causal=False, blockmask=None, out=None, lse=None,
                     with_lse=True):
    """rf_attn_fwd_rowwise (STOF's row-wise kernel); arguments as attn_fwd."""
    return attn_fwd(q, k, v, scale, causal, blockmask, out, lse, with_lse, kernel="row")


def choose_kernel(B, H, Sq, Sk, d, listed_tiles, partial_tiles, visible_pairs, num_sms=None,
                  device=None):
    """rf_attn_choose_kernel: RF_KERNEL_BLOCKWISE or RF_KERNEL_ROWWISE."""
    if num_sms is None:
        num_sms = _num_sms(device)
    r = lib().rf_attn_choose_kernel(B, H, Sq, Sk, d, int(listed_tiles), int(partial_tiles),
                                    int(visible_pairs), int(num_sms))
    if r < 0:
        raise ValueError("rf_attn_choose_kernel: invalid arguments")
    return r


def estimate_us(B, H, Sq, Sk, d, listed_tiles, partial_tiles, visible_pairs, num_sms=None,
                device=None):
    """rf_attn_estimate_us: (block-wise, row-wise) model times in microseconds."""
    if num_sms is None:
        num_sms = _num_sms(device)
    b, r = ctypes.c_double(), ctypes.c_double()
    _check(lib().rf_attn_estimate_us(B, H, Sq, Sk, d, int(listed_tiles), int(partial_tiles),
                                     int(visible_pairs), int(num_sms), ctypes.byref(b),
                                     ctypes.byref(r)))
    return b.value, r.value


def _num_sms(device):
    if torch.cuda.is_available():
        dev = torch.cuda.current_device() if device is None else torch.device(device).index or 0
        return torch.cuda.get_device_properties(dev).multi_processor_count
    return 152


def selector_counts(B, H, Sq, Sk, causal, blockmask=None, device=None):
    """rf_blockmask_counts: (listed_tiles, partial_tiles, visible_pairs) over
    all B*H heads, the selector's inputs, counted on the device from the tile
    lists (dense when blockmask is None); waits for the three numbers."""
    dev = blockmask.row_ptr.device if blockmask is not None else (
        torch.device("cuda", torch.cuda.current_device()) if device is None else device)
    counts = torch.empty(3, dtype=torch.int64, device=dev)
    bm = ctypes.byref(blockmask.as_struct()) if blockmask is not None else None
    with torch.cuda.device(dev):
        _check(lib().rf_blockmask_counts(bm, B, H, Sq, Sk, 1 if causal else 0, _ptr(counts),
                                         _stream()))
        listed, partial, pairs = (int(x) for x in counts.cpu().tolist())
    return listed, partial, pairs


def attn_fwd_host_workspace_bytes(B, H, Hkv, Sq, Sk, d, dtype=torch.bfloat16):
    return int(lib().rf_attn_fwd_host_workspace_bytes(
        B, H, Hkv, Sq, Sk, d, RF_F32 if dtype == torch.float32 else RF_BF16))


def attn_fwd_host(q, k, v, scale=None, causal=False, blockmask=None, out=None, lse=None,
                  with_lse=True, workspace=None, device=None):
    """rf_attn_fwd_host: q [B,H,Sq,d], k/v [B,Hkv,Sk,d] in HOST memory (pinned for
    overlap) -> (o, lse) in host memory; copies and kernels pipelined by chunks.
    The call is asynchronous on the current stream of `device`."""
    for t in (q, k, v):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous host tensors")
    B, H, Sq, d = q.shape
    Hkv, Sk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    pin = q.is_pinned()
    o = torch.empty(q.shape, dtype=q.dtype, pin_memory=pin) if out is None else out
    if lse is None and with_lse:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, pin_memory=pin)
    nbytes = attn_fwd_host_workspace_bytes(B, H, Hkv, Sq, Sk, d, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(1, nbytes), dtype=torch.uint8, device=dev)
    _cuda(workspace)
    bm = ctypes.byref(blockmask.as_struct()) if blockmask is not None else None
    with torch.cuda.device(dev):
        _check(lib().rf_attn_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv,
                                      Sq, Sk, d, float(scale), 1 if causal else 0, bm, _dt(q),
                                      _ptr(workspace), workspace.numel(), _stream()))
    return o, lse


def decode_workspace_bytes(B, H, nsplit, d):
    return int(lib().rf_decode_workspace_bytes(B, H, nsplit, d))


def attn_decode_splitk(q, k, v, nsplit, scale=None, workspace=None, out=None, lse=None):
    """rf_attn_decode_splitk: q [B,H,1,d], k/v [B,Hkv,Sk,d] -> (o, lse)."""
    _cuda(q, k, v)
    B, H, Sq, d = q.shape
    Hkv, Sk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    nbytes = decode_workspace_bytes(B, H, nsplit, d)
    if workspace is None:
        workspace = torch.empty(max(1, nbytes // 4), dtype=torch.float32, device=q.device)
    o = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty(B, H, Sq, dtype=torch.float32, device=q.device)
    _cuda(workspace, o, lse)
    _check(lib().rf_attn_decode_splitk(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv,
                                       Sk, d, float(scale), nsplit, _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _dt(q),
                                       _stream()))
    return o, lse


def attn_decode_splitk_noalloc(q, k, v, nsplit, scale=None, out=None, lse=None):
    """rf_attn_decode_splitk_noalloc: the split-K decode with the library's own
    fixed 16 MiB device workspace (for callers that cannot allocate; calls on
    one device share that workspace and must not overlap on the GPU)."""
    _cuda(q, k, v)
    B, H, Sq, d = q.shape
    Hkv, Sk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty(B, H, Sq, dtype=torch.float32, device=q.device)
    _cuda(o, lse)
    _check(lib().rf_attn_decode_splitk_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B,
                                               H, Hkv, Sk, d, float(scale), nsplit, _dt(q),
                                               _stream()))
    return o, lse


def attn_decode_partials(q, k, v, nsplit, scale=None, workspace=None):
    """rf_attn_decode_partials: q [B,H,1,d], k/v [B,Hkv,Sk,d] bf16 -> (o_part
    float32 [B*H, nsplit, d], lse_part float32 [B*H, nsplit]), views of the
    workspace."""
    _cuda(q, k, v)
    B, H, _, d = q.shape
    Hkv, Sk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    nbytes = decode_workspace_bytes(B, H, nsplit, d)
    ws = torch.empty(nbytes // 4, dtype=torch.float32, device=q.device) \
        if workspace is None else workspace
    _cuda(ws)
    _check(lib().rf_attn_decode_partials(_ptr(q), _ptr(k), _ptr(v), _ptr(ws),
                                         ws.numel() * ws.element_size(), B, H, Hkv, Sk, d,
                                         float(scale), int(nsplit), _dt(q), _stream()))
    n = B * H * nsplit
    return ws[:n * d].view(B * H, nsplit, d), ws[n * d:n * d + n].view(B * H, nsplit)


def splitk_merge(o_part, lse_part, out_dtype=torch.bfloat16):
    """rf_splitk_merge: o_part [rows, nsplit, d] f32, lse_part [rows, nsplit] f32.

    Contiguous partials go to rf_splitk_merge; strided views (for instance
    ``gathered.permute(1, 0, 2)`` of split-major [nsplit, rows, d] partials,
    with d contiguous) go to rf_splitk_merge_strided with their strides."""
    for t in (o_part, lse_part):
        if not t.is_cuda or t.dtype != torch.float32:
            raise ValueError("partials must be float32 CUDA tensors")
    rows, nsplit, d = o_part.shape
    if lse_part.shape != (rows, nsplit):
        raise ValueError("lse_part must be [rows, nsplit]")
    o = torch.empty(rows, d, dtype=out_dtype, device=o_part.device)
    lse = torch.empty(rows, dtype=torch.float32, device=o_part.device)
    out_dt = RF_F32 if out_dtype == torch.float32 else RF_BF16
    if o_part.is_contiguous() and lse_part.is_contiguous():
        _check(lib().rf_splitk_merge(_ptr(o_part), _ptr(lse_part), _ptr(o), _ptr(lse), rows,
                                     nsplit, d, out_dt, _stream()))
    else:
        if o_part.stride(2) != 1:
            raise ValueError("o_part's last dimension must be contiguous")
        _check(lib().rf_splitk_merge_strided(
            _ptr(o_part), _ptr(lse_part), _ptr(o), _ptr(lse), rows, nsplit, d, o_part.stride(1),
            o_part.stride(0), lse_part.stride(1), lse_part.stride(0), out_dt, _stream()))
    return o, lse


# The paged serving calls run once a layer or once a token, where the host's
# share of a call shows: their arguments are marshalled by a native module
# (csrc/serving_binding.cpp, over the same C entry points), which answers None
# for tensors that do not fit and the status of a refused call.

_SERVING = None


def _serving():
    """The native binding of the paged serving calls; raises if it has not been
    built."""
    global _SERVING
    if _SERVING is None:
        lib()
        path = _build.BINDING_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                "_rf_serving.so is not built (%s); run `python -m "
                "online_softmax_attention_rf_gb300.build`" % path)
        loader = importlib.machinery.ExtensionFileLoader("_rf_serving", path)
        spec = importlib.util.spec_from_file_location("_rf_serving", path, loader=loader)
        _SERVING = importlib.util.module_from_spec(spec)
        loader.exec_module(_SERVING)
    return _SERVING


def _launch(index, fn, *args):
    """fn(*args, the current stream of device `index`), with that device current."""
    with torch.cuda.device(index):
        _check(fn(*args, _stream()))


def _same_device(*ts):
    """The one CUDA device of the tensors that are given."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensors must live on one device")
    return dev


def _expect(t, name, dtype, shape, optional=False):
    """A contiguous tensor of this dtype and shape (None where that is allowed)."""
    if t is None and optional:
        return
    if t is None or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s"
                         % (name, dtype, tuple(shape)))


def _expect_pool(cache, name, Hkv, d, dtype):
    if cache.dim() != 4 or tuple(cache.shape[2:]) != (Hkv, d) or cache.dtype != dtype:
        raise ValueError("%s must be a %s pool [pages, page, %d, %d]" % (name, dtype, Hkv, d))
    if cache.stride(3) != 1:
        raise ValueError("%s's last dimension must be contiguous" % name)


def _expect_rows(x, name, T, heads, d, dtype):
    if x.dim() != 3 or tuple(x.shape) != (T, heads, d) or x.dtype != dtype:
        raise ValueError("%s must be a %s tensor [%d, %d, %d]" % (name, dtype, T, heads, d))
    if x.stride(2) != 1 or (heads > 1 and x.stride(1) != d):
        raise ValueError("%s: a token's heads must lie back to back" % name)


def _expect_table(block_table, B):
    if block_table.dim() != 2 or block_table.shape[0] != B or block_table.dtype != torch.int32 or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be int32 [B, max_pages] with contiguous rows")


def paged_slots(cu_q, kv_len, block_table, page_size, num_pages, total_q):
    """rf_paged_slots: where a step's new tokens go -> (pos int32 [T], slots int64
    [T]). cu_q int32 [B + 1], kv_len int32 [B] (with the new tokens),
    block_table int32 [B, max_pages] (rows may be strided)."""
    dev = _same_device(cu_q, kv_len, block_table)
    B = kv_len.shape[0]
    _expect(cu_q, "cu_q", torch.int32, (B + 1,))
    _expect(kv_len, "kv_len", torch.int32, (B,))
    _expect_table(block_table, B)
    width = block_table.shape[1]
    pos = torch.empty(total_q, dtype=torch.int32, device=dev)
    slots = torch.empty(total_q, dtype=torch.int64, device=dev)
    _launch(dev.index, lib().rf_paged_slots, cu_q.data_ptr(), kv_len.data_ptr(),
            block_table.data_ptr(), block_table.stride(0) if B > 1 else width, B, int(total_q),
            width, int(page_size), int(num_pages), pos.data_ptr(), slots.data_ptr())
    return pos, slots


def _refuse_append(q, k, v, k_cache, v_cache, slots, pos, cos_sin, q_weight, k_weight, q_out):
    _same_device(q, k, v, k_cache, v_cache, slots, pos, cos_sin, q_weight, k_weight, q_out)
    if k.dim() != 3:
        raise ValueError("k must be [T, Hkv, d]")
    T, Hkv, d = k.shape
    _expect_rows(k, "k", T, Hkv, d, k.dtype)
    _expect_rows(v, "v", T, Hkv, d, k.dtype)
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [T, H, d]")
        _expect_rows(q, "q", T, q.shape[1], d, k.dtype)
        _expect(q_out, "q_out", k.dtype, (T, q.shape[1], d), optional=True)
    _expect_pool(k_cache, "k_cache", Hkv, d, k.dtype)
    _expect_pool(v_cache, "v_cache", Hkv, d, k.dtype)
    if v_cache.shape[:2] != k_cache.shape[:2]:
        raise ValueError("k_cache and v_cache must have the same pages")
    _expect(slots, "slots", torch.int64, (T,))
    _expect(q_weight, "q_weight", k.dtype, (d,), optional=True)
    _expect(k_weight, "k_weight", k.dtype, (d,), optional=True)
    if cos_sin is not None:
        if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be a contiguous float32 tensor [max_pos, rot]")
        _expect(pos, "pos", torch.int32, (T,))
    raise ValueError("kv_append_paged: unsupported tensors")


def kv_append_paged(q, k, v, k_cache, v_cache, slots, pos=None, cos_sin=None, q_weight=None,
                    k_weight=None, eps=1e-6, interleaved=False, q_out=None):
    """rf_kv_append_paged: write a step's keys and values into their pages, with
    the head norm (q_weight, k_weight [d]) and the rotation (cos_sin float32
    [max_pos, rot], pos int32 [T]) of queries and keys on the way.

    q [T, H, d] (or None), k, v [T, Hkv, d] (views of a fused projection fit),
    k_cache, v_cache [pages, page, Hkv, d] (any strides with d contiguous),
    slots int64 [T] (negative: skipped) -> q_out [T, H, d], or None without q.
    q_out may be q itself when q is contiguous. bf16 or float32, d a multiple of
    16 up to 256; ``attn_paged`` reads bf16 pools with d 64 or 128 and pages of a
    multiple of 8 tokens only."""
    r = _serving().kv_append_paged(q, k, v, k_cache, v_cache, slots, pos, cos_sin, q_weight,
                                   k_weight, eps, interleaved, q_out)
    if r.__class__ is tuple:
        return r[0]
    if r is None:
        _refuse_append(q, k, v, k_cache, v_cache, slots, pos, cos_sin, q_weight, k_weight, q_out)
    _check(r)


class PagedPlan:
    """rf_paged_plan: a step's paged attention divided among the SMs, on the device.

    Made once a step from cu_q int32 [B + 1] and kv_len int32 [B] (with the new
    tokens) and read by the ``attn_paged`` of every layer; it keeps its own
    copy of the lengths. ``update`` makes it again in place, for a captured
    step whose lengths change."""

    def __init__(self, cu_q, kv_len, total_q, H, Hkv, page_size, max_pages, causal=True):
        self.B, self.T, self.H, self.Hkv = kv_len.shape[0], int(total_q), int(H), int(Hkv)
        self.page, self.max_pages, self.causal = int(page_size), int(max_pages), bool(causal)
        dev = _same_device(cu_q, kv_len)
        self.buf = torch.empty(int(lib().rf_paged_plan_bytes(self.B)), dtype=torch.uint8,
                               device=dev)
        self.update(cu_q, kv_len)

    def update(self, cu_q, kv_len):
        """The plan for new lengths of the same batch size."""
        dev = _same_device(cu_q, kv_len, self.buf)
        _expect(cu_q, "cu_q", torch.int32, (self.B + 1,))
        _expect(kv_len, "kv_len", torch.int32, (self.B,))
        _launch(dev.index, lib().rf_paged_plan, cu_q.data_ptr(), kv_len.data_ptr(), self.B, self.T,
                self.H, self.Hkv, self.page, self.max_pages, 1 if self.causal else 0,
                self.buf.data_ptr(), self.buf.numel())
        return self


def attn_paged_workspace(d, device="cuda"):
    """A workspace for ``attn_paged`` with head dimension d (calls that may
    overlap need one each)."""
    n = int(lib().rf_attn_paged_workspace_bytes(int(d)))
    return torch.empty(max(1, n // 4), dtype=torch.float32, device=device)


def _refuse_attn(q, k_cache, v_cache, block_table, plan, out, lse, workspace, tree_mask):
    _same_device(q, k_cache, v_cache, block_table, plan.buf, out, lse, workspace, tree_mask)
    if q.dim() != 3 or q.shape[:2] != (plan.T, plan.H):
        raise ValueError("q must be [%d, %d, d], as the plan was made for" % (plan.T, plan.H))
    T, H, d = q.shape
    _expect_rows(q, "q", T, H, d, q.dtype)
    _expect_pool(k_cache, "k_cache", plan.Hkv, d, q.dtype)
    _expect_pool(v_cache, "v_cache", plan.Hkv, d, q.dtype)
    if v_cache.shape[:2] != k_cache.shape[:2] or k_cache.shape[1] != plan.page:
        raise ValueError("k_cache and v_cache must have the same pages, of the plan's size")
    _expect_table(block_table, plan.B)
    if block_table.shape[1] != plan.max_pages:
        raise ValueError("block_table must be as wide as the plan's max_pages")
    _expect(out, "out", q.dtype, (T, H, d), optional=True)
    _expect(lse, "lse", torch.float32, (T, H), optional=True)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if tree_mask is not None:
        _expect(tree_mask, "tree_mask", torch.int64, (T,) + tuple(tree_mask.shape[1:2]))
    raise ValueError("attn_paged: unsupported tensors")


def attn_paged(q, k_cache, v_cache, block_table, plan, scale=None, out=None, lse=None,
               with_lse=True, workspace=None, tree_mask=None):
    """rf_attn_paged, or rf_attn_paged_tree with a tree_mask int64 [T, words] (bit j
    of a token's words: it sees the sequence's new token j; ``tree_mask`` makes
    it), which takes a plan made with causal=False: q [T, H, d] bf16 (a strided view of a fused projection
    fits), k_cache, v_cache [pages, page, Hkv, d] (any strides with d
    contiguous), block_table int32 [B, max_pages], plan a ``PagedPlan`` of the
    step -> (o [T, H, d], lse float32 [T, H] or None). d 64 or 128, pages of a
    multiple of 8 tokens. Rows outside every sequence are left as they are
    (uninitialised without `out`). Without `workspace` each call takes a new one
    from torch's allocator; a loop keeps one (``attn_paged_workspace``)."""
    if workspace is None:
        workspace = attn_paged_workspace(q.shape[-1], q.device)
    if tree_mask is not None and plan.causal:
        raise ValueError("attn_paged: a tree_mask takes a plan made with causal=False")
    r = _serving().attn_paged(q, k_cache, v_cache, block_table, plan.buf, plan.B, plan.T, plan.H,
                              plan.Hkv, plan.page, plan.max_pages, scale, out, lse, with_lse,
                              workspace, tree_mask)
    if r.__class__ is tuple:
        return r
    if r is None:
        _refuse_attn(q, k_cache, v_cache, block_table, plan, out, lse, workspace, tree_mask)
    _check(r)


def draft_verify_workspace(B, S, device="cuda"):
    """A workspace for ``draft_verify`` of B sequences and up to S drafts."""
    n = int(lib().rf_draft_verify_workspace_bytes(int(B), int(S)))
    return torch.empty(max(1, n), dtype=torch.uint8, device=device)


def _refuse_verify(target, draft, tokens, u, expo, n_draft, temperature, workspace):
    _same_device(target, draft, tokens, u, expo, n_draft, temperature, workspace)
    if target.dim() != 3 or target.shape[1] < 2:
        raise ValueError("target must be [B, S + 1, V] with S >= 1")
    B, S, V = target.shape[0], target.shape[1] - 1, target.shape[2]
    _expect(target, "target", target.dtype, (B, S + 1, V))
    _expect(draft, "draft", target.dtype, (B, S, V), optional=True)
    _expect(tokens, "tokens", torch.int32, (B, S))
    _expect(u, "u", torch.float32, (B, S))
    _expect(expo, "expo", torch.float32, (B, V))
    _expect(n_draft, "n_draft", torch.int32, (B,), optional=True)
    _expect(temperature, "temperature", torch.float32, (B,), optional=True)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    raise ValueError("draft_verify: unsupported tensors")


def draft_verify(target, draft, tokens, u, expo, n_draft=None, temperature=None, workspace=None):
    """rf_draft_verify: target logits [B, S + 1, V], draft logits [B, S, V] (or
    None: drafts with certainty), tokens int32 [B, S], u float32 [B, S] in
    [0, 1), expo float32 [B, V] exponential variates (2^-126 to 2^32), n_draft
    int32 [B], temperature float32 [B] (0: greedy) -> (out int32 [B, S + 1],
    n_accepted int32 [B])."""
    r = _serving().draft_verify(target, draft, tokens, u, expo, n_draft, temperature, workspace)
    if r.__class__ is tuple:
        return r
    if r is None:
        _refuse_verify(target, draft, tokens, u, expo, n_draft, temperature, workspace)
    _check(r)


def _returned(r, refuse, *args):
    """What a native call returned; refuse(*args) names the fault of tensors that it
    did not accept."""
    if r is None:
        refuse(*args)
    if r.__class__ is not tuple:
        _check(r)
    return r


def _refuse_nodes(fn, nodes, cu_q, kv_len):
    _same_device(*nodes.values(), cu_q, kv_len)
    if kv_len.dim() != 1 or nodes["parent"].dim() != 1:
        raise ValueError("parent must be int32 [T] and kv_len int32 [B]")
    for name, t in nodes.items():
        _expect(t, name, torch.int32, (nodes["parent"].shape[0],))
    _expect(kv_len, "kv_len", torch.int32, kv_len.shape)
    _expect(cu_q, "cu_q", torch.int32, (kv_len.shape[0] + 1,))
    raise ValueError("%s: unsupported tensors" % fn)


def tree_mask(parent, cu_q, kv_len, words=1):
    """rf_tree_mask: parent int32 [T] (a node's parent within its sequence, before
    it; -1: a root), cu_q int32 [B + 1], kv_len int32 [B] (with the nodes) -> (mask
    int64 [T, words] for ``attn_paged``, pos int32 [T] for ``kv_append_paged``).
    Up to 64 * words nodes a sequence, words up to 16."""
    return _returned(_serving().tree_mask(parent, cu_q, kv_len, words), _refuse_nodes, "tree_mask",
                     {"parent": parent}, cu_q, kv_len)


def tree_accept(parent, tokens, sampled, cu_q, kv_len):
    """rf_tree_accept: the walk down each tree from node 0 along the tokens drawn at
    its nodes. parent, tokens, sampled int32 [T], cu_q int32 [B + 1], kv_len int32
    [B] (with the nodes) -> (path int32 [T]: the walk's nodes from row cu_q[b] on,
    then -1; out int32 [T]: the tokens drawn at them; n_path, base, new_len int32
    [B]). ``kv_compact_paged(k_cache, v_cache, block_table, path, cu_q, n_path,
    base)`` then leaves new_len tokens in the cache."""
    return _returned(_serving().tree_accept(parent, tokens, sampled, cu_q, kv_len), _refuse_nodes,
                     "tree_accept", {"parent": parent, "tokens": tokens, "sampled": sampled}, cu_q,
                     kv_len)


def _refuse_sample(logits, expo, temperature, top_k, top_p, min_p):
    _same_device(logits, expo, temperature, top_k, top_p, min_p)
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [B, V] with contiguous rows")
    _dt(logits)
    B, V = logits.shape
    _expect(expo, "expo", torch.float32, (B, V))
    _expect(temperature, "temperature", torch.float32, (B,), optional=True)
    _expect(top_k, "top_k", torch.int32, (B,), optional=True)
    _expect(top_p, "top_p", torch.float32, (B,), optional=True)
    _expect(min_p, "min_p", torch.float32, (B,), optional=True)
    raise ValueError("sample_rows: unsupported tensors")


def sample_rows(logits, expo, temperature=None, top_k=None, top_p=None, min_p=None):
    """rf_sample_rows: a token drawn from each row of logits [B, V] (float32 or bf16;
    rows may be strided), expo float32 [B, V] exponential variates (2^-126 to
    2^32), temperature float32 [B] (0: greedy), top_k int32 [B] (0: no limit), top_p
    float32 [B] (1: no limit), min_p float32 [B] (0: no limit) -> (token int32 [B],
    logprob float32 [B] under the distribution that is left)."""
    return _returned(_serving().sample_rows(logits, expo, temperature, top_k, top_p, min_p),
                     _refuse_sample, logits, expo, temperature, top_k, top_p, min_p)


def _refuse_pool(fn, k_cache, v_cache, block_table, ints):
    _same_device(k_cache, v_cache, block_table, *(t for t, _ in ints.values()))
    if k_cache.dim() not in (4, 5) or k_cache.shape != v_cache.shape or \
            k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must be pools [pages, page, Hkv, d] or "
                         "[layers, pages, page, Hkv, d] of one shape and type")
    _dt(k_cache)
    if k_cache.stride(-1) != 1 or v_cache.stride(-1) != 1:
        raise ValueError("the pools' last dimension must be contiguous")
    if block_table is not None:
        _expect_table(block_table, block_table.shape[0])
    for name, (t, shape) in ints.items():
        _expect(t, name, torch.int32, shape, optional=name in ("n_keep", "base"))
    raise ValueError("%s: unsupported tensors" % fn)


def kv_compact_paged(k_cache, v_cache, block_table, keep, cu_keep, n_keep=None, base=None):
    """rf_kv_compact_paged: kept tokens of a paged cache moved together, in place:
    row base[b] + keep[cu_keep[b] + i] to row base[b] + i, i < n_keep[b].

    k_cache, v_cache [pages, page, Hkv, d] or [layers, pages, page, Hkv, d] (any
    strides with d contiguous, bf16 or float32), block_table int32 [B, max_pages],
    keep int32 [N] ascending within each sequence, cu_keep int32 [B + 1], n_keep
    int32 [B] (None: all of the sequence's), base int32 [B] (None: 0)."""
    r = _serving().kv_compact_paged(k_cache, v_cache, block_table, keep, cu_keep, n_keep, base)
    if r is None:
        B = block_table.shape[0]
        _refuse_pool("kv_compact_paged", k_cache, v_cache, block_table,
                     {"keep": (keep, (keep.numel(),)), "cu_keep": (cu_keep, (B + 1,)),
                      "n_keep": (n_keep, (B,)), "base": (base, (B,))})
    _returned(r, None)


def kv_copy_pages(k_cache, v_cache, src, dst):
    """rf_kv_copy_pages: page src[i] copied to page dst[i] (int32 [n]; a pair with a
    negative number is skipped) in pools [pages, page, Hkv, d] or [layers, pages,
    page, Hkv, d] (any strides with d contiguous, bf16 or float32). No page may be
    the dst of one pair and in another one."""
    r = _serving().kv_copy_pages(k_cache, v_cache, src, dst)
    if r is None:
        n = src.numel()
        _refuse_pool("kv_copy_pages", k_cache, v_cache, None, {"src": (src, (n,)),
                                                              "dst": (dst, (n,))})
    _returned(r, None)


def _refuse_pages(fn, tables, refs, ints):
    _same_device(*(t for t, _ in tables), refs, *(t for t, _ in ints.values()))
    for t, n in tables:
        if t.dim() != 2 or t.shape[0] != n:
            raise ValueError("a block table must be int32 [%d, max_pages]" % n)
        _expect_table(t, n)
    if tables[0][0].shape[1] != tables[-1][0].shape[1]:
        raise ValueError("the block tables must be of one width")
    _expect(refs, "refs", torch.int32, (refs.numel(),))
    for name, (t, shape) in ints.items():
        _expect(t, name, torch.int32, shape,
                optional=name == "new_len" and fn == "pages_release")
    raise ValueError("%s: unsupported tensors" % fn)


def pages_fork(block_table, kv_len, src, out, refs, page_size):
    """rf_pages_fork: row i of ``out`` int32 [n, max_pages] becomes a copy of row
    src[i] of block_table int32 [B, max_pages], and each of its pages gets an owner
    more in refs int32 [num_pages] (a page without one is free: it stays so, and is
    reported) -> kv_len[src] int32 [n]. ``pages_grow`` gives
    the rows pages of their own before they are written to."""
    r = _serving().pages_fork(block_table, kv_len, src, out, refs, page_size)
    if r is None:
        B, n = kv_len.numel(), src.numel()
        _refuse_pages("pages_fork", [(block_table, B), (out, n)], refs,
                      {"kv_len": (kv_len, (B,)), "src": (src, (n,))})
    return _returned(r, None)[0]


def pages_grow(block_table, kv_len, new_len, refs, page_size):
    """rf_pages_grow: the pages that new_len int32 [n] tokens need where kv_len int32
    [n] are there, written into block_table int32 [n, max_pages] and refs int32
    [num_pages] -> (copy_src int32 [n], copy_dst int32 [n], left int32 [1]). A
    partly filled last page that has other owners is replaced: ``kv_copy_pages(
    k_cache, v_cache, copy_src, copy_dst)`` has to follow before the row is used.
    left: free pages that remain, or, below 0, that are missing; then nothing was
    changed. A row whose partly filled last page has no owner gets nothing and is
    reported."""
    r = _serving().pages_grow(block_table, kv_len, new_len, refs, page_size)
    if r is None:
        n = kv_len.numel()
        _refuse_pages("pages_grow", [(block_table, n)], refs,
                      {"kv_len": (kv_len, (n,)), "new_len": (new_len, (n,))})
    return _returned(r, None)


def pages_release(block_table, kv_len, refs, page_size, new_len=None):
    """rf_pages_release: each page of a row behind its new_len int32 [n] tokens (None:
    0) of kv_len int32 [n] loses an owner in refs int32 [num_pages]; pages without
    one are free. The table keeps its entries."""
    r = _serving().pages_release(block_table, kv_len, refs, page_size, new_len)
    if r is None:
        n = kv_len.numel()
        _refuse_pages("pages_release", [(block_table, n)], refs,
                      {"kv_len": (kv_len, (n,)), "new_len": (new_len, (n,))})
    _returned(r, None)


def set_debug_visited(buf):
    """Record visited tiles of later attn_fwd calls on this thread into a uint8
    CUDA tensor (None turns it off)."""
    if buf is None:
        _check(lib().rf_debug_set_visited(None, 0))
    else:
        _cuda(buf)
        _check(lib().rf_debug_set_visited(_ptr(buf), buf.numel()))


def inject_fault(site):
    """Test aid: later calls on this thread skip one step at ``site`` so that
    a bounded device wait runs out (rf_debug_inject_fault); 0 turns it off."""
    _check(lib().rf_debug_inject_fault(int(site)))


def device_status():
    """Synchronise the current stream; return the device status code (0 = none)
    and clear it. Raises RFError for a nonzero code."""
    code = ctypes.c_int(0)
    st = lib().rf_device_status(_stream(), ctypes.byref(code))
    if st != RF_OK:
        raise RFError(st, lib().rf_last_error().decode(errors="replace"))
    return code.value
