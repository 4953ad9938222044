"""Tile-scheduled GEMM for GB300 (sm_103a): Python binding of libtstgemm.so.

Every step of C = A x B runs in the library's CUDA kernels; this module only
marshals arguments into the C ABI declared in include/tstgemm.h (same names).
PyTorch is used for device memory and streams: tensors passed to gemm_run must
already live on the GPU.  If the library is missing, importing the binding
raises; there is no CPU or PyTorch fallback.
"""
from __future__ import annotations

import ctypes

from . import _capi
from ._capi import (TST_BF16, TST_E4M3, TST_E5M2, TST_E4M3_E5M2, TST_E5M2_E4M3,  # noqa: F401
                    TST_OUT_F32, TST_OUT_BF16, TST_OUT_E4M3, TST_OUT_INT8, TST_LAYOUT_A_ROW_B_NK,
                    TST_SCORE_SOFTMAX, TST_SCORE_SIGMOID,
                    TST_ACT_NONE, TST_ACT_RELU, TST_ACT_GELU, TST_ACT_SILU, TST_BIAS_NONE, TST_BIAS_COL,
                    TST_BIAS_ROW,
                    TST_MAP_LINEAR_NFAST, TST_MAP_LINEAR_MFAST, TST_MAP_GROUPED_M, TST_MAP_GROUPED_N,
                    TST_STATIC, TST_PERSISTENT, TST_STREAMK, TST_STREAMK_HYBRID, TST_HYTIS,
                    TST_DEBUG_TRACE, TST_DEBUG_FAULT_SKIP_LOAD, TST_DEBUG_FAULT_SKIP_LOCK, TST_DEBUG_ROLE_CYCLES,
                    TST_SK_DETERMINISTIC, TST_SK_ATOMIC, TST_SK_SEPARATE,
                    TST_OK, TST_ERR_INVALID_ARG, TST_ERR_UNSUPPORTED, TST_ERR_ALIGNMENT, TST_ERR_OOM,
                    TST_ERR_CUDA, TST_ERR_TIMEOUT, TST_ERR_DEVICE_CHECK, TST_ERR_NO_DEVICE,
                    TST_NOALLOC_SCRATCH_BYTES)

lib = _capi.load()

_DTYPES = {"bf16": TST_BF16, "e4m3": TST_E4M3, "e5m2": TST_E5M2, "e4m3_e5m2": TST_E4M3_E5M2,
           "e5m2_e4m3": TST_E5M2_E4M3}
_OUT = {"f32": TST_OUT_F32, "bf16": TST_OUT_BF16, "e4m3": TST_OUT_E4M3}
_ACT = {"none": TST_ACT_NONE, "relu": TST_ACT_RELU, "gelu": TST_ACT_GELU, "silu": TST_ACT_SILU}
_BIAS = {"none": TST_BIAS_NONE, "col": TST_BIAS_COL, "row": TST_BIAS_ROW}
_MAPS = {"linear_nfast": TST_MAP_LINEAR_NFAST, "linear_mfast": TST_MAP_LINEAR_MFAST,
         "grouped_m": TST_MAP_GROUPED_M, "grouped_n": TST_MAP_GROUPED_N,
         "block_2d": _capi.TST_MAP_BLOCK_2D, "morton": _capi.TST_MAP_MORTON}
_FIXUP = {"deterministic": TST_SK_DETERMINISTIC, "atomic": TST_SK_ATOMIC, "separate": TST_SK_SEPARATE,
          "tma": _capi.TST_SK_TMA}
_L2 = {"none": _capi.TST_L2_NONE, "keep_a": _capi.TST_L2_KEEP_A, "keep_b": _capi.TST_L2_KEEP_B,
       "auto": _capi.TST_L2_AUTO}
_BOXES = {"auto": _capi.TST_BOXES_AUTO, "2d": _capi.TST_BOXES_2D, "3d": _capi.TST_BOXES_3D}
_STORE = {"auto": _capi.TST_STORE_AUTO, "direct": _capi.TST_STORE_DIRECT, "tma": _capi.TST_STORE_TMA}
_SCHED = {"static": TST_STATIC, "persistent": TST_PERSISTENT, "streamk": TST_STREAMK,
          "streamk_hybrid": TST_STREAMK_HYBRID, "hytis": TST_HYTIS}


class TstError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gemm_status_string(status)}")


def gemm_status_string(status: int) -> str:
    return lib.gemm_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != TST_OK:
        raise TstError(status, where)


def _enum(table, v, what):
    if isinstance(v, str):
        if v not in table:
            raise ValueError(f"unknown {what} {v!r}; expected one of {sorted(table)}")
        return table[v]
    return int(v)


class Plan:
    """Owns a tst_plan*; destroyed with the object (or explicitly via destroy())."""

    def __init__(self, handle: int, info):
        self.handle = handle
        self.info = info

    def destroy(self):
        if self.handle:
            _check(lib.gemm_plan_destroy(ctypes.c_void_p(self.handle)), "gemm_plan_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    @property
    def _h(self):
        if not self.handle:
            raise ValueError("plan was destroyed")
        return ctypes.c_void_p(self.handle)


def gemm_plan_create(M: int, N: int, K: int, dtype="bf16", mapping=("linear_nfast", 1), schedule="static",
                     out_dtype="f32", alpha: float = 1.0, has_bias: bool = False, relu: bool = False,
                     use_scales: bool = False, bn: int = 0, num_ctas: int = 0, sk_forward: bool = False,
                     host_only: bool = False, num_sms: int = 0, timeout_ns: int = 0, cta_group: int = 0,
                     stages: int = 0, bk: int = 0, sk_groups: int = 0, sk_fixup="deterministic", pdl: bool = False,
                     l2_hint="none", tma_boxes="auto", beta: float = 0.0, has_c: bool = False, c_dtype="f32",
                     bias_mode=None, activation=None,
                     row_scale: bool = False, col_scale: bool = False, d_scale: bool = False,
                     amax: bool = False, aux: bool = False, aux_dtype="f32", block_scale: bool = False,
                     cluster_n: int = 0, epilogue_store="auto", l2_prefetch: int = 0, ab_block=None) -> Plan:
    """Plan C = epilogue(A x B).  The basic epilogue is alpha, a column bias (has_bias),
    ReLU and the tensor-wise scales; any of beta/has_c, bias_mode='row', activation
    'gelu'/'silu', row_scale, col_scale, d_scale, amax, aux, block_scale or out_dtype 'e4m3'
    selects the extended one (gemm_plan_create_epi).  block_scale: an e4m3 D with one
    power-of-two scale per 32 x 32 tile, whose exponents gemm_run writes to block_exp.
    ab_block=(br, bk): block-scaled FP8 operands, one scale per br x bk tile of A and of B;
    (br, bk, br_b): B's tiles of br_b rows (gemm_run's a_block_scales, ceil(M / br) x
    ceil(K / bk), and b_block_scales, ceil(N / br_b) x ceil(K / bk), FP32 row-major)."""
    kind, group = mapping if isinstance(mapping, (tuple, list)) else (mapping, 1)
    m = _capi.tst_mapping(_enum(_MAPS, kind, "mapping"), int(group))
    opts = _capi.tst_plan_options(int(bn), int(num_ctas), int(bool(sk_forward)), int(bool(host_only)),
                                  int(num_sms), int(cta_group), int(timeout_ns), int(stages), int(bk),
                                  int(sk_groups), _enum(_FIXUP, sk_fixup, "sk_fixup"), int(bool(pdl)),
                                  _enum(_L2, l2_hint, "l2_hint"),
                                  _enum(_BOXES, tma_boxes, "tma_boxes"), int(cluster_n),
                                  _enum(_STORE, epilogue_store, "epilogue_store"), int(l2_prefetch))
    bmode = _enum(_BIAS, bias_mode, "bias_mode") if bias_mode is not None else \
        (TST_BIAS_COL if has_bias else TST_BIAS_NONE)
    act = _enum(_ACT, activation, "activation") if activation is not None else \
        (TST_ACT_RELU if relu else TST_ACT_NONE)
    extended = bool(has_c or bmode == TST_BIAS_ROW or act in (TST_ACT_GELU, TST_ACT_SILU) or row_scale or
                    col_scale or d_scale or amax or aux or block_scale)
    h = ctypes.c_void_p()
    br, bk, br_b = (tuple(ab_block) + (0,))[:3] if ab_block is not None else (0, 0, 0)
    if extended or ab_block is not None:
        epi = _capi.tst_epilogue_ex(_enum(_OUT, out_dtype, "out_dtype"), float(alpha), float(beta),
                                    int(bool(has_c)), _enum(_OUT, c_dtype, "c_dtype"), bmode, act,
                                    int(bool(use_scales)), int(bool(row_scale)), int(bool(col_scale)),
                                    int(bool(d_scale)), int(bool(amax)), int(bool(aux)),
                                    _enum(_OUT, aux_dtype, "aux_dtype"), int(bool(block_scale)), int(br), int(bk),
                                    int(br_b))
        _check(lib.gemm_plan_create_epi(ctypes.byref(h), int(M), int(N), int(K), _enum(_DTYPES, dtype, "dtype"),
                                        TST_LAYOUT_A_ROW_B_NK, m, _enum(_SCHED, schedule, "schedule"),
                                        ctypes.byref(epi), ctypes.byref(opts)), "gemm_plan_create_epi")
    else:
        epi = _capi.tst_epilogue(_enum(_OUT, out_dtype, "out_dtype"), float(alpha), int(bmode == TST_BIAS_COL),
                                 int(act == TST_ACT_RELU), int(bool(use_scales)))
        _check(lib.gemm_plan_create_ex(ctypes.byref(h), int(M), int(N), int(K), _enum(_DTYPES, dtype, "dtype"),
                                       TST_LAYOUT_A_ROW_B_NK, m, _enum(_SCHED, schedule, "schedule"),
                                       ctypes.byref(epi), ctypes.byref(opts)), "gemm_plan_create")
    info = _capi.tst_plan_info()
    _check(lib.gemm_plan_get_info(h, ctypes.byref(info)), "gemm_plan_get_info")
    return Plan(h.value, info)


def gemm_grouped_plan_create(groups: int, M: int, N: int, K: int, dtype="bf16", mapping=("grouped_m", 8),
                             out_dtype="bf16", alpha: float = 1.0, beta: float = 0.0, has_c: bool = False,
                             c_dtype="f32", has_bias: bool = False, bias_mode=None, relu: bool = False,
                             activation=None, use_scales: bool = False, row_scale: bool = False,
                             col_scale: bool = False, d_scale: bool = False, amax: bool = False, aux: bool = False,
                             aux_dtype="f32", bn: int = 0, num_ctas: int = 0, host_only: bool = False,
                             num_sms: int = 0, timeout_ns: int = 0, cta_group: int = 0, stages: int = 0,
                             bk: int = 0, pdl: bool = False, l2_hint="none", tma_boxes="auto",
                             block_scale: bool = False, ab_block=None) -> Plan:
    """Plan `groups` GEMMs sharing N and K in one persistent launch: A holds the groups'
    rows one after another (at most M in all), B one N x K matrix per group; the row
    counts are given to gemm_grouped_run as a device int32 array.  ab_block as in
    gemm_plan_create: A's scales are ceil(M / br) x ceil(K / bk), B's groups x
    ceil(N / br_b) x ceil(K / bk)."""
    kind, group = mapping if isinstance(mapping, (tuple, list)) else (mapping, 1)
    m = _capi.tst_mapping(_enum(_MAPS, kind, "mapping"), int(group))
    opts = _capi.tst_plan_options(int(bn), int(num_ctas), 0, int(bool(host_only)), int(num_sms), int(cta_group),
                                  int(timeout_ns), int(stages), int(bk), 0, 0, int(bool(pdl)),
                                  _enum(_L2, l2_hint, "l2_hint"),
                                  _enum(_BOXES, tma_boxes, "tma_boxes"))
    bmode = _enum(_BIAS, bias_mode, "bias_mode") if bias_mode is not None else \
        (TST_BIAS_COL if has_bias else TST_BIAS_NONE)
    act = _enum(_ACT, activation, "activation") if activation is not None else \
        (TST_ACT_RELU if relu else TST_ACT_NONE)
    br, ab_k, br_b = (tuple(ab_block) + (0,))[:3] if ab_block is not None else (0, 0, 0)
    epi = _capi.tst_epilogue_ex(_enum(_OUT, out_dtype, "out_dtype"), float(alpha), float(beta), int(bool(has_c)),
                                _enum(_OUT, c_dtype, "c_dtype"), bmode, act, int(bool(use_scales)),
                                int(bool(row_scale)), int(bool(col_scale)), int(bool(d_scale)), int(bool(amax)),
                                int(bool(aux)), _enum(_OUT, aux_dtype, "aux_dtype"), int(bool(block_scale)), int(br),
                                int(ab_k), int(br_b))
    h = ctypes.c_void_p()
    _check(lib.gemm_grouped_plan_create(ctypes.byref(h), int(groups), int(M), int(N), int(K),
                                        _enum(_DTYPES, dtype, "dtype"), TST_LAYOUT_A_ROW_B_NK, m, ctypes.byref(epi),
                                        ctypes.byref(opts)), "gemm_grouped_plan_create")
    info = _capi.tst_plan_info()
    _check(lib.gemm_plan_get_info(h, ctypes.byref(info)), "gemm_plan_get_info")
    return Plan(h.value, info)


def gemm_grouped_run(plan: Plan, group_rows, A, B, D, bias=None, scales=None, c=None, row_scale=None,
                     col_scale=None, d_scale=None, amax=None, aux=None, stream=None, a_block_scales=None,
                     b_block_scales=None):
    """Enqueue a grouped GEMM; group_rows is a CUDA int32 tensor of the groups' row counts."""
    if hasattr(group_rows, "dtype") and str(group_rows.dtype) != "torch.int32":
        raise ValueError("group_rows must be an int32 CUDA tensor")
    args = _capi.tst_epilogue_args(_ptr(c), _ptr(bias), _ptr(scales), _ptr(row_scale), _ptr(col_scale),
                                   _ptr(d_scale), _ptr(amax), _ptr(aux), None, _ptr(a_block_scales),
                                   _ptr(b_block_scales))
    _check(lib.gemm_grouped_run(plan._h, _ptr(group_rows), _ptr(A), _ptr(B), _ptr(D), ctypes.byref(args),
                                _stream(stream)), "gemm_grouped_run")


def gemm_grouped_array_plan_create(shapes, dtype="bf16", mapping=("grouped_m", 8), out_dtype="bf16",
                                   alpha: float = 1.0, relu: bool = False, activation=None, use_scales: bool = False,
                                   d_scale: bool = False, amax: bool = False, bn: int = 0, num_ctas: int = 0,
                                   host_only: bool = False, num_sms: int = 0, timeout_ns: int = 0, cta_group: int = 0,
                                   stages: int = 0, bk: int = 0, pdl: bool = False, l2_hint="none",
                                   tma_boxes="auto") -> Plan:
    """Plan a grouped GEMM over groups of different shapes: `shapes` is a list of
    (M_g, N_g, K_g); each group has its own A, B and D (gemm_grouped_array_run)."""
    G = len(shapes)
    Ms = (ctypes.c_int64 * max(G, 1))(*[int(m) for m, _, _ in shapes])
    Ns = (ctypes.c_int64 * max(G, 1))(*[int(n) for _, n, _ in shapes])
    Ks = (ctypes.c_int64 * max(G, 1))(*[int(k) for _, _, k in shapes])
    kind, group = mapping if isinstance(mapping, (tuple, list)) else (mapping, 1)
    m = _capi.tst_mapping(_enum(_MAPS, kind, "mapping"), int(group))
    opts = _capi.tst_plan_options(int(bn), int(num_ctas), 0, int(bool(host_only)), int(num_sms), int(cta_group),
                                  int(timeout_ns), int(stages), int(bk), 0, 0, int(bool(pdl)),
                                  _enum(_L2, l2_hint, "l2_hint"),
                                  _enum(_BOXES, tma_boxes, "tma_boxes"))
    act = _enum(_ACT, activation, "activation") if activation is not None else \
        (TST_ACT_RELU if relu else TST_ACT_NONE)
    epi = _capi.tst_epilogue_ex(_enum(_OUT, out_dtype, "out_dtype"), float(alpha), 0.0, 0, 0, TST_BIAS_NONE, act,
                                int(bool(use_scales)), 0, 0, int(bool(d_scale)), int(bool(amax)), 0, 0)
    h = ctypes.c_void_p()
    _check(lib.gemm_grouped_array_plan_create(ctypes.byref(h), G, Ms, Ns, Ks, _enum(_DTYPES, dtype, "dtype"),
                                              TST_LAYOUT_A_ROW_B_NK, m, ctypes.byref(epi), ctypes.byref(opts)),
           "gemm_grouped_array_plan_create")
    info = _capi.tst_plan_info()
    _check(lib.gemm_plan_get_info(h, ctypes.byref(info)), "gemm_plan_get_info")
    return Plan(h.value, info)


def gemm_grouped_array_run(plan: Plan, A, B, D, scales=None, d_scale=None, amax=None, stream=None):
    """Enqueue a grouped GEMM of different shapes; A, B, D are lists of CUDA tensors (or None
    for groups without rows or columns)."""
    def arr(xs):
        return (ctypes.c_void_p * max(len(xs), 1))(*[_ptr(x) for x in xs])
    args = _capi.tst_epilogue_args(None, None, _ptr(scales), None, None, _ptr(d_scale), _ptr(amax), None)
    _check(lib.gemm_grouped_array_run(plan._h, arr(A), arr(B), arr(D), ctypes.byref(args), _stream(stream)),
           "gemm_grouped_array_run")


def gemm_grouped_work_items(plan: Plan, group_rows, cta: int):
    """[(tile, m, n, k_begin, k_count, flags), ...] of one CTA of a grouped plan for the given
    host row counts, in device order."""
    rows = (ctypes.c_int32 * max(len(group_rows), 1))(*[int(r) for r in group_rows])
    count = ctypes.c_int64()
    _check(lib.gemm_grouped_work_items(plan._h, rows, int(cta), None, 0, ctypes.byref(count)),
           "gemm_grouped_work_items")
    arr = (_capi.tst_work_item * max(count.value, 1))()
    _check(lib.gemm_grouped_work_items(plan._h, rows, int(cta), arr, count.value, ctypes.byref(count)),
           "gemm_grouped_work_items")
    return [(w.tile, w.m, w.n, w.k_begin, w.k_count, w.flags) for w in arr[:count.value]]


def gemm_plan_get_info(plan: Plan):
    info = _capi.tst_plan_info()
    _check(lib.gemm_plan_get_info(plan._h, ctypes.byref(info)), "gemm_plan_get_info")
    return info


def gemm_tile_map(plan: Plan, i: int):
    m, n = ctypes.c_int32(), ctypes.c_int32()
    _check(lib.gemm_tile_map(plan._h, int(i), ctypes.byref(m), ctypes.byref(n)), "gemm_tile_map")
    return m.value, n.value


def gemm_work_items(plan: Plan, cta: int):
    """[(tile, m, n, k_begin, k_count, flags), ...] of one CTA, in device order."""
    count = ctypes.c_int64()
    _check(lib.gemm_work_items(plan._h, int(cta), None, 0, ctypes.byref(count)), "gemm_work_items")
    arr = (_capi.tst_work_item * max(count.value, 1))()
    _check(lib.gemm_work_items(plan._h, int(cta), arr, count.value, ctypes.byref(count)), "gemm_work_items")
    return [(w.tile, w.m, w.n, w.k_begin, w.k_count, w.flags) for w in arr[:count.value]]


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if not x.is_cuda:
            raise ValueError("tensors passed to the GEMM must be CUDA tensors (no host fallback)")
        if not x.is_contiguous():
            raise ValueError("tensors passed to the GEMM must be contiguous")
        return x.data_ptr()
    raise TypeError(f"expected a CUDA tensor or a device pointer, got {type(x)}")


_torch = None   # torch, once a call has needed its current stream


def _stream(stream):
    if stream is None:
        # the raw handle: making torch's Stream object costs 2.7 us a call, as much as a kernel launch
        global _torch
        if _torch is None:
            import torch
            _torch = torch
        return _torch._C._cuda_getCurrentRawStream(_torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def gemm_run(plan: Plan, A, B, C, bias=None, scales=None, stream=None, c=None, row_scale=None, col_scale=None,
             d_scale=None, amax=None, aux=None, block_exp=None, a_block_scales=None, b_block_scales=None):
    """Enqueue C = epilogue(A x B) on `stream` (default: torch's current stream).  The
    extended epilogue's operands (c: the addend of beta * C; row_scale, col_scale,
    d_scale, amax, aux; block_exp, int32 [ceil(M/32), ceil(N/32)] written by a
    block-scaled e4m3 D) go through gemm_run_epi."""
    if all(x is None for x in (c, row_scale, col_scale, d_scale, amax, aux, block_exp, a_block_scales,
                               b_block_scales)):
        _check(lib.gemm_run(plan._h, _ptr(A), _ptr(B), _ptr(C), _ptr(bias), _ptr(scales), _stream(stream)),
               "gemm_run")
        return
    args = _capi.tst_epilogue_args(_ptr(c), _ptr(bias), _ptr(scales), _ptr(row_scale), _ptr(col_scale),
                                   _ptr(d_scale), _ptr(amax), _ptr(aux), _ptr(block_exp), _ptr(a_block_scales),
                                   _ptr(b_block_scales))
    _check(lib.gemm_run_epi(plan._h, _ptr(A), _ptr(B), _ptr(C), ctypes.byref(args), _stream(stream)),
           "gemm_run_epi")


def _host_ptr(x):
    if not hasattr(x, "data_ptr") or x.is_cuda:
        raise ValueError("gemm_run_host takes host (CPU) tensors; pinned ones overlap the copies")
    if not x.is_contiguous():
        raise ValueError("tensors passed to the GEMM must be contiguous")
    return x.data_ptr()


def gemm_run_host(plan: Plan, A, B, D, panels: int = 0, stream=None, bias=None, scales=None, c=None,
                  row_scale=None, col_scale=None, d_scale=None, amax=None, aux=None, block_exp=None,
                  a_block_scales=None, b_block_scales=None):
    """End to end on host tensors A, B, D (CPU, contiguous; pinned for the copies to
    overlap the computation): row panels of A stream in, each panel's GEMM runs as soon as
    it has landed, its rows of D stream back.  Epilogue operands are CUDA tensors."""
    args = _capi.tst_epilogue_args(_ptr(c), _ptr(bias), _ptr(scales), _ptr(row_scale), _ptr(col_scale),
                                   _ptr(d_scale), _ptr(amax), _ptr(aux), _ptr(block_exp), _ptr(a_block_scales),
                                   _ptr(b_block_scales))
    _check(lib.gemm_run_host(plan._h, _host_ptr(A), _host_ptr(B), _host_ptr(D), ctypes.byref(args), int(panels),
                             _stream(stream)), "gemm_run_host")


def gemm_status_query(plan: Plan):
    """(status, raw status word) of the last run; synchronises that run's stream."""
    word = ctypes.c_uint32()
    st = lib.gemm_status_query(plan._h, ctypes.byref(word))
    return st, word.value


def gemm_plan_set_debug(plan: Plan, flags: int = 0, trace=None, cap: int = 0, timeout_ns: int = 0):
    _check(lib.gemm_plan_set_debug(plan._h, int(flags), _ptr(trace), int(cap), int(timeout_ns)),
           "gemm_plan_set_debug")


def gemm_plan_destroy(plan: Plan):
    plan.destroy()


def gemm_streamk_noalloc(M: int, N: int, K: int, A, B, C, dtype="bf16", mapping=("linear_nfast", 1),
                         schedule="streamk", out_dtype="f32", alpha: float = 1.0, has_bias: bool = False,
                         relu: bool = False, use_scales: bool = False, bn: int = 0, num_ctas: int = 0,
                         bias=None, scales=None, device_status=None, stream=None):
    """Stream-K GEMM that allocates no device memory: its partial tiles and locks live in the
    library's fixed scratch array (TST_NOALLOC_SCRATCH_BYTES).  For callers that cannot call
    cudaMalloc.  Calls that may overlap on the GPU share that array and must be serialised."""
    kind, group = mapping if isinstance(mapping, (tuple, list)) else (mapping, 1)
    m = _capi.tst_mapping(_enum(_MAPS, kind, "mapping"), int(group))
    epi = _capi.tst_epilogue(_enum(_OUT, out_dtype, "out_dtype"), float(alpha), int(bool(has_bias)),
                             int(bool(relu)), int(bool(use_scales)))
    _check(lib.gemm_streamk_noalloc(int(M), int(N), int(K), _enum(_DTYPES, dtype, "dtype"), m,
                                    _enum(_SCHED, schedule, "schedule"), ctypes.byref(epi), int(bn), int(num_ctas),
                                    _ptr(A), _ptr(B), _ptr(C), _ptr(bias), _ptr(scales), _ptr(device_status),
                                    _stream(stream)), "gemm_streamk_noalloc")


# ---------------------------------------------------------------- 8-bit integers
class Int8Plan:
    """Owns a tst_int8_plan*; destroyed with the object (or explicitly via destroy())."""

    def __init__(self, handle: int, info, out_dtype: int, has_bias: bool):
        self.handle = handle
        self.info = info
        self.M, self.N, self.K, self.groups = info.M, info.N, info.K, info.groups
        self.out_dtype, self.has_bias = out_dtype, has_bias

    def destroy(self):
        if self.handle:
            _check(lib.gemm_int8_plan_destroy(ctypes.c_void_p(self.handle)), "gemm_int8_plan_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    @property
    def _h(self):
        if not self.handle:
            raise ValueError("plan was destroyed")
        return self.handle


def gemm_int8_plan_create(M: int, N: int, K: int, groups: int = 0, out_dtype="bf16", has_bias: bool = False,
                          relu: bool = False, host_only: bool = False, num_sms: int = 0, tile_rows: int = 0,
                          timeout_ns: int = 0) -> Int8Plan:
    """Plan D = relu?(row_scale * col_scale * (A x B) + bias) of int8 A (M x K) and B (N x K), the integer
    sum exact.  groups > 0: that many GEMMs sharing N and K, A and D holding the groups' rows one after
    another (at most M), B, col_scale and bias one part per group.  tile_rows: the tile's rows of A (0: the plan
    chooses; the results are the same)."""
    out = _enum(_OUT, out_dtype, "out_dtype")
    opts = _capi.tst_int8_options(int(groups), out, int(bool(has_bias)), int(bool(relu)), int(bool(host_only)),
                                  int(num_sms), int(tile_rows), int(timeout_ns))
    h = ctypes.c_void_p()
    _check(lib.gemm_int8_plan_create(ctypes.byref(h), int(M), int(N), int(K), ctypes.byref(opts)),
           "gemm_int8_plan_create")
    info = _capi.tst_int8_plan_info()
    _check(lib.gemm_int8_plan_get_info(h, ctypes.byref(info)), "gemm_int8_plan_get_info")
    return Int8Plan(h.value, info, out, bool(has_bias))


def gemm_int8_run(plan: Int8Plan, A, B, D, row_scale, col_scale, bias=None, group_rows=None, stream=None):
    """Enqueue the int8 GEMM: A M x K, B N x K (grouped: groups * N rows, or groups x N x K), D M x N of the
    plan's type, row_scale FP32[M], col_scale and bias FP32[N] (grouped: [groups * N]), group_rows int32[groups]."""
    parts = max(plan.groups, 1) * plan.N
    if (plan.groups > 0) != (group_rows is not None):
        raise ValueError("a grouped plan needs group_rows, and no other plan takes them")
    if plan.has_bias and bias is None:
        raise ValueError("the plan needs a bias")
    _check(lib.gemm_int8_run(plan._h, None if group_rows is None else _array(group_rows, "group_rows", "int32", plan.groups),
                             _array(A, "A", "int8", plan.M * plan.K), _array(B, "B", "int8", parts * plan.K),
                             _array(D, "D", "float32" if plan.out_dtype == TST_OUT_F32 else "bfloat16", plan.M * plan.N),
                             _array(row_scale, "row_scale", "float32", plan.M),
                             _array(col_scale, "col_scale", "float32", parts),
                             _array(bias, "bias", "float32", parts) if plan.has_bias else None, _stream(stream)),
           "gemm_int8_run")


def gemm_int8_status_query(plan: Int8Plan) -> int:
    """Status recorded by the runs since the last query (TST_ERR_DEVICE_CHECK: the groups' rows add up to more
    than M); synchronises the last run's stream."""
    return lib.gemm_int8_status_query(plan._h)


def gemm_int8_plan_destroy(plan: Int8Plan):
    plan.destroy()


# ---------------------------------------------------------------- mixture of experts
class MoePlan:
    """Owns a tst_moe_plan*; destroyed with the object (or explicitly via destroy())."""

    def __init__(self, handle: int, max_tokens: int, experts: int, top_k: int, scored: bool = False):
        self.handle = handle
        self.max_tokens, self.experts, self.top_k = max_tokens, experts, top_k
        self.scored = scored   # routes by scores (moe_plan_create's score)

    def destroy(self):
        if self.handle:
            _check(lib.moe_plan_destroy(ctypes.c_void_p(self.handle)), "moe_plan_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    @property
    def _h(self):
        if not self.handle:
            raise ValueError("plan was destroyed")
        return self.handle


_SCORE = {"softmax": TST_SCORE_SOFTMAX, "sigmoid": TST_SCORE_SIGMOID}


def moe_plan_create(max_tokens: int, experts: int, top_k: int, normalize: bool = True, balance_coef: float = 0.01,
                    host_only: bool = False, score=None, groups: int = 1, top_groups=None, group_best: int = 1,
                    weight_scale: float = 1.0) -> MoePlan:
    """Plan the calls around a grouped GEMM whose groups are experts: up to max_tokens tokens per
    call, each sent to top_k of `experts` experts.  normalize: a token's weights are divided by
    their sum; balance_coef: factor of the balance loss.

    score ('softmax' or 'sigmoid'): moe_route chooses by scores and takes a bias per expert.  Of `groups`
    groups of adjacent experts each token uses the top_groups (None: all) whose group_best (1 or 2)
    largest values have the largest sum; the weights, scores without the bias, are multiplied by
    weight_scale."""
    h = ctypes.c_void_p()
    if score is None:
        if groups != 1 or top_groups not in (None, 1) or group_best != 1 or weight_scale != 1.0:
            raise ValueError("groups, top_groups, group_best and weight_scale need a score, 'softmax' or 'sigmoid'")
        opts = _capi.tst_moe_options(int(bool(normalize)), float(balance_coef), int(bool(host_only)))
        _check(lib.moe_plan_create(ctypes.byref(h), int(max_tokens), int(experts), int(top_k), ctypes.byref(opts)),
               "moe_plan_create")
    else:
        opts = _capi.tst_moe_score_options(_enum(_SCORE, score, "score"), int(groups),
                                           int(groups if top_groups is None else top_groups), int(group_best),
                                           int(bool(normalize)), float(weight_scale), float(balance_coef),
                                           int(bool(host_only)))
        _check(lib.moe_plan_create_scored(ctypes.byref(h), int(max_tokens), int(experts), int(top_k),
                                          ctypes.byref(opts)), "moe_plan_create_scored")
    return MoePlan(h.value, int(max_tokens), int(experts), int(top_k), score is not None)


def moe_plan_get_info(plan: MoePlan):
    info = _capi.tst_moe_plan_info()
    _check(lib.moe_plan_get_info(plan._h, ctypes.byref(info)), "moe_plan_get_info")
    return info


def moe_plan_destroy(plan: MoePlan):
    plan.destroy()


def moe_status_query(plan: MoePlan) -> int:
    """TST_OK, or TST_ERR_DEVICE_CHECK when a run since the last query met a row index outside its
    matrix; synchronises the last run's stream."""
    return lib.moe_status_query(plan._h)


_OUT_OF = {"torch.float32": TST_OUT_F32, "torch.bfloat16": TST_OUT_BF16, "torch.float8_e4m3fn": TST_OUT_E4M3,
           "torch.uint8": TST_OUT_E4M3, "torch.int8": TST_OUT_INT8}
_out_cache = {}   # torch dtype -> tst_out_dtype, so that a call does not print a dtype's name each time


def _out_of(x, what: str) -> int:
    code = _out_cache.get(x.dtype)
    if code is None:
        code = _OUT_OF.get(str(x.dtype))
        if code is None:
            raise ValueError(f"{what}: {x.dtype} is not one of {sorted(_OUT_OF)}")
        _out_cache[x.dtype] = code
    return code


def _matrix(x, what: str, rows=None, cols=None):
    """(pointer, rows, columns, row stride) of a 2-D CUDA tensor whose columns are adjacent."""
    shape = x.shape
    if not x.is_cuda or len(shape) != 2:
        raise ValueError(f"{what} must be a CUDA tensor of two dimensions (no host fallback)")
    m, n = shape
    if (rows is not None and m != rows) or (cols is not None and n != cols):
        raise ValueError(f"{what} must be {'any' if rows is None else rows} x {'any' if cols is None else cols}, "
                         f"not {m} x {n}")
    sr, sc = x.stride()
    if (sc != 1 and n > 1) or (sr < n and m > 1):
        raise ValueError(f"{what}: a row's elements must be adjacent and its rows apart (strides {sr}, {sc})")
    return x.data_ptr(), m, n, (sr if m > 1 else n)


_type_names = {}   # torch dtype -> its name without "torch."


def _array(x, what: str, dtype: str, size: int):
    """Pointer of a contiguous CUDA tensor of `size` elements."""
    if _type_names.get(x.dtype) != dtype:
        name = _type_names[x.dtype] = str(x.dtype)[6:]
        if name != dtype:
            raise ValueError(f"{what} must hold {dtype}, not {name}")
    if x.numel() != size or not x.is_contiguous() or not x.is_cuda:
        raise ValueError(f"{what} must be a contiguous CUDA tensor of {size} elements (no host fallback)")
    return x.data_ptr()


def _token_mask(mask, tokens: int):
    if mask is None:
        return None
    if not mask.is_cuda or mask.numel() != tokens or mask.element_size() != 1 or not mask.is_contiguous():
        raise ValueError(f"mask must be a contiguous CUDA tensor of {tokens} bytes (uint8 or bool)")
    return mask.data_ptr()


def moe_route(plan: MoePlan, logits, expert, weight, row, counts, totals, loss, mask=None, stream=None, bias=None):
    """Route each row of logits (tokens x experts, FP32 or BF16) to its top_k experts.  Written:
    expert, row (int32) and weight (FP32), tokens x top_k; counts (int32, per expert: the grouped
    GEMM's group_rows); totals (int32 {rows in all, tokens routed}); loss (FP32, one element).  mask:
    one byte per token, 0 for a token that is not routed.  bias (plans with a score): FP32 per expert,
    added to the scores for the choice alone."""
    ptr, t, _, ld = _matrix(logits, "logits", cols=plan.experts)
    n = t * plan.top_k
    args = (_array(expert, "expert", "int32", n), _array(weight, "weight", "float32", n), _array(row, "row", "int32", n),
            _array(counts, "counts", "int32", plan.experts), _array(totals, "totals", "int32", 2),
            _array(loss, "loss", "float32", 1), _stream(stream))
    if plan.scored:
        b = None if bias is None else _array(bias, "bias", "float32", plan.experts)
        _check(lib.moe_route_scored(plan._h, t, ptr, _out_of(logits, "logits"), ld, _token_mask(mask, t), b, *args),
               "moe_route_scored")
        return
    if bias is not None:
        raise ValueError("a bias needs a plan with a score")
    _check(lib.moe_route(plan._h, t, ptr, _out_of(logits, "logits"), ld, _token_mask(mask, t), *args), "moe_route")


def moe_route_backward(plan: MoePlan, logits, expert, counts, totals, d_logits, d_weight=None, d_loss=None, mask=None,
                       stream=None):
    """The logits' gradient (d_logits, of the logits' type) from those of the weights (d_weight) and of
    the loss (d_loss, one FP32 element on the device); the other arguments as moe_route had and gave
    them."""
    ptr, t, _, ld = _matrix(logits, "logits", cols=plan.experts)
    dptr, _, _, d_ld = _matrix(d_logits, "d_logits", t, plan.experts)
    if d_logits.dtype != logits.dtype:
        raise ValueError(f"d_logits must have the logits' type, {logits.dtype}")
    n = t * plan.top_k
    call, name = (lib.moe_route_scored_backward, "moe_route_scored_backward") if plan.scored else \
        (lib.moe_route_backward, "moe_route_backward")
    _check(call(plan._h, t, ptr, _out_of(logits, "logits"), ld, _token_mask(mask, t),
                _array(expert, "expert", "int32", n), _array(counts, "counts", "int32", plan.experts),
                _array(totals, "totals", "int32", 2),
                None if d_weight is None else _array(d_weight, "d_weight", "float32", n),
                None if d_loss is None else _array(d_loss, "d_loss", "float32", 1), dptr, d_ld, _stream(stream)), name)


def _whole_rows(x, what: str, cols=None):
    """(pointer, rows, columns) of a contiguous 2-D CUDA tensor."""
    shape = x.shape
    if not x.is_cuda or len(shape) != 2 or not x.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor of two dimensions (no host fallback)")
    m, n = shape
    if cols is not None and n != cols:
        raise ValueError(f"{what} must have {cols} columns, not {n}")
    return x.data_ptr(), m, n


def moe_dispatch(plan: MoePlan, x, row, rows, scales=None, stream=None):
    """rows[row[t][j]] = x[t].  rows of x's type: copied; rows of float8_e4m3fn (or uint8): quantized
    with one FP32 scale per 128 elements, written to scales (rows x ceil(hidden / 128)); rows of int8: with
    one per row, written to scales (one per row).  row None: row t is token t."""
    ptr, t, h, ld = _matrix(x, "x")
    out, n, _ = _whole_rows(rows, "rows", h)
    code = _out_of(rows, "rows")
    if code in (TST_OUT_E4M3, TST_OUT_INT8):
        if scales is None:
            raise ValueError("e4m3 and int8 rows need scales")
        sptr = _array(scales, "scales", "float32", n * (1 if code == TST_OUT_INT8 else -(-h // 128)))
    else:
        sptr = None
    _check(lib.moe_dispatch(plan._h, t, h, ptr, _out_of(x, "x"), ld,
                            None if row is None else _array(row, "row", "int32", t * plan.top_k), out, code, n, sptr,
                            _stream(stream)), "moe_dispatch")


def moe_combine(plan: MoePlan, rows, row, out, weight=None, stream=None):
    """out[t] = sum_j weight[t][j] * rows[row[t][j]] (weight None: 1), in FP32."""
    ptr, n, h = _whole_rows(rows, "rows")
    optr, t, _, ld = _matrix(out, "out", cols=h)
    k = t * plan.top_k
    _check(lib.moe_combine(plan._h, t, h, ptr, _out_of(rows, "rows"), n, _array(row, "row", "int32", k),
                           None if weight is None else _array(weight, "weight", "float32", k), optr,
                           _out_of(out, "out"), ld, _stream(stream)), "moe_combine")


def moe_combine_backward(plan: MoePlan, rows, row, weight, d_out, d_rows, d_weight, stream=None):
    """d_rows[row[t][j]] = weight[t][j] * d_out[t] (of rows' type) and d_weight[t][j] =
    <d_out[t], rows[row[t][j]]> (FP32)."""
    ptr, n, h = _whole_rows(rows, "rows")
    dptr, m, _ = _whole_rows(d_rows, "d_rows", h)
    if m != n or d_rows.dtype != rows.dtype:
        raise ValueError(f"d_rows must be {n} x {h} of rows' type, {rows.dtype}")
    optr, t, _, ld = _matrix(d_out, "d_out", cols=h)
    k = t * plan.top_k
    _check(lib.moe_combine_backward(plan._h, t, h, ptr, _out_of(rows, "rows"), n, _array(row, "row", "int32", k),
                                    _array(weight, "weight", "float32", k), optr, _out_of(d_out, "d_out"), ld, dptr,
                                    _array(d_weight, "d_weight", "float32", k), _stream(stream)),
           "moe_combine_backward")
