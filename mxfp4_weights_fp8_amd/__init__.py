"""Routed MoE FFN with MXFP4 expert weights and online FP8 activations on MI355X.

Thin Python binding over the C-ABI library ``libmoe_mxfp4.so`` (declared in
``include/moe_mxfp4.h``). This module only marshals arguments: torch supplies
device memory and the current HIP stream, every step of the path runs in the
library's HIP kernels. There is no fallback: if the library is missing or a
call fails, an exception is raised.

    plan(topk_ids, E)                     -> Plan          (moe_plan)
    quant_act(x)                          -> (x_q, x_s)    (moe_quant_act)
    ffn(x, topk_weights, plan, weights)   -> y             (moe_ffn)
    ffn(..., static=True)                 -> y             (moe_ffn_static: no workspace)
    ffn_quantized(x_q, x_s, ...)          -> y             (moe_ffn_quantized: x quantized already)

In front of the FFN, each with its gradient as an explicit call:

    add_norm(x, weight, residual)         -> h, y, x_q, x_s            (moe_add_norm)
    add_norm_grad(dy, h, weight)          -> dx, dweight               (moe_add_norm_grad)
    linear(x, w, bias, act, residual)     -> y                         (moe_linear)
    linear_grad(dy, x, w)                 -> dx, dw, dbias             (moe_linear_grad)
    gate(logits, K)                       -> topk_ids, topk_weights    (moe_gate)
    gate_grad(logits, topk_ids, d_weights) -> d_logits                 (moe_gate_grad)
    balance_loss(logits, topk_ids, alpha) -> loss, counts, d_logits    (moe_balance_loss)

Training the experts (bf16 weights), along a plan:

    sort_rows(x, p)                       -> rows by expert            (moe_sort_rows)
    expert_linear(rows, w, p)             -> y                         (moe_expert_linear)
    glu(z)                                -> h, z_q, z_s               (moe_glu: z saved in 8 bits)
    return_rows(rows, p, weights)         -> y by token                (moe_return_rows)
    return_rows_grad(dy, rows, p, weights) -> d_rows, d_weights        (moe_return_rows_grad)
    glu_grad(dh, z_q, z_s)                -> dz, h                     (moe_glu_grad)
    expert_linear_grad(dy, rows, w, p)    -> dx, dw                    (moe_expert_linear_grad)
    sort_rows(x_q, p, scales=x_s), restore_act(x_q, x_s)               (rows, tokens from add_norm's codes)
"""

from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_mxfp4.so")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EWORKSPACE, MOE_EHIP, MOE_ESCRATCH = 0, -1, -2, -3, -4, -5
#: workspace bytes moe_ffn_static can serve (MOE_FFN_STATIC_MAX_BYTES)
FFN_STATIC_MAX_BYTES = 64 << 20
EV_START, EV_QUANT_DONE, EV_W13_DONE, EV_W2_DONE, EV_SHARED_DONE, EV_END = range(6)
NUM_EVENTS = 6


class MoEError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("K", ctypes.c_int32), ("Is", ctypes.c_int32), ("small_max", ctypes.c_int32),
                ("flags", ctypes.c_int32),
                ("tile_w13", ctypes.c_int32), ("tile_w2", ctypes.c_int32)]


#: moe_dims.flags bit: run decode shapes as one persistent W13 -> W2 -> combine launch
FLAG_DECODE_CHAIN = 1
#: moe_dims.flags bit: bf16 activations (MXFP4A16): x not quantized, bf16 SwiGLU rows
FLAG_A16 = 2
#: moe_dims.flags bit: NVFP4 expert weights with bf16 activations (ffn with NVFP4 weights)
FLAG_NVFP4 = 4


class Shared(ctypes.Structure):
    _fields_ = [("w13s", ctypes.c_void_p), ("w13s_s", ctypes.c_void_p), ("w2s", ctypes.c_void_p),
                ("w2s_s", ctypes.c_void_p)]


class Debug(ctypes.Structure):
    _fields_ = [("x_q", ctypes.c_void_p), ("x_s", ctypes.c_void_p), ("h_q", ctypes.c_void_p),
                ("h_s", ctypes.c_void_p), ("sh_q", ctypes.c_void_p), ("sh_s", ctypes.c_void_p),
                ("events", ctypes.POINTER(ctypes.c_void_p))]


class LinearDims(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("act", ctypes.c_int32),
                ("type", ctypes.c_int32)]


class GateDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("K", ctypes.c_int32), ("score", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("logits_type", ctypes.c_int32), ("scale", ctypes.c_float)]


class ExpertDims(ctypes.Structure):
    _fields_ = [("P", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("E", ctypes.c_int32),
                ("type", ctypes.c_int32)]


class GluDims(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32), ("act", ctypes.c_int32)]


#: MOE_TYPE_*, MOE_ACT_* and MOE_SCORE_* by what the functions below take
TYPES = {torch.bfloat16: 0, torch.float32: 1}
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "sigmoid": 4}
SCORES = {"softmax": 0, "sigmoid": 1, "sqrtsoftplus": 2}

_lib = None

#: every symbol the header declares, with its ctypes signature
_SIGNATURES = {
    "moe_validate": (ctypes.c_int, [ctypes.POINTER(Dims)]),
    "moe_plan_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Dims)]),
    "moe_plan": (ctypes.c_int, [ctypes.POINTER(Dims)] + [ctypes.c_void_p] * 6 + [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_quant_act": (ctypes.c_int, [ctypes.POINTER(Dims)] + [ctypes.c_void_p] * 4),
    "moe_pack_weights": (ctypes.c_int, [ctypes.POINTER(Dims)] + [ctypes.c_void_p] * 5),
    "moe_ffn_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Dims)]),
    "moe_ffn": (ctypes.c_int, [ctypes.POINTER(Dims)] + [ctypes.c_void_p] * 10 + [ctypes.POINTER(Shared),
                ctypes.c_void_p, ctypes.POINTER(Debug), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "moe_ffn_static": (ctypes.c_int, [ctypes.POINTER(Dims)] + [ctypes.c_void_p] * 10 + [ctypes.POINTER(Shared),
                       ctypes.c_void_p, ctypes.POINTER(Debug), ctypes.c_void_p]),
    "moe_ffn_nvfp4": (ctypes.c_int, [ctypes.POINTER(Dims)] + [ctypes.c_void_p] * 13 + [ctypes.POINTER(Debug),
                      ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "moe_ffn_quantized": (ctypes.c_int, [ctypes.POINTER(Dims)] + [ctypes.c_void_p] * 11 + [ctypes.POINTER(Shared),
                          ctypes.c_void_p, ctypes.POINTER(Debug), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "moe_add_norm": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.c_float] + [ctypes.c_void_p] * 3 +
                     [ctypes.c_int32] + [ctypes.c_void_p] * 5),
    "moe_add_norm_grad_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32]),
    "moe_add_norm_grad": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.c_float] + [ctypes.c_void_p] * 3 +
                          [ctypes.c_int32] + [ctypes.c_void_p] * 4 + [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_linear_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(LinearDims)]),
    "moe_linear": (ctypes.c_int, [ctypes.POINTER(LinearDims)] + [ctypes.c_void_p] * 7 +
                   [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_linear_grad_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(LinearDims)]),
    "moe_linear_grad": (ctypes.c_int, [ctypes.POINTER(LinearDims)] + [ctypes.c_void_p] * 8 +
                        [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_gate": (ctypes.c_int, [ctypes.POINTER(GateDims)] + [ctypes.c_void_p] * 6),
    "moe_gate_grad": (ctypes.c_int, [ctypes.POINTER(GateDims)] + [ctypes.c_void_p] * 6),
    "moe_balance_loss_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(GateDims), ctypes.c_int32]),
    "moe_balance_loss": (ctypes.c_int, [ctypes.POINTER(GateDims), ctypes.c_int32, ctypes.c_float] +
                         [ctypes.c_void_p] * 7 + [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_sort_rows": (ctypes.c_int, [ctypes.c_int32] * 3 + [ctypes.c_void_p] * 5),
    "moe_restore_act": (ctypes.c_int, [ctypes.c_int32] * 2 + [ctypes.c_void_p] * 4),
    "moe_return_rows": (ctypes.c_int, [ctypes.c_int32] * 3 + [ctypes.c_void_p] * 4 + [ctypes.c_int32] +
                        [ctypes.c_void_p] * 2),
    "moe_return_rows_grad": (ctypes.c_int, [ctypes.c_int32] * 3 + [ctypes.c_void_p, ctypes.c_int32] +
                             [ctypes.c_void_p] * 6),
    "moe_expert_linear_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(ExpertDims)]),
    "moe_expert_linear": (ctypes.c_int, [ctypes.POINTER(ExpertDims)] + [ctypes.c_void_p] * 5 +
                          [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_expert_linear_grad_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(ExpertDims)]),
    "moe_expert_linear_grad": (ctypes.c_int, [ctypes.POINTER(ExpertDims)] + [ctypes.c_void_p] * 7 +
                               [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_glu": (ctypes.c_int, [ctypes.POINTER(GluDims)] + [ctypes.c_void_p] * 6),
    "moe_glu_grad": (ctypes.c_int, [ctypes.POINTER(GluDims)] + [ctypes.c_void_p] * 8),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
}


def lib() -> ctypes.CDLL:
    """Load the C-ABI library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m mxfp4_weights_fp8_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().moe_status_string(code).decode()


def make_dims(T, H, I, E, K, Is=0, small_max=0, flags=0, tile_w13=0, tile_w2=0) -> Dims:
    """moe_dims. tile_w13 / tile_w2: exact-shape tiling per GEMM (0 = the library's
    tuned table, -1 = no 128-row item on the small-M tiles, 1..128 = row limit)."""
    return Dims(int(T), int(H), int(I), int(E), int(K), int(Is), int(small_max), int(flags), int(tile_w13),
                int(tile_w2))


def validate(d: Dims) -> int:
    return lib().moe_validate(ctypes.byref(d))


def plan_workspace_bytes(d: Dims) -> int:
    return lib().moe_plan_workspace_bytes(ctypes.byref(d))


def ffn_workspace_bytes(d: Dims) -> int:
    return lib().moe_ffn_workspace_bytes(ctypes.byref(d))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(rc: int, what: str):
    if rc != MOE_OK:
        raise MoEError(rc, what)


def _require(t: torch.Tensor, dtype, shape, name):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected contiguous cuda {dtype} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)} contiguous={t.is_contiguous()} device={t.device}")


@dataclasses.dataclass
class Plan:
    dims: Dims
    expert_offsets: torch.Tensor   # [E+1] int32
    sorted_pairs: torch.Tensor     # [P] int32
    pair_rows: torch.Tensor        # [P] int32
    status: torch.Tensor           # [1] int32 (dropped pairs)
    ws: torch.Tensor               # plan workspace (uint8)


def plan(topk_ids: torch.Tensor, E: int, H: int, I: int, small_max: int = 0, Is: int = 0,
         out: Optional[Plan] = None, flags: int = 0, tile_w13: int = 0, tile_w2: int = 0) -> Plan:
    """moe_plan on the current stream. topk_ids: cuda int32 [T, K]. H, I (and Is,
    flags, tile_w13, tile_w2) complete the dims that moe_ffn will use with this plan."""
    T, K = topk_ids.shape
    d = make_dims(T, H, I, E, K, Is, small_max, flags, tile_w13, tile_w2)
    _check(validate(d), "moe_plan dims")
    _require(topk_ids, torch.int32, (T, K), "topk_ids")
    dev = topk_ids.device
    if out is None:
        P = T * K
        out = Plan(d, torch.empty(E + 1, dtype=torch.int32, device=dev),
                   torch.empty(max(P, 1), dtype=torch.int32, device=dev),
                   torch.empty(max(P, 1), dtype=torch.int32, device=dev),
                   torch.zeros(1, dtype=torch.int32, device=dev),
                   torch.empty(plan_workspace_bytes(d), dtype=torch.uint8, device=dev))
    rc = lib().moe_plan(ctypes.byref(d), _ptr(topk_ids), _ptr(out.expert_offsets), _ptr(out.sorted_pairs),
                        _ptr(out.pair_rows), _ptr(out.status), _ptr(out.ws), out.ws.numel(), _stream(dev))
    _check(rc, "moe_plan")
    out.dims = d
    return out


def quant_act(x: torch.Tensor):
    """moe_quant_act: bf16 [T, H] -> (E4M3 codes uint8 [T, H], E8M0 scales uint8 [T, H/128])."""
    T, H = x.shape
    d = make_dims(T, H, 128, 1, 1)
    _check(validate(d), "moe_quant_act dims")
    _require(x, torch.bfloat16, (T, H), "x")
    x_q = torch.empty((T, H), dtype=torch.uint8, device=x.device)
    x_s = torch.empty((T, H // 128), dtype=torch.uint8, device=x.device)
    _check(lib().moe_quant_act(ctypes.byref(d), _ptr(x), _ptr(x_q), _ptr(x_s), _stream(x.device)), "moe_quant_act")
    return x_q, x_s


def pack_weights(weights: dict) -> dict:
    """moe_pack_weights on the current stream: a new weights dict whose w13 and w2
    codes are in the kernel-native layout that moe_ffn reads (the scale tensors are
    shared with the input dict). weights: dict w13 [E, 2I, H/2], w13_s, w2
    [E, H, I/2], w2_s (uint8 cuda, row-major codes as produced by MXFP4 packing)."""
    w13, w2 = weights["w13"], weights["w2"]
    E, I2, Hh = w13.shape
    H, I = 2 * Hh, I2 // 2
    _require(w13, torch.uint8, (E, 2 * I, H // 2), "w13")
    _require(w2, torch.uint8, (E, H, I // 2), "w2")
    d = make_dims(1, H, I, E, 1)
    _check(validate(d), "moe_pack_weights dims")
    p13 = torch.empty_like(w13)
    p2 = torch.empty_like(w2)
    _check(lib().moe_pack_weights(ctypes.byref(d), _ptr(w13), _ptr(p13), _ptr(w2), _ptr(p2), _stream(w13.device)),
           "moe_pack_weights")
    out = dict(weights)
    out.update(w13=p13, w2=p2, layout="packed")
    return out


_hip = None


def _hip_rt() -> ctypes.CDLL:
    global _hip
    if _hip is None:
        _hip = ctypes.CDLL("libamdhip64.so")
        _hip.hipEventCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
        _hip.hipEventDestroy.argtypes = [ctypes.c_void_p]
        _hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p, ctypes.c_void_p]
    return _hip


class StageEvents:
    """NUM_EVENTS raw HIP events for moe_ffn's stage boundaries (recorded by the
    library on the stream it launches on)."""

    def __init__(self, only=None):
        """only: optional subset of stage indices to record (the others stay NULL)."""
        h = _hip_rt()
        self.handles = []
        for i in range(NUM_EVENTS):
            e = ctypes.c_void_p()
            if only is None or i in only:
                if h.hipEventCreate(ctypes.byref(e)) != 0:
                    raise RuntimeError("hipEventCreate failed")
            self.handles.append(e)
        self.array = (ctypes.c_void_p * NUM_EVENTS)(*[e.value for e in self.handles])

    def elapsed_ms(self, a: int, b: int) -> float:
        out = ctypes.c_float()
        rc = _hip_rt().hipEventElapsedTime(ctypes.byref(out), self.handles[a], self.handles[b])
        if rc != 0:
            raise RuntimeError(f"hipEventElapsedTime failed ({rc})")
        return float(out.value)

    def __del__(self):
        try:
            for e in self.handles:
                if e.value:
                    _hip_rt().hipEventDestroy(e)
        except Exception:
            pass


def ffn(x: torch.Tensor, topk_weights: torch.Tensor, p: Plan, weights: dict, shared: Optional[dict] = None,
        debug: bool = False, ws: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
        events=None, static: bool = False):
    """moe_ffn on the current stream. weights: dict from pack_weights (w13 and w2 in
    the kernel-native layout, w13_s and w2_s row-major; uint8 cuda); shared:
    optional dict w13s, w13s_s, w2s, w2s_s.
    Returns y (bf16 [T, H]); with debug=True returns (y, dict of x_q, x_s, h_q, h_s,
    sh_q, sh_s); with FLAG_A16 or FLAG_NVFP4 in the plan's flags, h_q holds the bf16
    SwiGLU rows (int16 [P, I]) and x_q, x_s, h_s are left as allocated.
    With FLAG_NVFP4 (moe_ffn_nvfp4) the weights dict holds NVFP4 tensors: w13 / w2
    codes (packed), w13_s [E, 2I, H/16] / w2_s [E, H, I/16] E4M3 block scales and
    w13_gs / w2_gs [E] float32 tensor scales. ``events``: optional StageEvents recorded at the stage boundaries.
    ``static``: call moe_ffn_static (the library's static scratch instead of a
    workspace; ``ws`` must then be None)."""
    d = p.dims
    T, H, I, E, K, Is = d.T, d.H, d.I, d.E, d.K, d.Is
    dev = x.device
    _require(x, torch.bfloat16, (T, H), "x")
    _require(topk_weights, torch.float32, (T, K), "topk_weights")
    if weights.get("layout") != "packed":
        raise ValueError("moe_ffn reads expert weights in the kernel-native layout: convert them with pack_weights")
    nv = bool(d.flags & FLAG_NVFP4)
    blk = 16 if nv else 32
    _require(weights["w13"], torch.uint8, (E, 2 * I, H // 2), "w13")
    _require(weights["w13_s"], torch.uint8, (E, 2 * I, H // blk), "w13_s")
    _require(weights["w2"], torch.uint8, (E, H, I // 2), "w2")
    _require(weights["w2_s"], torch.uint8, (E, H, I // blk), "w2_s")
    if nv:
        _require(weights["w13_gs"], torch.float32, (E,), "w13_gs")
        _require(weights["w2_gs"], torch.float32, (E,), "w2_gs")
        if static or (shared is not None and Is > 0):
            raise ValueError("NVFP4 weights run through moe_ffn_nvfp4: no static scratch, no shared expert")
    sh = None
    if shared is not None and Is > 0:
        _require(shared["w13s"], torch.uint8, (2 * Is, H), "w13s")
        _require(shared["w13s_s"], torch.uint8, (2 * Is // 128, H // 128), "w13s_s")
        _require(shared["w2s"], torch.uint8, (H, Is), "w2s")
        _require(shared["w2s_s"], torch.uint8, (H // 128, Is // 128), "w2s_s")
        sh = Shared(shared["w13s"].data_ptr(), shared["w13s_s"].data_ptr(), shared["w2s"].data_ptr(),
                    shared["w2s_s"].data_ptr())
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if static and ws is not None:
        raise ValueError("moe_ffn_static takes no workspace")
    if ws is None and not static:
        ws = torch.empty(ffn_workspace_bytes(d), dtype=torch.uint8, device=dev)
    dbg_t = None
    dbg = None
    ev_arr = None
    if debug or events is not None:
        dbg = Debug()
        if debug:
            P = T * K
            dbg_t = {"x_q": torch.empty((T, H), dtype=torch.uint8, device=dev),
                     "x_s": torch.empty((T, H // 128), dtype=torch.uint8, device=dev),
                     "h_q": torch.zeros((max(P, 1), I),
                                        dtype=torch.int16 if d.flags & (FLAG_A16 | FLAG_NVFP4) else torch.uint8,
                                        device=dev),
                     "h_s": torch.zeros((max(P, 1), I // 128), dtype=torch.uint8, device=dev),
                     "sh_q": torch.zeros((T, max(Is, 128)), dtype=torch.uint8, device=dev),
                     "sh_s": torch.zeros((T, max(Is, 128) // 128), dtype=torch.uint8, device=dev)}
            for k, v in dbg_t.items():
                setattr(dbg, k, v.data_ptr())
        if events is not None:
            ev_arr = events.array
            dbg.events = ctypes.cast(ev_arr, ctypes.POINTER(ctypes.c_void_p))
    args = [ctypes.byref(d), _ptr(x), _ptr(topk_weights), _ptr(p.expert_offsets), _ptr(p.sorted_pairs),
            _ptr(p.pair_rows), _ptr(p.ws), _ptr(weights["w13"]), _ptr(weights["w13_s"]), _ptr(weights["w2"]),
            _ptr(weights["w2_s"]), ctypes.byref(sh) if sh is not None else None, _ptr(y),
            ctypes.byref(dbg) if dbg is not None else None]
    if nv:
        _check(lib().moe_ffn_nvfp4(ctypes.byref(d), _ptr(x), _ptr(topk_weights), _ptr(p.expert_offsets),
                                   _ptr(p.sorted_pairs), _ptr(p.pair_rows), _ptr(p.ws), _ptr(weights["w13"]),
                                   _ptr(weights["w13_s"]), _ptr(weights["w13_gs"]), _ptr(weights["w2"]),
                                   _ptr(weights["w2_s"]), _ptr(weights["w2_gs"]), _ptr(y),
                                   ctypes.byref(dbg) if dbg is not None else None, _ptr(ws), ws.numel(),
                                   _stream(dev)), "moe_ffn_nvfp4")
    elif static:
        _check(lib().moe_ffn_static(*args, _stream(dev)), "moe_ffn_static")
    else:
        _check(lib().moe_ffn(*args, _ptr(ws), ws.numel(), _stream(dev)), "moe_ffn")
    if debug:
        return y, dbg_t
    return y


def ffn_quantized(x_q: torch.Tensor, x_s: torch.Tensor, topk_weights: torch.Tensor, p: Plan, weights: dict,
                  shared: Optional[dict] = None, ws: Optional[torch.Tensor] = None,
                  y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_ffn_quantized on the current stream: ffn for activations that are quantized
    already, x_q [T, H] E4M3 codes and x_s [T, H/128] E8M0 scales (uint8, from add_norm
    or quant_act). weights, shared, ws and y as in ffn."""
    d = p.dims
    T, H, I, E, K, Is = d.T, d.H, d.I, d.E, d.K, d.Is
    dev = x_q.device
    _require(x_q, torch.uint8, (T, H), "x_q")
    _require(x_s, torch.uint8, (T, H // 128), "x_s")
    _require(topk_weights, torch.float32, (T, K), "topk_weights")
    if weights.get("layout") != "packed":
        raise ValueError("moe_ffn reads expert weights in the kernel-native layout: convert them with pack_weights")
    for name, shape in (("w13", (E, 2 * I, H // 2)), ("w13_s", (E, 2 * I, H // 32)), ("w2", (E, H, I // 2)),
                        ("w2_s", (E, H, I // 32))):
        _require(weights[name], torch.uint8, shape, name)
    sh = None
    if shared is not None and Is > 0:
        for name, shape in (("w13s", (2 * Is, H)), ("w13s_s", (2 * Is // 128, H // 128)), ("w2s", (H, Is)),
                            ("w2s_s", (H // 128, Is // 128))):
            _require(shared[name], torch.uint8, shape, name)
        sh = Shared(shared["w13s"].data_ptr(), shared["w13s_s"].data_ptr(), shared["w2s"].data_ptr(),
                    shared["w2s_s"].data_ptr())
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    _require(y, torch.bfloat16, (T, H), "y")
    if ws is None:
        ws = torch.empty(ffn_workspace_bytes(d), dtype=torch.uint8, device=dev)
    _enqueue("moe_ffn_quantized", dev, ctypes.byref(d), x_q.data_ptr(), x_s.data_ptr(), topk_weights.data_ptr(),
             p.expert_offsets.data_ptr(), p.sorted_pairs.data_ptr(), p.pair_rows.data_ptr(), p.ws.data_ptr(),
             weights["w13"].data_ptr(), weights["w13_s"].data_ptr(), weights["w2"].data_ptr(),
             weights["w2_s"].data_ptr(), ctypes.byref(sh) if sh is not None else None, y.data_ptr(), None,
             ws.data_ptr(), ws.numel())
    return y


# ------------------------------------------------------------------ in front of the FFN

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # absent in CPU-only builds of torch


def _enqueue(name: str, dev: torch.device, *args):
    """Call an entry point with the current stream of `dev` as its last argument, with
    that device current, so that tensors may live on another than the current one."""
    fn = getattr(_lib or lib(), name)
    index = dev.index
    if index == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(index))
    if rc == MOE_EINVAL and name != "moe_ffn_quantized":   # whose scales may start anywhere
        odd = [hex(a) for a in args if isinstance(a, int) and a >> 32 > 0 and a % 16]
        if odd:
            raise MoEError(rc, f"{name}: tensors start at 16-byte aligned addresses, {', '.join(odd)} is not one")
    if rc != MOE_OK:
        raise MoEError(rc, name)


def _tensor(t, dtype, shape, dev, name):
    """Checks an argument (None passes) and gives its device address."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} contiguous={t.is_contiguous()} device={t.device}")
    return t.data_ptr()


def _new(rows, cols, dtype, dev):
    """An uninitialised [rows, cols] tensor (empty_strided takes 1.3 us, empty 2.2 us)."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=dev)


def _vector(n, dtype, dev):
    return torch.empty_strided((n,), (1,), dtype=dtype, device=dev)


def _first(t, dims, name):
    """Checks that the argument that sets sizes and device is a cuda tensor of `dims` dimensions."""
    if t.dim() != dims or not t.is_cuda:
        raise ValueError(f"{name}: expected a cuda tensor of {dims} dimensions, got {tuple(t.shape)} on {t.device}")
    return t.device


def _one_of(table, key, name):
    if key not in table:
        raise ValueError(f"{name}: {key!r} is none of {sorted(map(str, table))}")
    return table[key]


def _workspace(nbytes, dev, ws):
    if ws is None:
        return _vector(nbytes, torch.uint8, dev) if nbytes else None
    if ws.dtype != torch.uint8 or ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"ws: expected contiguous uint8 on {dev}, got {ws.dtype} on {ws.device}")
    return ws


class Normed(NamedTuple):
    h: torch.Tensor                  # [T, H] bf16 residual stream (x itself without a residual and without out.h)
    y: Optional[torch.Tensor]        # [T, H] bf16
    x_q: Optional[torch.Tensor]      # [T, H] uint8 E4M3 codes of y
    x_s: Optional[torch.Tensor]      # [T, H/128] uint8 E8M0 scales


def add_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             bf16: bool = True, fp8: bool = True, out: Optional[Normed] = None) -> Normed:
    """moe_add_norm on the current stream: h = x + residual, y = RMS norm of h times
    weight, and y's E4M3 codes and E8M0 scales for ffn_quantized. x, residual: bf16
    [T, H]; weight: bf16 or float32 [H]. bf16 / fp8 choose which forms of y are written
    (None in the other's place). out: tensors to write (None members are allocated;
    without a residual h is x itself unless out.h is given, which then receives a copy);
    out.h may be the residual or x, out.y may be x."""
    dev = _first(x, 2, "x")
    shape = x.shape
    T, H = shape
    xp = _tensor(x, torch.bfloat16, shape, dev, "x")
    rp = _tensor(residual, torch.bfloat16, shape, dev, "residual")
    wt = _one_of(TYPES, weight.dtype, "weight type")
    wp = _tensor(weight, weight.dtype, (H,), dev, "weight")
    h, y, q, s = out if out is not None else (None, None, None, None)
    hp = yp = qp = sp = None
    if h is not None:
        hp = _tensor(h, torch.bfloat16, shape, dev, "out.h")
        if residual is None and hp == xp:
            hp = None        # x is there already
    elif residual is None:
        h = x
    else:
        h = torch.empty_like(x)
        hp = h.data_ptr()
    if not bf16:
        y = None
    elif y is None:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    else:
        yp = _tensor(y, torch.bfloat16, shape, dev, "out.y")
    if not fp8:
        q = s = None
    else:
        if q is None:
            q = _new(T, H, torch.uint8, dev)
            qp = q.data_ptr()
        else:
            qp = _tensor(q, torch.uint8, shape, dev, "out.x_q")
        if s is None:
            s = _new(T, H // 128, torch.uint8, dev)
            sp = s.data_ptr()
        else:
            sp = _tensor(s, torch.uint8, (T, H // 128), dev, "out.x_s")
    _enqueue("moe_add_norm", dev, T, H, eps, xp, rp, wp, wt, hp, yp, qp, sp)
    return Normed(h, y, q, s)


def add_norm_grad(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                  dh: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                  ws: Optional[torch.Tensor] = None):
    """moe_add_norm_grad on the current stream. dy: bf16 [T, H] gradient of y; h: bf16
    [T, H] as add_norm returned it; dh: optional bf16 [T, H] gradient that h has from
    elsewhere. Returns (dx bf16 [T, H], the gradient of x and of the residual alike;
    dweight float32 [H]). dx: optional tensor to write (may be dy or dh)."""
    dev = _first(h, 2, "h")
    shape = h.shape
    T, H = shape
    wt = _one_of(TYPES, weight.dtype, "weight type")
    if dx is None:
        dx = torch.empty_like(h)
    dw = _vector(H, torch.float32, dev)
    ws = _workspace(lib().moe_add_norm_grad_workspace_bytes(T, H), dev, ws)
    _enqueue("moe_add_norm_grad", dev, T, H, eps, _tensor(dy, torch.bfloat16, shape, dev, "dy"),
             _tensor(h, torch.bfloat16, shape, dev, "h"), _tensor(weight, weight.dtype, (H,), dev, "weight"), wt,
             _tensor(dh, torch.bfloat16, shape, dev, "dh"), _tensor(dx, torch.bfloat16, shape, dev, "dx"),
             dw.data_ptr(), *_ws_args(ws))
    return dx, dw


def _ws_args(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel())


def linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
           residual: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
           y: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
           ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_linear on the current stream: act(x w^T + bias) + residual. x: bf16 [M, K];
    w: bf16 [N, K]; bias: float32 [N]; act: a key of ACTS; residual: [M, N] of the
    output's type; dtype: torch.bfloat16 or torch.float32 (a router's logits). y:
    optional tensor to write (may be the residual); z: optional float32 [M, N] that
    receives the values before the activation, for linear_grad."""
    dev = _first(x, 2, "x")
    M, K = x.shape
    _first(w, 2, "w")
    N = w.shape[0]
    d = LinearDims(M, N, K, _one_of(ACTS, act, "act"), _one_of(TYPES, dtype, "dtype"))
    if y is None:
        y = _new(M, N, dtype, dev)
    ws = _workspace(lib().moe_linear_workspace_bytes(d), dev, ws)
    _enqueue("moe_linear", dev, d, _tensor(x, torch.bfloat16, (M, K), dev, "x"),
             _tensor(w, torch.bfloat16, (N, K), dev, "w"), _tensor(bias, torch.float32, (N,), dev, "bias"),
             _tensor(residual, dtype, (M, N), dev, "residual"), _tensor(y, dtype, (M, N), dev, "y"),
             _tensor(z, torch.float32, (M, N), dev, "z"), *_ws_args(ws))
    return y


def linear_grad(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, act: str = "none",
                z: Optional[torch.Tensor] = None, need=(True, True, True), ws: Optional[torch.Tensor] = None):
    """moe_linear_grad on the current stream. dy: bf16 or float32 [M, N]; x, w as in
    linear; z: float32 [M, N] from linear (for an activation). need: which of the
    results are computed. Returns (dx bf16 [M, K], dw bf16 [N, K], dbias float32 [N]),
    None where not needed."""
    dev = _first(x, 2, "x")
    M, K = x.shape
    _first(w, 2, "w")
    N = w.shape[0]
    d = LinearDims(M, N, K, _one_of(ACTS, act, "act"), _one_of(TYPES, dy.dtype, "dy type"))
    dx = torch.empty_like(x) if need[0] else None
    dw = torch.empty_like(w) if need[1] else None
    db = _vector(N, torch.float32, dev) if need[2] else None
    ws = _workspace(lib().moe_linear_grad_workspace_bytes(d), dev, ws)
    _enqueue("moe_linear_grad", dev, d, _tensor(dy, dy.dtype, (M, N), dev, "dy"),
             _tensor(x, torch.bfloat16, (M, K), dev, "x"), _tensor(w, torch.bfloat16, (N, K), dev, "w"),
             _tensor(z, torch.float32, (M, N), dev, "z"), dx.data_ptr() if need[0] else None,
             dw.data_ptr() if need[1] else None, db.data_ptr() if need[2] else None, *_ws_args(ws))
    return dx, dw, db


def _gate_dims(logits, K, score, renorm, scale):
    T, E = logits.shape
    return GateDims(T, E, K, _one_of(SCORES, score, "score"), 1 if renorm else 0,
                    _one_of(TYPES, logits.dtype, "logits type"), scale)


def gate(logits: torch.Tensor, K: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
         renorm: bool = True, scale: float = 1.0, n_valid: Optional[torch.Tensor] = None,
         topk_ids: Optional[torch.Tensor] = None, topk_weights: Optional[torch.Tensor] = None):
    """moe_gate on the current stream. logits: float32 or bf16 [T, E]; score: a key of
    SCORES; bias: optional float32 [E], added to the scores for the choice alone;
    n_valid: optional int32 [1] on the device (16-byte aligned, as every tensor here: not any
    element of a larger one), rows from there on are padding. Returns
    (topk_ids int32 [T, K], topk_weights float32 [T, K]), ready for plan and ffn; picks
    that do not exist have id -1 and weight 0."""
    dev = _first(logits, 2, "logits")
    T, E = logits.shape
    d = _gate_dims(logits, K, score, renorm, scale)
    shape = (T, K)
    if topk_ids is None:
        topk_ids = _new(T, K, torch.int32, dev)
    if topk_weights is None:
        topk_weights = _new(T, K, torch.float32, dev)
    _enqueue("moe_gate", dev, d, _tensor(logits, logits.dtype, (T, E), dev, "logits"),
             _tensor(bias, torch.float32, (E,), dev, "bias"), _tensor(n_valid, torch.int32, (1,), dev, "n_valid"),
             _tensor(topk_ids, torch.int32, shape, dev, "topk_ids"),
             _tensor(topk_weights, torch.float32, shape, dev, "topk_weights"))
    return topk_ids, topk_weights


def gate_grad(logits: torch.Tensor, topk_ids: torch.Tensor, d_weights: torch.Tensor, score: str = "softmax",
              renorm: bool = True, scale: float = 1.0, add: Optional[torch.Tensor] = None,
              d_logits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_gate_grad on the current stream: float32 [T, E] gradient of the logits from
    d_weights float32 [T, K], the gradient of gate's weights, the picks held fixed. add:
    optional float32 [T, E] added to it (balance_loss's); d_logits: optional tensor to
    write (may be add)."""
    dev = _first(logits, 2, "logits")
    _first(topk_ids, 2, "topk_ids")
    T, E = logits.shape
    K = topk_ids.shape[1]
    d = _gate_dims(logits, K, score, renorm, scale)
    if d_logits is None:
        d_logits = _new(T, E, torch.float32, dev)
    _enqueue("moe_gate_grad", dev, d, _tensor(logits, logits.dtype, (T, E), dev, "logits"),
             _tensor(topk_ids, torch.int32, (T, K), dev, "topk_ids"),
             _tensor(d_weights, torch.float32, (T, K), dev, "d_weights"),
             _tensor(add, torch.float32, (T, E), dev, "add"),
             _tensor(d_logits, torch.float32, (T, E), dev, "d_logits"))
    return d_logits


def balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor, alpha: float, score: str = "softmax",
                 seq_offsets: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """moe_balance_loss on the current stream. logits: float32 or bf16 [T, E]; topk_ids:
    int32 [T, K]; seq_offsets: optional int32 [B + 1], sequence b is the tokens from
    seq_offsets[b] up to seq_offsets[b + 1] (default: one sequence of all tokens).
    Returns (loss float32 [1], counts int32 [B, E], d_logits float32 [T, E], the
    gradient of the loss)."""
    dev = _first(logits, 2, "logits")
    _first(topk_ids, 2, "topk_ids")
    T, E = logits.shape
    K = topk_ids.shape[1]
    if seq_offsets is not None:
        _first(seq_offsets, 1, "seq_offsets")
    B = 1 if seq_offsets is None else seq_offsets.shape[0] - 1
    d = _gate_dims(logits, K, score, False, 1.0)
    loss = _vector(1, torch.float32, dev)
    counts = _new(max(B, 0), E, torch.int32, dev)
    d_logits = _new(T, E, torch.float32, dev)
    ws = _workspace(lib().moe_balance_loss_workspace_bytes(d, B), dev, ws)
    _enqueue("moe_balance_loss", dev, d, B, alpha, _tensor(logits, logits.dtype, (T, E), dev, "logits"),
             _tensor(topk_ids, torch.int32, (T, K), dev, "topk_ids"),
             _tensor(seq_offsets, torch.int32, (B + 1,), dev, "seq_offsets"), loss.data_ptr(), counts.data_ptr(),
             d_logits.data_ptr(), *_ws_args(ws))
    return loss, counts, d_logits


# ------------------------------------------------------------------ training the experts

BF16 = torch.bfloat16


def _pairs(p: Plan, dev):
    """(T, K, address of pair_rows) of a plan."""
    d = p.dims
    T, K = d.T, d.K
    return T, K, _tensor(p.pair_rows, torch.int32, (max(T * K, 1),), dev, "pair_rows")


def _offsets(p: Plan, dev):
    """(rows, experts, address of expert_offsets) of a plan."""
    d = p.dims
    return d.T * d.K, d.E, _tensor(p.expert_offsets, torch.int32, (d.E + 1,), dev, "expert_offsets")


def sort_rows(x: torch.Tensor, p: Plan, scales: Optional[torch.Tensor] = None,
              rows: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_sort_rows on the current stream: the rows of the plan's experts, bf16 [T K, H].
    x: bf16 [T, H], or with scales (uint8 [T, H/128]) uint8 E4M3 codes as add_norm or
    quant_act gave them. rows: optional tensor to write. Rows behind the last expert's are
    left as they were (uninitialised in a new tensor). Its gradient is return_rows."""
    dev = _first(x, 2, "x")
    T, K, pr = _pairs(p, dev)
    H = x.shape[1]
    if rows is None:
        rows = _new(T * K, H, BF16, dev)
    _enqueue("moe_sort_rows", dev, T, H, K, _tensor(x, BF16 if scales is None else torch.uint8, (T, H), dev, "x"),
             _tensor(scales, torch.uint8, (T, H // 128), dev, "scales"), pr, _tensor(rows, BF16, (T * K, H), dev, "rows"))
    return rows


def restore_act(x_q: torch.Tensor, x_s: torch.Tensor) -> torch.Tensor:
    """moe_restore_act on the current stream: bf16 [T, H] values of E4M3 codes x_q uint8
    [T, H] and E8M0 scales x_s uint8 [T, H/128], as add_norm or quant_act gave them."""
    dev = _first(x_q, 2, "x_q")
    T, H = x_q.shape
    x = _new(T, H, BF16, dev)
    _enqueue("moe_restore_act", dev, T, H, _tensor(x_q, torch.uint8, (T, H), dev, "x_q"),
             _tensor(x_s, torch.uint8, (T, H // 128), dev, "x_s"), x.data_ptr())
    return x


def return_rows(rows: torch.Tensor, p: Plan, weights: Optional[torch.Tensor] = None,
                add: Optional[torch.Tensor] = None, dtype: torch.dtype = BF16,
                y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_return_rows on the current stream: [T, H] of dtype (torch.bfloat16 or
    torch.float32), the sum over a token's picks of weights float32 [T, K] (default: 1)
    times their rows (bf16 [T K, H] in the plan's order), plus add ([T, H] of dtype). y:
    optional tensor to write (may be add)."""
    dev = _first(rows, 2, "rows")
    T, K, pr = _pairs(p, dev)
    H = rows.shape[1]
    t = _one_of(TYPES, dtype, "dtype")
    if y is None:
        y = _new(T, H, dtype, dev)
    _enqueue("moe_return_rows", dev, T, H, K, _tensor(rows, BF16, (T * K, H), dev, "rows"), pr,
             _tensor(weights, torch.float32, (T, K), dev, "weights"), _tensor(add, dtype, (T, H), dev, "add"), t,
             _tensor(y, dtype, (T, H), dev, "y"))
    return y


def return_rows_grad(dy: torch.Tensor, rows: Optional[torch.Tensor], p: Plan, weights: Optional[torch.Tensor] = None,
                     need=(True, True), d_rows: Optional[torch.Tensor] = None):
    """moe_return_rows_grad on the current stream. dy: bf16 or float32 [T, H]; rows and
    weights as in return_rows (rows may be None where d_weights is not needed). Returns
    (d_rows bf16 [T K, H], d_weights float32 [T, K], gate_grad's), None where not needed.
    d_rows: optional tensor to write (may be rows); rows behind the last expert's are left
    as they were."""
    dev = _first(dy, 2, "dy")
    T, K, pr = _pairs(p, dev)
    H = dy.shape[1]
    t = _one_of(TYPES, dy.dtype, "dy type")
    if not need[0]:
        d_rows = None
    elif d_rows is None:
        d_rows = _new(T * K, H, BF16, dev)
    dw = _new(T, K, torch.float32, dev) if need[1] else None
    _enqueue("moe_return_rows_grad", dev, T, H, K, _tensor(dy, dy.dtype, (T, H), dev, "dy"), t,
             _tensor(rows, BF16, (T * K, H), dev, "rows"), pr,
             _tensor(weights, torch.float32, (T, K), dev, "weights"),
             _tensor(d_rows, BF16, (T * K, H), dev, "d_rows"), dw.data_ptr() if need[1] else None)
    return d_rows, dw


def expert_linear(x: torch.Tensor, w: torch.Tensor, p: Plan, dtype: torch.dtype = BF16,
                  y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_expert_linear on the current stream: y[r] = w[e] x[r] for the plan's rows r of
    expert e. x: bf16 [T K, K'] (sort_rows's); w: bf16 [E, N, K']; y: [T K, N] of dtype
    (torch.bfloat16 or torch.float32), optionally a tensor to write; rows behind the last
    expert's are left as they were (uninitialised in a new tensor)."""
    dev = _first(x, 2, "x")
    _first(w, 3, "w")
    P, E, off = _offsets(p, dev)
    N, K = w.shape[1:]
    d = ExpertDims(P, N, K, E, _one_of(TYPES, dtype, "dtype"))
    if y is None:
        y = _new(P, N, dtype, dev)
    ws = _workspace(lib().moe_expert_linear_workspace_bytes(d), dev, ws)
    _enqueue("moe_expert_linear", dev, d, _tensor(x, BF16, (P, K), dev, "x"), _tensor(w, BF16, (E, N, K), dev, "w"),
             off, _tensor(y, dtype, (P, N), dev, "y"), *_ws_args(ws))
    return y


def expert_linear_grad(dy: torch.Tensor, x: Optional[torch.Tensor], w: Optional[torch.Tensor], p: Plan,
                       need=(True, True), dtype: torch.dtype = BF16, dx: Optional[torch.Tensor] = None,
                       dw: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """moe_expert_linear_grad on the current stream. dy: bf16 [T K, N]; x, w as in
    expert_linear (x may be None where dw is not needed, w where dx is not). Returns (dx
    bf16 [T K, K'], dw [E, N, K'] of dtype, zero for an expert without rows), None where
    not needed; dx, dw: optional tensors to write (rows of dx behind the last expert's are
    left as they were)."""
    dev = _first(dy, 2, "dy")
    P, E, off = _offsets(p, dev)
    N = dy.shape[1]
    if w is not None:
        _first(w, 3, "w")
    elif x is None or need[0]:
        raise ValueError("w: needed for dx, and one of x and w for the sizes")
    else:
        _first(x, 2, "x")
    K = w.shape[2] if w is not None else x.shape[1]
    d = ExpertDims(P, N, K, E, _one_of(TYPES, dtype, "dtype"))
    if not need[0]:
        dx = None
    elif dx is None:
        dx = _new(P, K, BF16, dev)
    if not need[1]:
        dw = None
    elif dw is None:
        dw = torch.empty_strided((E, N, K), (N * K, K, 1), dtype=dtype, device=dev)
    ws = _workspace(lib().moe_expert_linear_grad_workspace_bytes(d), dev, ws)
    _enqueue("moe_expert_linear_grad", dev, d, _tensor(dy, BF16, (P, N), dev, "dy"), _tensor(x, BF16, (P, K), dev, "x"),
             _tensor(w, BF16, (E, N, K), dev, "w"), off, _tensor(dx, BF16, (P, K), dev, "dx"),
             _tensor(dw, dtype, (E, N, K), dev, "dw"), *_ws_args(ws))
    return dx, dw


def _glu_dims(R, I, act, p, dev):
    if p is None:
        return GluDims(R, I, 0, _one_of(ACTS, act, "act")), None
    P, E, off = _offsets(p, dev)
    if P != R:
        raise ValueError(f"a plan of {P} rows for {R}")
    return GluDims(R, I, E, _one_of(ACTS, act, "act")), off


def glu(z: torch.Tensor, act: str = "silu", save: bool = True, p: Optional[Plan] = None, out=None):
    """moe_glu on the current stream: (h, z_q, z_s) with h = act(g) u bf16 [R, I] of z = (g,
    u) bf16 [R, 2I], and z's E4M3 codes uint8 [R, 2I] and E8M0 scales uint8 [R, 2I/128] to
    keep for glu_grad in place of z (None without save). p: rows behind the plan's last
    expert's are left as they were (default: every row counts). out: (h, z_q, z_s) tensors
    to write, None members are allocated."""
    dev = _first(z, 2, "z")
    R, I = z.shape[0], z.shape[1] // 2
    if z.shape[1] % 2:
        raise ValueError(f"z: two halves, got {z.shape[1]} columns")
    d, off = _glu_dims(R, I, act, p, dev)
    h, q, s = out if out is not None else (None, None, None)
    if h is None:
        h = _new(R, I, BF16, dev)
    if not save:
        q = s = None
    else:
        if q is None:
            q = _new(R, 2 * I, torch.uint8, dev)
        if s is None:
            s = _new(R, 2 * I // 128, torch.uint8, dev)
    _enqueue("moe_glu", dev, d, _tensor(z, BF16, (R, 2 * I), dev, "z"), off, _tensor(h, BF16, (R, I), dev, "out h"),
             _tensor(q, torch.uint8, (R, 2 * I), dev, "out z_q"), _tensor(s, torch.uint8, (R, 2 * I // 128), dev, "out z_s"))
    return h, q, s


def glu_grad(dh: torch.Tensor, z: torch.Tensor, scales: Optional[torch.Tensor] = None, act: str = "silu",
             p: Optional[Plan] = None, need_h: bool = True, out=None):
    """moe_glu_grad on the current stream: (dz bf16 [R, 2I], h bf16 [R, I] or None) from dh
    bf16 [R, I] and z: glu's codes uint8 [R, 2I] with their scales, or bf16 z itself. h is
    act(g) u at the same values, for the second product's dw. p as in glu. out: (dz, h)
    tensors to write (dz may be a bf16 z, h may be dh), None members are allocated."""
    dev = _first(dh, 2, "dh")
    R, I = dh.shape
    d, off = _glu_dims(R, I, act, p, dev)
    dz, h = out if out is not None else (None, None)
    if dz is None:
        dz = _new(R, 2 * I, BF16, dev)
    if not need_h:
        h = None
    elif h is None:
        h = _new(R, I, BF16, dev)
    zp = _tensor(z, BF16 if scales is None else torch.uint8, (R, 2 * I), dev, "z")
    sp = _tensor(scales, torch.uint8, (R, 2 * I // 128), dev, "scales")
    _enqueue("moe_glu_grad", dev, d, _tensor(dh, BF16, (R, I), dev, "dh"), None if scales is not None else zp,
             zp if scales is not None else None, sp, off, _tensor(dz, BF16, (R, 2 * I), dev, "out dz"),
             _tensor(h, BF16, (R, I), dev, "out h"))
    return dz, h
