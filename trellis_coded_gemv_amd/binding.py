"""ctypes binding of libtrellis_gemv.so -- argument marshalling only.

Every step of the computation runs in the library's HIP kernels; PyTorch is
used only to own device memory and to supply the current HIP stream. The
functions mirror the C ABI of include/trellis_gemv.h name for name. If the
library is missing or fails to load, every entry point raises: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtrellis_gemv.so")

TG_FLAG_ROUND_WEIGHTS = 1
TG_FLAG_INT8_ACT = 2
TG_STATUS_SPLITK_TIMEOUT = 1
ABI_VERSION = 4

STATUS = {0: "TG_OK", -1: "TG_ERR_NULL", -2: "TG_ERR_SHAPE", -3: "TG_ERR_KBITS", -4: "TG_ERR_ALIGN",
          -5: "TG_ERR_WORKSPACE", -6: "TG_ERR_CODE_ID", -7: "TG_ERR_LAUNCH", -8: "TG_ERR_ARG"}

# every symbol the header declares
EXPORTS = ("tg_abi_version", "tg_build_id", "tg_workspace_status", "tg_status_str", "tg_workspace_size",
           "trellis_gemv", "trellis_gemv_noalloc", "tg_noalloc_scratch_bytes", "trellis_gemv_fused",
           "tg_fused_workspace_size", "trellis_gemm_small",
           "tg_decode_ceiling",
           "rht_apply", "trellis_gemv_grouped", "tg_grouped_workspace_size", "trellis_decode", "tg_code_table",
           "trellis_encode", "tg_encode_workspace_size", "trellis_gemm_prefill", "tg_prefill_workspace_size",
           "trellis_moe_block", "tg_moe_workspace_size",
           "moe_route", "moe_group", "int8_quantize", "int8_gemm", "tg_int8_workspace_size", "int8_gemm_grouped",
           "tg_int8_plan")

TG_ROUTE_SIGMOID = 1
TG_ROUTE_RENORM = 2
TG_ZERO_UNROUTED = 0x100


class TgLayer(ctypes.Structure):
    """Mirror of tg_layer."""
    _fields_ = [("m", ctypes.c_int32), ("n", ctypes.c_int32), ("k_bits", ctypes.c_int32),
                ("code_id", ctypes.c_int32), ("flags", ctypes.c_int32), ("splits", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("sign_in", ctypes.c_void_p), ("sign_out", ctypes.c_void_p)]


class TgError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_status_str(status)})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load the HIP library (once). Raises if it is not built, or was built from other sources
    than the ones in this tree (its tg_build_id differs from their hash)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m trellis_coded_gemv_amd.build`")
    from .build import source_hash
    L = ctypes.CDLL(LIB_PATH)
    L.tg_build_id.restype = ctypes.c_char_p
    L.tg_build_id.argtypes = []
    built, want = L.tg_build_id().decode(), source_hash()
    if built != want:
        raise RuntimeError(f"{LIB_PATH} was built from other sources (build id {built}, sources {want}): "
                           "rebuild it with `python -m trellis_coded_gemv_amd.build`")
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    LP = ctypes.POINTER(TgLayer)
    sig = {
        "tg_abi_version": (I32, []),
        "tg_build_id": (ctypes.c_char_p, []),
        "tg_workspace_status": (I32, [P, I32, ctypes.POINTER(ctypes.c_uint32), P]),
        "tg_status_str": (ctypes.c_char_p, [I32]),
        "tg_workspace_size": (SZ, [LP, I32]),
        "trellis_gemv": (I32, [LP, P, P, P, SZ, P]),
        "trellis_gemv_noalloc": (I32, [LP, P, P, P]),
        "trellis_gemv_fused": (I32, [LP, I32, P, P, P, SZ, P]),
        "tg_fused_workspace_size": (SZ, [LP, I32]),
        "tg_noalloc_scratch_bytes": (SZ, []),
        "trellis_gemm_small": (I32, [LP, I32, P, I64, P, I64, P, SZ, P]),
        "rht_apply": (I32, [I32, I32, P, P, P, I32, P]),
        "trellis_gemv_grouped": (I32, [LP, P, I32, P, I32, P, I64, P, I64, P, SZ, P]),
        "tg_grouped_workspace_size": (SZ, [LP, I32, I32]),
        "trellis_decode": (I32, [LP, P, P]),
        "tg_code_table": (I32, [I32, P, P]),
        "tg_decode_ceiling": (I32, [I32, I32, I32, I32, I32, P, P]),
        "trellis_encode": (I32, [I32, I32, I32, ctypes.c_float, P, P, P, P, SZ, P]),
        "tg_encode_workspace_size": (SZ, [I32, I32, I32]),
        "trellis_gemm_prefill": (I32, [LP, I32, P, I64, P, I64, P, SZ, P]),
        "tg_prefill_workspace_size": (SZ, [LP, I32]),
        "trellis_moe_block": (I32, [LP, P, I32, LP, P, I32, P, P, I32, P, P, P, SZ, P]),
        "tg_moe_workspace_size": (SZ, [LP, I32, LP, I32, I32]),
        "moe_route": (I32, [I32, I32, I32, P, I32, I64, P, I32, I32, I32, I32, ctypes.c_float, P, P, P]),
        "moe_group": (I32, [I32, I32, P, P, P, P]),
        "int8_quantize": (I32, [I32, I32, P, I32, I64, P, I64, P, P]),
        "int8_gemm": (I32, [I32, I32, I32, P, I64, P, P, I64, P, P, I32, I64, P, SZ, P]),
        "tg_int8_workspace_size": (SZ, [I32, I32, I32]),
        "tg_int8_plan": (I32, [I32, I32, I32, I32, ctypes.POINTER(I32)]),
        "int8_gemm_grouped": (I32, [I32, I32, I32, I32, P, I64, P, I32, P, P, P, P, P, I32, I64, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    if L.tg_abi_version() != ABI_VERSION:
        raise RuntimeError(f"{LIB_PATH} has ABI version {L.tg_abi_version()}, the binding expects {ABI_VERSION}")
    _lib = L
    return L


def _status_str(status: int) -> str:
    try:
        return lib().tg_status_str(status).decode()
    except Exception:  # noqa: BLE001 - message only
        return "?"


def _check(status: int, where: str) -> None:
    if status != 0:
        raise TgError(status, where)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class DeviceLayer:
    """A layer's arrays in device memory plus its tg_layer descriptor."""

    def __init__(self, arrays, device="cuda", flags: int = 0, splits: int = 0):
        torch = _torch()
        self.m, self.n, self.k_bits = int(arrays.m), int(arrays.n), int(arrays.k_bits)
        self.code_id, self.flags, self.splits = int(getattr(arrays, "code_id", 0)), int(flags), int(splits)
        self.codes = torch.from_numpy(np.ascontiguousarray(arrays.codes).view(np.int32)).to(device)
        self.scales = torch.from_numpy(np.ascontiguousarray(arrays.scales).view(np.int16)).to(device)
        self.sign_in = torch.from_numpy(np.ascontiguousarray(arrays.sign_in).view(np.int32)).to(device)
        self.sign_out = torch.from_numpy(np.ascontiguousarray(arrays.sign_out).view(np.int32)).to(device)

    def desc(self) -> TgLayer:
        return TgLayer(self.m, self.n, self.k_bits, self.code_id, self.flags, self.splits,
                       self.codes.data_ptr(), self.scales.data_ptr(),
                       self.sign_in.data_ptr(), self.sign_out.data_ptr())

    @property
    def code_bytes(self) -> int:
        return self.codes.numel() * 4


def fp16_tensor(bits: np.ndarray, device="cuda"):
    """Host uint16 fp16 patterns -> device float16 tensor (same bits)."""
    torch = _torch()
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.float16)).to(device)


def build_id() -> str:
    return lib().tg_build_id().decode()


def workspace_status(ws, clear: bool = False, stream=None) -> int:
    """The workspace's status word (TG_STATUS_* bits); waits for the stream."""
    word = ctypes.c_uint32(0)
    _check(lib().tg_workspace_status(_ptr(ws), int(clear), ctypes.byref(word), _stream(stream)), "tg_workspace_status")
    return int(word.value)


def workspace_size(layer: DeviceLayer, M: int = 1) -> int:
    d = layer.desc()
    return int(lib().tg_workspace_size(ctypes.byref(d), M))


def workspace(layer: DeviceLayer, M: int = 1, device="cuda"):
    """Zero-filled workspace for trellis_gemv (M == 1) / trellis_gemm_small."""
    size = workspace_size(layer, M)
    if size == 0:
        raise TgError(-8, "tg_workspace_size")
    return _torch().zeros(size, dtype=_torch().uint8, device=device)


def trellis_gemv(layer: DeviceLayer, x, y=None, ws=None, stream=None):
    """y = W x for fp16 x [n] on the device; returns fp32 y [m]."""
    torch = _torch()
    if y is None:
        y = torch.empty(layer.m, dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(layer, 1, x.device)
    d = layer.desc()
    _check(lib().trellis_gemv(ctypes.byref(d), _ptr(x), _ptr(y), _ptr(ws), ws.numel(), _stream(stream)),
           "trellis_gemv")
    return y


def _layer_array(layers):
    arr = (TgLayer * len(layers))(*[L.desc() for L in layers])
    return arr


def fused_workspace(layers, device="cuda"):
    """Zero-filled workspace for trellis_gemv_fused over these layers."""
    size = int(lib().tg_fused_workspace_size(_layer_array(layers), len(layers)))
    if size == 0:
        raise TgError(-8, "tg_fused_workspace_size")
    return _torch().zeros(size, dtype=_torch().uint8, device=device)


def trellis_gemv_fused(layers, x, ys=None, ws=None, stream=None):
    """y_l = W_l x for layers that share the fp16 input x [n]; returns the list of fp32 outputs."""
    torch = _torch()
    if ys is None:
        ys = [torch.empty(L.m, dtype=torch.float32, device=x.device) for L in layers]
    if ws is None:
        ws = fused_workspace(layers, x.device)
    arr = _layer_array(layers)
    yp = (ctypes.c_void_p * len(layers))(*[y.data_ptr() for y in ys])
    _check(lib().trellis_gemv_fused(arr, len(layers), _ptr(x), yp, _ptr(ws), ws.numel() * ws.element_size(),
                                    _stream(stream)), "trellis_gemv_fused")
    return ys


def trellis_gemm_small(layer: DeviceLayer, X, Y=None, ws=None, stream=None):
    """Y[r] = W X[r] for fp16 X [M, n] (row stride X.stride(0)); returns fp32 Y [M, m]."""
    torch = _torch()
    M = X.shape[0]
    if Y is None:
        Y = torch.empty(M, layer.m, dtype=torch.float32, device=X.device)
    if ws is None:
        ws = workspace(layer, M, X.device)
    d = layer.desc()
    ldx = X.stride(0) if M > 1 else X.shape[1]      # a single row's stride is meaningless (may be 0)
    ldy = Y.stride(0) if M > 1 else Y.shape[1]
    _check(lib().trellis_gemm_small(ctypes.byref(d), M, _ptr(X), ldx, _ptr(Y), ldy,
                                    _ptr(ws), ws.numel(), _stream(stream)), "trellis_gemm_small")
    return Y


def rht_apply(x, signs, inverse: bool = False, out=None, stream=None):
    """Randomized Hadamard transform on 128-blocks of fp16 rows x [rows, n] -> fp32."""
    torch = _torch()
    x2 = x.reshape(-1, x.shape[-1])
    if out is None:
        out = torch.empty(x2.shape, dtype=torch.float32, device=x.device)
    _check(lib().rht_apply(x2.shape[1], x2.shape[0], _ptr(x2), _ptr(out), _ptr(signs), int(bool(inverse)),
                           _stream(stream)), "rht_apply")
    return out.reshape(x.shape)


class LayerTable:
    """Host and device copies of an array of tg_layer descriptors (for the grouped path)."""

    def __init__(self, layers: Sequence[DeviceLayer], device="cuda"):
        torch = _torch()
        self.layers = list(layers)
        self.host = (TgLayer * len(self.layers))(*[l.desc() for l in self.layers])
        raw = np.frombuffer(bytes(self.host), dtype=np.uint8)
        self.device = torch.from_numpy(raw.copy()).to(device)

    def __len__(self):
        return len(self.layers)


def grouped_workspace(table: LayerTable, n_sel: int, device="cuda"):
    size = int(lib().tg_grouped_workspace_size(table.host, len(table), n_sel))
    if size == 0:
        raise TgError(-8, "tg_grouped_workspace_size")
    return _torch().zeros(size, dtype=_torch().uint8, device=device)


def trellis_gemv_grouped(table: LayerTable, sel, X, x_stride: int, Y, y_stride: int, ws=None, stream=None):
    """For each e < len(sel): Y[e*y_stride : ...][:m] = W_{sel[e]} X[e*x_stride : ...] (x_stride 0 = shared x)."""
    n_sel = int(sel.numel())
    if ws is None:
        ws = grouped_workspace(table, n_sel, X.device)
    _check(lib().trellis_gemv_grouped(table.host, _ptr(table.device), len(table), _ptr(sel), n_sel,
                                      _ptr(X), x_stride, _ptr(Y), y_stride, _ptr(ws), ws.numel(), _stream(stream)),
           "trellis_gemv_grouped")
    return Y


def trellis_decode(layer: DeviceLayer, out=None, stream=None):
    """All decoded weights as fp16 patterns, int16 tensor [m, n]."""
    torch = _torch()
    if out is None:
        out = torch.empty(layer.m, layer.n, dtype=torch.int16, device=layer.codes.device)
    d = layer.desc()
    _check(lib().trellis_decode(ctypes.byref(d), _ptr(out), _stream(stream)), "trellis_decode")
    return out


def decode_ceiling(k_bits: int, code_id: int, workgroups: int, steps: int, out=None, stream=None, flags: int = 0):
    """Launch the decode-only rate probe; returns its fp32 output [workgroups * 512]."""
    torch = _torch()
    if out is None:
        out = torch.empty(workgroups * 512, dtype=torch.float32, device="cuda")
    _check(lib().tg_decode_ceiling(k_bits, code_id, int(flags), workgroups, steps, _ptr(out), _stream(stream)),
           "tg_decode_ceiling")
    return out


def code_table(device="cuda", code_id: int = 0, stream=None):
    """The code for all 65536 states: int16 [65536] (code 0) or [65536, 2] (pair code)."""
    torch = _torch()
    shape = (1 << 16, 2) if code_id == 1 else (1 << 16,)
    out = torch.empty(shape, dtype=torch.int16, device=device)
    _check(lib().tg_code_table(int(code_id), _ptr(out), _stream(stream)), "tg_code_table")
    return out


def encode_workspace(n_tiles: int, k_bits: int, code_id: int = 0, device="cuda"):
    torch = _torch()
    n = lib().tg_encode_workspace_size(int(n_tiles), int(k_bits), int(code_id))
    if n == 0:
        raise TgError(-8, "tg_encode_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def trellis_encode(targets, k_bits: int, code_id: int = 0, scale: float = 1.0, codes=None, sq_err=None, ws=None,
                   stream=None):
    """Viterbi-encode tiles: targets fp32 [n_tiles, 256] (sequence order) -> (codes int32 [n_tiles, 8K], sq_err)."""
    torch = _torch()
    if targets.dtype != torch.float32 or not targets.is_contiguous() or targets.shape[-1] != 256:
        raise ValueError("targets must be a contiguous float32 tensor [n_tiles, 256]")
    n_tiles = int(targets.shape[0])
    dev = targets.device
    if codes is None:
        codes = torch.empty(n_tiles, 8 * k_bits, dtype=torch.int32, device=dev)
    if sq_err is None:
        sq_err = torch.empty(n_tiles, dtype=torch.float32, device=dev)
    if ws is None:
        ws = encode_workspace(n_tiles, k_bits, code_id, dev)
    _check(lib().trellis_encode(n_tiles, int(k_bits), int(code_id), float(scale), _ptr(targets),
                                _ptr(codes), _ptr(sq_err), _ptr(ws), ws.numel(), _stream(stream)), "trellis_encode")
    return codes, sq_err


def prefill_workspace(layer: DeviceLayer, M: int, device="cuda"):
    torch = _torch()
    d = layer.desc()
    n = lib().tg_prefill_workspace_size(ctypes.byref(d), int(M))
    if n == 0:
        raise TgError(-2, "tg_prefill_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def trellis_gemm_prefill(layer: DeviceLayer, X, Y=None, ws=None, stream=None):
    """Y [M, m] fp32 = W X[r] for every row of fp16 X [M, n] (row stride X.stride(0)); each weight decoded once per 512 rows into MFMA operands."""
    torch = _torch()
    M = int(X.shape[0])
    if Y is None:
        Y = torch.empty(M, layer.m, dtype=torch.float32, device=X.device)
    if ws is None:
        ws = prefill_workspace(layer, M, X.device)
    d = layer.desc()
    ldx = X.stride(0) if M > 1 else X.shape[1]
    ldy = Y.stride(0) if M > 1 else Y.shape[1]
    _check(lib().trellis_gemm_prefill(ctypes.byref(d), M, _ptr(X), ldx, _ptr(Y), ldy, _ptr(ws), ws.numel(),
                                      _stream(stream)), "trellis_gemm_prefill")
    return Y


def moe_workspace(gate_up: "LayerTable", down: "LayerTable", top_k: int, device="cuda"):
    torch = _torch()
    n = lib().tg_moe_workspace_size(gate_up.host, len(gate_up), down.host, len(down), int(top_k))
    if n == 0:
        raise TgError(-8, "tg_moe_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def trellis_moe_block(gate_up: "LayerTable", down: "LayerTable", sel, weights, x, y=None, ws=None, stream=None):
    """y [hidden] fp32 = sum_i w_i down_{sel_i}(fp16(silu(gate(x)) * up(x))); sel int32 / weights fp32 on device."""
    torch = _torch()
    top_k = int(sel.numel())
    hidden = down.layers[0].m
    if y is None:
        y = torch.empty(hidden, dtype=torch.float32, device=x.device)
    if ws is None:
        ws = moe_workspace(gate_up, down, top_k, x.device)
    _check(lib().trellis_moe_block(gate_up.host, _ptr(gate_up.device), len(gate_up), down.host, _ptr(down.device),
                                   len(down), _ptr(sel), _ptr(weights), top_k, _ptr(x), _ptr(y), _ptr(ws),
                                   ws.numel(), _stream(stream)), "trellis_moe_block")
    return y


# ---- routing and 8-bit products ------------------------------------------------------------
# These entry points look at every tensor they are given -- type, shape, innermost stride, device --
# so that nothing of the wrong layout reaches a kernel. The work runs on the tensors' own device: on
# `stream`, or on that device's current stream. Small calls take a few microseconds on the GPU, so
# the common way through (no stream named, the tensors on the current device) is kept short; any
# other call enters its device and stream and comes back on the common way, and what it allocates
# belongs to that stream. The C entry points take sizes of 32 bits and ctypes would cut larger ones to
# their low half, so those (and negative ones) are refused here.

_DTYPES = {}


def _dtype_code(dtype, where: str) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        torch = _torch()
        _DTYPES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
        code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"{where}: expected float32, float16 or bfloat16, got {dtype}")
    return code


def _expect(ok: bool, where: str, what: str) -> None:
    if not ok:
        raise ValueError(f"{where}: {what}")


def _common_device(where: str, first, *others) -> int:
    """Index of the GPU that holds every tensor (None among the others is skipped)."""
    at = first.get_device()
    if at < 0:
        raise ValueError(f"{where}: expected tensors on a GPU, got {first.device}")
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError(f"{where}: tensors on {first.device} and {t.device}")
    return at


class _Entered:
    """The device and stream of a call, as the current ones."""

    def __init__(self, at: int, stream):
        torch = _torch()
        self._enter = [torch.cuda.device(at)]
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=torch.device("cuda", at))
            if stream.device.index != at:
                raise ValueError(f"a stream of {stream.device} for tensors on cuda:{at}")
            self._enter.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self._enter:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self._enter):
            c.__exit__(*exc)


def moe_route(logits, top_k: int, bias=None, sigmoid: bool = False, n_group: int = 1, topk_group: int = 1,
              group_top: int = 1, renormalize: bool = True, scale: float = 1.0, sel=None, weights=None, stream=None):
    """Expert ids int32 [tokens, top_k] and weights fp32 [tokens, top_k] of router logits [tokens, experts] (fp32, fp16 or
    bf16): scores by softmax or sigmoid, selection by score + bias within the best topk_group of n_group groups (a group's
    value: its group_top largest, summed), weights from the scores alone. Ids of slots without an expert are -1, weight 0."""
    torch = _torch()
    w = "moe_route"
    dtype = _dtype_code(logits.dtype, w)
    if logits.dim() != 2:
        raise ValueError(f"{w}: expected logits [tokens, experts]")
    tokens, experts = logits.shape
    if (tokens | experts | top_k | n_group | topk_group | group_top) >> 31:
        raise TgError(-2 if (tokens | experts) >> 31 else -8, w)
    ld, inner = logits.stride()
    if inner != 1 and experts != 1:
        raise ValueError(f"{w}: a token's logits have to be neighbours")
    if bias is not None:
        _expect(bias.dtype == torch.float32 and bias.shape == (experts,) and bias.is_contiguous(), w, f"expected a float32 bias [{experts}]")
    at = _common_device(w, logits, bias, sel, weights)
    if stream is not None or at != torch._C._cuda_getDevice():
        with _Entered(at, stream):
            return moe_route(logits, top_k, bias, sigmoid, n_group, topk_group, group_top, renormalize, scale, sel, weights)
    if sel is None:
        sel = torch.empty(tokens, top_k, dtype=torch.int32, device=logits.device)
    else:
        _expect(sel.dtype == torch.int32 and sel.shape == (tokens, top_k) and sel.is_contiguous(), w, f"expected sel int32 [{tokens}, {top_k}]")
    if weights is None:
        weights = torch.empty(tokens, top_k, dtype=torch.float32, device=logits.device)
    else:
        _expect(weights.dtype == torch.float32 and weights.shape == (tokens, top_k) and weights.is_contiguous(), w,
                f"expected weights float32 [{tokens}, {top_k}]")
    flags = (TG_ROUTE_SIGMOID if sigmoid else 0) | (TG_ROUTE_RENORM if renormalize else 0)
    status = (_lib or lib()).moe_route(tokens, experts, top_k, logits.data_ptr(), dtype, ld if tokens > 1 else experts, None if bias is None else bias.data_ptr(),
                           n_group, topk_group, group_top, flags, scale, sel.data_ptr(), weights.data_ptr(), torch._C._cuda_getCurrentRawStream(at))
    if status:
        raise TgError(status, w)
    return sel, weights


def moe_group(sel, experts: int, offsets=None, order=None, stream=None):
    """The routed pairs (token * top_k + slot) in expert order: offsets int32 [experts + 1] and order int32 [pairs], of
    int32 ids of any shape; the pairs whose id is no expert come last, behind offsets[experts]. The three do not overlap."""
    torch = _torch()
    w = "moe_group"
    if sel.dtype != torch.int32 or not sel.is_contiguous():
        raise ValueError(f"{w}: expected contiguous int32 ids")
    pairs = sel.numel()
    if (pairs | experts) >> 31:
        raise TgError(-2, w)
    at = _common_device(w, sel, offsets, order)
    if stream is not None or at != torch._C._cuda_getDevice():
        with _Entered(at, stream):
            return moe_group(sel, experts, offsets, order)
    if offsets is None:
        offsets = torch.empty(experts + 1, dtype=torch.int32, device=sel.device)
    else:
        _expect(offsets.dtype == torch.int32 and offsets.shape == (experts + 1,) and offsets.is_contiguous(), w,
                f"expected offsets int32 [{experts + 1}]")
    if order is None:
        order = torch.empty(pairs, dtype=torch.int32, device=sel.device)
    else:
        _expect(order.dtype == torch.int32 and order.shape == (pairs,) and order.is_contiguous(), w, f"expected order int32 [{pairs}]")
    status = (_lib or lib()).moe_group(pairs, experts, sel.data_ptr(), offsets.data_ptr(), order.data_ptr(), torch._C._cuda_getCurrentRawStream(at))
    if status:
        raise TgError(status, w)
    return offsets, order


def int8_quantize(x, q=None, scales=None, stream=None):
    """Rows x [..., n] (fp32, fp16 or bf16) as int8 [..., n] with a scale for each row (fp32 [...]): x is about q * scale. q and
    scales do not overlap x."""
    torch = _torch()
    w = "int8_quantize"
    dtype = _dtype_code(x.dtype, w)
    shape = x.shape
    if len(shape) < 1 or x.numel() == 0:
        raise ValueError(f"{w}: expected rows [..., n]")
    if (x.numel() // shape[-1] | shape[-1]) >> 31:
        raise TgError(-2, w)
    at = _common_device(w, x, q, scales)
    if stream is not None or at != torch._C._cuda_getDevice():
        with _Entered(at, stream):
            return int8_quantize(x, q, scales)
    lead, n = shape[:-1], shape[-1]
    x2 = x if len(shape) == 2 else x.reshape(-1, n)
    rows, ldq = x2.shape[0], n
    ldx, inner = x2.stride()
    if inner != 1 and n > 1:
        x2 = x2.contiguous()
        ldx = n
    if q is None:
        q = torch.empty(rows, n, dtype=torch.int8, device=x.device)
        if x2 is not x:
            q = q.view(shape)
    else:
        _expect(q.dtype == torch.int8 and q.shape == shape and (q.is_contiguous() or (q.dim() == 2 and q.stride(1) == 1 and q.stride(0) >= n)),
                w, "expected q int8 in the shape of x, with neighbouring values")
        if q.dim() == 2 and rows > 1:
            ldq = q.stride(0)
    if scales is None:
        scales = torch.empty(rows, dtype=torch.float32, device=x.device)
        if x2 is not x:
            scales = scales.view(lead)
    else:
        _expect(scales.dtype == torch.float32 and scales.shape == lead and scales.is_contiguous(), w, "expected a float32 scale for each row")
    status = (_lib or lib()).int8_quantize(rows, n, x2.data_ptr(), dtype, ldx if rows > 1 else n, q.data_ptr(), ldq, scales.data_ptr(),
                               torch._C._cuda_getCurrentRawStream(at))
    if status:
        raise TgError(status, w)
    return q, scales


class Int8Layer:
    """A linear layer kept at 8 bits: q int8 [m, n] with a scale for each output channel (fp32 [m])."""

    def __init__(self, q, scales):
        torch = _torch()
        w = "Int8Layer"
        _expect(q.dtype == torch.int8 and q.dim() == 2 and q.stride(1) == 1, w, "expected q int8 [m, n] with neighbouring inputs")
        _expect(scales.dtype == torch.float32 and scales.shape == q.shape[:1] and scales.is_contiguous(), w, "expected float32 scales [m]")
        _common_device(w, q, scales)
        self.q, self.scales, self.device = q, scales, q.device
        self.m, self.n = int(q.shape[0]), int(q.shape[1])
        self.ldw = q.stride(0) if self.m > 1 else self.n

    @classmethod
    def from_dense(cls, weight, stream=None):
        """The nearest 8-bit layer of a dense weight [m, n] (fp32, fp16 or bf16)."""
        return cls(*int8_quantize(weight, stream=stream))


class Int8Experts:
    """The experts of a block, kept at 8 bits: q int8 [experts, m, n], scales fp32 [experts, m]."""

    def __init__(self, q, scales):
        torch = _torch()
        w = "Int8Experts"
        _expect(q.dtype == torch.int8 and q.dim() == 3 and q.is_contiguous(), w, "expected contiguous q int8 [experts, m, n]")
        _expect(scales.dtype == torch.float32 and scales.shape == q.shape[:2] and scales.is_contiguous(), w, "expected float32 scales [experts, m]")
        _common_device(w, q, scales)
        self.q, self.scales, self.device = q, scales, q.device
        self.experts, self.m, self.n = (int(v) for v in q.shape)

    @classmethod
    def from_dense(cls, weight, stream=None):
        """The nearest 8-bit experts of dense weights [experts, m, n]."""
        return cls(*int8_quantize(weight, stream=stream))


def int8_workspace(layer: "Int8Layer", M: int):
    """Zero-filled workspace for int8_gemm with M rows of this layer."""
    torch = _torch()
    if (int(M) | layer.m | layer.n) >> 31:
        raise TgError(-2, "tg_int8_workspace_size")
    size = int(lib().tg_int8_workspace_size(int(M), layer.m, layer.n))
    if size == 0:
        raise TgError(-2, "tg_int8_workspace_size")
    return torch.zeros(size, dtype=torch.uint8, device=layer.device)


def _int8_rows(torch, where: str, n: int, xq, xs):
    if xq.dtype != torch.int8 or xq.dim() != 2:
        raise ValueError(f"{where}: expected xq int8 [rows, {n}]")
    rows, width = xq.shape
    ldx, inner = xq.stride()
    if width != n or inner != 1:
        raise ValueError(f"{where}: expected xq int8 [rows, {n}] with neighbouring values")
    if xs.dtype != torch.float32 or xs.shape != (rows,) or not xs.is_contiguous():
        raise ValueError(f"{where}: expected a float32 scale for each row of xq")
    return rows, (ldx if rows > 1 else n)


def _int8_out(torch, where: str, Y, rows: int, m: int, out_dtype, xq):
    if Y is None:
        dtype = torch.float32 if out_dtype is None else out_dtype
        code = _dtype_code(dtype, where)
        return torch.empty(rows, m, dtype=dtype, device=xq.device), code, m
    code = _dtype_code(Y.dtype, where)
    _expect(out_dtype is None or out_dtype == Y.dtype, where, "Y is not of out_dtype")
    _expect(Y.shape == (rows, m) and (Y.stride(1) == 1 or m == 1) and (rows == 1 or Y.stride(0) >= m), where, f"expected Y [{rows}, {m}] with neighbouring outputs")
    return Y, code, (Y.stride(0) if rows > 1 else m)


def int8_gemm(layer: "Int8Layer", xq, xs, Y=None, out_dtype=None, ws=None, stream=None):
    """Y [M, m] = (xq wq^T) * xs[r] * scales[o] of 8-bit rows xq [M, n] with scales xs [M]; out_dtype (or Y's type) float32,
    float16 or bfloat16."""
    torch = _torch()
    w = "int8_gemm"
    m, n = layer.m, layer.n
    M, ldx = _int8_rows(torch, w, n, xq, xs)
    if (M | m | n) >> 31:
        raise TgError(-2, w)
    at = _common_device(w, xq, xs, layer.q, Y, ws)
    if stream is not None or at != torch._C._cuda_getDevice():
        with _Entered(at, stream):
            return int8_gemm(layer, xq, xs, Y, out_dtype, ws)
    Y, code, ldy = _int8_out(torch, w, Y, M, m, out_dtype, xq)
    if ws is None:
        ws = int8_workspace(layer, M)
    elif not ws.is_contiguous():
        raise ValueError(f"{w}: expected a contiguous workspace")
    status = (_lib or lib()).int8_gemm(M, m, n, xq.data_ptr(), ldx, xs.data_ptr(), layer.q.data_ptr(), layer.ldw, layer.scales.data_ptr(),
                           Y.data_ptr(), code, ldy, ws.data_ptr(), ws.numel() * ws.element_size(), torch._C._cuda_getCurrentRawStream(at))
    if status:
        raise TgError(status, w)
    return Y


def int8_gemm_grouped(experts: "Int8Experts", xq, xs, offsets, order, pairs_per_row: int = 1, Y=None, out_dtype=None, stream=None):
    """Y [pairs, m]: row p = order[j], offsets[e] <= j < offsets[e + 1], is expert e's product with the 8-bit row
    xq[p // pairs_per_row]. Rows of pairs without an expert, which order lists behind offsets[-1], are zero in an output that
    the call makes, and left as they were in a Y of the caller's."""
    torch = _torch()
    w = "int8_gemm_grouped"
    m, n, count = experts.m, experts.n, experts.experts
    rows, ldx = _int8_rows(torch, w, n, xq, xs)
    pairs = rows * int(pairs_per_row)
    if (pairs | count | m | n) >> 31:
        raise TgError(-2, w)
    if order.dtype != torch.int32 or order.shape != (pairs,) or not order.is_contiguous():
        raise ValueError(f"{w}: expected order int32 [{pairs}]")
    if offsets.dtype != torch.int32 or offsets.shape != (count + 1,) or not offsets.is_contiguous():
        raise ValueError(f"{w}: expected offsets int32 [{count + 1}]")
    at = _common_device(w, xq, xs, experts.q, offsets, order, Y)
    if stream is not None or at != torch._C._cuda_getDevice():
        with _Entered(at, stream):
            return int8_gemm_grouped(experts, xq, xs, offsets, order, pairs_per_row, Y, out_dtype)
    zero = TG_ZERO_UNROUTED if Y is None else 0
    Y, code, ldy = _int8_out(torch, w, Y, pairs, m, out_dtype, xq)
    status = (_lib or lib()).int8_gemm_grouped(pairs, count, m, n, xq.data_ptr(), ldx, xs.data_ptr(), int(pairs_per_row), experts.q.data_ptr(),
                                   experts.scales.data_ptr(), offsets.data_ptr(), order.data_ptr(), Y.data_ptr(), code | zero, ldy,
                                   torch._C._cuda_getCurrentRawStream(at))
    if status:
        raise TgError(status, w)
    return Y


class Int8Linear:
    """An 8-bit linear layer used like a dense one, beside TrellisLinear: y = W x over the last axis.

    `forward(x)` takes fp32, fp16 or bf16 activations [..., n] on the device, quantises each row with a scale of its own
    (int8_quantize) and returns fp32 [..., m] (int8_gemm). The workspace is kept and replaced by a larger one when a row
    count needs it (the earlier ones live on, for graphs that were captured with them; a call under capture that needs a
    larger one takes the graph's own, cleared at each replay); calls are ordered on one stream.
    """

    def __init__(self, layer: "Int8Layer"):
        self.layer = layer
        self._ws, self._earlier = None, []

    def forward(self, x, stream=None):
        n, m = self.layer.n, self.layer.m
        _expect(x.dim() > 0 and x.shape[-1] == n, "Int8Linear", f"expected activations [..., {n}], got {tuple(x.shape)}")
        if stream is not None or _common_device("Int8Linear", x, self.layer.q) != _torch()._C._cuda_getDevice():
            with _Entered(x.get_device(), stream):
                return self.forward(x)
        xq, xs = int8_quantize(x)
        xq, xs = xq.view(-1, n), xs.view(-1)
        ws = self._ws
        if ws is None or ws.numel() < lib().tg_int8_workspace_size(xq.shape[0], m, n):
            ws = int8_workspace(self.layer, xq.shape[0])
            if not _torch().cuda.is_current_stream_capturing():   # else its zeros are the graph's, there at its replays alone
                self._earlier.append(self._ws)
                self._ws = ws
        return int8_gemm(self.layer, xq, xs, ws=ws).reshape(x.shape[:-1] + (m,))

    __call__ = forward


class TrellisLinear:
    """A trellis-coded linear layer used like a dense one: y = W x over the last axis.

    `forward(x)` takes fp16 activations [..., n] on the device and returns fp32 [..., m]. It
    picks the entry point by the number of rows R (the product of the leading axes), as the
    pages' drop-in linear does for its batch sizes ("Trellis Quantization" lecture, Part
    eleven: small batches decode per call, prefill decodes once):
      R == 1                 -> trellis_gemv
      R <= 64                -> trellis_gemm_small
      R <  prefill_min_rows  -> trellis_gemm_small on row chunks of 64
      otherwise              -> trellis_gemm_prefill (decode once per 512 rows into MFMA operands)
    The default threshold (128 rows) sits at the measured crossover of the last two on the
    8192 -> 28672 gate shape (96 rows: chunked small batch faster; 128: prefill faster). Workspaces are allocated on first use of each path and kept
    (the prefill one grows with the largest row count seen); calls are ordered on one stream.
    """

    SMALL_MAX_ROWS = 64

    def __init__(self, layer: DeviceLayer, prefill_min_rows: int = 128):
        self.layer = layer
        self.prefill_min_rows = int(prefill_min_rows)
        self._ws = None
        self._prefill_ws, self._prefill_rows = None, 0

    @classmethod
    def path_for_rows(cls, rows: int, prefill_min_rows: int = 128) -> str:
        if rows < 1:
            raise ValueError("no rows")
        if rows == 1:
            return "gemv"
        if rows <= cls.SMALL_MAX_ROWS:
            return "small"
        return "small_chunked" if rows < prefill_min_rows else "prefill"

    def _layer_ws(self, device):
        if self._ws is None:   # one buffer for every row count up to 64 (the split count varies with it)
            size = max(workspace_size(self.layer, M) for M in range(1, self.SMALL_MAX_ROWS + 1))
            self._ws = _torch().zeros(size, dtype=_torch().uint8, device=device)
        return self._ws

    def forward(self, x, stream=None):
        torch = _torch()
        n, m = self.layer.n, self.layer.m
        if x.dtype != torch.float16 or x.shape[-1] != n:
            raise ValueError(f"expected float16 activations [..., {n}], got {tuple(x.shape)} {x.dtype}")
        lead = tuple(x.shape[:-1])
        X = x.reshape(-1, n).contiguous()
        rows = X.shape[0]
        path = self.path_for_rows(rows, self.prefill_min_rows)
        Y = torch.empty(rows, m, dtype=torch.float32, device=x.device)
        if path == "gemv":
            trellis_gemv(self.layer, X[0], Y[0], self._layer_ws(x.device), stream)
        elif path == "prefill":
            if rows > self._prefill_rows:
                self._prefill_ws, self._prefill_rows = prefill_workspace(self.layer, rows, x.device), rows
            trellis_gemm_prefill(self.layer, X, Y, self._prefill_ws, stream)
        else:
            ws = self._layer_ws(x.device)
            for r0 in range(0, rows, self.SMALL_MAX_ROWS):
                r1 = min(rows, r0 + self.SMALL_MAX_ROWS)
                trellis_gemm_small(self.layer, X[r0:r1], Y[r0:r1], ws, stream)
        return Y.reshape(lead + (m,))

    __call__ = forward
