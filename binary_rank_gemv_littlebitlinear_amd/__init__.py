"""Python binding of the LittleBit linear-forward C ABI (``include/lb.h``).

Argument marshalling only: every step of the forward runs in the HIP
library ``liblb.so`` built next to this file.  There is no fallback: if
the library is missing, loading fails loudly.  torch is used for device
memory and streams only (tensors are passed as raw pointers).

Functions keep the C names (``lb_create``, ``lb_pack_signs``, ...);
``Layer`` and ``Stack`` are thin owners that call them.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblb.so")

LB_F16, LB_F32 = 0, 1
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
LB_OK, LB_EINVAL, LB_ENOMEM, LB_EHIP, LB_ENOTREADY, LB_EUNSUPPORTED, LB_ETIMEOUT = 0, -1, -2, -3, -4, -5, -6


class LBError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_status_name(status)}: {msg}")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH):
    """Load liblb.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"HIP library not built: {path} is missing "
                           "(run python -m binary_rank_gemv_littlebitlinear_amd.build)")
    lib = C.CDLL(path)
    vp, i64, i32, u64 = C.c_void_p, C.c_int64, C.c_int, C.c_uint64
    P = C.POINTER
    sig = {
        "lb_create": ([i64, i64, i64, i32, P(vp)], i32),
        "lb_pack_signs": ([vp, i32, vp, vp], i32),
        "lb_set_scales": ([vp, i32, vp, vp, vp], i32),
        "lb_forward": ([vp, vp, vp, i64, vp], i32),
        "lb_forward_noalloc": ([vp, vp, vp, i64, vp], i32),
        "lb_unpack_signs": ([vp, i32, vp, vp], i32),
        "lb_get_scales": ([vp, i32, vp, vp, vp], i32),
        "lb_init_from_factors": ([vp, i32, vp, vp, vp, vp], i32),
        "lb_joint_itq": ([vp, vp, i64, i64, i64, i32, vp, vp, vp], i32),
        "lb_layer_shape": ([vp, P(i64), P(i64), P(i64), P(i32)], i32),
        "lb_prepare": ([vp, i64], i32),
        "lb_layer_device_bytes": ([vp, P(u64), P(u64)], i32),
        "lb_destroy": ([vp], i32),
        "lb_forward_stage1": ([vp, vp, vp, i64, vp], i32),
        "lb_forward_stage2": ([vp, vp, vp, i64, vp], i32),
        "lb_eff_bits": ([i64, i64, i64, i32, P(u64), P(u64)], i32),
        "lb_rank_for_bpw": ([i64, i64, u64, u64, i32, P(i64)], i32),
        "lb_stack_create": ([vp, i32, vp, i32, C.c_float, P(vp)], i32),
        "lb_stack_forward": ([vp, vp, vp, vp, i64, vp], i32),
        "lb_stack_trace_elems": ([vp, i64, P(i64)], i32),
        "lb_stack_reserve": ([vp, i64], i32),
        "lb_stack_set_mode": ([vp, i32], i32),
        "lb_stack_check": ([vp], i32),
        "lb_stack_test_wait_failure": ([vp, i32], i32),
        "lb_stack_test_delay": ([vp, C.c_uint32, C.c_uint32], i32),
        "lb_stack_timeline": ([vp, vp, i64, P(i64)], i32),
        "lb_stack_destroy": ([vp], i32),
        "lb_bank_create": ([vp, vp, i32, P(vp)], i32),
        "lb_bank_shape": ([vp, P(i32), P(i32), P(i64), P(i64), P(i32)], i32),
        "lb_bank_reserve": ([vp, i64], i32),
        "lb_bank_forward": ([vp, i32, vp, i64, vp, i64, i32, i64, i32, vp, vp, vp, i64, vp], i32),
        "lb_bank_grouped": ([vp, vp, i64, i64, vp, vp, i64, vp, i64, i32, i32, vp, vp, vp, i64, vp], i32),
        "lb_bank_destroy": ([vp], i32),
        "lb_route_ws_bytes": ([i64, i32, i32, P(u64)], i32),
        "lb_route": ([vp, i32, i64, i64, i32, i32, i32, vp, vp, vp, vp, vp, vp, u64, vp], i32),
        "lb_route_combine": ([vp, i64, i64, vp, vp, i64, i32, i64, vp, i64, vp, i64, i32, vp], i32),
        "lb_norm": ([i32, vp, i32, i64, i32, vp, vp, vp, i64, vp, i64, C.c_float, i32, vp, vp, C.c_float, vp, i64, vp,
                     i64, i64, i64, vp], i32),
        "lb_cache_create": ([i64, i32, i32, i32, P(vp)], i32),
        "lb_cache_shape": ([vp, P(i64), P(i32), P(i32), P(i32), P(i32)], i32),
        "lb_cache_append": ([vp, vp, i64, vp, i64, vp, i64, vp, i64, i32, vp, i64, i32, i32, vp, vp, vp, i64, i32, i32,
                             i64, vp], i32),
        "lb_cache_read": ([vp, vp, i64, vp, i64, vp, vp, vp, i64, i32, i32, i64, vp], i32),
        "lb_cache_reserve": ([vp, i64, i32, i64, i64], i32),
        "lb_cache_attend": ([vp, vp, i64, i32, vp, i64, vp, vp, vp, i64, i32, i32, i64, i64, C.c_float, i32, i32, vp],
                            i32),
        "lb_cache_destroy": ([vp], i32),
        "lb_status_str": ([i32], C.c_char_p),
        "lb_last_error": ([], C.c_char_p),
        "lb_version": ([], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


EXPORTED = ("lb_create", "lb_pack_signs", "lb_set_scales", "lb_forward", "lb_forward_noalloc",
            "lb_unpack_signs",
            "lb_get_scales", "lb_init_from_factors", "lb_joint_itq",
            "lb_layer_shape", "lb_prepare", "lb_layer_device_bytes", "lb_destroy", "lb_forward_stage1", "lb_forward_stage2",
            "lb_eff_bits", "lb_rank_for_bpw", "lb_stack_create", "lb_stack_forward",
            "lb_stack_trace_elems", "lb_stack_reserve", "lb_stack_set_mode", "lb_stack_check",
            "lb_stack_test_wait_failure", "lb_stack_test_delay",
            "lb_stack_timeline", "lb_stack_destroy",
            "lb_bank_create", "lb_bank_shape", "lb_bank_reserve", "lb_bank_forward", "lb_bank_grouped", "lb_bank_destroy",
            "lb_route_ws_bytes", "lb_route", "lb_route_combine",
            "lb_norm", "lb_cache_create", "lb_cache_shape", "lb_cache_append", "lb_cache_read", "lb_cache_reserve",
            "lb_cache_attend", "lb_cache_destroy", "lb_status_str", "lb_last_error", "lb_version")


def _status_name(st: int) -> str:
    names = {0: "LB_OK", -1: "LB_EINVAL", -2: "LB_ENOMEM", -3: "LB_EHIP", -4: "LB_ENOTREADY",
             -5: "LB_EUNSUPPORTED", -6: "LB_ETIMEOUT"}
    return names.get(st, f"status {st}")


def _check(st: int):
    if st != LB_OK:
        msg = load_library().lb_last_error().decode(errors="replace")
        raise LBError(st, msg)


def _ptr(t) -> int | None:
    """Device pointer of a torch tensor / raw int / None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        try:
            import torch
            if torch.cuda.is_available():
                return torch.cuda.current_stream().cuda_stream
        except Exception:
            pass
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _host(arr, dtype) -> np.ndarray:
    a = np.ascontiguousarray(arr)
    if a.dtype != dtype:
        a = np.ascontiguousarray(a.view(dtype) if a.dtype.itemsize == np.dtype(dtype).itemsize else a.astype(dtype))
    return a


# ------------------------------------------------------------ raw calls
def lb_create(a: int, b: int, s: int, residual: bool) -> int:
    out = C.c_void_p()
    _check(load_library().lb_create(a, b, s, int(bool(residual)), C.byref(out)))
    return out.value


def lb_pack_signs(layer: int, path: int, su_words, sv_words):
    su = _host(su_words, np.uint32)
    sv = _host(sv_words, np.uint32)
    _check(load_library().lb_pack_signs(layer, path, su.ctypes.data, sv.ctypes.data))


def lb_set_scales(layer: int, path: int, h, g, l):
    hh = _host(np.asarray(h, np.float16), np.uint16)
    gg = _host(np.asarray(g, np.float16), np.uint16)
    ll = _host(np.asarray(l, np.float16), np.uint16)
    _check(load_library().lb_set_scales(layer, path, hh.ctypes.data, gg.ctypes.data, ll.ctypes.data))


def lb_forward(layer: int, x, y, M: int, stream=None):
    _check(load_library().lb_forward(layer, _ptr(x), _ptr(y), int(M), _stream(stream)))


def lb_forward_noalloc(layer: int, x, y, M: int, stream=None):
    _check(load_library().lb_forward_noalloc(layer, _ptr(x), _ptr(y), int(M), _stream(stream)))


def lb_forward_stage1(layer: int, x, w, M: int, stream=None):
    _check(load_library().lb_forward_stage1(layer, _ptr(x), _ptr(w), int(M), _stream(stream)))


def lb_forward_stage2(layer: int, w, y, M: int, stream=None):
    _check(load_library().lb_forward_stage2(layer, _ptr(w), _ptr(y), int(M), _stream(stream)))


def lb_unpack_signs(layer: int, path: int):
    a, b, s, _ = lb_layer_shape(layer)
    wk = (s + 31) // 32
    su = np.zeros((b, wk), np.uint32)
    sv = np.zeros((a, wk), np.uint32)
    _check(load_library().lb_unpack_signs(layer, path, su.ctypes.data, sv.ctypes.data))
    return su, sv


def lb_get_scales(layer: int, path: int):
    """(h, g, l) of one path as fp16 arrays."""
    a, b, s, _ = lb_layer_shape(layer)
    h = np.zeros(b, np.uint16)
    g = np.zeros(a, np.uint16)
    l = np.zeros(s, np.uint16)
    _check(load_library().lb_get_scales(layer, path, h.ctypes.data, g.ctypes.data, l.ctypes.data))
    return h.view(np.float16), g.view(np.float16), l.view(np.float16)


def _check_dev(name, t, shape, dtype):
    if isinstance(t, int) or t is None:
        return
    if (t.dtype != dtype or not t.is_contiguous() or t.device.type != "cuda"
            or tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must be a contiguous {dtype} device tensor of shape {shape}")


def lb_init_from_factors(layer: int, path: int, U, V, R=None, stream=None):
    """Signs and scales of one path from device fp32 factors U (b x s), V (a x s),
    rotated first by the device fp64 rotation R (s x s) when given."""
    import torch
    a, b, s, _ = lb_layer_shape(layer)
    _check_dev("U", U, (b, s), torch.float32)
    _check_dev("V", V, (a, s), torch.float32)
    _check_dev("R", R, (s, s), torch.float64)
    _check(load_library().lb_init_from_factors(layer, path, _ptr(U), _ptr(V), _ptr(R),
                                               _stream(stream)))


def lb_joint_itq(U, V, iters: int = 50, R0=None, stream=None):
    """Joint-ITQ rotation (device fp64 s x s tensor) of device fp32 factors U (b x s), V (a x s)."""
    import torch
    b, s = U.shape
    a = V.shape[0]
    _check_dev("U", U, (b, s), torch.float32)
    _check_dev("V", V, (a, s), torch.float32)
    _check_dev("R0", R0, (s, s), torch.float64)
    R = torch.empty((s, s), dtype=torch.float64, device=U.device)
    _check(load_library().lb_joint_itq(_ptr(U), _ptr(V), a, b, s, int(iters), _ptr(R0), _ptr(R),
                                       _stream(stream)))
    return R


def lb_layer_shape(layer: int):
    a, b, s, r = C.c_int64(), C.c_int64(), C.c_int64(), C.c_int()
    _check(load_library().lb_layer_shape(layer, C.byref(a), C.byref(b), C.byref(s), C.byref(r)))
    return a.value, b.value, s.value, bool(r.value)


def lb_prepare(layer: int, M: int):
    _check(load_library().lb_prepare(layer, int(M)))


def lb_layer_device_bytes(layer: int):
    sb, tb = C.c_uint64(), C.c_uint64()
    _check(load_library().lb_layer_device_bytes(layer, C.byref(sb), C.byref(tb)))
    return sb.value, tb.value


def lb_destroy(layer: int):
    _check(load_library().lb_destroy(layer))


def lb_eff_bits(a: int, b: int, s: int, residual: bool):
    n, d = C.c_uint64(), C.c_uint64()
    _check(load_library().lb_eff_bits(a, b, s, int(bool(residual)), C.byref(n), C.byref(d)))
    return n.value, d.value


def lb_rank_for_bpw(a: int, b: int, bpw_num: int, bpw_den: int, residual: bool) -> int:
    s = C.c_int64()
    _check(load_library().lb_rank_for_bpw(a, b, bpw_num, bpw_den, int(bool(residual)), C.byref(s)))
    return s.value


def lb_stack_create(layers, unit_sizes, kappa: float) -> int:
    arr = (C.c_void_p * len(layers))(*layers)
    us = np.ascontiguousarray(unit_sizes, dtype=np.int32)
    out = C.c_void_p()
    _check(load_library().lb_stack_create(C.cast(arr, C.c_void_p), len(layers), us.ctypes.data,
                                          len(us), float(kappa), C.byref(out)))
    return out.value


def lb_stack_forward(stack: int, x0, y, trace, M: int, stream=None):
    _check(load_library().lb_stack_forward(stack, _ptr(x0), _ptr(y), _ptr(trace), int(M),
                                           _stream(stream)))


def lb_stack_trace_elems(stack: int, M: int) -> int:
    n = C.c_int64()
    _check(load_library().lb_stack_trace_elems(stack, int(M), C.byref(n)))
    return n.value


def lb_stack_reserve(stack: int, M: int):
    _check(load_library().lb_stack_reserve(stack, int(M)))


def lb_stack_set_mode(stack: int, mode: int):
    _check(load_library().lb_stack_set_mode(stack, int(mode)))


def lb_stack_test_wait_failure(stack: int, enable: bool):
    _check(load_library().lb_stack_test_wait_failure(stack, int(bool(enable))))


def lb_stack_test_delay(stack: int, seed: int, max_ticks: int):
    _check(load_library().lb_stack_test_delay(stack, int(seed), int(max_ticks)))


def lb_stack_check(stack: int):
    _check(load_library().lb_stack_check(stack))


def lb_stack_timeline(stack: int, buf=None, capacity: int = 0) -> int:
    n = C.c_int64()
    _check(load_library().lb_stack_timeline(stack, _ptr(buf), int(capacity), C.byref(n)))
    return n.value


def lb_stack_destroy(stack: int):
    _check(load_library().lb_stack_destroy(stack))


def lb_bank_create(layers, gates=None) -> int:
    arr = (C.c_void_p * len(layers))(*layers)
    if gates is not None and len(gates) != len(layers):
        raise ValueError("a bank needs as many gates as layers")
    gar = (C.c_void_p * len(gates))(*gates) if gates is not None else None
    out = C.c_void_p()
    _check(load_library().lb_bank_create(C.cast(arr, C.c_void_p), C.cast(gar, C.c_void_p) if gar else None,
                                         len(layers), C.byref(out)))
    return out.value


def lb_bank_shape(bank: int):
    """(layers, gated, a, b, device) of a bank."""
    n, g, d, a, b = C.c_int(), C.c_int(), C.c_int(), C.c_int64(), C.c_int64()
    _check(load_library().lb_bank_shape(bank, C.byref(n), C.byref(g), C.byref(a), C.byref(b), C.byref(d)))
    return n.value, bool(g.value), a.value, b.value, d.value


def lb_bank_reserve(bank: int, rows: int):
    _check(load_library().lb_bank_reserve(bank, int(rows)))


def _say(t) -> str:
    return f"{tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}"


# The checks below run on every call of operators that take microseconds: they read each attribute once, compare
# device numbers (-1: not on a GPU) and leave the wording of errors to the failing case.
def _rows(name, t, width, dtypes, dev):
    """(rows, row stride) of a 2-d tensor of `width` columns with unit column stride on GPU `dev`."""
    shape = t.shape
    if len(shape) == 2:
        rows, cols = shape
        ld, unit = t.stride()
        if cols == width and (unit == 1 or width == 1) and t.dtype in dtypes and t.get_device() == dev:
            # a single row's stride is never used; torch leaves it arbitrary
            return rows, ld if rows > 1 else width
    raise ValueError(f"{name} must be 2-d with {width} unit-stride columns, of {dtypes}, on GPU {dev}, not {_say(t)}")


def _flat(name, t, shape, dtype, dev):
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on GPU {dev}, not {_say(t)}")
    return t.data_ptr()


def _stream_of(stream, dev):
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _on_device(dev, fn, *args):
    """Calls the library with GPU `dev` current (for calls that have no object to take the device from)."""
    import torch
    if torch._C._cuda_getDevice() == dev:
        return _check(fn(*args))
    with torch.cuda.device(dev):
        _check(fn(*args))


_f16 = _f32 = _i32 = _f16_f32 = _only_f16 = None


def _types():
    global _f16, _f32, _i32, _f16_f32, _only_f16
    if _f16 is None:
        import torch
        _f16, _f32, _i32 = torch.float16, torch.float32, torch.int32
        _f16_f32, _only_f16 = (_f16, _f32), (_f16,)


def _epilogue(bank, y, act, bias, gate_bias, residual):
    """The arguments that lb_bank_forward and lb_bank_grouped share: GPU, rows, then in the C order."""
    _types()
    dev, b, n = bank.device, bank.b, bank.n
    rows, ldy = _rows("y", y, b, _f16_f32, dev)
    dtype = y.dtype
    if act is None:
        act = 0
    else:
        try:
            act = ACTIVATIONS[act]
        except KeyError:
            raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, not {act!r}") from None
    pb = pg = pr = None
    ldr = 0
    if bias is not None:
        pb = _flat("bias", bias, (n, b), _f16, dev)
    if gate_bias is not None:
        pg = _flat("gate_bias", gate_bias, (n, b), _f16, dev)
    if residual is not None:
        rr, ldr = _rows("residual", residual, b, (dtype,), dev)
        if rr != rows:
            raise ValueError("residual must have y's rows")
        pr = residual.data_ptr()
    return dev, rows, y.data_ptr(), ldy, LB_F32 if dtype is _f32 else LB_F16, act, pb, pg, pr, ldr


def lb_bank_forward(bank, x, y, expert: int = 0, act=None, bias=None, gate_bias=None, residual=None, stream=None):
    """``Bank`` owner and tensors: y = act(layer(x) + bias) + residual (see include/lb.h)."""
    dev, rows, py, ldy, yt, act, pb, pg, pr, ldr = _epilogue(bank, y, act, bias, gate_bias, residual)
    xr, ldx = _rows("x", x, bank.a, _only_f16, dev)
    if xr != rows:
        raise ValueError("x and y must have the same number of rows")
    _check(_lib.lb_bank_forward(bank.handle, int(expert), x.data_ptr(), ldx, py, ldy, yt, rows, act, pb, pg, pr, ldr,
                                _stream_of(stream, dev)))


def lb_bank_grouped(bank, x, offsets, y, index=None, act=None, bias=None, gate_bias=None, residual=None,
                    stream=None):
    """``Bank`` owner and tensors: rows offsets[e]..offsets[e+1]-1 through layer e (see include/lb.h)."""
    dev, rows, py, ldy, yt, act, pb, pg, pr, ldr = _epilogue(bank, y, act, bias, gate_bias, residual)
    xr, ldx = _rows("x", x, bank.a, _only_f16, dev)
    po = _flat("offsets", offsets, (bank.n + 1,), _i32, dev)
    pi = _flat("index", index, (rows,), _i32, dev) if index is not None else None
    _check(_lib.lb_bank_grouped(bank.handle, x.data_ptr(), xr, ldx, pi, po, rows, py, ldy, yt, act, pb, pg, pr, ldr,
                                _stream_of(stream, dev)))


def lb_bank_destroy(bank: int):
    _check(load_library().lb_bank_destroy(bank))


def lb_route_ws_bytes(tokens: int, experts: int, k: int) -> int:
    n = C.c_uint64()
    _check(load_library().lb_route_ws_bytes(int(tokens), int(experts), int(k), C.byref(n)))
    return n.value


def lb_route(logits, k: int, renormalise: bool, ids, weights, offsets, token, row, ws, stream=None):
    """Tensors of include/lb.h's lb_route; ws is a device byte tensor of lb_route_ws_bytes bytes, or None."""
    _types()
    dev = logits.get_device()
    if logits.dim() != 2 or dev < 0:
        raise ValueError("logits must be a 2-d device tensor")
    e = logits.shape[1]
    t, ld = _rows("logits", logits, e, _f16_f32, dev)
    n, pw = 0, None
    if ws is not None:
        import torch
        n = ws.numel()
        pw = _flat("ws", ws, (n,), torch.uint8, dev)
    _on_device(dev, load_library().lb_route, logits.data_ptr(), LB_F32 if logits.dtype is _f32 else LB_F16, ld, t, e, k,
               1 if renormalise else 0, _flat("ids", ids, (t, k), _i32, dev), _flat("weights", weights, (t, k), _f32, dev),
               _flat("offsets", offsets, (e + 1,), _i32, dev), _flat("token", token, (t * k,), _i32, dev),
               _flat("row", row, (t, k), _i32, dev), pw, n, _stream_of(stream, dev))


def lb_route_combine(y, row, weights, out, residual=None, stream=None):
    """out[t] = residual[t] + sum_j weights[t, j] * y[row[t, j]] (see include/lb.h)."""
    _types()
    dev = out.get_device()
    if out.dim() != 2 or row.dim() != 2 or dev < 0:
        raise ValueError("out must be a 2-d device tensor and row a 2-d tensor")
    width, k, dtype = out.shape[1], row.shape[1], out.dtype
    t, ldo = _rows("out", out, width, _f16_f32, dev)
    yr, ldy = _rows("y", y, width, _only_f16, dev)
    pr, ldr = None, 0
    if residual is not None:
        rr, ldr = _rows("residual", residual, width, (dtype,), dev)
        if rr != t:
            raise ValueError("residual must have out's rows")
        pr = residual.data_ptr()
    _on_device(dev, load_library().lb_route_combine, y.data_ptr(), yr, ldy, _flat("row", row, (t, k), _i32, dev),
               _flat("weights", weights, (t, k), _f32, dev), t, k, width, pr, ldr, out.data_ptr(), ldo,
               LB_F32 if dtype is _f32 else LB_F16, _stream_of(stream, dev))


NORMS = {"rms": 0, "layer": 1}


def _like(name, t, rows, width, dtypes, dev):
    """(pointer, row stride) of a tensor that must have `rows` rows (see _rows)."""
    n, ld = _rows(name, t, width, dtypes, dev)
    if n != rows:
        raise ValueError(f"{name} must have {rows} rows, not {n}")
    return t.data_ptr(), ld


def lb_norm(r, x=None, y=None, out=None, kind="rms", weight=None, bias=None, post=False, post_weight=None,
            post_bias=None, gate=None, scale=1.0, eps=1e-5, stream=None):
    """out = scale * r + gate * (norm of) y, x = its norm (see include/lb.h).

    r and y may be None, not both; gate has one row or a row for each of r's."""
    _types()
    lead = y if r is None else r
    if lead is None:
        raise ValueError("lb_norm needs r or y")
    dev = lead.get_device()
    if lead.dim() != 2 or dev < 0:
        raise ValueError("r and y must be 2-d device tensors")
    k = NORMS.get(kind)
    if k is None:
        raise ValueError(f"kind must be one of {sorted(NORMS)}, not {kind!r}")
    rows, width = lead.shape
    like = out if r is None else r
    rtype = _f16 if like is None else like.dtype
    if rtype is not _f16 and rtype is not _f32:
        raise ValueError(f"the residual must be {_f16} or {_f32}, not {rtype}")
    py = pr = po = px = pg = w = b = pw = pb = None
    ldy = ldr = ldo = ldx = ldg = ytype = 0
    if y is not None:
        py, ldy = _like("y", y, rows, width, _f16_f32, dev)
        ytype = LB_F32 if y.dtype is _f32 else LB_F16
    if r is not None:
        pr, ldr = _like("r", r, rows, width, _f16_f32, dev)
    if out is not None:
        po, ldo = _like("out", out, rows, width, (rtype,), dev)
    if x is not None:
        px, ldx = _like("x", x, rows, width, _only_f16, dev)
    if gate is not None:
        n, ldg = _rows("gate", gate, width, _only_f16, dev)
        if n == 1:
            ldg = 0
        elif n != rows:
            raise ValueError(f"gate must have 1 or {rows} rows, not {n}")
        pg = gate.data_ptr()
    if weight is not None:
        w = _flat("weight", weight, (width,), _f16, dev)
    if bias is not None:
        b = _flat("bias", bias, (width,), _f16, dev)
    if post_weight is not None:
        pw = _flat("post_weight", post_weight, (width,), _f16, dev)
    if post_bias is not None:
        pb = _flat("post_bias", post_bias, (width,), _f16, dev)
    _on_device(dev, load_library().lb_norm, k, py, ytype, ldy, 1 if post else 0, pw, pb, pg, ldg, pr, ldr, scale,
               LB_F32 if rtype is _f32 else LB_F16, w, b, eps, po, ldo, px, ldx, rows, width, _stream_of(stream, dev))


def _int32(name, v):
    """A number for a C int, which ctypes would cut to its lower bits."""
    v = int(v)
    if not -0x80000000 <= v <= 0x7fffffff:
        raise ValueError(f"{name} must fit 32 bits, not {v}")
    return v


def lb_cache_create(pages: int, page_tokens: int, kv_heads: int, head_dim: int) -> int:
    out = C.c_void_p()
    _check(load_library().lb_cache_create(int(pages), _int32("page_tokens", page_tokens), _int32("kv_heads", kv_heads),
                                          _int32("head_dim", head_dim), C.byref(out)))
    return out.value


def lb_cache_shape(cache: int):
    """(pages, page_tokens, kv_heads, head_dim, device) of a cache."""
    n, p, k, d, dev = C.c_int64(), C.c_int(), C.c_int(), C.c_int(), C.c_int()
    _check(load_library().lb_cache_shape(cache, C.byref(n), C.byref(p), C.byref(k), C.byref(d), C.byref(dev)))
    return n.value, p.value, k.value, d.value, dev.value


def lb_cache_reserve(cache: int, rows: int, heads: int, sequences: int, max_length: int):
    _check(load_library().lb_cache_reserve(cache, int(rows), _int32("heads", heads), int(sequences), int(max_length)))


def _sequences(rows, lengths, table, start, dev):
    """start, lengths, table, its row stride, columns, sequences, rows: the C order."""
    if table.dim() != 2 or table.dtype is not _i32 or table.get_device() != dev:
        raise ValueError(f"table must be a 2-d {_i32} tensor on GPU {dev}, not {_say(table)}")
    (n, columns), (ld, unit) = table.shape, table.stride()
    if unit != 1 and columns > 1:
        raise ValueError(f"table must have unit-stride columns, not {_say(table)}")
    if start is not None:
        start = _flat("start", start, (n + 1,), _i32, dev)
    elif rows != n:
        raise ValueError(f"without start there is a row for each sequence: {n}, not {rows}")
    return start, _flat("lengths", lengths, (n,), _i32, dev), table.data_ptr(), ld if n > 1 else columns, columns, n, rows


def _heads(name, t, dim, dev):
    """(pointer, row stride, rows, heads) of a 2-d tensor with `dim` columns for each head."""
    width = t.shape[1] if t.dim() == 2 else 0
    if not width or width % dim:
        raise ValueError(f"{name} must be 2-d with {dim} columns for each head, not {_say(t)}")
    rows, ld = _rows(name, t, width, _only_f16, dev)
    return t.data_ptr(), ld, rows, width // dim


def lb_cache_append(cache, k, v, lengths, table, start=None, q=None, q_out=None, rope=None, interleaved=False,
                    stream=None):
    """``Cache`` owner and tensors: the rows of k and v into the pages of their sequences (see include/lb.h)."""
    _types()
    dev, width = cache.device, cache.width
    rows, ldk = _rows("k", k, width, _only_f16, dev)
    pv, ldv = _like("v", v, rows, width, _only_f16, dev)
    pq = po = pr = None
    ldq = ldo = heads = positions = rot = 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        pq, ldq, qr, heads = _heads("q", q, cache.head_dim, dev)
        if qr != rows:
            raise ValueError("q must have k's rows")
        po, ldo = _like("q_out", q_out, rows, heads * cache.head_dim, _only_f16, dev)
    if rope is not None:
        if rope.dim() != 2:
            raise ValueError("rope must be 2-d: positions x rot")
        positions, rot = rope.shape
        pr = _flat("rope", rope, (positions, rot), _f32, dev)
    _check(_lib.lb_cache_append(cache.handle, k.data_ptr(), ldk, pv, ldv, pq, ldq, po, ldo, heads, pr, positions, rot,
                                1 if interleaved else 0, *_sequences(rows, lengths, table, start, dev),
                                _stream_of(stream, dev)))


def lb_cache_read(cache, k, v, lengths, table, start=None, stream=None):
    """``Cache`` owner and tensors: k and v receive the values of the sequences' last tokens (see include/lb.h)."""
    _types()
    dev, width = cache.device, cache.width
    rows, ldk = _rows("k", k, width, _only_f16, dev)
    pv, ldv = _like("v", v, rows, width, _only_f16, dev)
    _check(_lib.lb_cache_read(cache.handle, k.data_ptr(), ldk, pv, ldv,
                              *_sequences(rows, lengths, table, start, dev), _stream_of(stream, dev)))


def lb_cache_attend(cache, q, out, lengths, table, start=None, max_length=None, scale=None, causal=True, window=0,
                    stream=None):
    """``Cache`` owner and tensors: out = attention of q over the cache (see include/lb.h); scale defaults to
    1 / sqrt(head_dim)."""
    _types()
    dev = cache.device
    pq, ldq, rows, heads = _heads("q", q, cache.head_dim, dev)
    po, ldo = _like("out", out, rows, heads * cache.head_dim, _only_f16, dev)
    _check(_lib.lb_cache_attend(cache.handle, pq, ldq, heads, po, ldo, *_sequences(rows, lengths, table, start, dev),
                                int(max_length or 0), cache.head_dim ** -0.5 if scale is None else scale,
                                1 if causal else 0, max(-1, min(window, 0x7fffffff)),  # (any wider one hides nothing)
                                _stream_of(stream, dev)))


def lb_cache_destroy(cache: int):
    _check(load_library().lb_cache_destroy(cache))


# --------------------------------------------------------------- owners
class Layer:
    """Owner of one lb_layer handle."""

    def __init__(self, a: int, b: int, s: int, residual: bool):
        self.a, self.b, self.s, self.residual = a, b, s, bool(residual)
        self.handle = lb_create(a, b, s, residual)

    @classmethod
    def from_paths(cls, paths):
        p0 = paths[0]
        L = cls(p0["a"], p0["b"], p0["s"], len(paths) == 2)
        for i, p in enumerate(paths):
            lb_pack_signs(L.handle, i, p["su"], p["sv"])
            lb_set_scales(L.handle, i, p["h"], p["g"], p["l"])
        return L

    def forward(self, x, y, M=None, stream=None):
        lb_forward(self.handle, x, y, x.shape[0] if M is None else M, stream)

    def prepare(self, M: int):
        lb_prepare(self.handle, M)

    def device_bytes(self):
        """(sign bytes, total bytes) the layer holds on the device."""
        return lb_layer_device_bytes(self.handle)

    def close(self):
        if self.handle:
            lb_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Stack:
    """Owner of one lb_stack handle (keeps its layers alive)."""

    def __init__(self, layers, unit_sizes, kappa: float):
        self.layers = list(layers)
        self.unit_sizes = list(unit_sizes)
        self.handle = lb_stack_create([L.handle for L in self.layers], self.unit_sizes, kappa)

    def forward(self, x0, y, trace=None, M=None, stream=None):
        lb_stack_forward(self.handle, x0, y, trace, x0.shape[0] if M is None else M, stream)

    def trace_elems(self, M: int) -> int:
        return lb_stack_trace_elems(self.handle, M)

    def set_mode(self, mode: int):
        lb_stack_set_mode(self.handle, mode)

    def reserve(self, M: int):
        lb_stack_reserve(self.handle, M)

    def check(self):
        lb_stack_check(self.handle)

    def close(self):
        if self.handle:
            lb_stack_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Bank:
    """Owner of one lb_bank handle (keeps its layers alive).

    ``layers`` and ``gates`` are ``Layer`` objects of one shape; without gates a call computes
    act(layer(x) + bias) + residual, with them act(gate(x) + gate_bias) * (layer(x) + bias) + residual.
    Biases are fp16 tensors of (layers, b).
    """

    def __init__(self, layers, gates=None):
        self.handle = None
        self.layers = list(layers)
        self.gates = list(gates) if gates is not None else None
        if not self.layers:
            raise ValueError("a bank needs at least one layer")
        self.handle = lb_bank_create([L.handle for L in self.layers],
                                     [L.handle for L in self.gates] if self.gates is not None else None)
        self.n, _, self.a, self.b, self.device = lb_bank_shape(self.handle)

    def reserve(self, rows: int):
        lb_bank_reserve(self.handle, rows)

    def forward(self, x, y, expert: int = 0, act=None, bias=None, gate_bias=None, residual=None, stream=None):
        lb_bank_forward(self, x, y, expert, act, bias, gate_bias, residual, stream)

    def grouped(self, x, offsets, y, index=None, act=None, bias=None, gate_bias=None, residual=None, stream=None):
        lb_bank_grouped(self, x, offsets, y, index, act, bias, gate_bias, residual, stream)

    def close(self):
        if self.handle:
            lb_bank_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Route:
    """The routing of a fixed number of tokens: owner of lb_route's outputs and scratch.

    After ``run(logits)`` the device tensors ``experts``, ``weights`` and ``row`` (tokens, k), ``offsets``
    (experts + 1) and ``token`` (tokens * k) hold the result; a later run overwrites them.
    """

    def __init__(self, tokens: int, experts: int, k: int, renormalise: bool = True, device=None):
        import torch
        self.k, self.renormalise = int(k), bool(renormalise)
        n = lb_route_ws_bytes(tokens, experts, k)
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.experts = torch.empty((tokens, k), dtype=torch.int32, device=dev)
        self.weights = torch.empty((tokens, k), dtype=torch.float32, device=dev)
        self.offsets = torch.empty(experts + 1, dtype=torch.int32, device=dev)
        self.token = torch.empty(tokens * k, dtype=torch.int32, device=dev)
        self.row = torch.empty((tokens, k), dtype=torch.int32, device=dev)
        self.ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None

    def run(self, logits, stream=None) -> "Route":
        lb_route(logits, self.k, self.renormalise, self.experts, self.weights, self.offsets, self.token, self.row,
                 self.ws, stream)
        return self

    def combine(self, y, out, residual=None, stream=None):
        lb_route_combine(y, self.row, self.weights, out, residual, stream)


class Cache:
    """Owner of one lb_cache handle: keys and values in 8 bits, in pages, on the current GPU.

    Rows are tokens: k and v (rows, kv_heads * head_dim), q and out (rows, heads * head_dim), fp16.  ``table``
    (sequences, columns), ``lengths`` (sequences) and ``start`` (sequences + 1, or None for a row each) are int32.
    """

    def __init__(self, pages: int, page_tokens: int, kv_heads: int, head_dim: int):
        self.handle = None
        self.handle = lb_cache_create(pages, page_tokens, kv_heads, head_dim)
        self.pages, self.page_tokens, self.kv_heads, self.head_dim, self.device = lb_cache_shape(self.handle)
        self.width = self.kv_heads * self.head_dim

    def reserve(self, rows: int, heads: int, sequences: int, max_length: int):
        lb_cache_reserve(self.handle, rows, heads, sequences, max_length)

    def append(self, k, v, lengths, table, start=None, q=None, q_out=None, rope=None, interleaved=False, stream=None):
        lb_cache_append(self, k, v, lengths, table, start, q, q_out, rope, interleaved, stream)

    def read(self, k, v, lengths, table, start=None, stream=None):
        lb_cache_read(self, k, v, lengths, table, start, stream)

    def attend(self, q, out, lengths, table, start=None, max_length=None, scale=None, causal=True, window=0, stream=None):
        lb_cache_attend(self, q, out, lengths, table, start, max_length, scale, causal, window, stream)

    def close(self):
        if self.handle:
            lb_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def lb_status_str(status: int) -> str:
    return load_library().lb_status_str(int(status)).decode()


def lb_last_error() -> str:
    return load_library().lb_last_error().decode(errors="replace")


def lb_version() -> int:
    return load_library().lb_version()
