"""Python binding of libqdr (include/qdr.h, include/qdr_mixer.h, include/qdr_cache.h): argument
marshalling only.

Every function here has the name of the C entry point it calls.  Tensors are
torch tensors on the current HIP device; the library receives their device
pointers and the current stream.  There is no fallback: if libqdr.so is not
built, or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqdr.so")

DIM = 128
GATE_SCALAR, GATE_DIAG = 0, 1
UNIT_HEAD, UNIT_ROW = 0, 1
SCALE_DUAL, SCALE_ROW_ABSMAX = 0, 1
K_INT2, K_INT4, K_INT6, K_INT8, K_FP16, K_FP32 = 2, 4, 6, 8, 16, 32
DEVERR_SLOT, DEVERR_LENGTH, DEVERR_PAGE, DEVERR_FULL = 1, 2, 4, 8
RULE_DELTA, RULE_SUM = 0, 1
KV_INT8, KV_BF16 = 8, 16
ROTARY_HALF, ROTARY_PAIRS = 0, 1
ROTARY_PLAIN, ROTARY_LINEAR, ROTARY_TURNS, ROTARY_INDEX = 0, 1, 2, 3

_STATUS = {0: "QDR_OK", -1: "QDR_E_INVAL", -2: "QDR_E_NOMEM", -3: "QDR_E_DEVICE",
           -4: "QDR_E_SLOT", -5: "QDR_E_UNSUPPORTED"}


class QdrError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn}: {_STATUS.get(status, status)}: {msg}")
        self.status = status


class PoolDesc(ctypes.Structure):
    _fields_ = [("num_slots", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("unit", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("scale_mode", ctypes.c_int32), ("fit_iters", ctypes.c_int32),
                ("kinds", ctypes.c_void_p), ("omega", ctypes.c_void_p),
                ("scale_bits", ctypes.c_int32)]


class Layout(ctypes.Structure):
    _fields_ = [("slot_stride", ctypes.c_uint64), ("total_bytes", ctypes.c_uint64),
                ("num_slots", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("head_off", ctypes.POINTER(ctypes.c_uint64)),
                ("head_bytes", ctypes.POINTER(ctypes.c_uint32)),
                ("code_bytes", ctypes.POINTER(ctypes.c_uint32)),
                ("base", ctypes.c_void_p), ("bits_per_value", ctypes.c_double)]


class KVDesc(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("d", ctypes.c_int32), ("kind", ctypes.c_int32)]


class RotaryDesc(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("channels", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("freq", ctypes.c_void_p), ("amplitude", ctypes.c_double)]


EXPORTS = ["qdr_pool_bytes", "qdr_pool_create", "qdr_pool_destroy", "qdr_slot_reset",
           "qdr_pack", "qdr_unpack", "qdr_decode_step", "qdr_decode_step_split", "qdr_decode_step_bf16", "qdr_get_layout", "qdr_read_raw",
           "qdr_write_raw", "qdr_poll_device_error", "qdr_last_error", "qdr_clock_probe"]

MIXER_EXPORTS = ["qdr_prompt_workspace", "qdr_prompt", "qdr_linear_step", "qdr_linear_step_bf16", "qdr_kv_bytes",
                 "qdr_kv_create", "qdr_kv_destroy", "qdr_kv_write", "qdr_kv_read", "qdr_kv_attend_workspace",
                 "qdr_kv_attend", "qdr_kv_poll_device_error"]

CACHE_EXPORTS = ["qdr_rotary_frequencies", "qdr_rotary_create", "qdr_rotary_destroy", "qdr_rotate", "qdr_rotate_bf16",
                 "qdr_kv_write_rotary", "qdr_kv_copy", "qdr_slot_copy", "qdr_kv_assign_workspace", "qdr_kv_assign",
                 "qdr_kv_compact_workspace", "qdr_kv_compact", "qdr_kv_attend_shared_workspace", "qdr_kv_attend_shared"]

_lib = None
_raw_stream = None


def load():
    """Load libqdr.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with quantized_delta_rule_decode_amd/build.py")
    # torch's HIP runtime must be the process's HIP runtime: importing torch
    # first makes libqdr.so bind to the already loaded libamdhip64.so.7
    # instead of loading a second runtime instance.
    import torch
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ, F64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_double
    sig = {
        "qdr_pool_bytes": [ctypes.POINTER(PoolDesc), ctypes.POINTER(SZ)],
        "qdr_pool_create": [ctypes.POINTER(PoolDesc), P, SZ, ctypes.POINTER(P)],
        "qdr_pool_destroy": [P],
        "qdr_slot_reset": [P, P, I32, P],
        "qdr_pack": [P, P, I32, P, P],
        "qdr_unpack": [P, P, I32, P, P],
        "qdr_decode_step": [P, P, I32, P, P, P, P, P, P, P],
        "qdr_decode_step_split": [P, P, I32, P, P, P, P, P, P, P, P],
        "qdr_decode_step_bf16": [P, P, I32, P, P, P, P, P, P, P],
        "qdr_get_layout": [P, ctypes.POINTER(Layout)],
        "qdr_read_raw": [P, I32, P, SZ, P],
        "qdr_write_raw": [P, I32, P, SZ, P],
        "qdr_poll_device_error": [P, ctypes.POINTER(ctypes.c_uint32)],
        "qdr_clock_probe": [P, I32, P],
        "qdr_prompt_workspace": [P, I32, I32, ctypes.POINTER(SZ)],
        "qdr_prompt": [P, I32, P, P, P, I32, I32, P, P, P, P, P, P, P, SZ, P],
        "qdr_linear_step": [P, P, I32, P, P, P, P, P, P],
        "qdr_linear_step_bf16": [P, P, I32, P, P, P, P, P, P],
        "qdr_kv_bytes": [ctypes.POINTER(KVDesc), ctypes.POINTER(SZ)],
        "qdr_kv_create": [ctypes.POINTER(KVDesc), P, SZ, ctypes.POINTER(P)],
        "qdr_kv_destroy": [P],
        "qdr_kv_write": [P, P, I32, P, P, I32, I32, P, P, P],
        "qdr_kv_read": [P, P, I32, P, P, I32, I32, P, P, P],
        "qdr_kv_attend_workspace": [P, I32, I32, I32, I32, ctypes.POINTER(SZ)],
        "qdr_kv_attend": [P, P, I32, P, P, I32, I32, I32, P, ctypes.c_float, P, P, SZ, P],
        "qdr_kv_poll_device_error": [P, ctypes.POINTER(ctypes.c_uint32)],
        "qdr_rotary_frequencies": [I32, I32, F64, F64, F64, F64, F64, P, ctypes.POINTER(F64)],
        "qdr_rotary_create": [ctypes.POINTER(RotaryDesc), ctypes.POINTER(P)],
        "qdr_rotary_destroy": [P],
        "qdr_rotate": [P, P, I32, I32, P, I64, P, I64, P],
        "qdr_rotate_bf16": [P, P, I32, I32, P, I64, P, I64, P],
        "qdr_kv_write_rotary": [P, P, P, I32, P, P, I32, I32, P, I64, I32, P, P, I64, P, I64, P],
        "qdr_kv_copy": [P, P, P, P, I32, P],
        "qdr_slot_copy": [P, P, P, I32, P],
        "qdr_kv_assign_workspace": [P, I32, ctypes.POINTER(SZ)],
        "qdr_kv_assign": [P, P, P, I32, I32, P, P, I32, P, P, P, P, P, SZ, P],
        "qdr_kv_compact_workspace": [P, ctypes.POINTER(SZ)],
        "qdr_kv_compact": [P, P, P, I32, I32, P, P, P, P, SZ, P],
        "qdr_kv_attend_shared_workspace": [P, I32, I32, I32, I32, I32, ctypes.POINTER(SZ)],
        "qdr_kv_attend_shared": [P, P, I32, P, P, I32, I32, P, P, I32, I32, P, ctypes.c_float, P, P, SZ, P],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    # the current stream's handle without building a Stream object (4 us a call)
    global _raw_stream
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    L.qdr_last_error.argtypes = []
    L.qdr_last_error.restype = ctypes.c_char_p
    _lib = L
    return L


def _check(fn, status):
    if status != 0:
        raise QdrError(fn, status, load().qdr_last_error().decode())


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    import torch
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch._C._cuda_getDevice())


def _dptr(t, dtype, name, numel=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


def _ptr(t, dtype, name, shape):
    """Address of a contiguous device tensor of this type and shape; one test
    where all is well (a call of small tensors takes as long as its launch)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dptr(t, dtype, name)
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _strided(t, dtype, name, heads):
    """Address and distance between rows of a device tensor [T][heads][128] whose rows are contiguous."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != 3 or t.shape[2] != DIM or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected (T, {'heads' if heads is None else heads}, {DIM})")
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != DIM):
        raise ValueError(f"{name} must have contiguous rows of [heads][{DIM}]")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else t.shape[1] * DIM


def _sequences(cu):
    """n of the cumulative counts."""
    if cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError("cu must be one-dimensional with n + 1 elements")
    return cu.shape[0] - 1


def _workspace(given, need, stream):
    """Pointer and bytes of a call's workspace; without one, memory of torch's
    that is not reused before the call's stream is done with it."""
    if given is not None:
        return _ptr(given, given.dtype, "workspace", given.shape), given.nbytes, given
    import torch
    with torch.cuda.stream(torch.cuda.current_stream() if stream is None else stream):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    return ws.data_ptr(), need, ws


def _desc(num_slots, num_heads, kinds, omega, unit, gate, scale_mode, fit_iters, scale_bits=32):
    kinds = np.ascontiguousarray(kinds, np.uint8)
    om = None if omega is None else np.ascontiguousarray(omega, np.float32)
    d = PoolDesc(num_slots, num_heads, DIM, DIM, unit, gate, scale_mode, fit_iters,
                 kinds.ctypes.data, None if om is None else om.ctypes.data, scale_bits)
    return d, (kinds, om)


def qdr_pool_bytes(num_slots, num_heads, kinds, omega, unit=UNIT_HEAD, gate=GATE_SCALAR,
                   scale_mode=SCALE_DUAL, fit_iters=0, scale_bits=32) -> int:
    d, keep = _desc(num_slots, num_heads, kinds, omega, unit, gate, scale_mode, fit_iters, scale_bits)
    n = ctypes.c_size_t(0)
    _check("qdr_pool_bytes", load().qdr_pool_bytes(ctypes.byref(d), ctypes.byref(n)))
    return int(n.value)


def qdr_clock_probe(out, iters, stream=None):
    """Enqueue the shader-clock probe; out: torch.int64 device tensor of >= 5
    elements (see include/qdr.h).  Returns nothing; read out after the
    stream completes: MHz = 100 * (out[2] - out[0]) / (out[3] - out[1])."""
    import torch
    if out.numel() < 5:
        raise ValueError(f"out has {out.numel()} elements, expected at least 5")
    _check("qdr_clock_probe", load().qdr_clock_probe(_dptr(out, torch.int64, "out"), int(iters), _stream(stream)))


class Pool:
    """A state pool (qdr_pool_create ... qdr_pool_destroy)."""

    def __init__(self, num_slots, num_heads, kinds, omega, unit=UNIT_HEAD, gate=GATE_SCALAR,
                 scale_mode=SCALE_DUAL, fit_iters=0, dev_mem=None, scale_bits=32):
        self.num_slots, self.num_heads = int(num_slots), int(num_heads)
        self.unit, self.gate, self.scale_mode, self.fit_iters = unit, gate, scale_mode, fit_iters
        self.scale_bits = scale_bits
        d, keep = _desc(num_slots, num_heads, kinds, omega, unit, gate, scale_mode, fit_iters, scale_bits)
        h = ctypes.c_void_p(None)
        mem_ptr, mem_bytes = None, 0
        if dev_mem is not None:
            mem_ptr, mem_bytes = ctypes.c_void_p(dev_mem.data_ptr()), dev_mem.numel() * dev_mem.element_size()
        self._dev_mem = dev_mem
        _check("qdr_pool_create", load().qdr_pool_create(ctypes.byref(d), mem_ptr, mem_bytes, ctypes.byref(h)))
        self._h = h
        lay = Layout()
        _check("qdr_get_layout", load().qdr_get_layout(self._h, ctypes.byref(lay)))
        H = self.num_heads
        self.slot_stride = int(lay.slot_stride)
        self.total_bytes = int(lay.total_bytes)
        self.head_off = np.ctypeslib.as_array(lay.head_off, shape=(H,)).copy()
        self.head_bytes = np.ctypeslib.as_array(lay.head_bytes, shape=(H,)).copy()
        self.code_bytes = np.ctypeslib.as_array(lay.code_bytes, shape=(H,)).copy()
        self.base = int(lay.base)
        self.bits_per_value = float(lay.bits_per_value)

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            _check("qdr_pool_destroy", load().qdr_pool_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    # ---- entry points (same names as the C ABI)
    def qdr_slot_reset(self, slots, stream=None):
        import torch
        _check("qdr_slot_reset", load().qdr_slot_reset(
            self._h, _dptr(slots, torch.int32, "slots"), slots.numel(), _stream(stream)))

    def qdr_pack(self, slots, S, stream=None):
        import torch
        n = slots.numel()
        _check("qdr_pack", load().qdr_pack(
            self._h, _dptr(slots, torch.int32, "slots"), n,
            _dptr(S, torch.float32, "S", n * self.num_heads * DIM * DIM), _stream(stream)))

    def qdr_unpack(self, slots, S_out, stream=None):
        import torch
        n = slots.numel()
        _check("qdr_unpack", load().qdr_unpack(
            self._h, _dptr(slots, torch.int32, "slots"), n,
            _dptr(S_out, torch.float32, "S_out", n * self.num_heads * DIM * DIM), _stream(stream)))

    def qdr_decode_step(self, slots, q, k, v, beta, gate, o, stream=None):
        import torch
        B, H = slots.numel(), self.num_heads
        f32 = torch.float32
        gn = B * H if self.gate == GATE_SCALAR else B * H * DIM
        _check("qdr_decode_step", load().qdr_decode_step(
            self._h, _dptr(slots, torch.int32, "slots"), B,
            _dptr(q, f32, "q", B * H * DIM), _dptr(k, f32, "k", B * H * DIM),
            _dptr(v, f32, "v", B * H * DIM), _dptr(beta, f32, "beta", B * H),
            _dptr(gate, f32, "gate", gn), _dptr(o, f32, "o", B * H * DIM), _stream(stream)))

    def qdr_decode_step_bf16(self, slots, q, k, v, beta, gate, o, stream=None):
        """q, k, v, o: torch.bfloat16 [B][H][128]; beta, gate fp32."""
        import torch
        B, H = slots.numel(), self.num_heads
        bf, f32 = torch.bfloat16, torch.float32
        gn = B * H if self.gate == GATE_SCALAR else B * H * DIM
        _check("qdr_decode_step_bf16", load().qdr_decode_step_bf16(
            self._h, _dptr(slots, torch.int32, "slots"), B,
            _dptr(q, bf, "q", B * H * DIM), _dptr(k, bf, "k", B * H * DIM),
            _dptr(v, bf, "v", B * H * DIM), _dptr(beta, f32, "beta", B * H),
            _dptr(gate, f32, "gate", gn), _dptr(o, bf, "o", B * H * DIM), _stream(stream)))

    def qdr_decode_step_split(self, slots, q, k, v, beta, gate, o, stream_readout=None, stream_writeback=None):
        import torch
        B, H = slots.numel(), self.num_heads
        f32 = torch.float32
        gn = B * H if self.gate == GATE_SCALAR else B * H * DIM
        _check("qdr_decode_step_split", load().qdr_decode_step_split(
            self._h, _dptr(slots, torch.int32, "slots"), B,
            _dptr(q, f32, "q", B * H * DIM), _dptr(k, f32, "k", B * H * DIM),
            _dptr(v, f32, "v", B * H * DIM), _dptr(beta, f32, "beta", B * H),
            _dptr(gate, f32, "gate", gn), _dptr(o, f32, "o", B * H * DIM),
            _stream(stream_readout), _stream(stream_writeback)))

    # ---- token mixers over the pool's states (include/qdr_mixer.h)
    def qdr_prompt_workspace(self, n, T) -> int:
        """Bytes of the workspace of a prompt call over n sequences and T rows, for just these counts (fewer can need more)."""
        b = ctypes.c_size_t(0)
        _check("qdr_prompt_workspace", load().qdr_prompt_workspace(self._h, int(n), int(T), ctypes.byref(b)))
        return int(b.value)

    def qdr_prompt(self, rule, slots, cu, q, k, v, beta, gate, o, carry=None, workspace=None, stream=None):
        """Whole prompts into the pool's slots.  q, k, v, o: torch.bfloat16
        [T][H][128]; beta (None for RULE_SUM) and gate fp32 [T][H]; cu int32
        [n+1]; slots and carry int32 [n].  workspace: None, or a device tensor
        of at least qdr_prompt_workspace(n, T) bytes."""
        import torch
        bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
        n, T, H = _sequences(cu), q.shape[0], self.num_heads
        rows, gates = (T, H, DIM), (T, H)
        ws, size, keep = _workspace(workspace, 0 if workspace is not None else self.qdr_prompt_workspace(n, T), stream)
        _check("qdr_prompt", _lib.qdr_prompt(
            self._h, rule, _ptr(slots, i32, "slots", (n,)), None if carry is None else _ptr(carry, i32, "carry", (n,)),
            _ptr(cu, i32, "cu", (n + 1,)), n, T, _ptr(q, bf, "q", rows), _ptr(k, bf, "k", rows), _ptr(v, bf, "v", rows),
            None if beta is None else _ptr(beta, f32, "beta", gates), _ptr(gate, f32, "gate", gates),
            _ptr(o, bf, "o", rows), ws, size, _stream(stream)))

    def _linear_step(self, fn, dtype, slots, q, k, v, gate, o, stream):
        import torch
        B, H = slots.numel(), self.num_heads
        rows = (B, H, DIM)
        _check(fn, getattr(_lib, fn)(
            self._h, _ptr(slots, torch.int32, "slots", (B,)), B, _ptr(q, dtype, "q", rows), _ptr(k, dtype, "k", rows),
            _ptr(v, dtype, "v", rows), _ptr(gate, torch.float32, "gate", (B, H)), _ptr(o, dtype, "o", rows), _stream(stream)))

    def qdr_linear_step(self, slots, q, k, v, gate, o, stream=None):
        """q, k, v, o: fp32 [B][H][128]; gate fp32 [B][H]; an uncompressed pool."""
        import torch
        self._linear_step("qdr_linear_step", torch.float32, slots, q, k, v, gate, o, stream)

    def qdr_linear_step_bf16(self, slots, q, k, v, gate, o, stream=None):
        """The same with torch.bfloat16 q, k, v, o."""
        import torch
        self._linear_step("qdr_linear_step_bf16", torch.bfloat16, slots, q, k, v, gate, o, stream)

    def qdr_slot_copy(self, src_slots, dst_slots, stream=None):
        """Stored states of src_slots to dst_slots (int32 [m]; -1 on either side: the pair is skipped)."""
        import torch
        m = src_slots.numel()
        _check("qdr_slot_copy", load().qdr_slot_copy(
            self._h, _ptr(src_slots, torch.int32, "src_slots", (m,)), _ptr(dst_slots, torch.int32, "dst_slots", (m,)), m, _stream(stream)))

    def qdr_read_raw(self, slot, stream=None) -> np.ndarray:
        out = np.empty(self.slot_stride, np.uint8)
        _check("qdr_read_raw", load().qdr_read_raw(
            self._h, int(slot), out.ctypes.data_as(ctypes.c_void_p), out.size, _stream(stream)))
        return out

    def qdr_write_raw(self, slot, data, stream=None):
        data = np.ascontiguousarray(data, np.uint8)
        _check("qdr_write_raw", load().qdr_write_raw(
            self._h, int(slot), data.ctypes.data_as(ctypes.c_void_p), data.size, _stream(stream)))

    def qdr_poll_device_error(self) -> int:
        f = ctypes.c_uint32(0)
        _check("qdr_poll_device_error", load().qdr_poll_device_error(self._h, ctypes.byref(f)))
        return int(f.value)

    # ---- helpers over the raw bytes of one block
    def block(self, raw_slot: np.ndarray, h: int) -> np.ndarray:
        off = int(self.head_off[h])
        return raw_slot[off: off + int(self.head_bytes[h])]


def qdr_kv_bytes(num_pages, page_tokens, num_heads, kind=KV_INT8) -> int:
    d, n = KVDesc(num_pages, page_tokens, num_heads, DIM, kind), ctypes.c_size_t(0)
    _check("qdr_kv_bytes", load().qdr_kv_bytes(ctypes.byref(d), ctypes.byref(n)))
    return int(n.value)


class KVCache:
    """A paged key/value cache (qdr_kv_create ... qdr_kv_destroy)."""

    def __init__(self, num_pages, page_tokens, num_heads, kind=KV_INT8, dev_mem=None):
        self.num_pages, self.page_tokens, self.num_heads, self.kind = int(num_pages), int(page_tokens), int(num_heads), int(kind)
        d, h = KVDesc(self.num_pages, self.page_tokens, self.num_heads, DIM, self.kind), ctypes.c_void_p(None)
        mem_ptr, mem_bytes = None, 0
        if dev_mem is not None:
            mem_ptr, mem_bytes = _dptr(dev_mem, dev_mem.dtype, "dev_mem"), dev_mem.numel() * dev_mem.element_size()
        self._dev_mem = dev_mem
        _check("qdr_kv_create", load().qdr_kv_create(ctypes.byref(d), mem_ptr, mem_bytes, ctypes.byref(h)))
        self._h = h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            _check("qdr_kv_destroy", load().qdr_kv_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    # ---- entry points (same names as the C ABI)
    def _where(self, n, pages, cu, context):
        import torch
        i32 = torch.int32
        most = pages.shape[1] if pages.dim() == 2 else 0
        return _ptr(pages, i32, "pages", (n, most)), most, _ptr(cu, i32, "cu", (n + 1,)), _ptr(context, i32, "context", (n,)), n

    def _move(self, fn, pages, cu, context, k, v, stream):
        import torch
        n, rows = _sequences(cu), (k.shape[0], self.num_heads, DIM)
        _check(fn, getattr(_lib, fn)(self._h, *self._where(n, pages, cu, context), rows[0], _ptr(k, torch.bfloat16, "k", rows),
                                     _ptr(v, torch.bfloat16, "v", rows), _stream(stream)))

    def qdr_kv_write(self, pages, cu, context, k, v, stream=None):
        """pages int32 [n][max_pages], cu int32 [n+1], context int32 [n]; k, v
        torch.bfloat16 [T][heads][128]: each sequence's last cached tokens."""
        self._move("qdr_kv_write", pages, cu, context, k, v, stream)

    def qdr_kv_read(self, pages, cu, context, k, v, stream=None):
        """The same rows read back into k and v."""
        self._move("qdr_kv_read", pages, cu, context, k, v, stream)

    def qdr_kv_attend_workspace(self, n, T, q_heads, max_pages) -> int:
        """Bytes of the workspace of an attention call of just these counts (fewer sequences or rows can need more)."""
        b = ctypes.c_size_t(0)
        _check("qdr_kv_attend_workspace", load().qdr_kv_attend_workspace(
            self._h, int(n), int(T), int(q_heads), int(max_pages), ctypes.byref(b)))
        return int(b.value)

    def qdr_kv_attend(self, pages, cu, context, q, o, scale=None, workspace=None, stream=None):
        """q, o: torch.bfloat16 [T][q_heads][128]; scale: 1/sqrt(128) if None;
        workspace: None, or a device tensor of at least
        qdr_kv_attend_workspace(n, T, q_heads, max_pages) bytes."""
        import torch
        n, bf = _sequences(cu), torch.bfloat16
        if q.dim() != 3 or q.shape[2] != DIM:
            raise ValueError(f"q has shape {tuple(q.shape)}, expected (T, q_heads, {DIM})")
        T, heads, _ = rows = q.shape
        where = self._where(n, pages, cu, context)
        need = 0 if workspace is not None else self.qdr_kv_attend_workspace(n, T, heads, where[1])
        ws, size, keep = _workspace(workspace, need, stream)
        _check("qdr_kv_attend", _lib.qdr_kv_attend(
            self._h, *where, T, heads, _ptr(q, bf, "q", rows), DIM ** -0.5 if scale is None else scale, _ptr(o, bf, "o", rows),
            ws, size, _stream(stream)))

    # ---- around the cache (include/qdr_cache.h)
    def qdr_kv_write_rotary(self, rotary, pages, cu, context, k, v, q=None, q_out=None, stream=None):
        """qdr_kv_write of turned keys, and q [T][q_heads][128] turned into
        q_out (contiguous).  q, k and v may be parts of one projection's rows."""
        import torch
        bf = torch.bfloat16
        n, T, heads = _sequences(cu), k.shape[0], 0 if q is None else q.shape[1]
        (kp, ks), (vp, vs) = _strided(k, bf, "k", self.num_heads), _strided(v, bf, "v", self.num_heads)
        qp, qs, out = None, 0, None
        if q is not None:
            qp, qs = _strided(q, bf, "q", None)
            out = _ptr(q_out, bf, "q_out", (T, heads, DIM))
        if v.shape[0] != T or (q is not None and q.shape[0] != T):
            raise ValueError("q, k and v must have the same number of rows")
        _check("qdr_kv_write_rotary", _lib.qdr_kv_write_rotary(
            self._h, rotary._h, *self._where(n, pages, cu, context), T, qp, qs, heads, out, kp, ks, vp, vs, _stream(stream)))

    def qdr_kv_copy(self, src_pages, dst_pages, to=None, stream=None):
        """Pages src_pages to pages dst_pages (int32 [m]) of this cache, or of the cache `to`."""
        import torch
        m = src_pages.numel()
        _check("qdr_kv_copy", _lib.qdr_kv_copy(
            self._h, _ptr(src_pages, torch.int32, "src_pages", (m,)), (self if to is None else to)._h,
            _ptr(dst_pages, torch.int32, "dst_pages", (m,)), m, _stream(stream)))

    def qdr_kv_assign_workspace(self, m) -> int:
        """Bytes of the workspace of an assignment of m rows."""
        b = ctypes.c_size_t(0)
        _check("qdr_kv_assign_workspace", load().qdr_kv_assign_workspace(self._h, int(m), ctypes.byref(b)))
        return int(b.value)

    def qdr_kv_assign(self, pages, context, parent, add, refs, new_pages, new_context, new_refs, workspace=None, stream=None):
        """Page tables of the next step: row j goes on from row parent[j] (-1:
        from none) by add[j] tokens.  pages int32 [n][max_pages], context int32
        [n], parent, add int32 [m], refs int32 [num_pages]; the new arrays
        [m][max_pages], [m], [num_pages] are written."""
        import torch
        i32 = torch.int32
        if pages.dim() != 2 or parent.dim() != 1:
            raise ValueError("pages must have two dimensions and parent one")
        (n, most), m = pages.shape, parent.shape[0]
        ws, size, keep = _workspace(workspace, 0 if workspace is not None else self.qdr_kv_assign_workspace(m), stream)
        _check("qdr_kv_assign", _lib.qdr_kv_assign(
            self._h, _ptr(pages, i32, "pages", (n, most)), _ptr(context, i32, "context", (n,)), n, most,
            _ptr(parent, i32, "parent", (m,)), _ptr(add, i32, "add", (m,)), m, _ptr(refs, i32, "refs", (self.num_pages,)),
            _ptr(new_pages, i32, "new_pages", (m, most)), _ptr(new_context, i32, "new_context", (m,)),
            _ptr(new_refs, i32, "new_refs", (self.num_pages,)), ws, size, _stream(stream)))

    def qdr_kv_compact_workspace(self) -> int:
        """Bytes of qdr_kv_compact's workspace."""
        b = ctypes.c_size_t(0)
        _check("qdr_kv_compact_workspace", load().qdr_kv_compact_workspace(self._h, ctypes.byref(b)))
        return int(b.value)

    def qdr_kv_compact(self, refs, pages, moved, new_refs, new_pages, workspace=None, stream=None):
        """Pages in use (refs int32 [num_pages], not 0) to the lowest numbers.
        moved, new_refs int32 [num_pages] and new_pages like pages [n][max_pages] are written."""
        import torch
        i32, total = torch.int32, (self.num_pages,)
        if pages.dim() != 2:
            raise ValueError("pages must have two dimensions")
        n, most = pages.shape
        ws, size, keep = _workspace(workspace, 0 if workspace is not None else self.qdr_kv_compact_workspace(), stream)
        _check("qdr_kv_compact", _lib.qdr_kv_compact(
            self._h, _ptr(refs, i32, "refs", total), _ptr(pages, i32, "pages", (n, most)), n, most, _ptr(moved, i32, "moved", total),
            _ptr(new_refs, i32, "new_refs", total), _ptr(new_pages, i32, "new_pages", (n, most)), ws, size, _stream(stream)))

    def qdr_kv_attend_shared_workspace(self, n, T, groups, q_heads, max_pages) -> int:
        """Bytes of the workspace of such a call of just these counts (smaller counts can need more)."""
        b = ctypes.c_size_t(0)
        _check("qdr_kv_attend_shared_workspace", load().qdr_kv_attend_shared_workspace(
            self._h, int(n), int(T), int(groups), int(q_heads), int(max_pages), ctypes.byref(b)))
        return int(b.value)

    def qdr_kv_attend_shared(self, pages, cu, context, group_cu, shared, q, o, scale=None, workspace=None, stream=None):
        """qdr_kv_attend where the sequences group_cu[i] .. group_cu[i+1]-1 have
        their first shared[i] tokens in common.  group_cu int32 [groups+1], shared
        int32 [groups]."""
        import torch
        i32, n, bf = torch.int32, _sequences(cu), torch.bfloat16
        if q.dim() != 3 or q.shape[2] != DIM:
            raise ValueError(f"q has shape {tuple(q.shape)}, expected (T, q_heads, {DIM})")
        if shared.dim() != 1:
            raise ValueError("shared must be one-dimensional")
        T, heads, _ = rows = q.shape
        where, groups = self._where(n, pages, cu, context), shared.shape[0]
        need = 0 if workspace is not None else self.qdr_kv_attend_shared_workspace(n, T, groups, heads, where[1])
        ws, size, keep = _workspace(workspace, need, stream)
        _check("qdr_kv_attend_shared", _lib.qdr_kv_attend_shared(
            self._h, *where, T, _ptr(group_cu, i32, "group_cu", (groups + 1,)), _ptr(shared, i32, "shared", (groups,)), groups, heads,
            _ptr(q, bf, "q", rows), DIM ** -0.5 if scale is None else scale, _ptr(o, bf, "o", rows), ws, size, _stream(stream)))

    def qdr_kv_poll_device_error(self) -> int:
        f = ctypes.c_uint32(0)
        _check("qdr_kv_poll_device_error", load().qdr_kv_poll_device_error(self._h, ctypes.byref(f)))
        return int(f.value)


def qdr_rotary_frequencies(rule, channels, base=10000.0, factor=1.0, context=8192.0, low=1.0, high=32.0):
    """Frequencies (float64 [channels/2], radians a token) and amplitude of a ROTARY_ rule."""
    freq, amplitude = np.empty(max(0, int(channels) // 2)), ctypes.c_double(0)
    _check("qdr_rotary_frequencies", load().qdr_rotary_frequencies(
        int(rule), int(channels), base, factor, context, low, high, freq.ctypes.data, ctypes.byref(amplitude)))
    return freq, amplitude.value


class Rotary:
    """A rotation (qdr_rotary_create ... qdr_rotary_destroy): frequencies of the
    pairs of a head's first 2 len(freq) channels."""

    def __init__(self, freq, layout=ROTARY_HALF, amplitude=1.0):
        freq = np.ascontiguousarray(freq, np.float64)
        if freq.ndim != 1:
            raise ValueError("freq must be one-dimensional")
        self.channels, self.layout, self.amplitude = 2 * freq.size, int(layout), float(amplitude)
        d, h = RotaryDesc(DIM, self.channels, self.layout, freq.ctypes.data, self.amplitude), ctypes.c_void_p(None)
        _check("qdr_rotary_create", load().qdr_rotary_create(ctypes.byref(d), ctypes.byref(h)))
        self._h = h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            _check("qdr_rotary_destroy", load().qdr_rotary_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _turn(self, fn, dtype, positions, x, y, stream):
        import torch
        xp, xs = _strided(x, dtype, "x", None)
        yp, ys = _strided(y, dtype, "y", x.shape[1])
        T = x.shape[0]
        if y.shape[0] != T:
            raise ValueError(f"y has {y.shape[0]} rows, expected {T}")
        _check(fn, getattr(_lib, fn)(self._h, _ptr(positions, torch.int32, "positions", (T,)), T, x.shape[1], xp, xs, yp, ys, _stream(stream)))

    def qdr_rotate(self, positions, x, y, stream=None):
        """y = x turned by positions (int32 [T]); x, y fp32 [T][heads][128], rows any distance apart; y may be x."""
        import torch
        self._turn("qdr_rotate", torch.float32, positions, x, y, stream)

    def qdr_rotate_bf16(self, positions, x, y, stream=None):
        """The same with torch.bfloat16 x and y."""
        import torch
        self._turn("qdr_rotate_bf16", torch.bfloat16, positions, x, y, stream)


def qdr_last_error() -> str:
    return load().qdr_last_error().decode()
