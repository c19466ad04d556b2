"""decode_gemv_tensor_gb300 -- thin Python binding of libdgt (C ABI in include/dgt.h).

Lossless BF16 exponent-rank weight compression decoded inside the matrix
product, for one GB300 (sm_103a).  Every step runs in libdgt: the host packer
and container in C++, the transcode, rebuild and product kernels in CUDA.
This module only marshals arguments: numpy arrays for host data, torch tensors
for device memory and streams.  It fails loudly when libdgt.so is missing.

Names follow the C ABI: pack, unpack, write, read, upload, load_r4,
load_r4_into, r4_to_bf16, gemv, gemv_bf16, gemv_slices, moe_gemv,
moe_gemv_bf16, gemm, gemm_bf16, gemm_rebuild, gemm_plan, moe_gemm, moe_gemm_bf16,
add_rmsnorm, silu_mul, silu_mul_rows, repeat, weighted_sum, exponent_stats,
rotate, kv_append, kv_read, kv_attention, kv_reserve, kv_fork, kv_free,
kv_copy_pages, kv_compact, read_status; Rotary and KvCache hold a rotation's
frequencies and a paged 8-bit cache; DecodeStep and MoeDecodeStep compose a
batch-1 decode step from them, with a StepAttention over a cache or without,
and capture it in a CUDA graph.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdgt.so")

DGT_OK = 0
STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported shape", -3: "corrupt packed data",
          -4: "CUDA error", -5: "device wait timed out", -6: "out of host memory", -7: "I/O error",
          -8: "unsupported device or configuration", -9: "no room left in the cache"}


class DgtError(RuntimeError):
    def __init__(self, code, where):
        super().__init__(f"{where}: {STATUS.get(code, 'unknown')} ({code})")
        self.code = code


class PackedView(C.Structure):
    _fields_ = [
        ("rows", C.c_uint64), ("cols", C.c_uint64), ("format", C.c_int32), ("rice_k", C.c_int32),
        ("n_table", C.c_int32), ("reserved", C.c_int32), ("table", C.c_uint8 * 256),
        ("n_esc15", C.c_uint64), ("sm", C.c_void_p), ("words", C.c_void_p), ("n_words", C.c_uint64),
        ("blkq", C.c_void_p), ("n_blocks", C.c_uint64), ("grp", C.c_void_p), ("n_groups", C.c_uint64),
        ("payload", C.c_void_p), ("payload_bytes", C.c_uint64), ("tw", C.c_void_p), ("tesc", C.c_void_p),
        ("n_tiles", C.c_uint64), ("esc1", C.c_void_p), ("n_esc1", C.c_uint64), ("grp1", C.c_void_p),
        ("n_groups1", C.c_uint64),
    ]


class R4Struct(C.Structure):
    _fields_ = [
        ("rows", C.c_uint64), ("cols", C.c_uint64), ("n_table", C.c_int32), ("reserved", C.c_int32),
        ("table", C.c_uint8 * 256), ("n_esc", C.c_uint64), ("sm", C.c_void_p), ("nib", C.c_void_p),
        ("esc", C.c_void_p), ("seg", C.c_void_p),
    ]


class GemmPlan(C.Structure):
    _fields_ = [("m_tile", C.c_int32), ("split_k", C.c_int32), ("test_flags", C.c_uint32), ("schedule", C.c_int32)]


class HeadsStruct(C.Structure):
    _fields_ = [("data", C.c_void_p), ("token_stride", C.c_int64), ("head_stride", C.c_int64), ("heads", C.c_uint32),
                ("reserved", C.c_uint32)]


_pack_heads = struct.Struct("=QqqII").pack     # the same as bytes, which ctypes passes by address


class RotaryStruct(C.Structure):
    _fields_ = [("rot_dim", C.c_uint32), ("axes", C.c_uint32), ("interleaved", C.c_uint32), ("reserved", C.c_uint32),
                ("d_freq", C.c_void_p), ("d_axis", C.c_void_p)]


class KvCacheStruct(C.Structure):
    _fields_ = [("layers", C.c_uint32), ("pages", C.c_uint32), ("kv_heads", C.c_uint32), ("head_dim", C.c_uint32),
                ("max_seqs", C.c_uint32), ("max_pages", C.c_uint32), ("k", C.c_void_p), ("v", C.c_void_p),
                ("k_scale", C.c_void_p), ("v_scale", C.c_void_p), ("refs", C.c_void_p), ("table", C.c_void_p),
                ("lens", C.c_void_p)]


_lib = None


def lib():
    """The loaded libdgt (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libdgt.so is not built ({LIB_PATH}); run "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = C.CDLL(LIB_PATH)
        vp, u64, i32 = C.c_void_p, C.c_uint64, C.c_int
        hp = kp = vp     # dgt_heads as packed bytes, dgt_kv_cache by address: half the cost of a pointer type
        sig = {
            "dgt_status_string": (C.c_char_p, [i32]),
            "dgt_version": (i32, []),
            "dgt_pack": (i32, [vp, u64, u64, i32, i32, C.POINTER(vp)]),
            "dgt_packed_free": (None, [vp]),
            "dgt_packed_get_view": (i32, [vp, C.POINTER(PackedView)]),
            "dgt_packed_bits_per_weight": (C.c_double, [vp]),
            "dgt_unpack": (i32, [C.POINTER(PackedView), vp, i32]),
            "dgt_write": (i32, [C.c_char_p, C.POINTER(vp), C.POINTER(C.c_char_p), i32]),
            "dgt_read": (i32, [C.c_char_p, C.POINTER(C.POINTER(vp)), C.POINTER(C.POINTER(C.c_char_p)),
                               C.POINTER(i32)]),
            "dgt_read_free": (None, [C.POINTER(vp), C.POINTER(C.c_char_p), i32]),
            "dgt_r4_nseg": (u64, [u64]),
            "dgt_r4_rsum_offset": (u64, [u64, u64]),
            "dgt_r4_sizes": (i32, [u64, u64, u64, C.POINTER(u64), C.POINTER(u64), C.POINTER(u64)]),
            "dgt_r4_init_from_view": (i32, [C.POINTER(PackedView), vp, vp, vp, C.POINTER(R4Struct)]),
            "dgt_load_r4": (i32, [C.POINTER(PackedView), C.POINTER(R4Struct), vp, vp]),
            "dgt_r4_to_bf16": (i32, [C.POINTER(R4Struct), vp, vp, vp]),
            "dgt_read_status": (i32, [vp, vp, C.POINTER(C.c_int32)]),
            "dgt_gemv_slices": (i32, [u64, u64]),
            "dgt_gemv": (i32, [C.POINTER(R4Struct), vp, vp, vp, vp, vp]),
            "dgt_gemv_bf16": (i32, [vp, u64, u64, vp, vp, vp, vp, vp]),
            "dgt_gemv_ex": (i32, [C.POINTER(R4Struct), vp, vp, vp, vp, C.c_uint, vp]),
            "dgt_gemv_bf16_ex": (i32, [vp, u64, u64, vp, vp, vp, vp, C.c_uint, vp]),
            "dgt_gemm_default_plan": (i32, [u64, u64, u64, C.POINTER(GemmPlan)]),
            "dgt_gemm_workspace_bytes": (C.c_size_t, [u64, u64, C.POINTER(GemmPlan)]),
            "dgt_gemm": (i32, [C.POINTER(R4Struct), vp, u64, vp, vp, C.POINTER(GemmPlan), vp, C.c_size_t, vp, vp]),
            "dgt_gemm_bf16": (i32, [vp, u64, u64, vp, u64, vp, vp, C.POINTER(GemmPlan), vp, C.c_size_t, vp, vp]),
            "dgt_gemm_rebuild": (i32, [C.POINTER(R4Struct), vp, u64, vp, vp, C.POINTER(GemmPlan), vp, vp, C.c_size_t,
                                       vp, vp]),
            "dgt_moe_workspace_bytes": (C.c_size_t, [C.c_uint32, u64, u64, C.c_uint32, C.c_uint32]),
            "dgt_moe_gemv": (i32, [C.POINTER(R4Struct), C.c_uint32, vp, vp, C.c_uint32, C.c_uint32, vp, vp, vp,
                                   vp, vp, C.c_size_t, vp, vp]),
            "dgt_moe_gemv_ex": (i32, [C.POINTER(R4Struct), C.c_uint32, vp, vp, C.c_uint32, C.c_uint32, vp, vp, vp,
                                      vp, vp, C.c_size_t, vp, C.c_uint, vp]),
            "dgt_moe_gemv_bf16": (i32, [vp, u64, u64, C.c_uint32, vp, vp, C.c_uint32, C.c_uint32, vp, vp, vp,
                                        vp, vp, C.c_size_t, vp, vp]),
            "dgt_moe_gemv_noalloc": (i32, [C.POINTER(R4Struct), C.c_uint32, vp, vp, C.c_uint32, C.c_uint32, vp,
                                           vp, vp, vp, vp, vp]),
            "dgt_moe_gemm_workspace_bytes": (C.c_size_t, [C.c_uint32, u64, u64, C.c_uint32, C.c_uint32]),
            "dgt_moe_gemm": (i32, [C.POINTER(R4Struct), C.c_uint32, vp, vp, vp, C.c_uint32, C.c_uint32, vp, vp, vp,
                                   vp, C.c_size_t, vp, vp]),
            "dgt_moe_gemm_bf16": (i32, [vp, u64, u64, C.c_uint32, vp, vp, vp, C.c_uint32, C.c_uint32, vp, vp, vp,
                                        vp, C.c_size_t, vp, vp]),
            "dgt_add_rmsnorm": (i32, [vp, vp, vp, u64, C.c_float, vp, vp]),
            "dgt_silu_mul": (i32, [vp, vp, u64, vp, vp]),
            "dgt_silu_mul_rows": (i32, [vp, C.c_uint32, u64, vp, vp]),
            "dgt_repeat": (i32, [vp, u64, u64, vp, vp]),
            "dgt_weighted_sum": (i32, [vp, vp, C.c_uint32, u64, vp, vp]),
            "dgt_rotary_freqs": (i32, [C.c_double, C.c_uint32, vp]),
            "dgt_rotate": (i32, [vp, hp, hp, hp, hp, C.c_uint32, u64, vp, vp]),
            "dgt_kv_append": (i32, [kp, C.c_uint32, hp, hp, u64, vp, vp, vp, C.c_uint32, vp, vp]),
            "dgt_kv_read": (i32, [kp, C.c_int32, vp, vp, vp, C.c_uint32, u64, vp, vp, vp, vp]),
            "dgt_kv_attention_workspace_bytes": (C.c_size_t, [kp, C.c_uint32, C.c_uint32, u64]),
            "dgt_kv_attention": (i32, [kp, C.c_uint32, hp, u64, vp, vp, C.c_uint32, C.c_float, C.c_uint32,
                                       C.c_uint32, vp, vp, vp, C.c_size_t, vp, vp]),
            "dgt_kv_attention_ex": (i32, [kp, C.c_uint32, hp, u64, vp, vp, C.c_uint32, C.c_float, C.c_uint32,
                                          C.c_uint32, vp, vp, vp, C.c_size_t, vp, C.c_uint, vp]),
            "dgt_kv_pages_workspace_bytes": (C.c_size_t, [kp]),
            "dgt_kv_copy_pages": (i32, [kp, vp, vp, C.c_uint32, vp, vp]),
            "dgt_kv_fork": (i32, [kp, vp, vp, C.c_uint32, vp, vp]),
            "dgt_kv_reserve": (i32, [kp, vp, vp, C.c_uint32, vp, vp, C.c_size_t, vp, vp]),
            "dgt_kv_free": (i32, [kp, vp, C.c_uint32, vp, vp]),
            "dgt_kv_compact": (i32, [kp, vp, vp, C.c_size_t, vp, vp]),
            "dgt_exponent_stats": (i32, [vp, u64, C.c_uint32, vp, vp, vp, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(rc, where):
    if rc != DGT_OK:
        raise DgtError(rc, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


_raw_stream = None


def _stream_on(x, stream):
    """The stream handle for work on tensor x.  torch's raw-handle query where
    it has one: 0.1 us instead of the 3 us of a Stream object, for calls whose
    kernels take as long as that."""
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw_stream(x.device.index)


def _new(shape, dtype, device, stream=None, zero=False, temp=False):
    """A tensor that a call allocates for its work on `stream` (None: the
    current stream).  With a stream given, memory and fill are that stream's: a
    block of the current stream's may still be written by work queued there,
    and nothing would order a fill there before the kernel.  temp: released
    when the call returns, to the stream that uses it; otherwise the current
    stream may read it too until it is released."""
    import torch
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = make(shape, dtype=dtype, device=device)
    if not temp:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


# ---------------------------------------------------------------------------
# host: pack / unpack / container
# ---------------------------------------------------------------------------
class Packed:
    """A library-owned packed tensor (host).  Arrays are numpy views into it."""

    _ARRAYS2 = [("sm", "sm", np.uint8, "n"), ("words", "words", np.uint32, "n_words"),
                ("blkq", "blkq", np.uint8, "n_blocks"), ("grp", "grp", np.uint32, "n_groups*2")]
    _ARRAYS1 = [("sm", "sm", np.uint8, "n"), ("payload", "payload", np.uint8, "payload_bytes"),
                ("tw", "tw", np.uint8, "n_tiles"), ("tesc", "tesc", np.uint8, "n_tiles"),
                ("esc1", "esc1", np.uint8, "n_esc1"), ("grp1", "grp1", np.uint32, "n_groups1*3")]

    def __init__(self, handle):
        self._h = C.c_void_p(handle)
        self.view = PackedView()
        _check(lib().dgt_packed_get_view(self._h, C.byref(self.view)), "dgt_packed_get_view")

    def __del__(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.dgt_packed_free(self._h)
            self._h = None

    @property
    def rows(self):
        return self.view.rows

    @property
    def cols(self):
        return self.view.cols

    @property
    def format(self):
        return self.view.format

    @property
    def table(self):
        return np.frombuffer(bytes(self.view.table), np.uint8)

    def _count(self, spec):
        v = self.view
        if spec == "n":
            return v.rows * v.cols
        if "*" in spec:
            f, m = spec.split("*")
            return getattr(v, f) * int(m)
        return getattr(v, spec)

    def arrays(self):
        """name -> numpy view (host memory owned by this object)."""
        out = {}
        for name, field, dt, spec in (self._ARRAYS2 if self.format == 2 else self._ARRAYS1):
            cnt = int(self._count(spec))
            p = getattr(self.view, field)
            if cnt == 0 or not p:
                out[name] = np.zeros(0, dt)
            else:
                buf = (C.c_uint8 * (cnt * np.dtype(dt).itemsize)).from_address(p)
                out[name] = np.frombuffer(buf, dt, count=cnt)
        return out

    def bits_per_weight(self):
        return float(lib().dgt_packed_bits_per_weight(self._h))


def pack(w, format: int = 2, nthreads: int = 0) -> Packed:
    """dgt_pack: a bf16 matrix given as uint16 bit patterns [rows, cols]."""
    w = np.ascontiguousarray(w, dtype=np.uint16)
    rows, cols = w.shape if w.ndim == 2 else (1, w.size)
    h = C.c_void_p()
    _check(lib().dgt_pack(w.ctypes.data if w.size else None, rows, cols, format, nthreads, C.byref(h)),
           "dgt_pack")
    return Packed(h.value)


def unpack(p: Packed, nthreads: int = 0) -> np.ndarray:
    """dgt_unpack on the host: the original bf16 bit patterns [rows, cols]."""
    out = np.empty((p.rows, p.cols), np.uint16)
    _check(lib().dgt_unpack(C.byref(p.view), out.ctypes.data if out.size else None, nthreads),
           "dgt_unpack")
    return out


def write(path: str, tensors: dict) -> None:
    """dgt_write: a safetensors container of packed tensors."""
    names = list(tensors)
    hs = (C.c_void_p * len(names))(*[tensors[n]._h.value for n in names])
    ns = (C.c_char_p * len(names))(*[n.encode() for n in names])
    _check(lib().dgt_write(path.encode(), hs, ns, len(names)), "dgt_write")


def read(path: str) -> dict:
    """dgt_read: name -> Packed."""
    L = lib()
    ts = C.POINTER(C.c_void_p)()
    ns = C.POINTER(C.c_char_p)()
    cnt = C.c_int()
    _check(L.dgt_read(path.encode(), C.byref(ts), C.byref(ns), C.byref(cnt)), "dgt_read")
    out = {}
    for i in range(cnt.value):
        out[ns[i].decode()] = Packed(ts[i])
        ts[i] = None          # ownership moves to the Packed object
    L.dgt_read_free(ts, ns, cnt.value)
    return out


def gemv_slices(rows: int, cols: int) -> int:
    return int(lib().dgt_gemv_slices(rows, cols))


def r4_nseg(cols: int) -> int:
    return int(lib().dgt_r4_nseg(cols))


# ---------------------------------------------------------------------------
# device
# ---------------------------------------------------------------------------
class DevicePacked:
    """The arrays of a packed tensor copied to device memory (torch uint8
    tensors), and the view with their device addresses."""

    def __init__(self, p: Packed, device="cuda", stream=None, pinned=False):
        import torch
        self.host = p
        self.tensors = {}
        for name, arr in p.arrays().items():
            t = torch.from_numpy(arr.view(np.uint8).copy() if arr.size else np.zeros(16, np.uint8))
            if pinned:
                t = t.pin_memory()
            self.tensors[name] = t.to(device, non_blocking=pinned)
        self.view = PackedView.from_buffer_copy(p.view)
        for name, t in self.tensors.items():
            setattr(self.view, name if name != "words" else "words", t.data_ptr())
        self.rows, self.cols = p.rows, p.cols


def upload(p: Packed, device="cuda") -> DevicePacked:
    return DevicePacked(p, device)


class R4:
    """R4 runtime tensor: torch device buffers (nib, esc, seg; sm aliases the
    packed upload) and the dgt_r4 descriptor."""

    def __init__(self, dev: DevicePacked, stream=None):
        import torch
        v = dev.view
        nb, eb, sb = C.c_uint64(), C.c_uint64(), C.c_uint64()
        _check(lib().dgt_r4_sizes(v.rows, v.cols, v.n_esc15, C.byref(nb), C.byref(eb), C.byref(sb)),
               "dgt_r4_sizes")
        d = dev.tensors["sm"].device
        self.nib = _new(max(nb.value, 16), torch.uint8, d, stream)
        self.esc = _new(max(eb.value, 16), torch.uint8, d, stream)
        self.seg = _new(max(sb.value // 4, 4), torch.int32, d, stream)
        self.sm = dev.tensors["sm"]
        self.dev = dev
        self.s = R4Struct()
        _check(lib().dgt_r4_init_from_view(C.byref(v), _ptr(self.nib), _ptr(self.esc), _ptr(self.seg),
                                           C.byref(self.s)), "dgt_r4_init_from_view")
        self.rows, self.cols = v.rows, v.cols
        self.n_esc = v.n_esc15

    def clone(self) -> "R4":
        """A copy in new device buffers (device-to-device copies)."""
        c = R4.__new__(R4)
        c.sm, c.nib, c.esc, c.seg = self.sm.clone(), self.nib.clone(), self.esc.clone(), self.seg.clone()
        c.dev = None
        c.s = R4Struct.from_buffer_copy(self.s)
        c.s.sm, c.s.nib, c.s.esc, c.s.seg = c.sm.data_ptr(), c.nib.data_ptr(), c.esc.data_ptr(), c.seg.data_ptr()
        c.rows, c.cols, c.n_esc = self.rows, self.cols, self.n_esc
        return c

    @property
    def rsum(self):
        """The per-round escape summaries inside seg (a view, rows*nseg words)."""
        off = lib().dgt_r4_rsum_offset(self.rows, self.cols)
        return self.seg[off:off + self.rows * lib().dgt_r4_nseg(self.cols)]


def load_r4(dev: DevicePacked, status=None, stream=None) -> R4:
    """dgt_load_r4: transcode the uploaded format-1/2 tensor into R4 on the GPU."""
    r4 = R4(dev, stream)
    _check(lib().dgt_load_r4(C.byref(dev.view), C.byref(r4.s), _ptr(status), _stream(stream)), "dgt_load_r4")
    return r4


def load_r4_into(dev: DevicePacked, r4: R4, status=None, stream=None) -> R4:
    """dgt_load_r4 into existing R4 buffers (no allocation)."""
    _check(lib().dgt_load_r4(C.byref(dev.view), C.byref(r4.s), _ptr(status), _stream(stream)), "dgt_load_r4")
    return r4


def share_sm(dst: DevicePacked, src: DevicePacked) -> None:
    """Let dst use src's device copy of the sign/mantissa bytes (same tensor)."""
    dst.tensors["sm"] = src.tensors["sm"]
    dst.view.sm = src.tensors["sm"].data_ptr()


def r4_to_bf16(r4: R4, out=None, status=None, stream=None):
    """dgt_r4_to_bf16: rebuild the bf16 matrix on the GPU (torch.bfloat16 [rows, cols])."""
    import torch
    if out is None:
        out = _new((r4.rows, r4.cols), torch.bfloat16, r4.sm.device, stream)
    _check(lib().dgt_r4_to_bf16(C.byref(r4.s), _ptr(out), _ptr(status), _stream(stream)), "dgt_r4_to_bf16")
    return out


def read_status(status, stream=None) -> int:
    v = C.c_int32()
    _check(lib().dgt_read_status(_ptr(status), _stream(stream), C.byref(v)), "dgt_read_status")
    return v.value


STATIC_WEIGHTS = 1
TEST_SHORT_WAITS = 2


def test_wait_flags(polls=None) -> int:
    """Launch flags of the failure-path test hook (DGT_TEST_SHORT_WAITS with
    DGT_TEST_WAIT_POLLS(polls)): waits for streamed data give up after
    `polls` polls.  None: 0 (no hook)."""
    if polls is None:
        return 0
    if not 0 <= int(polls) <= 0xFFFF:
        raise ValueError("polls must be in 0..65535")
    return TEST_SHORT_WAITS | (int(polls) << 16)


def gemv(W: R4, x, y=None, y32=None, status=None, stream=None, static_weights=False, test_wait_polls=None):
    """dgt_gemv_ex: y = W x with W in R4; x bf16 [cols] on the device.
    static_weights: no kernel still running writes W (DGT_GEMV_STATIC_WEIGHTS),
    so W may stream before the previous kernel ends.  test_wait_polls: the
    failure-path test hook (see test_wait_flags).
    Returns (y bf16 [rows], y32 float32 [rows])."""
    import torch
    dev = W.sm.device
    if y is None:
        y = _new(W.rows, torch.bfloat16, dev, stream)
    if y32 is None:
        y32 = _new(W.rows, torch.float32, dev, stream)
    flags = (STATIC_WEIGHTS if static_weights else 0) | test_wait_flags(test_wait_polls)
    _check(lib().dgt_gemv_ex(C.byref(W.s), _ptr(x), _ptr(y), _ptr(y32), _ptr(status), flags, _stream(stream)),
           "dgt_gemv")
    return y, y32


def gemv_bf16(W, x, y=None, y32=None, status=None, stream=None, static_weights=False, test_wait_polls=None):
    """dgt_gemv_bf16_ex: the same product and order with bf16 weights [rows, cols]."""
    import torch
    rows, cols = W.shape
    if y is None:
        y = _new(rows, torch.bfloat16, W.device, stream)
    if y32 is None:
        y32 = _new(rows, torch.float32, W.device, stream)
    flags = (STATIC_WEIGHTS if static_weights else 0) | test_wait_flags(test_wait_polls)
    _check(lib().dgt_gemv_bf16_ex(_ptr(W), rows, cols, _ptr(x), _ptr(y), _ptr(y32), _ptr(status), flags,
                                  _stream(stream)), "dgt_gemv_bf16")
    return y, y32


def moe_workspace_bytes(n_experts: int, expert_rows: int, cols: int, tokens: int, topk: int) -> int:
    return int(lib().dgt_moe_workspace_bytes(n_experts, expert_rows, cols, tokens, topk))


def _moe_outputs(tokens, topk, ne, dev, want_y, want_out, y32, out, out32, stream):
    import torch
    if want_y and y32 is None:
        y32 = _new((tokens, topk, ne), torch.float32, dev, stream)
    if want_out and out is None:
        out = _new((tokens, ne), torch.bfloat16, dev, stream)
    if want_out and out32 is None:
        out32 = _new((tokens, ne), torch.float32, dev, stream)
    return y32, out, out32


def moe_gemv(W: R4, n_experts: int, ids, p, x, ws=None, y32=None, out=None, out32=None, status=None,
             stream=None, want_y=True, test_wait_polls=None):
    """dgt_moe_gemv_ex: expert gather with stacked R4 experts.  ids int32 [T, topk],
    p float32 [T, topk] or None, x bf16 [T, K].  test_wait_polls: the
    failure-path test hook (see test_wait_flags).  Returns (y32, out, out32)."""
    import torch
    tokens, topk = ids.shape
    ne = W.rows // n_experts
    dev = W.sm.device
    y32, out, out32 = _moe_outputs(tokens, topk, ne, dev, want_y, p is not None, y32, out, out32, stream)
    nb = moe_workspace_bytes(n_experts, ne, W.cols, tokens, topk)
    if ws is None:
        ws = _new(max(nb, 256), torch.uint8, dev, stream, temp=True)
    _check(lib().dgt_moe_gemv_ex(C.byref(W.s), n_experts, _ptr(ids), _ptr(p), tokens, topk, _ptr(x), _ptr(y32),
                                 _ptr(out), _ptr(out32), _ptr(ws), ws.numel(), _ptr(status),
                                 test_wait_flags(test_wait_polls), _stream(stream)), "dgt_moe_gemv")
    return y32, out, out32


def moe_gemv_bf16(W, n_experts: int, ids, p, x, ws=None, y32=None, out=None, out32=None, status=None,
                  stream=None, want_y=True):
    """dgt_moe_gemv_bf16: the same gather with stacked bf16 experts W [E*Ne, K]."""
    import torch
    tokens, topk = ids.shape
    rows, cols = W.shape
    ne = rows // n_experts
    y32, out, out32 = _moe_outputs(tokens, topk, ne, W.device, want_y, p is not None, y32, out, out32, stream)
    nb = moe_workspace_bytes(n_experts, ne, cols, tokens, topk)
    if ws is None:
        ws = _new(max(nb, 256), torch.uint8, W.device, stream, temp=True)
    _check(lib().dgt_moe_gemv_bf16(_ptr(W), rows, cols, n_experts, _ptr(ids), _ptr(p), tokens, topk, _ptr(x),
                                   _ptr(y32), _ptr(out), _ptr(out32), _ptr(ws), ws.numel(), _ptr(status),
                                   _stream(stream)), "dgt_moe_gemv_bf16")
    return y32, out, out32


def moe_gemm_workspace_bytes(n_experts: int, expert_rows: int, cols: int, tokens: int, topk: int) -> int:
    return int(lib().dgt_moe_gemm_workspace_bytes(n_experts, expert_rows, cols, tokens, topk))


def moe_gemm(W: R4, n_experts: int, ids, p, X, ws=None, y32=None, out=None, out32=None, status=None,
             stream=None):
    """dgt_moe_gemm: the expert products of every (token, slot) pair on the
    tensor cores, experts stacked in one R4 tensor.  ids int32 [T, topk], p
    float32 [T, topk] or None, X bf16 [T, K].  Returns (y32 [T, topk, Ne],
    out bf16 [T, Ne], out32 [T, Ne]) (out and out32 None without p)."""
    import torch
    tokens, topk = ids.shape
    ne = W.rows // n_experts
    dev = W.sm.device
    y32, out, out32 = _moe_outputs(tokens, topk, ne, dev, True, p is not None, y32, out, out32, stream)
    nb = moe_gemm_workspace_bytes(n_experts, ne, W.cols, tokens, topk)
    if ws is None:
        ws = _new(max(nb, 256), torch.uint8, dev, stream, temp=True)
    _check(lib().dgt_moe_gemm(C.byref(W.s), n_experts, _ptr(ids), _ptr(p), _ptr(X), tokens, topk, _ptr(y32),
                              _ptr(out), _ptr(out32), _ptr(ws), ws.numel(), _ptr(status), _stream(stream)),
           "dgt_moe_gemm")
    return y32, out, out32


def moe_gemm_bf16(W, n_experts: int, ids, p, X, ws=None, y32=None, out=None, out32=None, status=None,
                  stream=None):
    """dgt_moe_gemm_bf16: the same products with stacked bf16 experts W [E*Ne, K]."""
    import torch
    tokens, topk = ids.shape
    rows, cols = W.shape
    ne = rows // n_experts
    y32, out, out32 = _moe_outputs(tokens, topk, ne, W.device, True, p is not None, y32, out, out32, stream)
    nb = moe_gemm_workspace_bytes(n_experts, ne, cols, tokens, topk)
    if ws is None:
        ws = _new(max(nb, 256), torch.uint8, W.device, stream, temp=True)
    _check(lib().dgt_moe_gemm_bf16(_ptr(W), rows, cols, n_experts, _ptr(ids), _ptr(p), _ptr(X), tokens, topk,
                                   _ptr(y32), _ptr(out), _ptr(out32), _ptr(ws), ws.numel(), _ptr(status),
                                   _stream(stream)), "dgt_moe_gemm_bf16")
    return y32, out, out32


def gemm_plan(M: int, N: int, K: int, m_tile=None, split_k=None, test_wait_polls=None, schedule=None) -> GemmPlan:
    """dgt_gemm_default_plan, optionally overridden (schedule: 0 auto, 1 one
    CTA per tile, 2 persistent; test_wait_polls: the failure-path test hook,
    see test_wait_flags)."""
    p = GemmPlan()
    _check(lib().dgt_gemm_default_plan(M, N, K, C.byref(p)), "dgt_gemm_default_plan")
    if m_tile is not None:
        p.m_tile = m_tile
    if split_k is not None:
        p.split_k = split_k
    if schedule is not None:
        p.schedule = schedule
    p.test_flags = test_wait_flags(test_wait_polls)
    return p


def _gemm_out(M, N, dev, Y32, Y, plan, ws, stream):
    import torch
    if Y32 is None:
        Y32 = _new((M, N), torch.float32, dev, stream)
    if Y is None:
        Y = _new((M, N), torch.bfloat16, dev, stream)
    nb = int(lib().dgt_gemm_workspace_bytes(M, N, C.byref(plan)))
    if ws is None and nb:
        ws = _new(nb, torch.uint8, dev, stream, temp=True)
    return Y32, Y, ws


def gemm(W: R4, X, plan=None, Y32=None, Y=None, ws=None, status=None, stream=None):
    """dgt_gemm: Y = X W^T on tcgen05 with W in R4; X bf16 [M, K].  Returns (Y32, Y)."""
    M, K = X.shape
    N = W.rows
    plan = plan or gemm_plan(M, N, K)
    Y32, Y, ws = _gemm_out(M, N, W.sm.device, Y32, Y, plan, ws, stream)
    _check(lib().dgt_gemm(C.byref(W.s), _ptr(X), M, _ptr(Y32), _ptr(Y), C.byref(plan), _ptr(ws),
                          0 if ws is None else ws.numel(), _ptr(status), _stream(stream)), "dgt_gemm")
    return Y32, Y


def gemm_bf16(W, X, plan=None, Y32=None, Y=None, ws=None, status=None, stream=None):
    """dgt_gemm_bf16: the same product, tiles, split and order with bf16 weights W [N, K]."""
    M, K = X.shape
    N = W.shape[0]
    plan = plan or gemm_plan(M, N, K)
    Y32, Y, ws = _gemm_out(M, N, W.device, Y32, Y, plan, ws, stream)
    _check(lib().dgt_gemm_bf16(_ptr(W), N, K, _ptr(X), M, _ptr(Y32), _ptr(Y), C.byref(plan), _ptr(ws),
                               0 if ws is None else ws.numel(), _ptr(status), _stream(stream)), "dgt_gemm_bf16")
    return Y32, Y


def gemm_rebuild(W: R4, X, scratch=None, plan=None, Y32=None, Y=None, ws=None, status=None, stream=None):
    """dgt_gemm_rebuild: the R4 weights rebuilt to bf16 in `scratch` (allocated
    when None), then the bf16 GEMM (for long prompts).  Returns (Y32, Y)."""
    import torch
    M, K = X.shape
    N = W.rows
    plan = plan or gemm_plan(M, N, K)
    if scratch is None:
        scratch = _new((N, K), torch.bfloat16, W.sm.device, stream, temp=True)
    Y32, Y, ws = _gemm_out(M, N, W.sm.device, Y32, Y, plan, ws, stream)
    _check(lib().dgt_gemm_rebuild(C.byref(W.s), _ptr(X), M, _ptr(Y32), _ptr(Y), C.byref(plan), _ptr(scratch),
                                  _ptr(ws), 0 if ws is None else ws.numel(), _ptr(status), _stream(stream)),
           "dgt_gemm_rebuild")
    return Y32, Y


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def _heads(x, name):
    """The dgt_heads view of a bf16 tensor [tokens, heads, dim] on the device (packed)."""
    import torch
    if x.dtype is not torch.bfloat16 or not x.is_cuda or x.dim() != 3:
        raise ValueError(f"{name}: a CUDA bfloat16 tensor [tokens, heads, dim]")
    (n, h, _), (ts, hs, es) = x.shape, x.stride()
    if es != 1 and x.numel():
        raise ValueError(f"{name}: a contiguous last dimension")
    # a stride that no element uses may be anything
    return _pack_heads(x.data_ptr(), ts if n > 1 else 0, hs if h > 1 else 0, h, 0)


def _i32(x, name, n=None):
    import torch
    if x.dtype is not torch.int32 or not x.is_cuda or not x.is_contiguous() or (n is not None and x.numel() != n):
        raise ValueError(f"{name}: a contiguous CUDA int32 tensor" + ("" if n is None else f" of {n} elements"))
    return x.data_ptr()


def _status(x):
    import torch
    if x is None:
        return None
    if x.dtype is not torch.int32 or not x.is_cuda or x.numel() == 0:
        raise ValueError("status: a CUDA int32 tensor")
    return x.data_ptr()


class Rotary:
    """What a rotation turns and by how much (dgt_rotary), its tables on the
    device.  The first rot_dim dimensions of a head are turned; pair i is
    dimensions (i, i + rot_dim/2), or (2i, 2i + 1) when interleaved, with
    frequency base^(-2i/rot_dim) radians per position, or inv_freq[i].
    sections: how many pairs each axis (time, height, width, ...) turns, in
    order (None: one axis); axis: the axis of each pair, instead."""

    def __init__(self, rot_dim: int, base: float = 10000.0, sections=None, interleaved: bool = False, inv_freq=None,
                 axis=None, device="cuda"):
        import math
        import torch
        half = rot_dim // 2
        freq = np.zeros(max(half, 1), np.uint64)
        if inv_freq is None:
            _check(lib().dgt_rotary_freqs(float(base), rot_dim, freq.ctypes.data), "dgt_rotary_freqs")
        else:
            if rot_dim % 2 or len(inv_freq) != half:
                raise ValueError("inv_freq: rot_dim / 2 frequencies")
            freq[:] = [round(math.ldexp(float(f) / (2 * math.pi), 64)) % 2 ** 64 for f in inv_freq]
        if axis is None:
            sections = [half] if sections is None else [int(n) for n in sections]
            if sum(sections) != half or min(sections) < 0:
                raise ValueError("sections: they add up to rot_dim / 2 pairs")
            axis = [i for i, n in enumerate(sections) for _ in range(n)]
            self.axes = len(sections)
        else:
            if len(axis) != half or min(axis) < 0:
                raise ValueError("axis: one for each of the rot_dim / 2 pairs")
            self.axes = max(axis) + 1
        self.rot_dim, self.interleaved = rot_dim, bool(interleaved)
        self.freq = torch.from_numpy(freq.view(np.int64).copy()).to(device)
        self.axis = torch.tensor(axis, dtype=torch.uint8, device=device)
        self.s = RotaryStruct(rot_dim, self.axes, int(self.interleaved), 0, self.freq.data_ptr(),
                              self.axis.data_ptr())
        self.ptr = C.addressof(self.s)


def rotate(rotary: Rotary, q, pos, k=None, q_out=None, k_out=None, stream=None):
    """dgt_rotate: q (and k) bf16 [tokens, heads, dim] turned to their
    positions, pos int32 [tokens] or [axes, tokens].  The outputs may be the
    inputs.  Returns (q_out, k_out) (k_out None without k)."""
    import torch
    tokens, nq, dim = q.shape
    p = _i32(pos, "pos", rotary.axes * tokens)
    hq, hk, ok = _heads(q, "q"), None, None
    if q_out is None:
        q_out = _new((tokens, nq, dim), torch.bfloat16, q.device, stream)
        oq = _pack_heads(q_out.data_ptr(), nq * dim, dim, nq, 0)
    else:
        oq = _heads(q_out, "q_out")
        if q_out.shape != q.shape:
            raise ValueError("q_out: the shape of q")
    if k is None:
        k_out = None
    else:
        hk, nk = _heads(k, "k"), k.shape[1]
        if k.shape[0] != tokens or k.shape[2] != dim:
            raise ValueError("k: the same tokens and head size as q")
        if k_out is None:
            k_out = _new((tokens, nk, dim), torch.bfloat16, q.device, stream)
            ok = _pack_heads(k_out.data_ptr(), nk * dim, dim, nk, 0)
        else:
            ok = _heads(k_out, "k_out")
            if k_out.shape != k.shape:
                raise ValueError("k_out: the shape of k")
    _check(lib().dgt_rotate(rotary.ptr, hq, hk, oq, ok, dim, tokens, p, _stream_on(q, stream)), "dgt_rotate")
    return q_out, k_out


# ---------------------------------------------------------------------------
# paged 8-bit cache of keys and values
# ---------------------------------------------------------------------------
KV_PAGE = 64


class KvCache:
    """A paged cache of keys and values as e4m3 codes with a power-of-two scale
    for each page and kv head (dgt_kv_cache; the block layout is in dgt.h).  A
    page holds 64 tokens in every layer.  Device tensors: k, v uint8 [layers,
    pages, kv_heads, 64 * head_dim], k_scale, v_scale float32 [layers, pages,
    kv_heads]; refs int32 [pages], table int32 [max_seqs, max_pages] and lens
    int32 [max_seqs] for the sequences, slots 0..max_seqs-1."""

    def __init__(self, layers: int, pages: int, kv_heads: int, head_dim: int, max_seqs: int, max_pages: int,
                 device="cuda"):
        import torch
        z = lambda dt, *s: torch.zeros(s, dtype=dt, device=device)
        block = KV_PAGE * head_dim
        self.layers, self.pages, self.kv_heads, self.head_dim = layers, pages, kv_heads, head_dim
        self.max_seqs, self.max_pages = max_seqs, max_pages
        self.k, self.v = (z(torch.uint8, layers, pages, kv_heads, block) for _ in range(2))
        self.k_scale, self.v_scale = (z(torch.float32, layers, pages, kv_heads) for _ in range(2))
        self.refs = z(torch.int32, pages)
        self.table = torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=device)
        self.lens = z(torch.int32, max_seqs)
        self.s = KvCacheStruct(layers, pages, kv_heads, head_dim, max_seqs, max_pages,
                               *(t.data_ptr() for t in (self.k, self.v, self.k_scale, self.v_scale, self.refs,
                                                        self.table, self.lens)))
        self.ptr = C.addressof(self.s)
        self.ws = torch.empty(max(int(lib().dgt_kv_pages_workspace_bytes(self.ptr)), 256), dtype=torch.uint8,
                              device=device)   # of the page operations


def kv_append(cache: KvCache, layer: int, k, v, seqs, start, cu=None, status=None, stream=None):
    """dgt_kv_append: new keys and values, bf16 [tokens, kv_heads, head_dim],
    quantised into the pages of the sequences `seqs` int32 [batch] from
    positions `start` int32 [batch] on.  cu int32 [batch + 1]: the rows of
    each (None: one row each)."""
    tokens, batch = k.shape[0], seqs.numel()
    if k.shape != v.shape or tuple(k.shape[1:]) != (cache.kv_heads, cache.head_dim):
        raise ValueError("k, v: [tokens, kv_heads, head_dim]")
    _check(lib().dgt_kv_append(cache.ptr, layer, _heads(k, "k"), _heads(v, "v"), tokens,
                               _i32(seqs, "seqs"), _i32(start, "start", batch),
                               None if cu is None else _i32(cu, "cu", batch + 1), batch, _status(status),
                               _stream_on(cache.k, stream)), "dgt_kv_append")


def kv_read(cache: KvCache, layer, seqs, first, cu, tokens: int, status=None, stream=None):
    """dgt_kv_read: the values of the sequences' positions first[b] .. as bf16
    (k, v), each [tokens, kv_heads, head_dim]; layer None: [layers, tokens,
    ...].  cu int32 [batch + 1] (None: one position each), tokens: their sum."""
    import torch
    batch = seqs.numel()
    if layer is not None and layer < 0:
        raise ValueError("layer: None or 0..layers - 1")
    shape = (tokens, cache.kv_heads, cache.head_dim)
    if layer is None:
        shape = (cache.layers, *shape)
    dev = cache.k.device
    out = [_new(shape, torch.bfloat16, dev, stream) for _ in range(2)]
    _check(lib().dgt_kv_read(cache.ptr, -1 if layer is None else layer, _i32(seqs, "seqs"),
                             _i32(first, "first", batch), None if cu is None else _i32(cu, "cu", batch + 1), batch,
                             tokens, _ptr(out[0]), _ptr(out[1]), _status(status), _stream_on(cache.k, stream)), "dgt_kv_read")
    return out


def _attention_workspace(cache, q_heads, batch, tokens, stream, temp):
    import torch
    nb = int(lib().dgt_kv_attention_workspace_bytes(cache.ptr, q_heads, batch, tokens))
    return _new(max(nb, 256), torch.uint8, cache.k.device, stream, zero=True, temp=temp)


def kv_attention_workspace(cache: KvCache, q_heads: int, batch: int, tokens: int, stream=None):
    """A workspace for kv_attention calls of these sizes on `stream` (zeroed, as its first use wants it)."""
    return _attention_workspace(cache, q_heads, batch, tokens, stream, False)


def kv_attention(cache: KvCache, layer: int, q, seqs, cu=None, scale=None, window: int = 0, sinks: int = 0, out=None,
                 lse=None, ws=None, status=None, stream=None, test_wait_polls=None):
    """dgt_kv_attention_ex: the new rows q, bf16 [tokens, q_heads, head_dim], the
    last ones of the sequences `seqs` int32 [batch], over the cache.  cu int32
    [batch + 1]: the rows of each (None: one row each).  scale: of the scores
    (None: head_dim^-0.5).  window > 0: a row sees its last `window` positions
    and the first `sinks`.  lse: float32 [tokens, q_heads] or None.
    test_wait_polls: the failure-path test hook (see test_wait_flags).
    Returns out, bf16 [tokens, q_heads, head_dim]."""
    import torch
    tokens, heads, dim = q.shape
    batch = seqs.numel()
    if dim != cache.head_dim:
        raise ValueError("q: [tokens, q_heads, head_dim] with the cache's head_dim")
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks: not negative")
    if out is None:
        out = _new((tokens, heads, dim), torch.bfloat16, q.device, stream)
    elif out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_cuda or not out.is_contiguous():
        raise ValueError("out: a contiguous CUDA bfloat16 tensor of q's shape")
    if lse is not None and (lse.numel() != tokens * heads or lse.dtype != torch.float32 or not lse.is_cuda or
                            not lse.is_contiguous()):
        raise ValueError("lse: a contiguous CUDA float32 tensor [tokens, q_heads]")
    if ws is not None and not (ws.is_cuda and ws.is_contiguous()):
        raise ValueError("ws: a contiguous CUDA tensor (kv_attention_workspace)")
    if ws is None:
        ws = _attention_workspace(cache, heads, batch, tokens, stream, True)
    _check(lib().dgt_kv_attention_ex(cache.ptr, layer, _heads(q, "q"), tokens, _i32(seqs, "seqs"),
                                     None if cu is None else _i32(cu, "cu", batch + 1), batch,
                                     dim ** -0.5 if scale is None else scale, min(window, 1 << 30), min(sinks, 1 << 30),
                                     _ptr(out), _ptr(lse),
                                     _ptr(ws), ws.numel(), _status(status), test_wait_flags(test_wait_polls),
                                     _stream_on(cache.k, stream)), "dgt_kv_attention")
    return out


def kv_reserve(cache: KvCache, seqs, count, start=None, status=None, stream=None):
    """dgt_kv_reserve: room for count[i] more tokens of sequence seqs[i] (int32
    on the device), copying a shared partly filled page first.  Returns start
    int32: the lengths before (-1 everywhere when there is too little room)."""
    import torch
    n = seqs.numel()
    if start is None:
        start = _new(n, torch.int32, seqs.device, stream)
    _check(lib().dgt_kv_reserve(cache.ptr, _i32(seqs, "seqs"), _i32(count, "count", n), n,
                                _i32(start, "start", n), _ptr(cache.ws), cache.ws.numel(), _status(status),
                                _stream_on(cache.k, stream)), "dgt_kv_reserve")
    return start


def kv_fork(cache: KvCache, src, dst, status=None, stream=None):
    """dgt_kv_fork: sequences dst[i] become copies of src[i] that share its pages."""
    _check(lib().dgt_kv_fork(cache.ptr, _i32(src, "src"), _i32(dst, "dst", src.numel()), src.numel(),
                             _status(status), _stream_on(cache.k, stream)), "dgt_kv_fork")


def kv_free(cache: KvCache, seqs, status=None, stream=None):
    """dgt_kv_free: the sequences give up their pages."""
    _check(lib().dgt_kv_free(cache.ptr, _i32(seqs, "seqs"), seqs.numel(), _status(status), _stream_on(cache.k, stream)),
           "dgt_kv_free")


def kv_copy_pages(cache: KvCache, src, dst, status=None, stream=None):
    """dgt_kv_copy_pages: pages src[i] -> dst[i] (int32 on the device) in every layer."""
    _check(lib().dgt_kv_copy_pages(cache.ptr, _i32(src, "src"), _i32(dst, "dst", src.numel()), src.numel(),
                                   _status(status), _stream_on(cache.k, stream)), "dgt_kv_copy_pages")


def kv_compact(cache: KvCache, live=None, status=None, stream=None):
    """dgt_kv_compact: the used pages move to the lowest numbers; live (int32
    [1] on the device) gets their count."""
    _check(lib().dgt_kv_compact(cache.ptr, None if live is None else _i32(live, "live", 1), _ptr(cache.ws),
                                cache.ws.numel(), _status(status), _stream_on(cache.k, stream)), "dgt_kv_compact")


# ---------------------------------------------------------------------------
# decoder-layer decode step (batch 1)
# ---------------------------------------------------------------------------
def add_rmsnorm(x32, gamma, eps, h=None, y32=None, stream=None):
    """dgt_add_rmsnorm: x32 += y32 (if given, in place), then h = bf16 RMS norm
    of x32 scaled by gamma (bf16).  Returns h."""
    import torch
    n = x32.numel()
    if h is None:
        h = _new(n, torch.bfloat16, x32.device, stream)
    _check(lib().dgt_add_rmsnorm(_ptr(x32), _ptr(y32), _ptr(gamma), n, C.c_float(eps), _ptr(h), _stream(stream)),
           "dgt_add_rmsnorm")
    return h


def silu_mul(g32, u32, out=None, stream=None):
    """dgt_silu_mul: bf16(silu(g) * u) from two float32 vectors."""
    import torch
    n = g32.numel()
    if out is None:
        out = _new(n, torch.bfloat16, g32.device, stream)
    _check(lib().dgt_silu_mul(_ptr(g32), _ptr(u32), n, _ptr(out), _stream(stream)), "dgt_silu_mul")
    return out


def silu_mul_rows(gu32, out=None, stream=None):
    """dgt_silu_mul_rows: gu32 float32 [rows, 2n] = [gate | up] per row ->
    bf16 [rows, n]."""
    import torch
    rows, n2 = gu32.shape
    n = n2 // 2
    if out is None:
        out = _new((rows, n), torch.bfloat16, gu32.device, stream)
    _check(lib().dgt_silu_mul_rows(_ptr(gu32), rows, n, _ptr(out), _stream(stream)), "dgt_silu_mul_rows")
    return out


def repeat(v, n_out, out=None, stream=None):
    """dgt_repeat: out[i] = v[i mod len(v)] (bf16)."""
    import torch
    if out is None:
        out = _new(n_out, torch.bfloat16, v.device, stream)
    _check(lib().dgt_repeat(_ptr(v), v.numel(), n_out, _ptr(out), _stream(stream)), "dgt_repeat")
    return out


DENSE_PROJ = ("q", "k", "v", "o", "gate", "up", "down")


class StepAttention:
    """The attention of a batch-1 decode step: the new token's q and k turned to
    its position, its k and v appended to sequence `seq` of a KvCache (layer l
    of the step is layer l of the cache), and attention over what the sequence
    holds, with an optional window and first tokens that stay visible.  For
    DecodeStep and MoeDecodeStep; the query heads have the cache's head_dim,
    their count a multiple of its kv_heads.  Positions and lengths live on the
    device, so a captured step moves on by one token with every replay, and
    every eager step appends its token too.  Several
    steps may share one, if they run one after the other: the tokens of each
    follow those of the others.
    self.status (int32 [1]) reports a pool or a table without room
    (DGT_ERR_FULL: nothing is appended) and bad pages."""

    def __init__(self, cache: KvCache, rotary: Rotary, seq: int = 0, window: int = 0, sinks: int = 0, scale=None):
        import torch
        if rotary.axes != 1:
            raise ValueError("rotary: one axis")
        i32 = lambda v: torch.tensor([v], dtype=torch.int32, device=cache.k.device)
        self.cache, self.rotary, self.window, self.sinks, self.scale = cache, rotary, window, sinks, scale
        self.seq, self.one, self.start, self.status = i32(seq), i32(1), i32(0), i32(0)
        self.ws = {}     # by query heads; kept, because captured steps hold their addresses

    def prepare(self, q_width: int, depth: int):
        """Workspace for steps of this query width; checks that the cache has room for the layers."""
        c = self.cache
        if q_width % (c.head_dim * c.kv_heads) or depth > c.layers:
            raise ValueError("the cache's heads or layers do not fit the step's")
        heads = q_width // c.head_dim
        if heads not in self.ws:
            self.ws[heads] = kv_attention_workspace(c, heads, 1, 1)

    def begin(self, stream=None):
        """Room for the step's token; its position to self.start."""
        kv_reserve(self.cache, self.seq, self.one, start=self.start, status=self.status, stream=stream)

    def __call__(self, layer: int, q, k, v, out, stream=None):
        """One layer: bf16 vectors q, k, v of the projections (q and k are
        rotated in place), out bf16 of q's width."""
        c = self.cache
        q, k, v = (x.view(1, -1, c.head_dim) for x in (q, k, v))
        rotate(self.rotary, q, self.start, k=k, q_out=q, k_out=k, stream=stream)
        kv_append(c, layer, k, v, self.seq, self.start, status=self.status, stream=stream)
        kv_attention(c, layer, q, self.seq, scale=self.scale, window=self.window, sinks=self.sinks,
                     out=out.view(q.shape), ws=self.ws[q.shape[1]], status=self.status, stream=stream)


class DecodeStep:
    """One batch-1 decode step through a stack of dense decoder layers, every
    op a kernel of this library.  Per layer, with the fp32 residual stream x:

        h = rmsnorm(x, g1);  q = Wq h;  k = Wk h;  v = Wv h
        a = repeat(v, rows of Wq);  x += Wo a
        h = rmsnorm(x, g2);  m = silu(Wgate h) * (Wup h);  x += Wdown m

    and a final h = rmsnorm(x, g_final).  Without `attention` the output
    projection reads the value vector repeated over the query heads, as above;
    with a StepAttention a is the attention of the new token over its cache,
    and every step appends one token.  layers: list of dicts proj -> R4 (or bf16 tensors [rows, cols] for
    the twin), either q, k, v, o, gate, up, down, or the stacked form qkv
    (rows of q, then k, then v; k and v of equal size), o, gate_up (rows of
    gate, then up) and down, which computes the same step with one product
    for q, k, v and one for gate and up; gammas: list of 2 * len(layers) + 1
    bf16 vectors.  Layer l of the step uses layers[l % len(layers)] and gammas
    for its index, so a few distinct layers can stand in for a deeper model.
    The R4 step and the BF16 step over the same weights give bit-identical
    outputs."""

    def __init__(self, layers, gammas, depth=None, eps=1e-5, device=None, attention=None):
        import torch
        self.attention = attention
        self.layers, self.gammas, self.eps = layers, gammas, eps
        self.depth = depth or len(layers)
        w0 = layers[0]
        self.fused = "qkv" in w0
        self.r4 = isinstance(w0["o"], R4)
        shape = (lambda w: (w.rows, w.cols)) if self.r4 else (lambda w: tuple(w.shape))
        hidden = shape(w0["o"])[0]
        dims = {p: shape(w0[p])[0] for p in w0}
        dev = device or (w0["o"].sm.device if self.r4 else w0["o"].device)
        self.hidden = hidden
        f32 = lambda n: torch.empty(n, dtype=torch.float32, device=dev)
        b16 = lambda n: torch.empty(n, dtype=torch.bfloat16, device=dev)
        self.x = f32(hidden)
        self.h = b16(hidden)
        self.y = {p: (b16(dims[p]), f32(dims[p])) for p in w0}
        nq = shape(w0["o"])[1]                       # query width: the output projection's input
        self.ffn = shape(w0["down"])[1]
        if self.fused:
            nkv = (dims["qkv"] - nq) // 2
            self.q16, self.k16 = self.y["qkv"][0][:nq], self.y["qkv"][0][nq:nq + nkv]
            self.v16 = self.y["qkv"][0][nq + nkv:nq + 2 * nkv]
            self.g32 = self.y["gate_up"][1][:self.ffn]
            self.u32 = self.y["gate_up"][1][self.ffn:]
        else:
            self.q16, self.k16, self.v16 = (self.y[p][0] for p in ("q", "k", "v"))
            self.g32, self.u32 = self.y["gate"][1], self.y["up"][1]
        self.a = b16(nq)
        self.m = b16(self.ffn)
        self.out = b16(hidden)
        self._graph = None
        if attention is not None:
            attention.prepare(nq, self.depth)
        # the step streams its weights before each product's dependency wait
        # (DGT_GEMV_STATIC_WEIGHTS): everything that wrote them must be done
        torch.cuda.synchronize(dev)

    def _gemv(self, W, x, p, stream):
        # the step's weights are only read: they stream while the previous kernel ends
        y, y32 = self.y[p]
        if self.r4:
            gemv(W, x, y, y32, stream=stream, static_weights=True)
        else:
            gemv_bf16(W, x, y, y32, stream=stream, static_weights=True)
        return y, y32

    def launch(self, stream=None):
        """Queue the step on `stream` (self.x holds the input, then the output
        residual stream; self.out the final normed vector)."""
        gi = 0
        if self.attention is not None:
            self.attention.begin(stream)
        for l in range(self.depth):
            W = self.layers[l % len(self.layers)]
            add_rmsnorm(self.x, self.gammas[gi % (len(self.gammas) - 1)], self.eps, self.h,
                        None if l == 0 else self.y["down"][1], stream)
            gi += 1
            for p in (("qkv",) if self.fused else ("q", "k", "v")):
                self._gemv(W[p], self.h, p, stream)
            if self.attention is not None:
                self.attention(l, self.q16, self.k16, self.v16, self.a, stream)
            else:
                repeat(self.v16, self.a.numel(), self.a, stream)
            self._gemv(W["o"], self.a, "o", stream)
            add_rmsnorm(self.x, self.gammas[gi % (len(self.gammas) - 1)], self.eps, self.h, self.y["o"][1], stream)
            gi += 1
            for p in (("gate_up",) if self.fused else ("gate", "up")):
                self._gemv(W[p], self.h, p, stream)
            silu_mul(self.g32, self.u32, self.m, stream)
            self._gemv(W["down"], self.m, "down", stream)
        add_rmsnorm(self.x, self.gammas[-1], self.eps, self.out, self.y["down"][1], stream)

    def __call__(self, x0, stream=None):
        """Eager step from the fp32 input x0: returns (x, out)."""
        import torch
        with torch.cuda.stream(stream):
            self.x.copy_(x0)
        self.launch(stream)
        return self.x, self.out

    def capture(self):
        """Capture launch() in a CUDA graph; replay() then runs the step on the
        current contents of self.x.  Nothing runs here and no eager step is
        needed before: with an attention that would leave a token in its
        sequence."""
        import torch
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                self.launch(s)
        torch.cuda.current_stream().wait_stream(s)
        self._graph = g
        return g

    def replay(self, x0=None):
        if x0 is not None:
            self.x.copy_(x0)
        self._graph.replay()
        return self.x, self.out


def weighted_sum(y32, p, out=None, stream=None):
    """dgt_weighted_sum: out = sum over slots j of p[j] * y32[j] (fmaf chain in
    slot order from +0); y32 float32 [slots, n], p float32 [slots]."""
    import torch
    slots = p.numel()
    n = y32.numel() // slots
    if out is None:
        out = _new(n, torch.float32, y32.device, stream)
    _check(lib().dgt_weighted_sum(_ptr(y32), _ptr(p), slots, n, _ptr(out), _stream(stream)), "dgt_weighted_sum")
    return out


class MoeDecodeStep:
    """A batch-1 decode step through a stack of mixture-of-experts decoder
    layers, every op a kernel of this library.  Per layer, with the fp32
    residual stream x and the layer's routing (expert ids[j], weights p[j],
    j < topk):

        h = rmsnorm(x, g1);  q, k, v = W h;  a = repeat(v, rows of Wq);  x += Wo a
        h = rmsnorm(x, g2);  for every slot j (one gather each):
            m_j = silu(Wgate[ids[j]] h) * (Wup[ids[j]] h);  d_j = Wdown[ids[j]] m_j
        x += sum_j p[j] d_j   (slot order)

    and a final rmsnorm.  Wgate, Wup ([E * ffn, hidden]) and Wdown
    ([E * hidden, ffn]) stack the experts; the gate and up gathers take the
    token's h once for all its slots, the down gather takes slot j's m_j as
    its own input.  Routing is an input (the router is not part of the
    format).  layers: dicts with q, k, v, o, gate, up, down (R4, or bf16
    tensors for the twin), or the stacked form qkv, o, gate_up, down, where
    gate_up stacks expert e's gate rows and then its up rows as expert e's
    block ([E * 2 ffn, hidden]): one product for q, k, v and one gather for
    gate and up.  routes: per layer (ids int32 [topk], p float32 [topk]) on
    the device; layer l uses layers[l % len] and routes[l % len].  attention: a
    StepAttention, as in DecodeStep.  The R4 step and the BF16 step give
    bit-identical outputs."""

    def __init__(self, layers, gammas, routes, n_experts, depth=None, eps=1e-5, attention=None):
        import torch
        self.attention = attention
        self.layers, self.gammas, self.routes, self.E, self.eps = layers, gammas, routes, n_experts, eps
        self.depth = depth or len(layers)
        w0 = layers[0]
        self.fused = "qkv" in w0
        self.r4 = isinstance(w0["o"], R4)
        shape = (lambda w: (w.rows, w.cols)) if self.r4 else (lambda w: tuple(w.shape))
        hidden = shape(w0["o"])[0]
        ffn = shape(w0["down"])[1]
        topk = routes[0][0].numel()
        dev = w0["o"].sm.device if self.r4 else w0["o"].device
        self.hidden, self.ffn, self.topk = hidden, ffn, topk
        f32 = lambda *s: torch.empty(s, dtype=torch.float32, device=dev)
        b16 = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=dev)
        self.x, self.h, self.out = f32(hidden), b16(hidden), b16(hidden)
        attn = ("qkv", "o") if self.fused else ("q", "k", "v", "o")
        self.y = {p: (b16(shape(w0[p])[0]), f32(shape(w0[p])[0])) for p in attn}
        nq = shape(w0["o"])[1]
        if self.fused:
            nkv = (shape(w0["qkv"])[0] - nq) // 2
            self.q16, self.k16 = self.y["qkv"][0][:nq], self.y["qkv"][0][nq:nq + nkv]
            self.v16 = self.y["qkv"][0][nq + nkv:nq + 2 * nkv]
            self.ygu = f32(1, topk, 2 * ffn)
        else:
            self.q16, self.k16, self.v16 = (self.y[p][0] for p in ("q", "k", "v"))
            self.yg, self.yu = f32(1, topk, ffn), f32(1, topk, ffn)
        self.a = b16(nq)
        self.m = b16(topk, ffn)
        self.yd = f32(topk, 1, hidden)
        self.comb = f32(hidden)
        nb_up = moe_workspace_bytes(n_experts, 2 * ffn if self.fused else ffn, hidden, 1, topk)
        nb_dn = moe_workspace_bytes(n_experts, hidden, ffn, topk, 1)
        self.ws_g = torch.empty(max(nb_up, 256), dtype=torch.uint8, device=dev)
        self.ws_u = torch.empty(max(nb_up, 256), dtype=torch.uint8, device=dev)
        self.ws_d = torch.empty(max(nb_dn, 256), dtype=torch.uint8, device=dev)
        self._graph = None
        if attention is not None:
            attention.prepare(nq, self.depth)
        torch.cuda.synchronize(dev)     # the products stream weights before their dependency wait

    def _gemv(self, W, x, p, stream):
        y, y32 = self.y[p]
        if self.r4:
            gemv(W, x, y, y32, stream=stream, static_weights=True)
        else:
            gemv_bf16(W, x, y, y32, stream=stream, static_weights=True)

    def _moe(self, W, ids, x, ws, y32, stream):
        f = moe_gemv if self.r4 else moe_gemv_bf16
        f(W, self.E, ids, None, x, ws=ws, y32=y32, stream=stream)

    def launch(self, stream=None):
        ng = len(self.gammas) - 1
        if self.attention is not None:
            self.attention.begin(stream)
        for l in range(self.depth):
            W = self.layers[l % len(self.layers)]
            ids, p = self.routes[l % len(self.routes)]
            add_rmsnorm(self.x, self.gammas[(2 * l) % ng], self.eps, self.h, None if l == 0 else self.comb, stream)
            for pr in (("qkv",) if self.fused else ("q", "k", "v")):
                self._gemv(W[pr], self.h, pr, stream)
            if self.attention is not None:
                self.attention(l, self.q16, self.k16, self.v16, self.a, stream)
            else:
                repeat(self.v16, self.a.numel(), self.a, stream)
            self._gemv(W["o"], self.a, "o", stream)
            add_rmsnorm(self.x, self.gammas[(2 * l + 1) % ng], self.eps, self.h, self.y["o"][1], stream)
            ids1 = ids.view(1, self.topk)
            if self.fused:
                self._moe(W["gate_up"], ids1, self.h.view(1, -1), self.ws_g, self.ygu, stream)
                silu_mul_rows(self.ygu.view(self.topk, 2 * self.ffn), self.m, stream)
            else:
                self._moe(W["gate"], ids1, self.h.view(1, -1), self.ws_g, self.yg, stream)
                self._moe(W["up"], ids1, self.h.view(1, -1), self.ws_u, self.yu, stream)
                silu_mul(self.yg, self.yu, self.m.view(-1), stream)
            self._moe(W["down"], ids.view(self.topk, 1), self.m, self.ws_d, self.yd, stream)
            weighted_sum(self.yd, p, self.comb, stream)
        add_rmsnorm(self.x, self.gammas[-1], self.eps, self.out, self.comb, stream)

    def __call__(self, x0, stream=None):
        import torch
        with torch.cuda.stream(stream):
            self.x.copy_(x0)
        self.launch(stream)
        return self.x, self.out

    def capture(self):
        """As DecodeStep.capture."""
        import torch
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                self.launch(s)
        torch.cuda.current_stream().wait_stream(s)
        self._graph = g
        return g

    def replay(self, x0=None):
        if x0 is not None:
            self.x.copy_(x0)
        self._graph.replay()
        return self.x, self.out


# ---------------------------------------------------------------------------
# exponent statistics
# ---------------------------------------------------------------------------
def exponent_stats(w, tile=128, stream=None):
    """dgt_exponent_stats on a device bf16 tensor (any shape, flat order):
    returns (hist int64 [256], tile_bits float64 [tiles] (both on the device),
    total tile bits, tensor exponent entropy in bits per weight)."""
    import torch
    n = w.numel()
    dev = w.device
    hist = _new(256, torch.int64, dev, stream)
    # an invalid tile gets a 1-element buffer; the C call rejects it
    tb = _new(max((n + tile - 1) // tile, 1) if tile > 0 else 1, torch.float64, dev, stream)
    tot = _new(2, torch.float64, dev, stream, temp=True)
    _check(lib().dgt_exponent_stats(_ptr(w), n, tile, _ptr(hist), _ptr(tb), _ptr(tot), _stream(stream)),
           "dgt_exponent_stats")
    with torch.cuda.stream(stream):
        t = tot.cpu()
    return hist, tb, float(t[0]), float(t[1])

