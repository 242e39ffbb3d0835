"""Thin Python binding over the C ABI of libkvq.so (include/kvq.h).

Argument marshalling only: tensors are checked and turned into raw device
pointers; all work runs in the library's CUDA kernels.  PyTorch supplies the
device memory and the stream.  There is no CPU fallback: importing this
module fails if libkvq.so has not been built
(``python -m rotated_int4_kv_kvq_b200.build``).
"""

from __future__ import annotations

import contextlib
import ctypes
import os

import torch

SRFT = 0
SRHT = 1

KVQ_OK = 0
STATUS = {
    0: "KVQ_OK", 1: "KVQ_ERR_NULL", 2: "KVQ_ERR_BAD_DIM", 3: "KVQ_ERR_BAD_GROUP",
    4: "KVQ_ERR_MISALIGNED", 5: "KVQ_ERR_BAD_ROT", 6: "KVQ_ERR_CUDA",
    7: "KVQ_ERR_BAD_SIZE", 8: "KVQ_ERR_DEVICE_TIMEOUT", 9: "KVQ_ERR_UNSUPPORTED_DEVICE",
    10: "KVQ_ERR_BAD_BITS", 11: "KVQ_ERR_BAD_INDEX", 12: "KVQ_ERR_BAD_DTYPE",
}

LIB_PATH = os.environ.get("KVQ_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libkvq.so")

EXPORTS = ("kvq_rot_quant_fwd", "kvq_dequant_rot_inv", "kvq_rot_quant_fwd_lambda",
           "kvq_dequant_rot_inv_lambda", "kvq_rot_quant_fwd_bits", "kvq_dequant_rot_inv_bits",
           "kvq_decode_step", "kvq_decode_step_windowed",
           "kvq_attend_decode", "kvq_qk_norm_rope", "kvq_paged_append", "kvq_paged_attend",
           "kvq_paged_attend_workspace", "kvq_status_string", "kvq_device_status", "kvq_version")

DTYPES = {torch.float16: 0, torch.bfloat16: 1}  # kvq_dtype


class _PagedCacheC(ctypes.Structure):  # kvq_paged_cache
    _fields_ = [("k_packed", ctypes.c_void_p), ("v_packed", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("n_kv_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("d", ctypes.c_int32), ("group", ctypes.c_int32),
                ("signs", ctypes.c_void_p), ("rot", ctypes.c_int32)]


class _RopeC(ctypes.Structure):  # kvq_rope
    _fields_ = [("cos_sin", ctypes.c_void_p), ("n_pos", ctypes.c_int64),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class KVQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({status_string(status)})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m rotated_int4_kv_kvq_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(LIB_PATH)
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    lib.kvq_rot_quant_fwd.argtypes = [p, i64, i32, i32, p, i32, p, p, p]
    lib.kvq_rot_quant_fwd.restype = i32
    lib.kvq_dequant_rot_inv.argtypes = [p, p, i64, i32, i32, p, i32, p, p]
    lib.kvq_dequant_rot_inv.restype = i32
    lib.kvq_rot_quant_fwd_lambda.argtypes = [p, i64, i32, i32, p, p, i32, p, p, p]
    lib.kvq_rot_quant_fwd_lambda.restype = i32
    lib.kvq_dequant_rot_inv_lambda.argtypes = [p, p, i64, i32, i32, p, p, i32, p, p]
    lib.kvq_dequant_rot_inv_lambda.restype = i32
    lib.kvq_decode_step.argtypes = [p, p, p, i64, i64, i64, i32, i32, p, i32, p, p]
    lib.kvq_decode_step.restype = i32
    lib.kvq_decode_step_windowed.argtypes = [p, p, p, p, i64, i64, i64, i32, i32, i32, p, i32, p]
    lib.kvq_decode_step_windowed.restype = i32
    lib.kvq_rot_quant_fwd_bits.argtypes = [p, i64, i32, i32, i32, p, i32, p, p, p]
    lib.kvq_rot_quant_fwd_bits.restype = i32
    lib.kvq_dequant_rot_inv_bits.argtypes = [p, p, i64, i32, i32, i32, p, i32, p, p]
    lib.kvq_dequant_rot_inv_bits.restype = i32
    lib.kvq_attend_decode.argtypes = [p, p, p, p, p, i64, i32, i64, i64, i32, i32, p, i32,
                                      ctypes.c_float, p, p]
    lib.kvq_attend_decode.restype = i32
    lib.kvq_qk_norm_rope.argtypes = [p, p, i32, i64, i32, i32, i32, i64, i64, p, p, p, p, p, p,
                                     i64, i64, p]
    lib.kvq_qk_norm_rope.restype = i32
    lib.kvq_paged_append.argtypes = [p, p, i32, i64, i64, i64, p, p, p, p, p, p, p, p]
    lib.kvq_paged_append.restype = i32
    lib.kvq_paged_attend.argtypes = [p, i32, i64, i64, p, p, p, p, i64, i64, i32, i32, i32,
                                     ctypes.c_float, p, i64, p, i64, p]
    lib.kvq_paged_attend.restype = i32
    lib.kvq_paged_attend_workspace.argtypes = [i64, i32, i32, i32, i32]
    lib.kvq_paged_attend_workspace.restype = i64
    lib.kvq_status_string.argtypes = [i32]
    lib.kvq_status_string.restype = ctypes.c_char_p
    lib.kvq_device_status.argtypes = [i32]
    lib.kvq_device_status.restype = i32
    lib.kvq_version.argtypes = []
    lib.kvq_version.restype = i32
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.kvq_status_string(int(status)).decode()


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


# torch's query of a device's current raw stream handle; building a
# torch.cuda.Stream object per call costs ~2 us, the raw query ~0.1 us.
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, dev: torch.device) -> int | None:
    """Raw handle of `stream`; None means the current stream of `dev`."""
    if stream is None:
        if _raw_current_stream is not None and dev.index is not None:
            return _raw_current_stream(dev.index)
        stream = torch.cuda.current_stream(dev)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _device_of(tensors, stream) -> torch.device:
    """The one CUDA device that every tensor argument lives on.

    The library launches on the calling thread's current device and builds
    its copy descriptors over the pointers it is given, so all operands of a
    call must share one device; an explicit torch stream must belong to it
    too.  Raises ValueError before anything is launched otherwise.  (A raw
    integer stream handle cannot be checked here; it must belong to the same
    device.)"""
    devs = {t.device for t in tensors if t is not None}
    if len(devs) != 1:
        raise ValueError("all tensor arguments must be on one CUDA device, got "
                         + ", ".join(sorted(str(d) for d in devs)))
    dev = devs.pop()
    if isinstance(stream, torch.cuda.Stream) and stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, tensors on {dev}")
    return dev


def _current(dev: torch.device):
    """Context that makes `dev` the current device for one library call."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _empty(like: torch.Tensor, shape, stream) -> torch.Tensor:
    """An uninitialized tensor of `like`'s type and device that belongs to the
    stream the call runs on: memory that the current stream's queued work still
    uses is not handed to a kernel of another stream."""
    if stream is None:
        return like.new_empty(shape)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return like.new_empty(shape)


def _check(t: torch.Tensor, name: str, dtype, shape):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != tuple(shape):  # torch.Size compares as a tuple
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _raise(fn: str, st: int):
    if st != KVQ_OK:
        raise KVQError(fn, st)


def kvq_rot_quant_fwd(x: torch.Tensor, signs: torch.Tensor, rot: int, group: int,
                      packed: torch.Tensor | None = None,
                      scales: torch.Tensor | None = None, stream=None,
                      lam: torch.Tensor | None = None):
    """Forward step on x [n_vec, d] fp16 -> (packed [n_vec, d/2] u8,
    scales [n_vec, d/group] f32).  Outputs are allocated when not given.
    With ``lam`` ([d] f32), x is scaled channel-wise first
    (kvq_rot_quant_fwd_lambda)."""
    n, d = x.shape
    _check(x, "x", torch.float16, (n, d))
    _check(signs, "signs", torch.int8, (d,))
    if packed is None:
        packed = torch.empty((n, d // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((n, d // group), dtype=torch.float32, device=x.device)
    _check(packed, "packed", torch.uint8, (n, d // 2))
    _check(scales, "scales", torch.float32, (n, d // group))
    if lam is not None:
        _check(lam, "lam", torch.float32, (d,))
    dev = _device_of((x, signs, packed, scales, lam), stream)
    with _current(dev):
        if lam is None:
            st = lib.kvq_rot_quant_fwd(_ptr(x), n, d, group, _ptr(signs), rot, _ptr(packed),
                                       _ptr(scales), _stream(stream, dev))
            _raise("kvq_rot_quant_fwd", st)
        else:
            st = lib.kvq_rot_quant_fwd_lambda(_ptr(x), n, d, group, _ptr(signs), _ptr(lam), rot,
                                              _ptr(packed), _ptr(scales), _stream(stream, dev))
            _raise("kvq_rot_quant_fwd_lambda", st)
    return packed, scales


def kvq_dequant_rot_inv(packed: torch.Tensor, scales: torch.Tensor, signs: torch.Tensor,
                        rot: int, group: int, out: torch.Tensor | None = None, stream=None,
                        lam: torch.Tensor | None = None):
    """Inverse step -> out [n_vec, d] fp16 (allocated when not given).  With
    ``lam`` ([d] f32) the result is divided channel-wise by it
    (kvq_dequant_rot_inv_lambda)."""
    n, half = packed.shape
    d = 2 * half
    _check(packed, "packed", torch.uint8, (n, half))
    _check(scales, "scales", torch.float32, (n, d // group))
    _check(signs, "signs", torch.int8, (d,))
    if out is None:
        out = torch.empty((n, d), dtype=torch.float16, device=packed.device)
    _check(out, "out", torch.float16, (n, d))
    if lam is not None:
        _check(lam, "lam", torch.float32, (d,))
    dev = _device_of((packed, scales, signs, out, lam), stream)
    with _current(dev):
        if lam is None:
            st = lib.kvq_dequant_rot_inv(_ptr(packed), _ptr(scales), n, d, group, _ptr(signs),
                                         rot, _ptr(out), _stream(stream, dev))
            _raise("kvq_dequant_rot_inv", st)
        else:
            st = lib.kvq_dequant_rot_inv_lambda(_ptr(packed), _ptr(scales), n, d, group,
                                                _ptr(signs), _ptr(lam), rot, _ptr(out),
                                                _stream(stream, dev))
            _raise("kvq_dequant_rot_inv_lambda", st)
    return out


def kvq_rot_quant_fwd_bits(x: torch.Tensor, signs: torch.Tensor, rot: int, group: int,
                           bits: int, packed: torch.Tensor | None = None,
                           scales: torch.Tensor | None = None, stream=None):
    """Forward step with b-bit codes: packed [n_vec, d*bits/8] u8 (little-endian
    bitstream per vector), scales [n_vec, d/group] f32."""
    n, d = x.shape
    qp = d * bits // 8
    _check(x, "x", torch.float16, (n, d))
    _check(signs, "signs", torch.int8, (d,))
    if packed is None:
        packed = torch.empty((n, qp), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((n, d // group), dtype=torch.float32, device=x.device)
    _check(packed, "packed", torch.uint8, (n, qp))
    _check(scales, "scales", torch.float32, (n, d // group))
    dev = _device_of((x, signs, packed, scales), stream)
    with _current(dev):
        st = lib.kvq_rot_quant_fwd_bits(_ptr(x), n, d, group, bits, _ptr(signs), rot,
                                        _ptr(packed), _ptr(scales), _stream(stream, dev))
    _raise("kvq_rot_quant_fwd_bits", st)
    return packed, scales


def kvq_dequant_rot_inv_bits(packed: torch.Tensor, scales: torch.Tensor, signs: torch.Tensor,
                             rot: int, group: int, bits: int, out: torch.Tensor | None = None,
                             stream=None):
    """Inverse step of kvq_rot_quant_fwd_bits -> out [n_vec, d] fp16."""
    n, qp = packed.shape
    d = qp * 8 // bits
    _check(packed, "packed", torch.uint8, (n, qp))
    _check(scales, "scales", torch.float32, (n, d // group))
    _check(signs, "signs", torch.int8, (d,))
    if out is None:
        out = torch.empty((n, d), dtype=torch.float16, device=packed.device)
    _check(out, "out", torch.float16, (n, d))
    dev = _device_of((packed, scales, signs, out), stream)
    with _current(dev):
        st = lib.kvq_dequant_rot_inv_bits(_ptr(packed), _ptr(scales), n, d, group, bits,
                                          _ptr(signs), rot, _ptr(out), _stream(stream, dev))
    _raise("kvq_dequant_rot_inv_bits", st)
    return out


def kvq_decode_step(x_new: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, pos: int,
                    signs: torch.Tensor, rot: int, group: int,
                    out: torch.Tensor | None = None, stream=None):
    """Decode step on a head-major cache: packed [H, cap, d/2] u8 and
    scales [H, cap, d/group] f32 get row ``pos``; returns out [H, pos+1, d]."""
    h, d = x_new.shape
    cap = packed.shape[1]
    _check(x_new, "x_new", torch.float16, (h, d))
    _check(packed, "packed", torch.uint8, (h, cap, d // 2))
    _check(scales, "scales", torch.float32, (h, cap, d // group))
    _check(signs, "signs", torch.int8, (d,))
    if out is None:
        out = torch.empty((h, pos + 1, d), dtype=torch.float16, device=x_new.device)
    _check(out, "out", torch.float16, (h, pos + 1, d))
    dev = _device_of((x_new, packed, scales, signs, out), stream)
    with _current(dev):
        st = lib.kvq_decode_step(_ptr(x_new), _ptr(packed), _ptr(scales), h, cap, pos, d, group,
                                 _ptr(signs), rot, _ptr(out), _stream(stream, dev))
    _raise("kvq_decode_step", st)
    return out


def kvq_decode_step_windowed(x_new: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                             kv: torch.Tensor, pos: int, signs: torch.Tensor, rot: int, group: int,
                             window: int = 16, stream=None):
    """Decode step with a dequantized-prefix cache: kv [H, cap, d] fp16 is the
    persistent attention view (row ``pos`` gets x_new; a completed window of
    ``window`` rows is quantized into packed/scales and replaced by its
    dequantized values).  Returns kv."""
    h, d = x_new.shape
    cap = packed.shape[1]
    _check(x_new, "x_new", torch.float16, (h, d))
    _check(packed, "packed", torch.uint8, (h, cap, d // 2))
    _check(scales, "scales", torch.float32, (h, cap, d // group))
    _check(kv, "kv", torch.float16, (h, cap, d))
    _check(signs, "signs", torch.int8, (d,))
    dev = _device_of((x_new, packed, scales, kv, signs), stream)
    with _current(dev):
        st = lib.kvq_decode_step_windowed(_ptr(x_new), _ptr(packed), _ptr(scales), _ptr(kv), h,
                                          cap, pos, window, d, group, _ptr(signs), rot,
                                          _stream(stream, dev))
    _raise("kvq_decode_step_windowed", st)
    return kv


def kvq_attend_decode(q: torch.Tensor, k_packed: torch.Tensor, k_scales: torch.Tensor,
                      v_packed: torch.Tensor, v_scales: torch.Tensor, length: int,
                      signs: torch.Tensor, rot: int, group: int, sm_scale: float | None = None,
                      out: torch.Tensor | None = None, stream=None):
    """Decode attention over the int4 cache: q [H, nq, d] fp16 against
    rows [0, length) of the K/V caches [H, cap, d/2] (+ scales); returns
    out [H, nq, d] fp16.  sm_scale defaults to 1/sqrt(d)."""
    h, nq, d = q.shape
    cap = k_packed.shape[1]
    _check(q, "q", torch.float16, (h, nq, d))
    for name, t in (("k_packed", k_packed), ("v_packed", v_packed)):
        _check(t, name, torch.uint8, (h, cap, d // 2))
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        _check(t, name, torch.float32, (h, cap, d // group))
    _check(signs, "signs", torch.int8, (d,))
    if out is None:
        out = torch.empty((h, nq, d), dtype=torch.float16, device=q.device)
    _check(out, "out", torch.float16, (h, nq, d))
    scale = float(sm_scale) if sm_scale is not None else d ** -0.5
    dev = _device_of((q, k_packed, k_scales, v_packed, v_scales, signs, out), stream)
    with _current(dev):
        st = lib.kvq_attend_decode(_ptr(q), _ptr(k_packed), _ptr(k_scales), _ptr(v_packed),
                                   _ptr(v_scales), h, nq, cap, length, d, group, _ptr(signs),
                                   rot, scale, _ptr(out), _stream(stream, dev))
    _raise("kvq_attend_decode", st)
    return out


def rope_table(n_pos: int, rot_dim: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """Table [n_pos, rot_dim] f32 of the position rotation: row p holds the
    rot_dim/2 cosines, then the sines, of p theta^(-2i/rot_dim).  The angles
    are formed in 64 bits: at far positions 32 lose the fraction of a turn."""
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
    p = torch.arange(n_pos, dtype=torch.float64, device=device)
    angle = p[:, None] * theta ** (-i / rot_dim)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def paged_rows(cu_q: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor,
               page_size: int, n_tokens: int):
    """Positions [n_tokens] int32 and slots [n_tokens] int64 of the new tokens
    that cu_q, kv_len (after the append) and page_table describe, for
    kvq_qk_norm_rope and kvq_paged_append; -1 for tokens of no sequence or
    before position 0.  A token whose page the table does not have (past its
    end, or a negative entry) gets a slot past every pool, which the append
    skips and reports.  The same for every layer: computed once a step, on the
    device, without a synchronization."""
    tok = torch.arange(n_tokens, device=cu_q.device)
    n_seqs, max_pages = page_table.shape
    if n_seqs == 0:
        return torch.full_like(tok, -1, dtype=torch.int32), torch.full_like(tok, -1)
    seq = torch.searchsorted(cu_q[1:], tok, right=True).clamp_(max=n_seqs - 1)
    end = cu_q[1:][seq]
    here = (tok >= cu_q[seq]) & (tok < end)
    pos = torch.where(here, kv_len[seq].long() - end + tok, -1)
    col = pos // page_size
    if max_pages:
        page = page_table[seq, col.clamp(0, max_pages - 1)].long()
    else:
        page = torch.full_like(tok, -1)
    slots = torch.where((col < max_pages) & (page >= 0), page * page_size + pos % page_size, 1 << 62)
    return pos.int(), torch.where(pos >= 0, slots, -1)


class PagedCache:
    """The int4 K/V cache of one layer in pages: k_packed, v_packed
    [pages, H, page_size, d/2] u8, k_scales, v_scales [pages, H, page_size,
    d/group] f32, the sign vector [d] i8 and the rotation.  A page row is a row
    of kvq_rot_quant_fwd.  The fields are fixed (calls use the tensors' addresses):
    other tensors want another PagedCache."""

    __slots__ = ("k_packed", "k_scales", "v_packed", "v_scales", "signs", "rot", "n_pages",
                 "n_kv_heads", "page_size", "d", "group", "device", "c", "ref")

    def __init__(self, k_packed: torch.Tensor, k_scales: torch.Tensor, v_packed: torch.Tensor,
                 v_scales: torch.Tensor, signs: torch.Tensor, rot: int = SRFT):
        if not isinstance(k_packed, torch.Tensor) or k_packed.dim() != 4:
            raise ValueError("k_packed must be a tensor [pages, heads, page_size, d/2]")
        if not isinstance(k_scales, torch.Tensor) or k_scales.dim() != 4 or k_scales.shape[3] < 1:
            raise ValueError("k_scales must be a tensor [pages, heads, page_size, d/group]")
        pages, heads, page, half = shape = tuple(k_packed.shape)
        d = 2 * half
        group = d // k_scales.shape[3]
        _check(k_packed, "k_packed", torch.uint8, shape)
        _check(v_packed, "v_packed", torch.uint8, shape)
        shape = (pages, heads, page, d // max(group, 1))
        _check(k_scales, "k_scales", torch.float32, shape)
        _check(v_scales, "v_scales", torch.float32, shape)
        _check(signs, "signs", torch.int8, (d,))
        dev = _one_device((k_packed, k_scales, v_packed, v_scales, signs))
        c = _PagedCacheC(k_packed.data_ptr(), v_packed.data_ptr(), k_scales.data_ptr(),
                         v_scales.data_ptr(), pages, heads, page, d, group, signs.data_ptr(), rot)
        fields = dict(k_packed=k_packed, k_scales=k_scales, v_packed=v_packed, v_scales=v_scales,
                      signs=signs, rot=rot, n_pages=pages, n_kv_heads=heads, page_size=page, d=d,
                      group=group, device=dev, c=c, ref=ctypes.addressof(c))
        for name, value in fields.items():
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        if getattr(self, name, None) is value and name in self.__slots__:
            return  # cache.k_scales *= 2 works in place, then assigns what is there
        raise AttributeError(f"the fields of a PagedCache are fixed ({name!r}): make another one")

    def __delattr__(self, name):
        raise AttributeError(f"the fields of a PagedCache are fixed ({name!r}): make another one")

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, page_size: int, d: int, group: int,
              signs: torch.Tensor, rot: int = SRFT) -> "PagedCache":
        """A pool of n_pages uninitialized pages on the device of `signs`."""
        if group < 1 or d % group != 0:
            raise ValueError(f"group {group} does not divide d = {d}")

        def codes():
            return torch.empty((n_pages, n_kv_heads, page_size, d // 2), dtype=torch.uint8,
                               device=signs.device)

        def scales():
            return torch.empty((n_pages, n_kv_heads, page_size, d // group), device=signs.device)
        return cls(codes(), scales(), codes(), scales(), signs, rot)

    def tensors(self):
        return self.k_packed, self.k_scales, self.v_packed, self.v_scales, self.signs


def _one_device(tensors) -> int:
    """Index of the one CUDA device that every tensor (None: absent) lives on.
    (Integer indexes: device objects cost a few hundred ns each to compare.)"""
    dev = -1
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if i != dev:
                if dev >= 0 or i < 0:
                    _device_of(tensors, None)  # says which
                    raise ValueError("all tensor arguments must be on one CUDA device")
                dev = i
    return dev


def _enter(dev: int, stream):
    """For a call on device index `dev`: (raw stream handle, context to leave).
    The context is None when the device is current already."""
    if isinstance(stream, torch.cuda.Stream) and stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, tensors on cuda:{dev}")
    if stream is None:
        raw = (_raw_current_stream(dev) if _raw_current_stream is not None
               else torch.cuda.current_stream(dev).cuda_stream)
    else:
        raw = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    guard = None
    if dev != torch.cuda.current_device():  # last: nothing after it can fail
        guard = torch.cuda.device(dev)
        guard.__enter__()
    return raw, guard


def _call(fn: str, dev: int, stream, args) -> None:
    raw, guard = _enter(dev, stream)
    try:
        st = getattr(lib, fn)(*args, raw)
    finally:
        if guard is not None:
            guard.__exit__(None, None, None)
    if st != KVQ_OK:
        raise KVQError(fn, st)


def _check_tokens(t: torch.Tensor, name: str, dtype, shape) -> int:
    """Checks rows [tokens, heads, d] whose tokens may lie apart (a part of a
    fused projection); returns the token stride."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype or dtype not in DTYPES:
        raise TypeError(f"{name} must be {dtype if dtype in DTYPES else 'float16 or bfloat16'}, "
                        f"got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    tokens, heads, d = shape
    st, sh, sd = t.stride()
    if sd != 1 or (sh != d and heads > 1):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return st if tokens > 1 else heads * d  # the stride of a single token says nothing


def _int32(x) -> int:
    """A whole number of rows or tokens for an int32 argument: beyond it as good
    as the largest, below 0 refused by the call.  (ctypes keeps the low 32 bits.)"""
    return max(-1, min(int(x), (1 << 31) - 1))


def _rope(positions, cos_sin, interleaved, eps, n_tokens):
    """(address of positions or None, kvq_rope) of a call."""
    pos = None
    if positions is not None:
        _check(positions, "positions", torch.int32, (n_tokens,))
        pos = positions.data_ptr()
    if cos_sin is None:
        return pos, _RopeC(None, 0, 0, 0, eps)
    if positions is None:
        raise ValueError("a rotation needs positions")
    if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2:
        raise ValueError("cos_sin must be a table [positions, rot_dim]")
    n_pos, rot_dim = shape = cos_sin.shape
    _check(cos_sin, "cos_sin", torch.float32, shape)
    return pos, _RopeC(cos_sin.data_ptr(), n_pos, rot_dim, bool(interleaved), eps)


def kvq_qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None = None, *,
                     positions: torch.Tensor | None = None, cos_sin: torch.Tensor | None = None,
                     interleaved: bool = False, q_weight: torch.Tensor | None = None,
                     k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                     q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                     stream=None):
    """Norm (weights [d] f32; none without a weight) and position rotation
    (table cos_sin [positions, rot_dim] f32, see rope_table; none without a
    table) of queries q [T, Hq, d] and keys k [T, Hk, d], fp16 or bf16, in one
    pass.  Returns (q_out, k_out), allocated when not given; they may be q and
    k themselves.  Rows of tokens at negative positions are left as they were,
    with or without a rotation."""
    t, hq, d = shape = q.shape
    dt = q.dtype
    qs = _check_tokens(q, "q", dt, shape)
    if q_out is None:
        q_out = _empty(q, shape, stream)
        qos = hq * d
    else:
        qos = _check_tokens(q_out, "q_out", dt, shape)
    hk = ks = kos = 0
    kp = kop = qwp = kwp = None
    if k is not None:
        hk = k.shape[1]
        kshape = (t, hk, d)
        ks = _check_tokens(k, "k", dt, kshape)
        if k_out is None:
            k_out = _empty(q, kshape, stream)
            kos = hk * d
        else:
            kos = _check_tokens(k_out, "k_out", dt, kshape)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    if q_weight is not None:
        _check(q_weight, "q_weight", torch.float32, (d,))
        qwp = q_weight.data_ptr()
    if k_weight is not None:
        _check(k_weight, "k_weight", torch.float32, (d,))
        kwp = k_weight.data_ptr()
    pos, rope = _rope(positions, cos_sin, interleaved, eps, t)
    dev = _one_device((q, k, positions, cos_sin, q_weight, k_weight, q_out, k_out))
    _call("kvq_qk_norm_rope", dev, stream,
          (q.data_ptr(), kp, DTYPES[dt], t, hq, hk, d, qs, ks, pos, qwp, kwp,
           ctypes.addressof(rope), q_out.data_ptr(), kop, qos, kos))
    return q_out, k_out


def kvq_paged_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: PagedCache, *,
                     positions: torch.Tensor | None = None, cos_sin: torch.Tensor | None = None,
                     interleaved: bool = False, k_weight: torch.Tensor | None = None,
                     eps: float = 1e-6, k_hat: torch.Tensor | None = None,
                     v_hat: torch.Tensor | None = None, stream=None) -> None:
    """Writes the new tokens' k, v [T, H, d] (fp16 or bf16) as rows `slots`
    [T] i64 (page * page_size + row in the page; negative: padding) of the
    cache, k after its norm and position rotation (as in kvq_qk_norm_rope).
    k_hat, v_hat [T, H, d], when given, receive the values the new rows stand
    for."""
    dt = k.dtype
    t = k.shape[0]
    shape = (t, cache.n_kv_heads, cache.d)
    ks = _check_tokens(k, "k", dt, shape)
    vs = _check_tokens(v, "v", dt, shape)
    _check(slots, "slots", torch.int64, (t,))
    kw = kh = vh = None
    if k_weight is not None:
        _check(k_weight, "k_weight", torch.float32, (cache.d,))
        kw = k_weight.data_ptr()
    if k_hat is not None:
        _check(k_hat, "k_hat", dt, shape)
        kh = k_hat.data_ptr()
    if v_hat is not None:
        _check(v_hat, "v_hat", dt, shape)
        vh = v_hat.data_ptr()
    pos, rope = _rope(positions, cos_sin, interleaved, eps, t)
    dev = _one_device((cache.signs, k, v, slots, positions, cos_sin, k_weight, k_hat, v_hat))
    _call("kvq_paged_append", dev, stream,
          (k.data_ptr(), v.data_ptr(), DTYPES[dt], t, ks, vs, slots.data_ptr(), pos, kw,
           ctypes.addressof(rope), cache.ref, kh, vh))


def kvq_paged_attend(q: torch.Tensor, cache: PagedCache, cu_q: torch.Tensor,
                     kv_len: torch.Tensor, page_table: torch.Tensor, *, max_q_len: int,
                     window: int = 0, sm_scale: float | None = None,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Causal attention of new tokens q [T, H * n_q, d] (fp16 or bf16) over
    the paged cache, which holds their keys and values already.  cu_q [S+1]
    i32: first token of each sequence; kv_len [S] i32: its cached rows;
    page_table [S, max_pages] i32; max_q_len: the most new tokens of a sequence
    (chooses the kernel); window: attend at most that many rows (0: all);
    sm_scale defaults to 1/sqrt(d).  Returns out [T, H * n_q, d]; rows of no
    sequence are left as they were.  The workspace (uint8) is allocated when
    not given; one that is given must not be used by another call before this
    one has finished on the device."""
    t, h, d = shape = q.shape
    dt = q.dtype
    n_q = h // cache.n_kv_heads
    if d != cache.d or n_q * cache.n_kv_heads != h or h == 0:
        raise ValueError(f"q [{t}, {h}, {d}] does not fit a cache of {cache.n_kv_heads} KV heads "
                         f"and d = {cache.d}")
    qs = _check_tokens(q, "q", dt, shape)
    if out is None:
        out = _empty(q, shape, stream)
        outs = h * d
    else:
        outs = _check_tokens(out, "out", dt, shape)
    max_q_len, window = _int32(max_q_len), _int32(window)
    n_seqs = kv_len.shape[0]
    max_pages = page_table.shape[-1]
    _check(kv_len, "kv_len", torch.int32, (n_seqs,))
    _check(cu_q, "cu_q", torch.int32, (n_seqs + 1,))
    _check(page_table, "page_table", torch.int32, (n_seqs, max_pages))
    if workspace is None:
        need = lib.kvq_paged_attend_workspace(t, cache.n_kv_heads, n_q, d, max_q_len)
        if need < 0:
            raise KVQError("kvq_paged_attend_workspace", -need)
        workspace = _empty(cache.k_packed, (need,), stream)
    else:
        need = workspace.numel()
        _check(workspace, "workspace", torch.uint8, (need,))
    dev = _one_device((cache.signs, q, out, cu_q, kv_len, page_table, workspace))
    _call("kvq_paged_attend", dev, stream,
          (q.data_ptr(), DTYPES[dt], t, qs, cache.ref, cu_q.data_ptr(), kv_len.data_ptr(),
           page_table.data_ptr(), n_seqs, max_pages, n_q, max_q_len, window,
           d ** -0.5 if sm_scale is None else float(sm_scale), out.data_ptr(), outs,
           workspace.data_ptr(), need))
    return out


def kvq_device_status(clear: bool = True) -> int:
    """Synchronize the device and return the kernels' device status code."""
    return int(lib.kvq_device_status(1 if clear else 0))


def kvq_version() -> int:
    return int(lib.kvq_version())
