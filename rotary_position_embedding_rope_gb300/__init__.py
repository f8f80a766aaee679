"""Python binding of librope: rotary position embedding on GB300 (sm_103a).

The functions named like the C ABI (``rope_tables_build``, ``rope_apply_qk``,
``rope_apply_q``, ``rope_check_errors``, ``rope_status_string``,
``rope_qk_kernel_variant``) take the same arguments as ``include/rope.h``,
with torch tensors (or raw integer addresses) in place of pointers and a
torch stream (or raw handle, or None for torch's current stream) in place of
``void* stream``.  They only marshal arguments: every step runs in the CUDA
library, and a missing library is an error, never a fallback.

``build_tables``, ``apply_qk``, ``apply_q`` and ``rotate_qk`` are conveniences
that read the sizes from tensor shapes and allocate tables and outputs with
torch; ``PreparedApply`` checks a rotation's arguments once for calls
repeated on tensors of one shape.  ``autograd.rotary_qk`` wraps the out-of-place call in a
``torch.autograd.Function`` (backward = rotation by the negated angle).
``build_tables_ex`` builds the table of a frequency mode ('lang', 'pixel',
'constant') at given positions, optionally XPOS-scaled; ``apply_qk_xpos``
rotates Q and K with their own XPOS tables.  ``attention`` calls
``rope_attention_fwd`` (``rope_attention_fwd_masked`` with an ``attn_mask``):
attention with the rotation fused into the Q/K tile loads (or, with a key
workspace, keys rotated once beforehand).
``cache_append`` writes new keys (rotated) and values into a paged cache,
``attention_packed`` attends over packed prompts of different lengths and
``attention_shared_prefix`` runs one new token per sequence over a prefix all
sequences share and each one's own pages; ``attention_paged`` attends from each sequence's
new tokens, one or a chunk of a prompt, to its keys in the cache.
``norm_rotate_qk`` normalises query and key heads (RMS norm) and rotates them in the same
pass (``norm_rotate_qk_backward`` and ``autograd.norm_rotary_qk`` give the gradients),
``norm_cache_append`` does it on the way into the paged cache.
``build_tables_scaled`` builds the tables of contexts longer than those trained on.
``host.HostRotator`` and ``host.HostAttention`` run the rotation and the
attention on tensors that live in pinned host memory, overlapping the copies
with the calls.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import _build

__all__ = [
    "RopeError", "ROPE_OK", "ROPE_ERR_INVALID_ARG", "ROPE_ERR_UNSUPPORTED", "ROPE_ERR_CUDA",
    "ROPE_ERR_POS_OUT_OF_RANGE", "ROPE_ERR_KERNEL_TIMEOUT", "ROPE_ERR_BAD_INDEX",
    "VARIANT_ELEMENTWISE", "VARIANT_VECTOR",
    "ROPE_SPLIT_HALF", "ROPE_INTERLEAVED", "ROPE_F32", "ROPE_BF16", "ROPE_F16", "ROPE_FREQ_LANG",
    "ROPE_FREQ_PIXEL", "ROPE_FREQ_CONSTANT", "ROPE_MASK_NONE", "ROPE_MASK_KEYS",
    "ROPE_MASK_QUERY_KEYS", "ROPE_SCALE_LINEAR", "ROPE_SCALE_NTK", "ROPE_SCALE_SMOOTH",
    "ROPE_SCALE_YARN", "library_path", "load_library",
    # the C ABI, same names
    "rope_tables_build", "rope_tables_build_ex", "rope_apply_qk", "rope_apply_q",
    "rope_apply_qk_out", "rope_attention_fwd", "rope_attention_fwd_masked",
    "rope_attention_fwd_noalloc", "rope_check_errors", "rope_probe_wait_expiry",
    "rope_status_string", "rope_qk_kernel_variant", "rope_force_kernel_variant",
    "rope_tune_rotation_launch", "rope_cache_append",
    "rope_attention_packed_fwd", "rope_attention_packed_workspace",
    "rope_attention_decode_fwd", "rope_attention_decode_workspace",
    "rope_tables_build_scaled", "rope_norm_qk_fwd", "rope_norm_qk_bwd", "rope_norm_qk_workspace",
    "rope_norm_cache_append", "rope_attention_paged_fwd", "rope_attention_paged_workspace",
    # conveniences
    "build_tables", "build_tables_ex", "apply_qk", "apply_q", "apply_qk_xpos", "rotate_qk",
    "attention", "attention_workspace", "PreparedApply", "cache_append",
    "attention_packed", "attention_shared_prefix", "build_tables_scaled", "norm_rotate_qk",
    "norm_rotate_qk_backward", "norm_cache_append", "attention_paged",
]

(ROPE_OK, ROPE_ERR_INVALID_ARG, ROPE_ERR_UNSUPPORTED, ROPE_ERR_CUDA, ROPE_ERR_POS_OUT_OF_RANGE,
 ROPE_ERR_KERNEL_TIMEOUT, ROPE_ERR_BAD_INDEX) = range(7)
VARIANT_ELEMENTWISE, VARIANT_VECTOR = 2, 3
ROPE_SPLIT_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_F32, ROPE_BF16, ROPE_F16 = 0, 1, 2
ROPE_FREQ_LANG, ROPE_FREQ_PIXEL, ROPE_FREQ_CONSTANT = 0, 1, 2
ROPE_MASK_NONE, ROPE_MASK_KEYS, ROPE_MASK_QUERY_KEYS = 0, 1, 2
ROPE_SCALE_LINEAR, ROPE_SCALE_NTK, ROPE_SCALE_SMOOTH, ROPE_SCALE_YARN = range(4)
_FREQ_CODE = {"lang": ROPE_FREQ_LANG, "pixel": ROPE_FREQ_PIXEL, "constant": ROPE_FREQ_CONSTANT}
_SCALE_CODE = {"linear": ROPE_SCALE_LINEAR, "ntk": ROPE_SCALE_NTK, "smooth": ROPE_SCALE_SMOOTH, "yarn": ROPE_SCALE_YARN}
_DTYPE_CODE = {torch.float32: ROPE_F32, torch.bfloat16: ROPE_BF16, torch.float16: ROPE_F16}
_LAYOUT_CODE = {"split_half": ROPE_SPLIT_HALF, "interleaved": ROPE_INTERLEAVED}


class RopeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, rope_status_string(status)))


_lib = None


def library_path() -> str:
    """lib/librope.so, or the library ROPE_LIBRARY names (a build of the same
    sources with other compile-time settings, made with
    ``_build.build(extra_flags=[...], output=...)``, for timing variants)."""
    return os.environ.get("ROPE_LIBRARY") or _build.LIBRARY


def load_library() -> ctypes.CDLL:
    """Load lib/librope.so (built by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path) and os.environ.get("ROPE_LIBRARY"):
        raise RuntimeError("ROPE_LIBRARY names %s, which does not exist" % path)
    if not os.path.exists(path):
        raise RuntimeError(
            "librope.so is not built (%s); run `python -c \"import __graft_entry__ as g; "
            "g.build()\"` first" % path)
    lib = ctypes.CDLL(path)
    c = ctypes
    P = c.c_void_p
    lib.rope_tables_build.argtypes = [c.c_double, c.c_int32, c.c_int64, c.c_double, P, P, P]
    lib.rope_tables_build.restype = c.c_int
    lib.rope_tables_build_ex.argtypes = [c.c_int32, c.c_double, c.c_double, c.c_int32, c.c_int64,
                                         c.c_double, c.c_double, c.c_int32, c.c_double, c.c_double,
                                         c.c_double, P, P, P]
    lib.rope_tables_build_ex.restype = c.c_int
    lib.rope_apply_qk.argtypes = [P, P, P, P, P, c.c_int64, c.c_int32, c.c_int32, c.c_int64,
                                  c.c_int32, c.c_int32, c.c_int32, c.c_int32, c.c_int32,
                                  c.c_int32, c.c_int64, P]
    lib.rope_apply_qk.restype = c.c_int
    lib.rope_apply_q.argtypes = [P, P, P, P, c.c_int64, c.c_int32, c.c_int64, c.c_int32,
                                 c.c_int32, c.c_int32, c.c_int32, c.c_int32, c.c_int32,
                                 c.c_int64, P]
    lib.rope_apply_q.restype = c.c_int
    lib.rope_check_errors.argtypes = [P]
    lib.rope_check_errors.restype = c.c_int
    lib.rope_probe_wait_expiry.argtypes = [c.c_int64, P]
    lib.rope_probe_wait_expiry.restype = c.c_int
    lib.rope_status_string.argtypes = [c.c_int]
    lib.rope_status_string.restype = c.c_char_p
    lib.rope_qk_kernel_variant.argtypes = [P, P, P, P, P, c.c_int64, c.c_int32, c.c_int32,
                                           c.c_int64, c.c_int32, c.c_int32, c.c_int32,
                                           c.c_int32, c.c_int32, c.c_int32, c.c_int64]
    lib.rope_qk_kernel_variant.restype = c.c_int32
    lib.rope_apply_qk_out.argtypes = [P, P, P, P, P, P, P, c.c_int64, c.c_int64, c.c_int32,
                                      c.c_int32, c.c_int64, c.c_int32, c.c_int32, c.c_int32,
                                      c.c_int32, c.c_int32, c.c_int32, c.c_int64, P]
    lib.rope_apply_qk_out.restype = c.c_int
    lib.rope_attention_fwd.argtypes = [P, P, P, P, P, P, P, P, c.c_int64, c.c_int32, c.c_int32,
                                       c.c_int64, c.c_int64, c.c_int32, c.c_int32, c.c_int32,
                                       c.c_int32, c.c_float, c.c_int32, c.c_int64, P,
                                       c.c_int64, P]
    lib.rope_attention_fwd.restype = c.c_int
    lib.rope_attention_fwd_masked.argtypes = [P, P, P, P, P, P, P, P, c.c_int64, c.c_int32,
                                              c.c_int32, c.c_int64, c.c_int64, c.c_int32,
                                              c.c_int32, c.c_int32, c.c_int32, c.c_float,
                                              c.c_int32, c.c_int64, P, c.c_int32, P, c.c_int64, P]
    lib.rope_attention_fwd_masked.restype = c.c_int
    lib.rope_attention_fwd_noalloc.argtypes = [P, P, P, P, P, P, P, P, c.c_int64, c.c_int32,
                                               c.c_int32, c.c_int64, c.c_int64, c.c_int32,
                                               c.c_int32, c.c_int32, c.c_int32, c.c_float,
                                               c.c_int32, c.c_int64, P]
    lib.rope_attention_fwd_noalloc.restype = c.c_int
    lib.rope_force_kernel_variant.argtypes = [c.c_int32]
    lib.rope_force_kernel_variant.restype = c.c_int
    lib.rope_tune_rotation_launch.argtypes = [c.c_int32, c.c_int32, c.c_int32]
    lib.rope_tune_rotation_launch.restype = c.c_int
    lib.rope_cache_append.argtypes = [P] * 10 + [c.c_int64] * 5 + [c.c_int32] * 5 + \
        [c.c_int64, c.c_int64, c.c_int32, c.c_int64, P]
    lib.rope_cache_append.restype = c.c_int
    lib.rope_attention_packed_fwd.argtypes = [P] * 10 + [c.c_int64] * 6 + [c.c_int32] * 6 + \
        [c.c_float, c.c_int32, c.c_int64, P, c.c_int64, P]
    lib.rope_attention_packed_fwd.restype = c.c_int
    lib.rope_attention_packed_workspace.argtypes = [c.c_int64] * 3 + [c.c_int32] * 3
    lib.rope_attention_packed_workspace.restype = c.c_int64
    lib.rope_attention_decode_fwd.argtypes = [P] * 7 + [c.c_int64, P, P, P, c.c_int64, c.c_int64] + \
        [c.c_int32] * 5 + [c.c_float, c.c_int32, c.c_int64, c.c_int64, c.c_int32, c.c_int64, P, c.c_int64, P]
    lib.rope_attention_decode_fwd.restype = c.c_int
    lib.rope_attention_decode_workspace.argtypes = [c.c_int64] + [c.c_int32] * 4 + [c.c_int64] * 2
    lib.rope_attention_decode_workspace.restype = c.c_int64
    lib.rope_tables_build_scaled.argtypes = [c.c_int32, c.c_double, c.c_int32, c.c_int64, c.c_int64, c.c_double,
                                             c.c_int64, c.c_double, c.c_double, c.c_double, P, P, P]
    lib.rope_tables_build_scaled.restype = c.c_int
    lib.rope_norm_qk_fwd.argtypes = [P] * 9 + [c.c_int64, c.c_int64, c.c_int32, c.c_int32, c.c_int64, c.c_int32, P, P,
                                               c.c_int32, c.c_int32, c.c_int32, c.c_float, c.c_int32, c.c_int32,
                                               c.c_int64, P]
    lib.rope_norm_qk_fwd.restype = c.c_int
    lib.rope_norm_qk_bwd.argtypes = [P] * 13 + [c.c_int64, c.c_int64, c.c_int32, c.c_int32, c.c_int64, c.c_int32, P, P,
                                                c.c_int32, c.c_int32, c.c_int32, c.c_float, c.c_int32, c.c_int32,
                                                c.c_int64, P, c.c_int64, P]
    lib.rope_norm_qk_bwd.restype = c.c_int
    lib.rope_norm_qk_workspace.argtypes = [c.c_int32]
    lib.rope_norm_qk_workspace.restype = c.c_int64
    lib.rope_norm_cache_append.argtypes = [P] * 14 + [c.c_int64] * 6 + [c.c_int32] * 5 + \
        [c.c_float, c.c_int32, c.c_int64, c.c_int64, c.c_int32, c.c_int32, c.c_int64, P]
    lib.rope_norm_cache_append.restype = c.c_int
    lib.rope_attention_paged_fwd.argtypes = [P] * 10 + [c.c_int64] * 3 + [c.c_int32] * 6 + \
        [c.c_float, c.c_int32, c.c_int64, c.c_int64, c.c_int32, c.c_int64, P, c.c_int64, P]
    lib.rope_attention_paged_fwd.restype = c.c_int
    lib.rope_attention_paged_workspace.argtypes = [c.c_int64] * 2 + [c.c_int32] * 4 + [c.c_int64]
    lib.rope_attention_paged_workspace.restype = c.c_int64
    _lib = lib
    return lib


# --------------------------------------------------------------------------
# marshalling
# --------------------------------------------------------------------------
def _addr(x, name: str, device_required: bool = True):
    """Device address of a tensor (checked contiguous, on CUDA) or a raw int."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if isinstance(x, torch.Tensor):
        if device_required and not x.is_cuda:
            raise ValueError("%s must be a CUDA tensor" % name)
        if not x.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
        return x.data_ptr() if x.numel() > 0 else None
    raise TypeError("%s: expected a tensor, an int address or None" % name)


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != ROPE_OK:
        raise RopeError(status, where)


# --------------------------------------------------------------------------
# functions of the C ABI, same names and arguments
# --------------------------------------------------------------------------
def rope_tables_build(theta, rotary_dim, max_pos, interpolate_factor, cos_out, sin_out,
                      stream=None):
    lib = load_library()
    for t, n in ((cos_out, "cos_out"), (sin_out, "sin_out")):
        if isinstance(t, torch.Tensor) and (t.dtype != torch.float32 or
                                            t.numel() < max_pos * (rotary_dim // 2)):
            raise ValueError("%s must be float32 with at least max_pos*rotary_dim/2 elements" % n)
    st = lib.rope_tables_build(float(theta), int(rotary_dim), int(max_pos),
                               float(interpolate_factor), _addr(cos_out, "cos_out"),
                               _addr(sin_out, "sin_out"), _stream(stream))
    _check(st, "rope_tables_build")


def rope_tables_build_ex(freq_mode, theta, max_freq, rotary_dim, rows, pos_offset, pos_divisor,
                         xpos_sign, xpos_scale_base, xpos_gamma, xpos_center, cos_out, sin_out,
                         stream=None):
    lib = load_library()
    for t, n in ((cos_out, "cos_out"), (sin_out, "sin_out")):
        if isinstance(t, torch.Tensor) and (t.dtype != torch.float32 or
                                            t.numel() < rows * (rotary_dim // 2)):
            raise ValueError("%s must be float32 with at least rows*rotary_dim/2 elements" % n)
    st = lib.rope_tables_build_ex(int(freq_mode), float(theta), float(max_freq), int(rotary_dim),
                                  int(rows), float(pos_offset), float(pos_divisor), int(xpos_sign),
                                  float(xpos_scale_base), float(xpos_gamma), float(xpos_center),
                                  _addr(cos_out, "cos_out"), _addr(sin_out, "sin_out"),
                                  _stream(stream))
    _check(st, "rope_tables_build_ex")


def rope_apply_qk(q, k, cos, sin, pos_idx, B, Hq, Hk, S, D, rotary_dim, layout,
                  seq_before_head, backward, dtype, table_rows, stream=None):
    lib = load_library()
    st = lib.rope_apply_qk(_addr(q, "q"), _addr(k, "k"), _addr(cos, "cos"), _addr(sin, "sin"),
                           _addr(pos_idx, "pos_idx"), int(B), int(Hq), int(Hk), int(S), int(D),
                           int(rotary_dim), int(layout), int(seq_before_head), int(backward),
                           int(dtype), int(table_rows), _stream(stream))
    _check(st, "rope_apply_qk")


def rope_apply_qk_out(q, k, q_out, k_out, cos, sin, pos_idx, pos_batch_stride, B, Hq, Hk, S, D,
                      rotary_dim, layout, seq_before_head, backward, dtype, table_rows,
                      stream=None):
    lib = load_library()
    st = lib.rope_apply_qk_out(_addr(q, "q"), _addr(k, "k"), _addr(q_out, "q_out"),
                               _addr(k_out, "k_out"), _addr(cos, "cos"), _addr(sin, "sin"),
                               _addr(pos_idx, "pos_idx"), int(pos_batch_stride), int(B), int(Hq),
                               int(Hk), int(S), int(D), int(rotary_dim), int(layout),
                               int(seq_before_head), int(backward), int(dtype), int(table_rows),
                               _stream(stream))
    _check(st, "rope_apply_qk_out")


def rope_apply_q(x, cos, sin, pos_idx, B, H, S, D, rotary_dim, layout, seq_before_head,
                 backward, dtype, table_rows, stream=None):
    lib = load_library()
    st = lib.rope_apply_q(_addr(x, "x"), _addr(cos, "cos"), _addr(sin, "sin"),
                          _addr(pos_idx, "pos_idx"), int(B), int(H), int(S), int(D),
                          int(rotary_dim), int(layout), int(seq_before_head), int(backward),
                          int(dtype), int(table_rows), _stream(stream))
    _check(st, "rope_apply_q")


def rope_check_errors(stream=None) -> int:
    """Synchronise the stream; returns the status (does not raise)."""
    return load_library().rope_check_errors(_stream(stream))


def rope_probe_wait_expiry(cycles: int, stream=None) -> int:
    """Launch one bounded wait that expires after `cycles` clock cycles and
    sets the timeout bit of the device flag (the next rope_check_errors
    returns ROPE_ERR_KERNEL_TIMEOUT).  Returns the launch status."""
    return load_library().rope_probe_wait_expiry(int(cycles), _stream(stream))


def rope_status_string(status: int) -> str:
    return load_library().rope_status_string(int(status)).decode()


def rope_qk_kernel_variant(q, k, cos, sin, pos_idx, B, Hq, Hk, S, D, rotary_dim, layout,
                           seq_before_head, backward, dtype, table_rows) -> int:
    lib = load_library()
    return lib.rope_qk_kernel_variant(
        _addr(q, "q", False), _addr(k, "k", False), _addr(cos, "cos", False),
        _addr(sin, "sin", False), _addr(pos_idx, "pos_idx", False), int(B), int(Hq), int(Hk),
        int(S), int(D), int(rotary_dim), int(layout), int(seq_before_head), int(backward),
        int(dtype), int(table_rows))


def rope_force_kernel_variant(variant: int):
    _check(load_library().rope_force_kernel_variant(int(variant)), "rope_force_kernel_variant")


def rope_tune_rotation_launch(ctas_per_sm: int = 0, min_units: int = 0, prefetch_next: int = 0):
    """Grid sizing of the vector rotation kernel (0 = defaults); results do
    not depend on it."""
    _check(load_library().rope_tune_rotation_launch(int(ctas_per_sm), int(min_units),
                                                    int(prefetch_next)),
           "rope_tune_rotation_launch")


# --------------------------------------------------------------------------
# conveniences
# --------------------------------------------------------------------------
def _allocated(make, stream, device):
    """What make() allocates, for a call on ``stream``.

    The caching allocator hands a block out again as soon as the host has
    dropped it, to work that runs behind its last use on the same stream: memory
    that a call on another stream writes at once has to be that stream's.  It is
    recorded on the current stream, where the caller uses it next.
    """
    if stream is None:
        return make()
    current = torch.cuda.current_stream(device)
    handle = _stream(stream)
    if handle == current.cuda_stream:
        return make()
    own = torch.cuda.ExternalStream(handle, current.device) if handle else \
        torch.cuda.default_stream(current.device)
    with torch.cuda.stream(own):
        made = make()
    for t in made if isinstance(made, tuple) else (made,):
        t.record_stream(current)
    return made


def build_tables(theta: float, rotary_dim: int, max_pos: int, interpolate_factor: float = 1.0,
                 device=None, stream=None):
    """Allocate and fill fp32 cos/sin tables [max_pos, rotary_dim // 2]."""
    device = torch.device("cuda") if device is None else torch.device(device)
    h = rotary_dim // 2
    cos, sin = _allocated(lambda: tuple(torch.empty((max_pos, h), dtype=torch.float32, device=device)
                                        for _ in range(2)), stream, device)
    rope_tables_build(theta, rotary_dim, max_pos, interpolate_factor, cos, sin, stream)
    return cos, sin


def build_tables_ex(freqs_for: str, rotary_dim: int, rows: int, theta: float = 10000.0,
                    max_freq: float = 10.0, pos_offset: float = 0.0, pos_divisor: float = 1.0,
                    xpos_sign: int = 0, xpos_scale_base: float = 512.0, xpos_gamma: float = 0.4,
                    xpos_center: float = 0.0, device=None, stream=None):
    """Allocate and fill fp32 cos/sin tables [rows, rotary_dim // 2] of the mode
    ``freqs_for`` ('lang', 'pixel' or 'constant'), row m at position
    pos_offset + m / pos_divisor, XPOS-scaled when xpos_sign is +1 (queries) or
    -1 (keys)."""
    device = torch.device("cuda") if device is None else torch.device(device)
    h = rotary_dim // 2
    cos, sin = _allocated(lambda: tuple(torch.empty((rows, h), dtype=torch.float32, device=device)
                                        for _ in range(2)), stream, device)
    rope_tables_build_ex(_FREQ_CODE[freqs_for], theta, max_freq, rotary_dim, rows, pos_offset,
                         pos_divisor, xpos_sign, xpos_scale_base, xpos_gamma, xpos_center, cos,
                         sin, stream)
    return cos, sin


def rope_tables_build_scaled(kind, theta, rotary_dim, rows, pos_offset, factor, original_positions, low_turns,
                             high_turns, value_scale, cos_out, sin_out, stream=None):
    lib = load_library()
    for t, n in ((cos_out, "cos_out"), (sin_out, "sin_out")):
        if isinstance(t, torch.Tensor) and (t.dtype != torch.float32 or
                                            t.numel() < rows * (rotary_dim // 2)):
            raise ValueError("%s must be float32 with at least rows*rotary_dim/2 elements" % n)
    st = lib.rope_tables_build_scaled(int(kind), float(theta), int(rotary_dim), int(rows), int(pos_offset),
                                      float(factor), int(original_positions), float(low_turns),
                                      float(high_turns), float(value_scale), _addr(cos_out, "cos_out"),
                                      _addr(sin_out, "sin_out"), _stream(stream))
    _check(st, "rope_tables_build_scaled")


def build_tables_scaled(kind: str, rotary_dim: int, rows: int, factor: float, original_positions: int = 0,
                        theta: float = 10000.0, pos_offset: int = 0, low_turns: float | None = None,
                        high_turns: float | None = None, value_scale: float | None = None, device=None,
                        stream=None):
    """Allocate and fill fp32 cos/sin tables [rows, rotary_dim // 2] for a context ``factor``
    times the ``original_positions`` a model was trained on; row m stands for position
    pos_offset + m.

    kind: "linear" (positions divided by the factor), "ntk" (a larger base), "smooth"
    (pairs that make fewer than low_turns = 1 turns over the trained context are slowed
    by the factor, those of more than high_turns = 4 kept, a ramp between) or "yarn" (the
    ramp along the pairs, between those of low_turns = 1 and high_turns = 32 turns).
    value_scale: factor of all values, above 0; None: 1, for "yarn" 0.1 ln(factor) + 1.
    """
    if value_scale == 0:                       # (the library's word for "none given")
        raise ValueError("value_scale must be above 0")
    at = -1
    if device is not None:
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("tables are built on a CUDA device, not on %s" % device)
        at = -1 if device.index is None else device.index
    o = (_serving or _native()).build_tables_scaled(
        _SCALE_CODE[kind], theta, rotary_dim, rows, pos_offset, factor, original_positions,
        1.0 if low_turns is None else low_turns,
        (32.0 if kind == "yarn" else 4.0) if high_turns is None else high_turns,
        0.0 if value_scale is None else value_scale, at, stream)
    if type(o) is int:
        raise RopeError(o, "rope_tables_build_scaled")
    return o


def _shape4(x: torch.Tensor, seq_before_head: bool):
    if x.dim() != 4:
        raise ValueError("expected a 4-D tensor, got shape %s" % (tuple(x.shape),))
    if seq_before_head:
        B, S, H, D = x.shape
    else:
        B, H, S, D = x.shape
    return B, H, S, D


def apply_qk(q: torch.Tensor, k: torch.Tensor | None, cos: torch.Tensor, sin: torch.Tensor,
             pos_idx: torch.Tensor | None = None, rotary_dim: int | None = None,
             layout: str = "split_half", seq_before_head: bool = False, backward: bool = False,
             stream=None):
    """Rotate q and k in place; sizes are read from the tensors.

    q: [B, Hq, S, D] (or [B, S, Hq, D] with seq_before_head); k likewise with
    Hk heads, or None.  cos/sin: float32 [rows, rotary_dim // 2].
    pos_idx: int32 [S] or None.  rotary_dim defaults to 2 * cos.shape[1].
    """
    B, Hq, S, D = _shape4(q, seq_before_head)
    Hk = 0
    if k is not None:
        Bk, Hk, Sk, Dk = _shape4(k, seq_before_head)
        if (Bk, Sk, Dk) != (B, S, D) or k.dtype != q.dtype:
            raise ValueError("q and k must agree in batch, sequence, head_dim and dtype")
    if q.dtype not in _DTYPE_CODE:
        raise TypeError("unsupported dtype %s" % q.dtype)
    if cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.shape != sin.shape:
        raise ValueError("cos and sin must be float32 tables of the same shape")
    rd = 2 * cos.shape[1] if rotary_dim is None else rotary_dim
    if cos.shape[1] != rd // 2:
        raise ValueError("table width %d does not match rotary_dim %d" % (cos.shape[1], rd))
    if pos_idx is not None and (pos_idx.dtype != torch.int32 or pos_idx.numel() != S):
        raise ValueError("pos_idx must be int32 with S elements")
    rope_apply_qk(q, k, cos, sin, pos_idx, B, Hq, Hk, S, D, rd, _LAYOUT_CODE[layout],
                  int(seq_before_head), int(backward), _DTYPE_CODE[q.dtype], cos.shape[0],
                  stream)
    return q, k


class PreparedApply:
    """rope_apply_qk with every argument but q and k checked and converted
    once, for calls repeated on tensors of one shape (a model layer, a decode
    loop): each call marshals two pointers and the fixed rest.

        f = PreparedApply(q, k, cos, sin, stream=s)   # shapes, tables, layout
        f(q, k)                  # forward, in place
        f(dq, dk, backward=True)

    q and k of later calls must have the shapes and dtype of the ones given
    here (their element counts are checked; raw integer addresses are passed
    as they are).  The stream is fixed here (None: torch's current stream at
    this point).  Only marshalling: the library does the work."""

    def __init__(self, q, k, cos, sin, pos_idx=None, rotary_dim=None, layout="split_half",
                 seq_before_head=False, stream=None):
        B, Hq, S, D = _shape4(q, seq_before_head)
        Hk = 0
        if k is not None:
            Bk, Hk, Sk, Dk = _shape4(k, seq_before_head)
            if (Bk, Sk, Dk) != (B, S, D) or k.dtype != q.dtype:
                raise ValueError("q and k must agree in batch, sequence, head_dim and dtype")
        if q.dtype not in _DTYPE_CODE:
            raise TypeError("unsupported dtype %s" % q.dtype)
        if cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.shape != sin.shape:
            raise ValueError("cos and sin must be float32 tables of the same shape")
        rd = 2 * cos.shape[1] if rotary_dim is None else rotary_dim
        if cos.shape[1] != rd // 2:
            raise ValueError("table width %d does not match rotary_dim %d" % (cos.shape[1], rd))
        if pos_idx is not None and (pos_idx.dtype != torch.int32 or pos_idx.numel() != S):
            raise ValueError("pos_idx must be int32 with S elements")
        c = ctypes
        self._fn = load_library().rope_apply_qk
        self._keep = (cos, sin, pos_idx)
        self._nq, self._nk = q.numel(), 0 if k is None else k.numel()
        head = [c.c_void_p(_addr(cos, "cos")), c.c_void_p(_addr(sin, "sin")),
                c.c_void_p(_addr(pos_idx, "pos_idx")), c.c_int64(B), c.c_int32(Hq),
                c.c_int32(Hk), c.c_int64(S), c.c_int32(D), c.c_int32(rd),
                c.c_int32(_LAYOUT_CODE[layout]), c.c_int32(int(seq_before_head))]
        tail = [c.c_int32(_DTYPE_CODE[q.dtype]), c.c_int64(cos.shape[0]),
                c.c_void_p(_stream(stream))]
        self._fwd = tuple(head + [c.c_int32(0)] + tail)
        self._bwd = tuple(head + [c.c_int32(1)] + tail)

    def __call__(self, q, k=None, backward: bool = False):
        if isinstance(q, int):
            qp = q
        else:
            if q.numel() != self._nq:
                raise ValueError("q does not have the prepared shape")
            qp = q.data_ptr()
        if k is None or isinstance(k, int):
            kp = k
        else:
            if k.numel() != self._nk:
                raise ValueError("k does not have the prepared shape")
            kp = k.data_ptr()
        st = self._fn(qp, kp, *(self._bwd if backward else self._fwd))
        if st != ROPE_OK:
            raise RopeError(st, "rope_apply_qk")


def apply_q(x: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor,
            pos_idx: torch.Tensor | None = None, rotary_dim: int | None = None,
            layout: str = "split_half", seq_before_head: bool = False, backward: bool = False,
            stream=None):
    """Rotate one tensor in place through the query-only entry point."""
    B, H, S, D = _shape4(x, seq_before_head)
    if x.dtype not in _DTYPE_CODE:
        raise TypeError("unsupported dtype %s" % x.dtype)
    if cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.shape != sin.shape:
        raise ValueError("cos and sin must be float32 tables of the same shape")
    rd = 2 * cos.shape[1] if rotary_dim is None else rotary_dim
    if cos.shape[1] != rd // 2:
        raise ValueError("table width %d does not match rotary_dim %d" % (cos.shape[1], rd))
    if pos_idx is not None and (pos_idx.dtype != torch.int32 or pos_idx.numel() != S):
        raise ValueError("pos_idx must be int32 with S elements")
    rope_apply_q(x, cos, sin, pos_idx, B, H, S, D, rd, _LAYOUT_CODE[layout],
                 int(seq_before_head), int(backward), _DTYPE_CODE[x.dtype], cos.shape[0], stream)
    return x


def apply_qk_xpos(q: torch.Tensor, k: torch.Tensor, tables_q, tables_k,
                  pos_idx: torch.Tensor | None = None, rotary_dim: int | None = None,
                  layout: str = "split_half", seq_before_head: bool = False,
                  backward: bool = False, stream=None):
    """XPOS: rotate Q with its table (xpos_sign +1) and K with its table
    (xpos_sign -1), in place: one launch per tensor."""
    apply_q(q, tables_q[0], tables_q[1], pos_idx, rotary_dim, layout, seq_before_head, backward,
            stream)
    apply_q(k, tables_k[0], tables_k[1], pos_idx, rotary_dim, layout, seq_before_head, backward,
            stream)
    return q, k


def _positions(pos_idx, B: int, S: int):
    """(tensor, batch stride) for an int32 [S] or [B, S'] (S' >= S) position tensor."""
    if pos_idx is None:
        return None, 0
    if pos_idx.dtype != torch.int32:
        raise ValueError("pos_idx must be int32")
    if pos_idx.dim() == 1:
        if pos_idx.numel() != S:
            raise ValueError("pos_idx [S] must have S elements")
        return pos_idx, 0
    if pos_idx.dim() == 2 and pos_idx.shape[0] == B and pos_idx.shape[1] >= S:
        return pos_idx, pos_idx.shape[1]
    raise ValueError("pos_idx must be [S] or [B, >=S]")


def rotate_qk(q: torch.Tensor, k: torch.Tensor | None, cos: torch.Tensor, sin: torch.Tensor,
              pos_idx: torch.Tensor | None = None, rotary_dim: int | None = None,
              layout: str = "split_half", seq_before_head: bool = False, backward: bool = False,
              q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Out-of-place rotation: returns (q_out, k_out), allocated when not given.

    pos_idx: int32 [S] (shared by all sequences) or [B, S] (one row per
    sequence).  Passing q_out=q (k_out=k) rotates that tensor in place.
    """
    B, Hq, S, D = _shape4(q, seq_before_head)
    Hk = 0
    if k is not None:
        Bk, Hk, Sk, Dk = _shape4(k, seq_before_head)
        if (Bk, Sk, Dk) != (B, S, D) or k.dtype != q.dtype:
            raise ValueError("q and k must agree in batch, sequence, head_dim and dtype")
    if q.dtype not in _DTYPE_CODE:
        raise TypeError("unsupported dtype %s" % q.dtype)
    if cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.shape != sin.shape:
        raise ValueError("cos and sin must be float32 tables of the same shape")
    rd = 2 * cos.shape[1] if rotary_dim is None else rotary_dim
    if cos.shape[1] != rd // 2:
        raise ValueError("table width %d does not match rotary_dim %d" % (cos.shape[1], rd))
    pos, stride = _positions(pos_idx, B, S)
    q_out = _allocated(lambda: torch.empty_like(q), stream, q.device) if q_out is None else q_out
    if k is not None and k_out is None:
        k_out = _allocated(lambda: torch.empty_like(k), stream, k.device)
    for o, x, n in ((q_out, q, "q_out"), (k_out, k, "k_out")):
        if x is not None and (o.shape != x.shape or o.dtype != x.dtype):
            raise ValueError("%s must match its input's shape and dtype" % n)
    rope_apply_qk_out(q, k, q_out, k_out if k is not None else None, cos, sin, pos, stride, B, Hq,
                      Hk, S, D, rd, _LAYOUT_CODE[layout], int(seq_before_head), int(backward),
                      _DTYPE_CODE[q.dtype], cos.shape[0], stream)
    return q_out, k_out


def rope_attention_fwd(q, k, v, o, cos, sin, pos_q, pos_k, B, Hq, Hk, Sq, Sk, D, rotary_dim,
                       layout, causal, softmax_scale, dtype, table_rows, k_workspace=None,
                       workspace_bytes=0, stream=None):
    lib = load_library()
    st = lib.rope_attention_fwd(_addr(q, "q"), _addr(k, "k"), _addr(v, "v"), _addr(o, "o"),
                                _addr(cos, "cos"), _addr(sin, "sin"), _addr(pos_q, "pos_q"),
                                _addr(pos_k, "pos_k"), int(B), int(Hq), int(Hk), int(Sq), int(Sk),
                                int(D), int(rotary_dim), int(layout), int(causal),
                                float(softmax_scale), int(dtype), int(table_rows),
                                _addr(k_workspace, "k_workspace"), int(workspace_bytes),
                                _stream(stream))
    _check(st, "rope_attention_fwd")


def rope_attention_fwd_masked(q, k, v, o, cos, sin, pos_q, pos_k, B, Hq, Hk, Sq, Sk, D, rotary_dim,
                              layout, causal, softmax_scale, dtype, table_rows, attn_mask,
                              mask_kind, k_workspace=None, workspace_bytes=0, stream=None):
    lib = load_library()
    st = lib.rope_attention_fwd_masked(_addr(q, "q"), _addr(k, "k"), _addr(v, "v"), _addr(o, "o"),
                                       _addr(cos, "cos"), _addr(sin, "sin"), _addr(pos_q, "pos_q"),
                                       _addr(pos_k, "pos_k"), int(B), int(Hq), int(Hk), int(Sq),
                                       int(Sk), int(D), int(rotary_dim), int(layout), int(causal),
                                       float(softmax_scale), int(dtype), int(table_rows),
                                       _addr(attn_mask, "attn_mask"), int(mask_kind),
                                       _addr(k_workspace, "k_workspace"), int(workspace_bytes),
                                       _stream(stream))
    _check(st, "rope_attention_fwd_masked")


def rope_attention_fwd_noalloc(q, k, v, o, cos, sin, pos_q, pos_k, B, Hq, Hk, Sq, Sk, D,
                               rotary_dim, layout, causal, softmax_scale, dtype, table_rows,
                               stream=None):
    """rope_attention_fwd with the rot(K) buffer taken from the library's own
    32 MiB device array: for callers that cannot allocate device memory when
    they call (their memory is all reserved by their own pool, or they may
    only use buffers their host framework gives them).  Allocates nothing."""
    lib = load_library()
    st = lib.rope_attention_fwd_noalloc(_addr(q, "q"), _addr(k, "k"), _addr(v, "v"),
                                        _addr(o, "o"), _addr(cos, "cos"), _addr(sin, "sin"),
                                        _addr(pos_q, "pos_q"), _addr(pos_k, "pos_k"), int(B),
                                        int(Hq), int(Hk), int(Sq), int(Sk), int(D),
                                        int(rotary_dim), int(layout), int(causal),
                                        float(softmax_scale), int(dtype), int(table_rows),
                                        _stream(stream))
    _check(st, "rope_attention_fwd_noalloc")


def attention_workspace(k: torch.Tensor, attn_mask: torch.Tensor | None = None) -> torch.Tensor:
    """A key workspace for rope_attention_fwd(_masked) on keys like k: rot(K)
    and, for a [B, Sk] attn_mask, the per-batch key-tile counts after it (with
    them the kernels skip the key tiles the mask hides entirely), then the
    per-batch prefix lengths (an entry whose mask shows exactly its first L
    keys, as padding does, is then computed without reading the mask)."""
    kb = k.numel() * k.element_size()
    n = kb
    if attn_mask is not None and attn_mask.dim() == 2:
        n = (kb + 15) // 16 * 16 + 8 * k.shape[0]
    return torch.empty(n, dtype=torch.uint8, device=k.device)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cos: torch.Tensor,
              sin: torch.Tensor, pos_q: torch.Tensor | None = None,
              pos_k: torch.Tensor | None = None, rotary_dim: int | None = None,
              layout: str = "split_half", causal: bool = False, scale: float | None = None,
              out: torch.Tensor | None = None, k_workspace="auto",
              attn_mask: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """softmax(scale * rot(q) rot(k)^T + mask) v with q [B,Hq,Sq,D], k/v [B,Hk,Sk,D].

    k_workspace: "auto" allocates a buffer (attention_workspace) that receives
    rot(K) (the keys are rotated once, then read rotated by the attention
    kernel); a tensor of at least k's size is used as that buffer; None
    rotates the key tiles inside the attention kernel instead (nothing extra
    is written).  The result is the same bit for bit.
    attn_mask: None, or a bool (or uint8) CUDA tensor [B, Sk] (one entry per
    key) or [B, Sq, Sk] (one per query and key); False hides the key from the
    query, together with the causal mask.
    """
    B, Hq, Sq, D = q.shape
    _, Hk, Sk, _ = k.shape
    if v.shape != k.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("k and v must have the same shape, and q, k, v the same dtype")
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("attention takes bf16 or fp16 q, k, v (the tensor-core products are 16-bit); "
                        "got %s: convert the inputs first (e.g. q.bfloat16()), a rounding that is "
                        "the caller's choice" % q.dtype)
    rd = 2 * cos.shape[1] if rotary_dim is None else rotary_dim
    o = _allocated(lambda: torch.empty_like(q), stream, q.device) if out is None else out
    if isinstance(k_workspace, str):
        if k_workspace != "auto":
            raise ValueError("k_workspace must be 'auto', None or a tensor")
        k_workspace = _allocated(lambda: attention_workspace(k, attn_mask), stream, k.device)
    ws_bytes = 0 if k_workspace is None else k_workspace.numel() * k_workspace.element_size()
    args = (q, k, v, o, cos, sin, pos_q, pos_k, B, Hq, Hk, Sq, Sk, D, rd, _LAYOUT_CODE[layout],
            int(causal), -1.0 if scale is None else scale, _DTYPE_CODE[q.dtype], cos.shape[0])
    if attn_mask is None:
        rope_attention_fwd(*args, k_workspace, ws_bytes, stream)
        return o
    if attn_mask.dtype not in (torch.bool, torch.uint8):
        raise TypeError("attn_mask must be bool or uint8")
    if tuple(attn_mask.shape) == (B, Sk):
        kind = ROPE_MASK_KEYS
    elif tuple(attn_mask.shape) == (B, Sq, Sk):
        kind = ROPE_MASK_QUERY_KEYS
    else:
        raise ValueError("attn_mask must be [B, Sk] or [B, Sq, Sk], got %s" %
                         (tuple(attn_mask.shape),))
    rope_attention_fwd_masked(*args, attn_mask, kind, k_workspace, ws_bytes, stream)
    return o


# --------------------------------------------------------------------------
# serving: packed sequences and a paged cache
# --------------------------------------------------------------------------
def rope_cache_append(k, v, k_pages, v_pages, block_table, cu_seqlens, cache_lens, cos, sin, pos,
                      pos_offset, n_seqs, total, k_stride, v_stride, Hk, D, rotary_dim, layout,
                      page_size, n_pages, max_blocks, dtype, table_rows, stream=None):
    st = load_library().rope_cache_append(
        _addr(k, "k"), _addr(v, "v"), _addr(k_pages, "k_pages"), _addr(v_pages, "v_pages"),
        _addr(block_table, "block_table"), _addr(cu_seqlens, "cu_seqlens"),
        _addr(cache_lens, "cache_lens"), _addr(cos, "cos"), _addr(sin, "sin"), _addr(pos, "pos"),
        int(pos_offset), int(n_seqs), int(total), int(k_stride), int(v_stride), int(Hk), int(D),
        int(rotary_dim), int(layout), int(page_size), int(n_pages), int(max_blocks), int(dtype),
        int(table_rows), _stream(stream))
    _check(st, "rope_cache_append")


def rope_attention_packed_fwd(q, k, v, o, cos, sin, pos_q, pos_k, cu_seqlens_q, cu_seqlens_k, n_seqs,
                              total_q, total_k, q_stride, k_stride, v_stride, Hq, Hk, D, rotary_dim,
                              layout, causal, softmax_scale, dtype, table_rows, workspace,
                              workspace_bytes, stream=None):
    st = load_library().rope_attention_packed_fwd(
        _addr(q, "q"), _addr(k, "k"), _addr(v, "v"), _addr(o, "o"), _addr(cos, "cos"),
        _addr(sin, "sin"), _addr(pos_q, "pos_q"), _addr(pos_k, "pos_k"),
        _addr(cu_seqlens_q, "cu_seqlens_q"), _addr(cu_seqlens_k, "cu_seqlens_k"), int(n_seqs),
        int(total_q), int(total_k), int(q_stride), int(k_stride), int(v_stride), int(Hq), int(Hk),
        int(D), int(rotary_dim), int(layout), int(causal), float(softmax_scale), int(dtype),
        int(table_rows), _addr(workspace, "workspace"), int(workspace_bytes), _stream(stream))
    _check(st, "rope_attention_packed_fwd")


def rope_attention_packed_workspace(n_seqs, total_q, total_k, Hq, Hk, D) -> int:
    """Bytes of workspace (-1 for sizes the call does not take)."""
    return load_library().rope_attention_packed_workspace(int(n_seqs), int(total_q), int(total_k),
                                                          int(Hq), int(Hk), int(D))


def rope_attention_decode_fwd(q, k_pages, v_pages, o, block_table, seq_lens, prefix_table, prefix_len,
                              cos, sin, pos_q, B, q_stride, Hq, Hk, D, rotary_dim, layout,
                              softmax_scale, page_size, n_pages, max_blocks, dtype, table_rows,
                              workspace, workspace_bytes, stream=None):
    st = load_library().rope_attention_decode_fwd(
        _addr(q, "q"), _addr(k_pages, "k_pages"), _addr(v_pages, "v_pages"), _addr(o, "o"),
        _addr(block_table, "block_table"), _addr(seq_lens, "seq_lens"),
        _addr(prefix_table, "prefix_table"), int(prefix_len), _addr(cos, "cos"), _addr(sin, "sin"),
        _addr(pos_q, "pos_q"), int(B), int(q_stride), int(Hq), int(Hk), int(D), int(rotary_dim),
        int(layout), float(softmax_scale), int(page_size), int(n_pages), int(max_blocks), int(dtype),
        int(table_rows), _addr(workspace, "workspace"), int(workspace_bytes), _stream(stream))
    _check(st, "rope_attention_decode_fwd")


def rope_attention_decode_workspace(B, Hq, Hk, D, page_size, max_blocks, prefix_len) -> int:
    """Bytes of workspace (-1 for sizes the call does not take)."""
    return load_library().rope_attention_decode_workspace(int(B), int(Hq), int(Hk), int(D),
                                                          int(page_size), int(max_blocks),
                                                          int(prefix_len))


def rope_attention_paged_fwd(q, k_pages, v_pages, o, block_table, cu_seqlens_q, seq_lens, cos, sin, pos_q, n_seqs, total_q,
                             q_stride, Hq, Hk, D, rotary_dim, layout, causal, softmax_scale, page_size, n_pages,
                             max_blocks, dtype, table_rows, workspace, workspace_bytes, stream=None):
    st = load_library().rope_attention_paged_fwd(
        _addr(q, "q"), _addr(k_pages, "k_pages"), _addr(v_pages, "v_pages"), _addr(o, "o"),
        _addr(block_table, "block_table"), _addr(cu_seqlens_q, "cu_seqlens_q"), _addr(seq_lens, "seq_lens"),
        _addr(cos, "cos"), _addr(sin, "sin"), _addr(pos_q, "pos_q"), int(n_seqs), int(total_q), int(q_stride), int(Hq),
        int(Hk), int(D), int(rotary_dim), int(layout), int(causal), float(softmax_scale), int(page_size), int(n_pages),
        int(max_blocks), int(dtype), int(table_rows), _addr(workspace, "workspace"), int(workspace_bytes),
        _stream(stream))
    _check(st, "rope_attention_paged_fwd")


def rope_attention_paged_workspace(n_seqs, total_q, Hq, Hk, D, page_size, max_blocks) -> int:
    """Bytes of workspace (-1 for sizes the call does not take)."""
    return load_library().rope_attention_paged_workspace(int(n_seqs), int(total_q), int(Hq), int(Hk), int(D),
                                                         int(page_size), int(max_blocks))


_serving = None


def _native():
    """The binding module of the serving and norm calls (csrc/serving_binding.cpp), given
    the entry points of the library that is loaded."""
    global _serving
    if _serving is None:
        lib = load_library()
        path = _build.BINDING
        if not os.path.exists(path):
            raise RuntimeError(
                "%s is not built; run `python -c \"import __graft_entry__ as g; g.build()\"` "
                "first" % path)
        spec = importlib.util.spec_from_file_location("_serving", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.rope_cache_append, lib.rope_attention_packed_fwd,
            lib.rope_attention_packed_workspace, lib.rope_attention_decode_fwd,
            lib.rope_attention_decode_workspace, lib.rope_norm_qk_fwd, lib.rope_norm_qk_bwd,
            lib.rope_norm_qk_workspace, lib.rope_norm_cache_append,
            lib.rope_tables_build_scaled, lib.rope_attention_paged_fwd,
            lib.rope_attention_paged_workspace)))
        _serving = module
    return _serving


def cache_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 block_table: torch.Tensor, cu_seqlens: torch.Tensor, cache_lens: torch.Tensor,
                 cos: torch.Tensor, sin: torch.Tensor, pos: torch.Tensor | None = None,
                 pos_offset: int = 0, rotary_dim: int | None = None, layout: str = "split_half",
                 stream=None) -> None:
    """Rotate new keys and write them, with their values, into a paged cache.

    k, v: [T, Hk, D] packed new tokens (views with a token stride are taken as
    they are); sequence b owns tokens cu_seqlens[b] .. cu_seqlens[b+1] - 1,
    which become its keys cache_lens[b], cache_lens[b] + 1, ...
    k_pages, v_pages: [pages, Hk, page_size, D], page_size 16, 32, 64 or 128.
    block_table: int32 [n_seqs, max_blocks]; cu_seqlens: int32 [n_seqs + 1];
    cache_lens: int32 [n_seqs] (not advanced by the call).
    pos: int32 [T] table rows (-1 = not rotated), or None for pos_offset + the
    key's index in its sequence.
    Not differentiable: the pools carry no graph of k and v, and count as
    written in place.
    """
    st = (_serving or _native()).cache_append(
        k, v, k_pages, v_pages, block_table, cu_seqlens, cache_lens, cos, sin, pos, pos_offset,
        rotary_dim, _LAYOUT_CODE[layout], stream)
    if st != ROPE_OK:
        raise RopeError(st, "rope_cache_append")


def norm_cache_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, wq: torch.Tensor | None,
                      wk: torch.Tensor | None, k_pages: torch.Tensor, v_pages: torch.Tensor,
                      block_table: torch.Tensor, cu_seqlens: torch.Tensor, cache_lens: torch.Tensor,
                      cos: torch.Tensor, sin: torch.Tensor, eps: float = 1e-6,
                      pos: torch.Tensor | None = None, pos_offset: int = 0, rotary_dim: int | None = None,
                      layout: str = "split_half", q_out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """cache_append of a model that normalises queries and keys (norm_rotate_qk): new keys,
    normalised and rotated, and values into the pages; returns the queries, normalised and
    rotated, [T, Hq, D] (rows of tokens of no sequence are not written).

    q: [T, Hq, D], the new tokens' queries (a view with a token stride is taken as it is);
    wq, wk: [D] weights in fp32 or q's type, 16-byte aligned, or None.  q_out: the output, which may be q
    itself where that is dense.  Everything else as cache_append; attention_paged takes the
    result without cos and sin.
    """
    o = (_serving or _native()).norm_cache_append(
        q, k, v, wq, wk, k_pages, v_pages, block_table, cu_seqlens, cache_lens, cos, sin, eps, pos, pos_offset,
        rotary_dim, _LAYOUT_CODE[layout], q_out, stream)
    if type(o) is int:
        raise RopeError(o, "rope_norm_cache_append")
    return o


def attention_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                    cu_seqlens_q: torch.Tensor, seq_lens: torch.Tensor, cos: torch.Tensor | None = None,
                    sin: torch.Tensor | None = None, pos_q: torch.Tensor | None = None,
                    rotary_dim: int | None = None, layout: str = "split_half", causal: bool = True,
                    scale: float | None = None, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of every sequence's new tokens, one or a chunk of a prompt, over its paged cache.

    q: [Tq, Hq, D] packed new tokens (a view with a token stride is taken as it is);
    returns [Tq, Hq, D].  Sequence b's queries are tokens cu_seqlens_q[b] ..
    cu_seqlens_q[b+1] - 1 (none is allowed), the last of its seq_lens[b] keys
    (cache_append or norm_cache_append them first): with causal, query i of Lq sees the
    keys j <= i + Lk - Lq.  A query that sees no key gets zeros; rows of ``out`` that
    belong to no sequence keep what they hold.
    k_pages, v_pages: the cache, [pages, Hk, page_size, D]; block_table: int32 [n_seqs,
    max_blocks]; cu_seqlens_q: int32 [n_seqs + 1]; seq_lens: int32 [n_seqs].
    cos, sin: the rotation table, or None where q is rotated already (norm_cache_append).
    pos_q: int32 [Tq] table rows (-1 = not rotated), or None for a query's index among its
    sequence's keys.
    workspace: None, or a uint8 tensor of rope_attention_paged_workspace(...) bytes to use
    (128-byte aligned; its contents do not matter).
    stream: as attention_packed.  Forward only, as well.
    """
    o = (_serving or _native()).attention_paged(
        q, k_pages, v_pages, block_table, cu_seqlens_q, seq_lens, cos, sin, pos_q, rotary_dim,
        _LAYOUT_CODE[layout], causal, scale, out, workspace, stream)
    if type(o) is int:
        raise RopeError(o, "rope_attention_paged_fwd")
    return o


def attention_packed(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                     cos: torch.Tensor, sin: torch.Tensor, cu_seqlens_k: torch.Tensor | None = None,
                     pos_q: torch.Tensor | None = None, pos_k: torch.Tensor | None = None,
                     rotary_dim: int | None = None, layout: str = "split_half", causal: bool = False,
                     scale: float | None = None, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """softmax(scale * rot(q) rot(k)^T + mask) v for packed sequences of different lengths.

    q: [Tq, Hq, D]; k, v: [Tk, Hk, D] (views with a token stride are taken as
    they are); returns [Tq, Hq, D].  Sequence b's queries are tokens
    cu_seqlens_q[b] .. cu_seqlens_q[b+1] - 1, its keys those of cu_seqlens_k
    (None: the same); both int32 [n_seqs + 1].  With causal, the queries are
    the last tokens of their sequence: query i of Lq sees the keys
    j <= i + Lk - Lq.  A query that sees no key gets zeros; rows of ``out``
    that belong to no sequence keep what they hold.
    pos_q, pos_k: int32 [Tq], [Tk] table rows (-1 = not rotated), or None for
    a token's index among its sequence's queries (keys).
    workspace: None, or a uint8 tensor of rope_attention_packed_workspace(...)
    bytes to use (128-byte aligned; its contents do not matter).
    stream: what the call runs on (None: the current stream); inputs have to be
    ready there and to stay until it is done with them.
    Forward only: the output carries no graph of the inputs.
    """
    o = (_serving or _native()).attention_packed(
        q, k, v, cu_seqlens_q, cos, sin, cu_seqlens_k, pos_q, pos_k, rotary_dim,
        _LAYOUT_CODE[layout], causal, scale, out, workspace, stream)
    if type(o) is int:
        raise RopeError(o, "rope_attention_packed_fwd")
    return o


def attention_shared_prefix(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                            block_table: torch.Tensor, seq_lens: torch.Tensor,
                            prefix_table: torch.Tensor | None, prefix_len: int, cos: torch.Tensor,
                            sin: torch.Tensor, pos_q: torch.Tensor | None = None,
                            rotary_dim: int | None = None, layout: str = "split_half",
                            scale: float | None = None, out: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of one new token per sequence over a shared prefix and its own suffix.

    q: [B, Hq, D] (a view with a row stride is taken as it is), one query per
    sequence; returns [B, Hq, D].  k_pages, v_pages: the cache that
    cache_append writes, [pages, Hk, page_size, D] of rotated keys.
    prefix_table: int32 pages of the prefix_len keys that all sequences share
    (None with prefix_len 0), read for the batch, not for every sequence.
    block_table: int32 [B, max_blocks]; seq_lens: int32 [B], the keys of each
    suffix, the new token's own among them (cache_append it first).
    pos_q: int32 [B] table rows (-1 = not rotated), or None for
    prefix_len + seq_lens - 1.
    workspace: None, or a uint8 tensor of rope_attention_decode_workspace(...)
    bytes to use (128-byte aligned; its contents do not matter).
    stream: as attention_packed.  Forward only, as well.
    """
    o = (_serving or _native()).attention_shared_prefix(
        q, k_pages, v_pages, block_table, seq_lens, prefix_table, prefix_len, cos, sin, pos_q,
        rotary_dim, _LAYOUT_CODE[layout], scale, out, workspace, stream)
    if type(o) is int:
        raise RopeError(o, "rope_attention_decode_fwd")
    return o


# --------------------------------------------------------------------------
# normalised queries and keys
# --------------------------------------------------------------------------
def rope_norm_qk_fwd(q, k, q_out, k_out, wq, wk, cos, sin, pos_idx, pos_batch_stride, B, Hq, Hk, S, D, q_strides,
                     k_strides, rotary_dim, layout, seq_before_head, eps, dtype, weight_dtype, table_rows, stream=None):
    """q_strides, k_strides: three integers (batch, token, head), or None for dense; q and k of
    other strides are given as addresses."""
    st = load_library().rope_norm_qk_fwd(
        _addr(q, "q"), _addr(k, "k"), _addr(q_out, "q_out"), _addr(k_out, "k_out"), _addr(wq, "wq"), _addr(wk, "wk"),
        _addr(cos, "cos"), _addr(sin, "sin"), _addr(pos_idx, "pos_idx"), int(pos_batch_stride), int(B), int(Hq),
        int(Hk), int(S), int(D), _strides3(q_strides), _strides3(k_strides), int(rotary_dim), int(layout),
        int(seq_before_head), float(eps), int(dtype), int(weight_dtype), int(table_rows), _stream(stream))
    _check(st, "rope_norm_qk_fwd")


def rope_norm_qk_bwd(q, k, gq, gk, dq, dk, wq, wk, dwq, dwk, cos, sin, pos_idx, pos_batch_stride, B, Hq, Hk, S, D,
                     q_strides, k_strides, rotary_dim, layout, seq_before_head, eps, dtype, weight_dtype, table_rows,
                     workspace, workspace_bytes, stream=None):
    st = load_library().rope_norm_qk_bwd(
        _addr(q, "q"), _addr(k, "k"), _addr(gq, "gq"), _addr(gk, "gk"), _addr(dq, "dq"), _addr(dk, "dk"),
        _addr(wq, "wq"), _addr(wk, "wk"), _addr(dwq, "dwq"), _addr(dwk, "dwk"), _addr(cos, "cos"), _addr(sin, "sin"),
        _addr(pos_idx, "pos_idx"), int(pos_batch_stride), int(B), int(Hq), int(Hk), int(S), int(D),
        _strides3(q_strides), _strides3(k_strides), int(rotary_dim), int(layout), int(seq_before_head), float(eps),
        int(dtype), int(weight_dtype), int(table_rows), _addr(workspace, "workspace"), int(workspace_bytes),
        _stream(stream))
    _check(st, "rope_norm_qk_bwd")


def _strides3(s):
    return None if s is None else (ctypes.c_int64 * 3)(*s)


def rope_norm_qk_workspace(D) -> int:
    """Bytes of workspace (-1 for a D the call does not take)."""
    return load_library().rope_norm_qk_workspace(int(D))


def rope_norm_cache_append(q, k, v, q_out, k_pages, v_pages, wq, wk, block_table, cu_seqlens, cache_lens, cos, sin, pos,
                           pos_offset, n_seqs, total, q_stride, k_stride, v_stride, Hq, Hk, D, rotary_dim, layout, eps,
                           page_size, n_pages, max_blocks, dtype, weight_dtype, table_rows, stream=None):
    st = load_library().rope_norm_cache_append(
        _addr(q, "q"), _addr(k, "k"), _addr(v, "v"), _addr(q_out, "q_out"), _addr(k_pages, "k_pages"),
        _addr(v_pages, "v_pages"), _addr(wq, "wq"), _addr(wk, "wk"), _addr(block_table, "block_table"),
        _addr(cu_seqlens, "cu_seqlens"), _addr(cache_lens, "cache_lens"), _addr(cos, "cos"), _addr(sin, "sin"),
        _addr(pos, "pos"), int(pos_offset), int(n_seqs), int(total), int(q_stride), int(k_stride), int(v_stride), int(Hq),
        int(Hk), int(D), int(rotary_dim), int(layout), float(eps), int(page_size), int(n_pages), int(max_blocks),
        int(dtype), int(weight_dtype), int(table_rows), _stream(stream))
    _check(st, "rope_norm_cache_append")


def norm_rotate_qk(q: torch.Tensor | None, k: torch.Tensor | None, wq: torch.Tensor | None,
                   wk: torch.Tensor | None, cos: torch.Tensor, sin: torch.Tensor, eps: float = 1e-6,
                   pos_idx: torch.Tensor | None = None, rotary_dim: int | None = None,
                   layout: str = "split_half", seq_before_head: bool = False,
                   q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """The RMS norm of every query and key head and the rotation, in one pass:
    y = R(t) (w * x / sqrt(mean(x^2) + eps)).  Returns (q_out, k_out), dense.

    q: [B, Hq, S, D] (or [B, S, Hq, D] with seq_before_head), k likewise with Hk heads, or
    either None; bf16, fp16 or fp32; views are taken as they are as long as features are
    dense and strides whole 16-byte vectors (a part of a fused projection's output).
    wq, wk: [D] weights of all query (key) heads, fp32 or the rows' type, 16-byte aligned, or
    None (ones).
    cos/sin: float32 [rows, rotary_dim // 2].  pos_idx: int32 [S] or [B, S] table rows (-1 =
    normalised, not rotated), or None.  q_out=q (k_out=k) works in place on a dense tensor.
    Carries no graph: ``autograd.norm_rotary_qk`` is the differentiable form.
    """
    o = (_serving or _native()).norm_rotate_qk(q, k, wq, wk, cos, sin, eps, pos_idx, rotary_dim,
                                               _LAYOUT_CODE[layout], seq_before_head, q_out, k_out, stream)
    if type(o) is int:
        raise RopeError(o, "rope_norm_qk_fwd")
    return o


def norm_rotate_qk_backward(gq: torch.Tensor | None, gk: torch.Tensor | None, q: torch.Tensor | None,
                            k: torch.Tensor | None, wq: torch.Tensor | None, wk: torch.Tensor | None,
                            cos: torch.Tensor, sin: torch.Tensor, eps: float = 1e-6,
                            pos_idx: torch.Tensor | None = None, rotary_dim: int | None = None,
                            layout: str = "split_half", seq_before_head: bool = False,
                            weight_grads: tuple[bool, bool] = (True, True), stream=None):
    """Gradients of norm_rotate_qk: (dq, dk, dwq, dwk), dense, None for what is not given or
    not wanted.  gq, gk: gradients of the outputs, dense; q, k and the rest: what the
    forward call was given."""
    o = (_serving or _native()).norm_rotate_qk_backward(
        gq, gk, q, k, wq, wk, cos, sin, eps, pos_idx, rotary_dim, _LAYOUT_CODE[layout], seq_before_head,
        weight_grads[0], weight_grads[1], stream)
    if type(o) is int:
        raise RopeError(o, "rope_norm_qk_bwd")
    return o
