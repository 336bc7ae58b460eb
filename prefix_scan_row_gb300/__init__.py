"""Python binding of libmtscan.so (include/mt_scan.h): prefix scans on one
NVIDIA GB300.

The functions here only marshal arguments (pointers, sizes, the current CUDA
stream) into the C ABI; every step of the scan runs in the library's CUDA
kernels. There is no fallback: if the shared library is missing or fails to
load, importing this package raises.

Names and arguments follow the C ABI:

* ``mt_scan_rows(inp, out, inclusive)`` -- row-wise sum scan of a contiguous
  [rows, n] f32/bf16/f16 CUDA tensor.
* ``mt_scan_rows_op(inp, out, op, inclusive)`` -- the same with op in
  add / mul / max / min.
* ``mt_exclusive_scan(arr, out, scratch, n_dev, op)`` -- device-wide exclusive
  add/min/max over i32/i64/f32 with the live count in a device int32.
* ``mt_inclusive_scan(arr, out, scratch, n_dev, op)`` -- the inclusive form
  (in place allowed).
* ``mt_reduce(arr, out, scratch, n_dev, op)`` -- out[0] = op(arr[0:n]).
* ``mt_select(arr, flags, out, num_out, scratch, n_dev)`` -- stream compaction
  (``mt_select_wide`` for 8-byte elements).
* ``mt_reduce_by_key_add(keys_in, values_in, keys_out, values_out, num_runs,
  scratch, n_dev)`` -- run-length sums of consecutive equal keys.
* ``mt_scan_scratch_slots(capacity, dtype, kind)`` -- scratch sizing.

Operators of sequence models (activations [batch, len, dim], f32/bf16/f16):

* ``mt_embed(tokens, table, out, scale)`` and ``mt_embed_grad(tokens, dout,
  dtable, scratch, scale, accumulate)`` -- embedding lookup, and the table's
  gradient by sorted tokens.
* ``mt_causal_conv(x, weight, out, ...)``, ``mt_causal_conv_step`` (one token
  of each sequence) and ``mt_causal_conv_grad`` -- short causal convolution with
  bias and SiLU.
* ``mt_selective_scan(u, delta, A, B, C, out, ...)``, ``mt_selective_scan_step``
  and ``mt_selective_scan_grad`` -- selective state space scan with gate.
* their scratch sizes: ``mt_embed_grad_scratch_slots``,
  ``mt_causal_conv_grad_scratch_slots``, ``mt_selective_scan_scratch_slots`` and
  ``mt_selective_scan_checkpoint_slots``, in 8-byte slots.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmtscan.so")
LIB_CHECKED_PATH = os.path.join(_HERE, "libmtscan_checked.so")  # the bounds-checked build

MT_F32, MT_BF16, MT_F16, MT_I32, MT_I64, MT_U32, MT_U64, MT_F64 = 0, 1, 2, 3, 4, 5, 6, 7
MT_ADD, MT_MIN, MT_MAX, MT_MUL = 0, 1, 2, 3
MT_SCRATCH_SCAN, MT_SCRATCH_SELECT, MT_SCRATCH_REDUCE, MT_SCRATCH_REDUCE_BY_KEY = 1, 2, 3, 4
MT_OK = 0
MT_ERR_ARG, MT_ERR_DTYPE, MT_ERR_ALIAS, MT_ERR_CUDA, MT_ERR_LOOKBACK_TIMEOUT, MT_ERR_ALIGN = (
    -1, -2, -3, -4, -5, -6)
MT_ERR_TOO_LARGE = -7
MT_ERR_MEMORY = -8
MT_ERR_BOUNDS = -9
MT_NOALLOC_SCRATCH_BYTES = 1 << 20

DTYPE_CODE = {torch.float32: MT_F32, torch.bfloat16: MT_BF16, torch.float16: MT_F16,
              torch.int32: MT_I32, torch.int64: MT_I64, torch.uint32: MT_U32, torch.uint64: MT_U64,
              torch.float64: MT_F64}
OP_CODE = {"add": MT_ADD, "min": MT_MIN, "max": MT_MAX, "mul": MT_MUL}

EXPORTS = ("mt_scan_rows", "mt_scan_rows_op", "mt_exclusive_scan", "mt_inclusive_scan", "mt_reduce", "mt_select",
           "mt_select_wide", "mt_reduce_by_key_add", "mt_scan_scratch_slots",
           "mt_scan_status", "mt_scan_launches", "mt_scan_strerror", "mt_scan_debug_lookback",
           "mt_scan_rows_noalloc", "mt_scan_rows_scratch_slots", "mt_scan_build_checked",
           "mt_embed", "mt_embed_grad", "mt_embed_grad_scratch_slots", "mt_causal_conv", "mt_causal_conv_step",
           "mt_causal_conv_grad", "mt_causal_conv_grad_scratch_slots", "mt_selective_scan", "mt_selective_scan_step",
           "mt_selective_scan_grad", "mt_selective_scan_scratch_slots", "mt_selective_scan_checkpoint_slots")


class ScanError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {mt_scan_strerror(code)} ({code})")


def _load(path: str):
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"`"
            " (the scan library has no CPU fallback)")
    L = ctypes.CDLL(path)
    p, i64, i32, u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint32
    L.mt_scan_rows.argtypes = [p, p, i64, i64, i32, i32, p]
    L.mt_scan_rows.restype = i32
    L.mt_scan_rows_op.argtypes = [p, p, i64, i64, i32, i32, i32, p]
    L.mt_scan_rows_op.restype = i32
    L.mt_exclusive_scan.argtypes = [p, p, p, p, i32, i32, p]
    L.mt_exclusive_scan.restype = i32
    L.mt_inclusive_scan.argtypes = [p, p, p, p, i32, i32, p]
    L.mt_inclusive_scan.restype = i32
    L.mt_reduce.argtypes = [p, p, p, p, i32, i32, p]
    L.mt_reduce.restype = i32
    L.mt_select.argtypes = [p, p, p, p, p, p, p]
    L.mt_select_wide.argtypes = [p, p, p, p, p, p, i32, p]
    L.mt_select_wide.restype = i32
    L.mt_reduce_by_key_add.argtypes = [p, p, p, p, p, p, p, i32, i32, p]
    L.mt_reduce_by_key_add.restype = i32
    L.mt_select.restype = i32
    L.mt_scan_scratch_slots.argtypes = [i64, i32, i32]
    L.mt_scan_scratch_slots.restype = i64
    L.mt_scan_status.argtypes = [p]
    L.mt_scan_status.restype = i32
    L.mt_scan_launches.argtypes = []
    L.mt_scan_launches.restype = ctypes.c_uint64
    L.mt_scan_strerror.argtypes = [i32]
    L.mt_scan_strerror.restype = ctypes.c_char_p
    L.mt_scan_debug_lookback.argtypes = [i64, u32]
    L.mt_scan_debug_lookback.restype = i32
    L.mt_scan_rows_noalloc.argtypes = [p, p, i64, i64, i32, i32, p]
    L.mt_scan_rows_noalloc.restype = i32
    L.mt_scan_rows_scratch_slots.argtypes = [i64, i64, i32]
    L.mt_scan_rows_scratch_slots.restype = i64
    L.mt_scan_build_checked.argtypes = []
    L.mt_scan_build_checked.restype = i32
    f32, args = ctypes.c_float, ctypes.c_char_p  # argument blocks are packed bytes
    L.mt_embed.argtypes = [p, i64, i32, p, i64, i64, i32, f32, p, p]
    L.mt_embed_grad.argtypes = [p, i64, i32, p, i32, i64, i64, f32, p, i32, i32, p, p]
    L.mt_embed_grad_scratch_slots.argtypes = [i64, i64, i64]
    L.mt_causal_conv_grad_scratch_slots.argtypes = [i64, i64, i64, i64]
    L.mt_selective_scan_scratch_slots.argtypes = [i64, i64, i64, i64, i64, i32]
    L.mt_selective_scan_checkpoint_slots.argtypes = [i64, i64, i64, i64]
    for name in ("mt_embed_grad_scratch_slots", "mt_causal_conv_grad_scratch_slots",
                 "mt_selective_scan_scratch_slots", "mt_selective_scan_checkpoint_slots"):
        getattr(L, name).restype = i64
    for name in ("mt_causal_conv", "mt_causal_conv_step", "mt_causal_conv_grad", "mt_selective_scan",
                 "mt_selective_scan_step", "mt_selective_scan_grad"):
        getattr(L, name).argtypes = [args, p]
        getattr(L, name).restype = i32
    return L


def _check(code: int, where: str) -> None:
    if code != MT_OK:
        raise ScanError(code, where)


def _stream(stream) -> int:
    if stream is None:
        if torch.cuda.is_initialized():  # the handle alone: a Stream object costs 3 us of host time a call
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t) -> int:
    return 0 if t is None else (t if isinstance(t, int) else t.data_ptr())


def _contiguous(**tensors) -> None:
    """The library sees flat memory: a strided view would be read as such."""
    for name, t in tensors.items():
        if isinstance(t, torch.Tensor) and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


# The argument blocks mt_conv_args and mt_ssm_args: eight bytes a field.
_CONV_ARGS = struct.Struct("=30q")
_SSM_ARGS = struct.Struct("=58q")
_NO_ACT = (0, 0, 0)  # an activation that is absent: pointer, batch and token strides


def _act(name, t, shape, dtype):
    """An activation's pointer and its batch and token strides; its innermost
    axis (two for B and C of a scan) must be contiguous."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} of {dtype}, not {list(t.shape)} of {t.dtype}")
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}'s innermost axis must be contiguous")
    if len(shape) == 4 and shape[2] > 1 and s[2] != shape[3]:
        raise ValueError(f"{name}'s two innermost axes must be contiguous")
    return t.data_ptr(), s[0], s[1]


def _act_step(name, t, shape, dtype):
    """The same of one token a sequence: the token stride does not count."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} of {dtype}, not {list(t.shape)} of {t.dtype}")
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}'s innermost axis must be contiguous")
    if len(shape) == 3 and shape[1] > 1 and s[1] != shape[2]:
        raise ValueError(f"{name}'s two innermost axes must be contiguous")
    return t.data_ptr(), s[0], 0


def _flat(name, t, shape, dtype):
    """The pointer of a contiguous tensor; 0 for None."""
    if t is None:
        return 0
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)} of {dtype}, not {list(t.shape)} of {t.dtype}")
    return t.data_ptr()


def _pool(name, state, row, dtype, batch, slots):
    """The pointer and the number of rows of a pool of states."""
    if state is None:
        return 0, batch
    if state.dtype != dtype or state.dim() != 3 or tuple(state.shape[1:]) != row or not state.is_contiguous():
        raise ValueError(f"{name} must be contiguous [slots, {row[0]}, {row[1]}] of {dtype}")
    if slots is None and state.shape[0] < batch:
        raise ValueError(f"{name} needs a row for every sequence")
    return state.data_ptr(), state.shape[0]


def _scratch(name, t, slots):
    """The pointer of a scratch tensor of at least `slots` 8-byte slots."""
    if t is None:
        if slots > 0:
            raise ValueError(f"{name} is needed: {slots} 8-byte slots")
        return 0
    if t.numel() * t.element_size() < 8 * slots or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and hold {slots} 8-byte slots")
    return t.data_ptr()


class Library:
    """The calls of one loaded build of the C ABI: the ordinary library, or
    (load_checked) its bounds-checked twin. Each method marshals torch
    tensors into the C call of the same name."""

    def __init__(self, path: str):
        self.path = path
        self.lib = _load(path)

    def mt_scan_strerror(self, code: int) -> str:
        return self.lib.mt_scan_strerror(int(code)).decode()

    def mt_scan_rows(self, inp: torch.Tensor, out: torch.Tensor, inclusive: bool, stream=None) -> None:
        """Row-wise sum scan of a contiguous 2-D (or 1-D = one row) CUDA tensor."""
        if inp.dim() == 1:
            rows, n = 1, inp.shape[0]
        else:
            rows, n = inp.shape
        if out.shape != inp.shape or out.dtype != inp.dtype:
            raise ValueError("out must match inp in shape and dtype")
        if not (inp.is_contiguous() and out.is_contiguous()):
            raise ValueError("inp and out must be contiguous")
        code = DTYPE_CODE.get(inp.dtype, -99)
        _check(self.lib.mt_scan_rows(_ptr(inp), _ptr(out), rows, n, code, int(bool(inclusive)),
                                     _stream(stream)), "mt_scan_rows")

    def mt_scan_rows_op(self, inp: torch.Tensor, out: torch.Tensor, op: str, inclusive: bool,
                        stream=None) -> None:
        """Row-wise scan with op in 'add' | 'mul' | 'max' | 'min'."""
        if inp.dim() == 1:
            rows, n = 1, inp.shape[0]
        else:
            rows, n = inp.shape
        if out.shape != inp.shape or out.dtype != inp.dtype:
            raise ValueError("out must match inp in shape and dtype")
        if not (inp.is_contiguous() and out.is_contiguous()):
            raise ValueError("inp and out must be contiguous")
        code = DTYPE_CODE.get(inp.dtype, -99)
        _check(self.lib.mt_scan_rows_op(_ptr(inp), _ptr(out), rows, n, code, OP_CODE[op],
                                        int(bool(inclusive)), _stream(stream)), "mt_scan_rows_op")

    def mt_exclusive_scan(self, arr: torch.Tensor, out: torch.Tensor, scratch: torch.Tensor,
                          n_dev: torch.Tensor, op: str, stream=None) -> None:
        """Exclusive scan of arr[0:*n_dev] into out (op: 'add' | 'min' | 'max')."""
        if out.dtype != arr.dtype:
            raise ValueError("out must have arr's dtype")
        if n_dev.dtype != torch.int32:
            raise ValueError("n_dev must be an int32 device tensor")
        _contiguous(arr=arr, out=out, scratch=scratch)
        code = DTYPE_CODE.get(arr.dtype, -99)
        _check(self.lib.mt_exclusive_scan(_ptr(arr), _ptr(out), _ptr(scratch), _ptr(n_dev), code,
                                          OP_CODE[op], _stream(stream)), "mt_exclusive_scan")

    def mt_inclusive_scan(self, arr: torch.Tensor, out: torch.Tensor, scratch: torch.Tensor,
                          n_dev: torch.Tensor, op: str, stream=None) -> None:
        """Inclusive scan of arr[0:*n_dev] into out (out may be arr)."""
        if out.dtype != arr.dtype:
            raise ValueError("out must have arr's dtype")
        if n_dev.dtype != torch.int32:
            raise ValueError("n_dev must be an int32 device tensor")
        _contiguous(arr=arr, out=out, scratch=scratch)
        code = DTYPE_CODE.get(arr.dtype, -99)
        _check(self.lib.mt_inclusive_scan(_ptr(arr), _ptr(out), _ptr(scratch), _ptr(n_dev), code,
                                          OP_CODE[op], _stream(stream)), "mt_inclusive_scan")

    def mt_reduce(self, arr: torch.Tensor, out: torch.Tensor, scratch: torch.Tensor, n_dev: torch.Tensor,
                  op: str, stream=None) -> None:
        """out[0] = op(arr[0:*n_dev]) (the identity for an empty input)."""
        if out.dtype != arr.dtype:
            raise ValueError("out must have arr's dtype")
        if n_dev.dtype != torch.int32:
            raise ValueError("n_dev must be an int32 device tensor")
        _contiguous(arr=arr, scratch=scratch)
        code = DTYPE_CODE.get(arr.dtype, -99)
        _check(self.lib.mt_reduce(_ptr(arr), _ptr(out), _ptr(scratch), _ptr(n_dev), code, OP_CODE[op],
                                  _stream(stream)), "mt_reduce")

    def mt_select(self, arr: torch.Tensor, flags: torch.Tensor, out: torch.Tensor, num_out: torch.Tensor,
                  scratch: torch.Tensor, n_dev: torch.Tensor, stream=None) -> None:
        """Stream compaction of 4-byte elements by exactly-0/1 uint8 flags."""
        if arr.element_size() != 4 or out.element_size() != 4:
            raise ValueError("select copies 4-byte elements")
        if flags.dtype != torch.uint8 or num_out.dtype != torch.int32 or n_dev.dtype != torch.int32:
            raise ValueError("flags must be uint8, num_out and n_dev int32")
        _contiguous(arr=arr, flags=flags, out=out, scratch=scratch)
        _check(self.lib.mt_select(_ptr(arr), _ptr(flags), _ptr(out), _ptr(num_out), _ptr(scratch),
                                  _ptr(n_dev), _stream(stream)), "mt_select")

    def mt_select_wide(self, arr: torch.Tensor, flags: torch.Tensor, out: torch.Tensor, num_out: torch.Tensor,
                       scratch: torch.Tensor, n_dev: torch.Tensor, stream=None) -> None:
        """Stream compaction of 4- or 8-byte elements, or of structs: a 1-D arr
        holds one element per entry, an [n, ...] arr one struct per row (its
        trailing dimensions), copied bit for bit."""
        eb = arr.element_size() * math.prod(arr.shape[1:])
        if out.element_size() * math.prod(out.shape[1:]) != eb:
            raise ValueError("out's elements must have arr's size")
        if flags.dtype != torch.uint8 or num_out.dtype != torch.int32 or n_dev.dtype != torch.int32:
            raise ValueError("flags must be uint8, num_out and n_dev int32")
        _contiguous(arr=arr, flags=flags, out=out, scratch=scratch)
        _check(self.lib.mt_select_wide(_ptr(arr), _ptr(flags), _ptr(out), _ptr(num_out), _ptr(scratch),
                                       _ptr(n_dev), eb, _stream(stream)), "mt_select_wide")

    def mt_reduce_by_key_add(self, keys_in: torch.Tensor, values_in: torch.Tensor, keys_out: torch.Tensor,
                             values_out: torch.Tensor, num_runs: torch.Tensor, scratch: torch.Tensor,
                             n_dev: torch.Tensor, stream=None) -> None:
        """Runs of consecutive equal keys -> (key, sum of values); i32/u32/f32."""
        if keys_out.dtype != keys_in.dtype or values_out.dtype != values_in.dtype:
            raise ValueError("outputs must have their inputs' dtypes")
        if num_runs.dtype != torch.int32 or n_dev.dtype != torch.int32:
            raise ValueError("num_runs and n_dev must be int32")
        _contiguous(keys_in=keys_in, values_in=values_in, keys_out=keys_out, values_out=values_out,
                    scratch=scratch)
        _check(self.lib.mt_reduce_by_key_add(_ptr(keys_in), _ptr(values_in), _ptr(keys_out), _ptr(values_out),
                                             _ptr(num_runs), _ptr(scratch), _ptr(n_dev),
                                             DTYPE_CODE.get(keys_in.dtype, -99), DTYPE_CODE.get(values_in.dtype, -99),
                                             _stream(stream)), "mt_reduce_by_key_add")

    def mt_scan_scratch_slots(self, capacity: int, dtype, kind: int) -> int:
        code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
        r = self.lib.mt_scan_scratch_slots(int(capacity), code, int(kind))
        if r < 0:
            raise ValueError("mt_scan_scratch_slots: bad capacity, dtype or kind")
        return r

    def mt_scan_rows_scratch_slots(self, rows: int, n: int, dtype) -> int:
        """8-byte slots of look-back workspace a [rows, n] row scan of `dtype`
        takes (from the library's pool, or from mt_scan_rows_noalloc's array);
        0 when every row fits in one tile."""
        code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
        r = self.lib.mt_scan_rows_scratch_slots(int(rows), int(n), code)
        if r < 0:
            raise ValueError("mt_scan_rows_scratch_slots: bad size or dtype")
        return r

    def alloc_scratch(self, capacity: int, dtype, kind: int, device="cuda") -> torch.Tensor:
        """Caller-owned scratch of mt_scan_scratch_slots(...) 8-byte slots."""
        return torch.empty(self.mt_scan_scratch_slots(capacity, dtype, kind), dtype=torch.int64,
                           device=device)

    def mt_scan_status(self, stream=None) -> int:
        """Synchronise the stream, then read and clear the device error words."""
        return self.lib.mt_scan_status(_stream(stream))

    def mt_scan_launches(self) -> int:
        return self.lib.mt_scan_launches()

    def mt_scan_build_checked(self) -> bool:
        return bool(self.lib.mt_scan_build_checked())

    def mt_scan_debug_lookback(self, skip_publish_tile: int = -1, spin_limit: int = 0) -> None:
        self.lib.mt_scan_debug_lookback(int(skip_publish_tile), int(spin_limit))

    def mt_scan_rows_noalloc(self, inp: torch.Tensor, out: torch.Tensor, inclusive: bool, stream=None) -> None:
        """mt_scan_rows without any device allocation, for callers that may not
        allocate: the look-back records of long rows live in a fixed 1 MiB array
        inside the library. Raises ScanError(MT_ERR_TOO_LARGE) for a shape that
        needs more (mt_scan_rows_scratch_slots(rows, n, dtype) * 8 above
        MT_NOALLOC_SCRATCH_BYTES). The first long-row call in a CUDA context
        looks up that array's address there; calls that overlap on the GPU must
        not be made."""
        if inp.dim() == 1:
            rows, n = 1, inp.shape[0]
        else:
            rows, n = inp.shape
        if out.shape != inp.shape or out.dtype != inp.dtype:
            raise ValueError("out must match inp in shape and dtype")
        if not (inp.is_contiguous() and out.is_contiguous()):
            raise ValueError("inp and out must be contiguous")
        code = DTYPE_CODE.get(inp.dtype, -99)
        _check(self.lib.mt_scan_rows_noalloc(_ptr(inp), _ptr(out), rows, n, code, int(bool(inclusive)),
                                             _stream(stream)), "mt_scan_rows_noalloc")

    # ---- operators of sequence models ------------------------------------------------

    def mt_embed(self, tokens: torch.Tensor, table: torch.Tensor, out: torch.Tensor, scale: float = 1.0,
                 stream=None) -> None:
        """out[..., :] = scale * table[tokens, :]; a token outside the table (padding) gives zeros."""
        vocab, dim = table.shape
        if out.dtype != table.dtype or out.shape != tokens.shape + (dim,):
            raise ValueError("out must have table's dtype and tokens' shape with the row length added")
        if not (tokens.is_contiguous() and table.is_contiguous() and out.is_contiguous()):
            raise ValueError("tokens, table and out must be contiguous")
        _check(self.lib.mt_embed(tokens.data_ptr(), tokens.numel(), DTYPE_CODE.get(tokens.dtype, -99), table.data_ptr(),
                                 vocab, dim, DTYPE_CODE.get(table.dtype, -99), scale, out.data_ptr(), _stream(stream)),
               "mt_embed")

    def mt_embed_grad(self, tokens: torch.Tensor, dout: torch.Tensor, dtable: torch.Tensor, scratch: torch.Tensor,
                      scale: float = 1.0, accumulate: bool = False, stream=None) -> None:
        """dtable[v, :] (+)= scale * the sum of dout's rows whose token is v."""
        vocab, dim = dtable.shape
        n = tokens.numel()
        if dout.shape != tokens.shape + (dim,):
            raise ValueError("dout must have tokens' shape with dtable's row length added")
        if not (tokens.is_contiguous() and dout.is_contiguous() and dtable.is_contiguous()):
            raise ValueError("tokens, dout and dtable must be contiguous")
        _check(self.lib.mt_embed_grad(tokens.data_ptr(), n, DTYPE_CODE.get(tokens.dtype, -99), dout.data_ptr(),
                                      DTYPE_CODE.get(dout.dtype, -99), vocab, dim, scale, dtable.data_ptr(),
                                      DTYPE_CODE.get(dtable.dtype, -99), int(bool(accumulate)),
                                      _scratch("scratch", scratch, self.mt_embed_grad_scratch_slots(n, vocab, dim)),
                                      _stream(stream)), "mt_embed_grad")

    @staticmethod
    def _slots(r: int, where: str) -> int:
        if r < 0:
            raise ValueError(f"{where}: a size out of range")
        return r

    def mt_embed_grad_scratch_slots(self, ntokens: int, vocab: int, dim: int) -> int:
        return self._slots(self.lib.mt_embed_grad_scratch_slots(ntokens, vocab, dim), "mt_embed_grad_scratch_slots")

    def mt_causal_conv_grad_scratch_slots(self, batch: int, length: int, dim: int, width: int) -> int:
        return self._slots(self.lib.mt_causal_conv_grad_scratch_slots(batch, length, dim, width),
                           "mt_causal_conv_grad_scratch_slots")

    def mt_selective_scan_scratch_slots(self, batch: int, length: int, dim: int, nstate: int, groups: int = 1,
                                        grad: bool = False) -> int:
        return self._slots(self.lib.mt_selective_scan_scratch_slots(batch, length, dim, nstate, groups, int(grad)),
                           "mt_selective_scan_scratch_slots")

    def mt_selective_scan_checkpoint_slots(self, batch: int, length: int, dim: int, nstate: int) -> int:
        return self._slots(self.lib.mt_selective_scan_checkpoint_slots(batch, length, dim, nstate),
                           "mt_selective_scan_checkpoint_slots")

    def mt_causal_conv(self, x: torch.Tensor, weight: torch.Tensor, out: torch.Tensor, bias=None, silu: bool = True,
                       state=None, carry_in: bool = False, slots=None, lens=None, stream=None) -> None:
        """The convolution of whole prompts, x and out [batch, len, dim]. `state`
        [slots, width - 1, dim] is left holding each sequence's last inputs and,
        with carry_in, gives those before its first token."""
        batch, length, dim = shape = tuple(x.shape)
        dt, width = x.dtype, weight.shape[1]
        wdt = weight.dtype
        sp, nslots = _pool("state", state, (width - 1, dim), dt, batch, slots)
        _check(self.lib.mt_causal_conv(_CONV_ARGS.pack(
            DTYPE_CODE.get(dt, -99), DTYPE_CODE.get(wdt, -99), batch, length, dim, width, bool(silu), bool(carry_in), nslots,
            *_act("x", x, shape, dt), _flat("weight", weight, (dim, width), wdt), _flat("bias", bias, (dim,), wdt), sp,
            _flat("slots", slots, (batch,), torch.int32), _flat("lens", lens, (batch,), torch.int32),
            *_act("out", out, shape, dt), *_NO_ACT, *_NO_ACT, 0, 0, 0, 0), _stream(stream)), "mt_causal_conv")

    def mt_causal_conv_step(self, x: torch.Tensor, weight: torch.Tensor, state, out: torch.Tensor, bias=None,
                            silu: bool = True, slots=None, stream=None) -> None:
        """One token of each sequence: x and out [batch, dim]; state is shifted by it."""
        batch, dim = shape = tuple(x.shape)
        dt, width = x.dtype, weight.shape[1]
        wdt = weight.dtype
        sp, nslots = _pool("state", state, (width - 1, dim), dt, batch, slots)
        _check(self.lib.mt_causal_conv_step(_CONV_ARGS.pack(
            DTYPE_CODE.get(dt, -99), DTYPE_CODE.get(wdt, -99), batch, 1, dim, width, bool(silu), 0, nslots,
            *_act_step("x", x, shape, dt), _flat("weight", weight, (dim, width), wdt), _flat("bias", bias, (dim,), wdt), sp,
            _flat("slots", slots, (batch,), torch.int32), 0, *_act_step("out", out, shape, dt),
            *_NO_ACT, *_NO_ACT, 0, 0, 0, 0), _stream(stream)), "mt_causal_conv_step")

    def mt_causal_conv_grad(self, x: torch.Tensor, weight: torch.Tensor, dout: torch.Tensor, dx: torch.Tensor,
                            dweight: torch.Tensor, scratch: torch.Tensor, bias=None, dbias=None, silu: bool = True,
                            state=None, dstate=None, lens=None, stream=None) -> None:
        """Gradients of mt_causal_conv from dout. `state` is the one that the
        forward call began from (with carry_in), dstate its gradient."""
        batch, length, dim = shape = tuple(x.shape)
        dt, width = x.dtype, weight.shape[1]
        wdt = weight.dtype
        sp, nslots = _pool("state", state, (width - 1, dim), dt, batch, None)
        need = self.mt_causal_conv_grad_scratch_slots(batch, length, dim, width)
        _check(self.lib.mt_causal_conv_grad(_CONV_ARGS.pack(
            DTYPE_CODE.get(dt, -99), DTYPE_CODE.get(wdt, -99), batch, length, dim, width, bool(silu), state is not None, nslots,
            *_act("x", x, shape, dt), _flat("weight", weight, (dim, width), wdt), _flat("bias", bias, (dim,), wdt), sp,
            0, _flat("lens", lens, (batch,), torch.int32), *_NO_ACT, *_act("dout", dout, shape, dt),
            *_act("dx", dx, shape, dt), _flat("dweight", dweight, (dim, width), torch.float32),
            _flat("dbias", dbias, (dim,), torch.float32), _flat("dstate", dstate, (batch, width - 1, dim), dt),
            _scratch("scratch", scratch, need)), _stream(stream)), "mt_causal_conv_grad")

    def mt_selective_scan(self, u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                          out: torch.Tensor, scratch=None, D=None, z=None, delta_bias=None, softplus: bool = True,
                          state=None, carry_in: bool = False, slots=None, lens=None, checkpoints=None, stream=None) -> None:
        """The scan of whole prompts: u, delta, z and out [batch, len, dim], B and
        C [batch, len, groups, nstate], A [dim, nstate] f32. `state` [slots, dim,
        nstate] f32 is left holding each sequence's last state and, with carry_in,
        gives its first; `checkpoints` are written for mt_selective_scan_grad."""
        batch, length, dim = shape = tuple(u.shape)
        dt, nstate, groups = u.dtype, A.shape[1], B.shape[2]
        f32 = torch.float32
        shared = (batch, length, groups, nstate)
        sp, nslots = _pool("state", state, (dim, nstate), f32, batch, slots)
        need = self.mt_selective_scan_scratch_slots(batch, length, dim, nstate, groups)
        ck = 0
        if checkpoints is not None:
            ck = _scratch("checkpoints", checkpoints, self.mt_selective_scan_checkpoint_slots(batch, length, dim, nstate))
        _check(self.lib.mt_selective_scan(_SSM_ARGS.pack(
            DTYPE_CODE.get(dt, -99), batch, length, dim, nstate, groups, bool(softplus), bool(carry_in), nslots,
            *_act("u", u, shape, dt), *_act("delta", delta, shape, dt), *(_NO_ACT if z is None else _act("z", z, shape, dt)),
            *_act("B", B, shared, dt), *_act("C", C, shared, dt), _flat("A", A, (dim, nstate), f32), _flat("D", D, (dim,), f32),
            _flat("delta_bias", delta_bias, (dim,), f32), sp, _flat("slots", slots, (batch,), torch.int32),
            _flat("lens", lens, (batch,), torch.int32), *_act("out", out, shape, dt), ck,
            _scratch("scratch", scratch, need), *_NO_ACT * 6, 0, 0, 0, 0, 0), _stream(stream)), "mt_selective_scan")

    def mt_selective_scan_step(self, u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                               state: torch.Tensor, out: torch.Tensor, D=None, z=None, delta_bias=None,
                               softplus: bool = True, slots=None, stream=None) -> None:
        """One token of each sequence: u, delta, z and out [batch, dim], B and C
        [batch, groups, nstate]; state is updated in place."""
        batch, dim = shape = tuple(u.shape)
        dt, nstate, groups = u.dtype, A.shape[1], B.shape[1]
        f32 = torch.float32
        shared = (batch, groups, nstate)
        sp, nslots = _pool("state", state, (dim, nstate), f32, batch, slots)
        _check(self.lib.mt_selective_scan_step(_SSM_ARGS.pack(
            DTYPE_CODE.get(dt, -99), batch, 1, dim, nstate, groups, bool(softplus), 0, nslots,
            *_act_step("u", u, shape, dt), *_act_step("delta", delta, shape, dt),
            *(_NO_ACT if z is None else _act_step("z", z, shape, dt)), *_act_step("B", B, shared, dt),
            *_act_step("C", C, shared, dt), _flat("A", A, (dim, nstate), f32), _flat("D", D, (dim,), f32),
            _flat("delta_bias", delta_bias, (dim,), f32), sp, _flat("slots", slots, (batch,), torch.int32), 0,
            *_act_step("out", out, shape, dt), 0, 0, *_NO_ACT * 6, 0, 0, 0, 0, 0), _stream(stream)), "mt_selective_scan_step")

    def mt_selective_scan_grad(self, u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                               dout: torch.Tensor, checkpoints: torch.Tensor, du: torch.Tensor, ddelta: torch.Tensor,
                               dA: torch.Tensor, dB: torch.Tensor, dC: torch.Tensor, scratch: torch.Tensor, D=None, dD=None,
                               z=None, dz=None, delta_bias=None, ddelta_bias=None, softplus: bool = True, dfinal=None,
                               dinit=None, lens=None, stream=None) -> None:
        """Every gradient of mt_selective_scan from dout and dfinal (the gradient of
        the last states), with the checkpoints that the forward call wrote."""
        batch, length, dim = shape = tuple(u.shape)
        dt, nstate, groups = u.dtype, A.shape[1], B.shape[2]
        f32 = torch.float32
        shared, states = (batch, length, groups, nstate), (batch, dim, nstate)
        if z is not None and dz is None:
            raise ValueError("dz is needed with z")
        need = self.mt_selective_scan_scratch_slots(batch, length, dim, nstate, groups, True)
        ck = _scratch("checkpoints", checkpoints, self.mt_selective_scan_checkpoint_slots(batch, length, dim, nstate))
        _check(self.lib.mt_selective_scan_grad(_SSM_ARGS.pack(
            DTYPE_CODE.get(dt, -99), batch, length, dim, nstate, groups, bool(softplus), 0, batch,
            *_act("u", u, shape, dt), *_act("delta", delta, shape, dt), *(_NO_ACT if z is None else _act("z", z, shape, dt)),
            *_act("B", B, shared, dt), *_act("C", C, shared, dt), _flat("A", A, (dim, nstate), f32), _flat("D", D, (dim,), f32),
            _flat("delta_bias", delta_bias, (dim,), f32), 0, 0, _flat("lens", lens, (batch,), torch.int32), *_NO_ACT, ck,
            _scratch("scratch", scratch, need), *_act("dout", dout, shape, dt), *_act("du", du, shape, dt),
            *_act("ddelta", ddelta, shape, dt), *(_NO_ACT if z is None else _act("dz", dz, shape, dt)),
            *_act("dB", dB, shared, dt), *_act("dC", dC, shared, dt), _flat("dA", dA, (dim, nstate), f32),
            _flat("dD", dD, (dim,), f32), _flat("ddelta_bias", ddelta_bias, (dim,), f32), _flat("dfinal", dfinal, states, f32),
            _flat("dinit", dinit, states, f32)), _stream(stream)), "mt_selective_scan_grad")


_default = Library(LIB_PATH)
lib = _default.lib
mt_scan_strerror = _default.mt_scan_strerror
mt_scan_rows = _default.mt_scan_rows
mt_scan_rows_op = _default.mt_scan_rows_op
mt_exclusive_scan = _default.mt_exclusive_scan
mt_inclusive_scan = _default.mt_inclusive_scan
mt_reduce = _default.mt_reduce
mt_select = _default.mt_select
mt_select_wide = _default.mt_select_wide
mt_reduce_by_key_add = _default.mt_reduce_by_key_add
mt_scan_scratch_slots = _default.mt_scan_scratch_slots
mt_scan_rows_scratch_slots = _default.mt_scan_rows_scratch_slots
alloc_scratch = _default.alloc_scratch
mt_scan_status = _default.mt_scan_status
mt_scan_launches = _default.mt_scan_launches
mt_scan_build_checked = _default.mt_scan_build_checked
mt_scan_debug_lookback = _default.mt_scan_debug_lookback
mt_scan_rows_noalloc = _default.mt_scan_rows_noalloc
mt_embed = _default.mt_embed
mt_embed_grad = _default.mt_embed_grad
mt_embed_grad_scratch_slots = _default.mt_embed_grad_scratch_slots
mt_causal_conv = _default.mt_causal_conv
mt_causal_conv_step = _default.mt_causal_conv_step
mt_causal_conv_grad = _default.mt_causal_conv_grad
mt_causal_conv_grad_scratch_slots = _default.mt_causal_conv_grad_scratch_slots
mt_selective_scan = _default.mt_selective_scan
mt_selective_scan_step = _default.mt_selective_scan_step
mt_selective_scan_grad = _default.mt_selective_scan_grad
mt_selective_scan_scratch_slots = _default.mt_selective_scan_scratch_slots
mt_selective_scan_checkpoint_slots = _default.mt_selective_scan_checkpoint_slots


def load_checked() -> Library:
    """The bounds-checked build (libmtscan_checked.so): the same calls, whose
    kernels check every store and shared-memory access against its buffer
    and report a bad one as MT_ERR_BOUNDS through mt_scan_status() instead of
    making it. For tests and debugging."""
    return Library(LIB_CHECKED_PATH)
