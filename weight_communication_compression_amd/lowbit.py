"""Thin ctypes binding of liblowbit (the C ABI in ``include/lowbit.h`` and, for
the training-step operators, ``include/lowbit_train.h``).

Argument marshalling only: every step runs in the gfx950 HIP kernels behind the
C ABI.  torch is used for device memory (tensors) and for
the current HIP stream.  If the library is missing or a call fails, a
``LowbitError`` is raised -- there is no CPU fallback.

Wire format of the returned tensors:
  codes  -- torch.int32 holding the packed uint32 words (bit patterns)
  scales -- torch.float16, one binary16 scale per block
"""
from __future__ import annotations

import ctypes
import os
import warnings
from typing import NamedTuple, Optional, Sequence

import torch

__all__ = [
    "LowbitError", "lib", "library_path", "num_words", "num_blocks", "QParams",
    "quantize_pack", "unpack_dequant", "ef_compress", "reduce_requant",
    "wdiff_compress", "wdiff_apply", "copy_f32", "xor_streams", "add_inplace_f32", "fold_f32",
    "dropout", "dropout_backward", "block_join", "block_join_backward", "BlockJoin",
    "BlockJoinGrads", "JoinParams", "linear_xent", "linear_xent_backward", "LinearXent",
    "LinearXentGrads", "XentParams",
    "stream_probe", "PROBE_READ", "PROBE_WRITE", "PROBE_COPY",
    "OK", "EINVAL", "EUNSUPPORTED", "EDEVICE", "F32", "BF16", "HINT_INPUT_REUSED",
]

OK, EINVAL, EUNSUPPORTED, EDEVICE = 0, 1, 2, 3
PROBE_READ, PROBE_WRITE, PROBE_COPY = 0, 1, 2
F32, BF16 = 0, 1
HINT_INPUT_REUSED = 1        # lowbit_qparams.hints: the input is read again soon

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "liblowbit.so")


class LowbitError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        name = {1: "invalid argument", 2: "unsupported combination",
                3: "device launch error"}.get(status, f"status {status}")
        super().__init__(f"{what}: {name}")


class QParams(ctypes.Structure):
    """lowbit_qparams"""
    _fields_ = [("bitwidth", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("stochastic", ctypes.c_int32), ("hints", ctypes.c_int32),
                ("seed", ctypes.c_uint64), ("index_offset", ctypes.c_uint64)]


class JoinParams(ctypes.Structure):
    """lowbit_join_params"""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("rows_per_gate", ctypes.c_int64), ("norm", ctypes.c_int32),
                ("block_type", ctypes.c_int32), ("stream_type", ctypes.c_int32),
                ("param_type", ctypes.c_int32), ("eps", ctypes.c_float),
                ("residual_scale", ctypes.c_float), ("p", ctypes.c_double),
                ("seed", ctypes.c_uint64)]


class XentParams(ctypes.Structure):
    """lowbit_xent_params"""
    _fields_ = [("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("hidden", ctypes.c_int64),
                ("ignore_index", ctypes.c_int64), ("type", ctypes.c_int32)]


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Load liblowbit.so (built in-tree by ``build.py``); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise LowbitError(-1, f"{library_path} is not built (run __graft_entry__.build())")
        L = ctypes.CDLL(library_path)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        f64, u64 = ctypes.c_double, ctypes.c_uint64
        QP, JP = ctypes.POINTER(QParams), ctypes.POINTER(JoinParams)
        XP = ctypes.POINTER(XentParams)
        sigs = {
            "lowbit_num_words": (i64, [i64, i32]),
            "lowbit_num_blocks": (i64, [i64, i32]),
            "lowbit_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "lowbit_version": (ctypes.c_char_p, []),
            "lowbit_quantize_pack": (ctypes.c_int, [P, ctypes.c_int, i64, QP, P, P, P]),
            "lowbit_unpack_dequant": (ctypes.c_int, [P, P, i64, QP, P, P]),
            "lowbit_ef_compress": (ctypes.c_int, [P, ctypes.c_int, P, i64, QP, P, P, P]),
            "lowbit_ef21_compress": (ctypes.c_int, [P, ctypes.c_int, P, i64, QP, P, P, P]),
            "lowbit_hadamard_quantize_pack": (ctypes.c_int, [P, ctypes.c_int, i64, QP, P, P, P]),
            "lowbit_hadamard_unpack_dequant": (ctypes.c_int, [P, P, i64, QP, P, P]),
            "lowbit_reduce_requant": (ctypes.c_int, [P, P, i32, i64, QP, QP, P, P, P, P]),
            "lowbit_reduce_requant_ef": (ctypes.c_int, [P, P, i32, i64, QP, QP, P, P, P, P, P]),
            "lowbit_wdiff_compress": (ctypes.c_int, [P, P, ctypes.c_int, i64, QP, P, P, P]),
            "lowbit_wdiff_apply": (ctypes.c_int, [P, P, P, i64, QP, P, ctypes.c_int, P]),
            "lowbit_copy_f32": (ctypes.c_int, [P, P, i64, P]),
            "lowbit_xor_streams_u32": (ctypes.c_int, [P, i32, i64, P, P]),
            "lowbit_add_inplace_f32": (ctypes.c_int, [P, P, i64, P]),
            "lowbit_fold_f32": (ctypes.c_int, [P, i64, i32, P, P]),
            "lowbit_dropout": (ctypes.c_int, [P, P, ctypes.c_int, i64, f64, u64, u64, P, P]),
            "lowbit_dropout_backward": (ctypes.c_int, [P, ctypes.c_int, i64, f64, u64, u64, P, P]),
            "lowbit_block_join": (ctypes.c_int, [P] * 7 + [JP] + [P] * 4),
            "lowbit_block_join_backward_workspace": (i64, [JP]),
            "lowbit_block_join_backward": (ctypes.c_int, [P] * 9 + [JP] + [P] * 8 + [i64, P]),
            "lowbit_linear_xent_workspace": (i64, [XP, i32]),
            "lowbit_linear_xent": (ctypes.c_int, [P, P, P, XP, P, P, P, i64, P]),
            "lowbit_linear_xent_backward": (ctypes.c_int, [P] * 6 + [XP] + [P] * 3 + [i64, P]),
            "lowbit_stream_probe_u32": (ctypes.c_int, [i32, P, P, i64, ctypes.c_uint32, i32, i32, P]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def num_words(n: int, bitwidth: int) -> int:
    v = lib().lowbit_num_words(n, bitwidth)
    if v < 0:
        raise LowbitError(EINVAL, "num_words")
    return int(v)


def num_blocks(n: int, block_size: int) -> int:
    v = lib().lowbit_num_blocks(n, block_size)
    if v < 0:
        raise LowbitError(EINVAL, "num_blocks")
    return int(v)


# ------------------------------------------------------------ marshalling --
def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise LowbitError(EINVAL, f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _dev(t: torch.Tensor, what: str) -> int:
    if not t.is_cuda:
        raise LowbitError(EINVAL, f"{what} must be a GPU tensor")
    if not t.is_contiguous():
        raise LowbitError(EINVAL, f"{what} must be contiguous")
    return t.data_ptr()


# The current stream's handle without the Stream object around it (0.15 instead of
# 2 us a call); torch versions without it take the long way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor) -> int:
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _qp(bitwidth, block_size, stochastic=False, seed=0, index_offset=0, hints=0) -> QParams:
    return QParams(int(bitwidth), int(block_size), int(bool(stochastic)), int(hints),
                   int(seed) & (2 ** 64 - 1), int(index_offset))


def _check(status: int, what: str) -> None:
    if status != OK:
        raise LowbitError(status, what)


def _need_codes(t: torch.Tensor, n: int, bitwidth: int, what: str) -> None:
    if t.dtype != torch.int32 or t.numel() < num_words(n, bitwidth):
        raise LowbitError(EINVAL, f"{what} must be int32 with >= {num_words(n, bitwidth)} words")


def _need_scales(t: torch.Tensor, n: int, block_size: int, what: str) -> None:
    if t.dtype != torch.float16 or t.numel() < num_blocks(n, block_size):
        raise LowbitError(EINVAL,
                          f"{what} must be float16 with >= {num_blocks(n, block_size)} entries")


def _out_codes(n, bitwidth, like, codes):
    if codes is None:
        codes = torch.empty(num_words(n, bitwidth), dtype=torch.int32, device=like.device)
    _need_codes(codes, n, bitwidth, "codes")
    return codes


def _out_scales(n, block_size, like, scales):
    if scales is None:
        scales = torch.empty(num_blocks(n, block_size), dtype=torch.float16, device=like.device)
    _need_scales(scales, n, block_size, "scales")
    return scales


# -------------------------------------------------------------- the codec --
def quantize_pack(x: torch.Tensor, bitwidth: int, block_size: int, stochastic: bool = False,
                  seed: int = 0, index_offset: int = 0, codes: Optional[torch.Tensor] = None,
                  scales: Optional[torch.Tensor] = None, input_reused: bool = False):
    """Compress x (float32 or bfloat16) -> (codes int32[num_words], scales float16[num_blocks]).

    input_reused: the caller reads x again soon (LOWBIT_HINT_INPUT_REUSED), so
    it is kept in the caches rather than streamed."""
    n = x.numel()
    codes = _out_codes(n, bitwidth, x, codes)
    scales = _out_scales(n, block_size, x, scales)
    qp = _qp(bitwidth, block_size, stochastic, seed, index_offset,
             HINT_INPUT_REUSED if input_reused else 0)
    _check(lib().lowbit_quantize_pack(_dev(x, "x"), _dtype_code(x), n, ctypes.byref(qp),
                                      _dev(codes, "codes"), _dev(scales, "scales"), _stream(x)),
           "lowbit_quantize_pack")
    return codes, scales


def unpack_dequant(codes: torch.Tensor, scales: torch.Tensor, n: int, bitwidth: int,
                   block_size: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Decompress -> float32[n]."""
    _need_codes(codes, n, bitwidth, "codes")
    _need_scales(scales, n, block_size, "scales")
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=codes.device)
    if out.dtype != torch.float32 or out.numel() < n:
        raise LowbitError(EINVAL, "out must be float32 with >= n elements")
    qp = _qp(bitwidth, block_size)
    _check(lib().lowbit_unpack_dequant(_dev(codes, "codes"), _dev(scales, "scales"), n,
                                       ctypes.byref(qp), _dev(out, "out"), _stream(codes)),
           "lowbit_unpack_dequant")
    return out


def hadamard_quantize_pack(x: torch.Tensor, bitwidth: int, block_size: int,
                           stochastic: bool = False, seed: int = 0, index_offset: int = 0,
                           codes: Optional[torch.Tensor] = None,
                           scales: Optional[torch.Tensor] = None, input_reused: bool = False):
    """Blockwise Walsh-Hadamard transform of x, then compress; a partial last
    block (x.numel() not a multiple of block_size) is compressed untransformed.

    input_reused: as for quantize_pack (LOWBIT_HINT_INPUT_REUSED)."""
    n = x.numel()
    codes = _out_codes(n, bitwidth, x, codes)
    scales = _out_scales(n, block_size, x, scales)
    qp = _qp(bitwidth, block_size, stochastic, seed, index_offset,
             HINT_INPUT_REUSED if input_reused else 0)
    _check(lib().lowbit_hadamard_quantize_pack(_dev(x, "x"), _dtype_code(x), n, ctypes.byref(qp),
                                               _dev(codes, "codes"), _dev(scales, "scales"),
                                               _stream(x)), "lowbit_hadamard_quantize_pack")
    return codes, scales


def hadamard_unpack_dequant(codes: torch.Tensor, scales: torch.Tensor, n: int, bitwidth: int,
                            block_size: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Decompress, then the inverse blockwise transform -> float32[n]."""
    _need_codes(codes, n, bitwidth, "codes")
    _need_scales(scales, n, block_size, "scales")
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=codes.device)
    if out.dtype != torch.float32 or out.numel() < n:
        raise LowbitError(EINVAL, "out must be float32 with >= n elements")
    qp = _qp(bitwidth, block_size)
    _check(lib().lowbit_hadamard_unpack_dequant(_dev(codes, "codes"), _dev(scales, "scales"), n,
                                                ctypes.byref(qp), _dev(out, "out"),
                                                _stream(codes)), "lowbit_hadamard_unpack_dequant")
    return out


def ef_compress(g: torch.Tensor, residual: torch.Tensor, bitwidth: int, block_size: int,
                stochastic: bool = False, seed: int = 0, index_offset: int = 0,
                codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
    """Error-feedback compress; `residual` (float32[n]) is updated in place."""
    n = g.numel()
    if residual.dtype != torch.float32 or residual.numel() != n:
        raise LowbitError(EINVAL, "residual must be float32 with g.numel() elements")
    codes = _out_codes(n, bitwidth, g, codes)
    scales = _out_scales(n, block_size, g, scales)
    qp = _qp(bitwidth, block_size, stochastic, seed, index_offset)
    _check(lib().lowbit_ef_compress(_dev(g, "g"), _dtype_code(g), _dev(residual, "residual"), n,
                                    ctypes.byref(qp), _dev(codes, "codes"),
                                    _dev(scales, "scales"), _stream(g)), "lowbit_ef_compress")
    return codes, scales


def ef21_compress(g: torch.Tensor, state: torch.Tensor, bitwidth: int, block_size: int,
                  stochastic: bool = False, seed: int = 0, index_offset: int = 0,
                  codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
    """EF21 compress of g - state; `state` (float32[n]) becomes state + deq, in place."""
    n = g.numel()
    if state.dtype != torch.float32 or state.numel() != n:
        raise LowbitError(EINVAL, "state must be float32 with g.numel() elements")
    codes = _out_codes(n, bitwidth, g, codes)
    scales = _out_scales(n, block_size, g, scales)
    qp = _qp(bitwidth, block_size, stochastic, seed, index_offset)
    _check(lib().lowbit_ef21_compress(_dev(g, "g"), _dtype_code(g), _dev(state, "state"), n,
                                      ctypes.byref(qp), _dev(codes, "codes"),
                                      _dev(scales, "scales"), _stream(g)), "lowbit_ef21_compress")
    return codes, scales


def _reduce(peer_codes, peer_scales, n, bitwidth, block_size, stochastic, seed, index_offset,
            out_codes, out_scales, out_sum, want_sum, out_bitwidth, out_block_size, residual,
            input_reused=False):
    P = len(peer_codes)
    if P != len(peer_scales):
        raise LowbitError(EINVAL, "peer_codes and peer_scales differ in length")
    if P < 1:
        raise LowbitError(EINVAL, "reduce_requant needs at least one peer")
    ob = bitwidth if out_bitwidth is None else out_bitwidth
    oB = block_size if out_block_size is None else out_block_size
    for c, sc in zip(peer_codes, peer_scales):
        _need_codes(c, n, bitwidth, "peer codes")
        _need_scales(sc, n, block_size, "peer scales")
    like = peer_codes[0]
    out_codes = _out_codes(n, ob, like, out_codes)
    out_scales = _out_scales(n, oB, like, out_scales)
    if want_sum and out_sum is None:
        out_sum = torch.empty(n, dtype=torch.float32, device=like.device)
    if out_sum is not None and (out_sum.dtype != torch.float32 or out_sum.numel() < n):
        raise LowbitError(EINVAL, "out_sum must be float32 with >= n elements")
    cp = (ctypes.c_void_p * P)(*[_dev(c, "peer codes") for c in peer_codes])
    sp = (ctypes.c_void_p * P)(*[_dev(s, "peer scales") for s in peer_scales])
    qi = _qp(bitwidth, block_size, hints=HINT_INPUT_REUSED if input_reused else 0)
    qo = _qp(ob, oB, stochastic, seed, index_offset)
    tail = (_dev(out_codes, "out_codes"), _dev(out_scales, "out_scales"),
            _dev(out_sum, "out_sum") if out_sum is not None else None, _stream(like))
    if residual is None:
        _check(lib().lowbit_reduce_requant(ctypes.cast(cp, ctypes.c_void_p),
                                           ctypes.cast(sp, ctypes.c_void_p), P, n,
                                           ctypes.byref(qi), ctypes.byref(qo), *tail),
               "lowbit_reduce_requant")
    else:
        if residual.dtype != torch.float32 or residual.numel() != n:
            raise LowbitError(EINVAL, "residual must be float32 with n elements")
        _check(lib().lowbit_reduce_requant_ef(ctypes.cast(cp, ctypes.c_void_p),
                                              ctypes.cast(sp, ctypes.c_void_p), P, n,
                                              ctypes.byref(qi), ctypes.byref(qo),
                                              _dev(residual, "residual"), *tail),
               "lowbit_reduce_requant_ef")
    return out_codes, out_scales, out_sum


def reduce_requant(peer_codes: Sequence[torch.Tensor], peer_scales: Sequence[torch.Tensor],
                   n: int, bitwidth: int, block_size: int, stochastic: bool = False,
                   seed: int = 0, index_offset: int = 0, out_codes=None, out_scales=None,
                   out_sum=None, want_sum: bool = False, out_bitwidth: Optional[int] = None,
                   out_block_size: Optional[int] = None, input_reused: bool = False):
    """Local reduce: dequantize npeers chunks packed with (bitwidth,
    block_size), sum in peer order, requantize with (out_bitwidth,
    out_block_size) (default: the same) and the rounding options.
    input_reused: the caller reads the peers' codes again soon
    (LOWBIT_HINT_INPUT_REUSED), so they are not streamed; results are the same.

    Returns (codes, scales, sum_or_None)."""
    return _reduce(peer_codes, peer_scales, n, bitwidth, block_size, stochastic, seed,
                   index_offset, out_codes, out_scales, out_sum, want_sum, out_bitwidth,
                   out_block_size, None, input_reused)


def reduce_requant_ef(peer_codes: Sequence[torch.Tensor], peer_scales: Sequence[torch.Tensor],
                      n: int, bitwidth: int, block_size: int, residual: torch.Tensor,
                      stochastic: bool = False, seed: int = 0, index_offset: int = 0,
                      out_codes=None, out_scales=None, out_sum=None, want_sum: bool = False,
                      out_bitwidth: Optional[int] = None, out_block_size: Optional[int] = None,
                      input_reused: bool = False):
    """Local reduce with stage-2 error feedback: the sum plus `residual`
    (float32[n], updated in place) is requantized.  Returns (codes, scales,
    sum_or_None); the sum is taken before the residual is added.
    input_reused: as for reduce_requant."""
    if residual is None:
        raise LowbitError(EINVAL, "reduce_requant_ef needs a residual")
    return _reduce(peer_codes, peer_scales, n, bitwidth, block_size, stochastic, seed,
                   index_offset, out_codes, out_scales, out_sum, want_sum, out_bitwidth,
                   out_block_size, residual, input_reused)


def wdiff_compress(w_new: torch.Tensor, w_old: torch.Tensor, bitwidth: int, block_size: int,
                   stochastic: bool = False, seed: int = 0, index_offset: int = 0,
                   codes=None, scales=None):
    """Compress the weight difference w_new - w_old."""
    n = w_new.numel()
    if w_old.dtype != w_new.dtype or w_old.numel() != n:
        raise LowbitError(EINVAL, "w_new and w_old must match in dtype and size")
    codes = _out_codes(n, bitwidth, w_new, codes)
    scales = _out_scales(n, block_size, w_new, scales)
    qp = _qp(bitwidth, block_size, stochastic, seed, index_offset)
    _check(lib().lowbit_wdiff_compress(_dev(w_new, "w_new"), _dev(w_old, "w_old"),
                                       _dtype_code(w_new), n, ctypes.byref(qp),
                                       _dev(codes, "codes"), _dev(scales, "scales"),
                                       _stream(w_new)), "lowbit_wdiff_compress")
    return codes, scales


def wdiff_apply(w_old: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, bitwidth: int,
                block_size: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """w_out = w_old + deq (rounded to w_old's dtype); `out` may be w_old itself."""
    n = w_old.numel()
    _need_codes(codes, n, bitwidth, "codes")
    _need_scales(scales, n, block_size, "scales")
    if out is None:
        out = torch.empty_like(w_old)
    if out.dtype != w_old.dtype or out.numel() != n:
        raise LowbitError(EINVAL, "out must match w_old")
    qp = _qp(bitwidth, block_size)
    _check(lib().lowbit_wdiff_apply(_dev(w_old, "w_old"), _dev(codes, "codes"),
                                    _dev(scales, "scales"), n, ctypes.byref(qp),
                                    _dev(out, "out"), _dtype_code(w_old), _stream(w_old)),
           "lowbit_wdiff_apply")
    return out


def copy_f32(x: torch.Tensor, y: torch.Tensor) -> torch.Tensor:
    """Plain float32 copy kernel (bandwidth reference, not a codec step)."""
    if x.dtype != torch.float32 or y.dtype != torch.float32 or y.numel() != x.numel():
        raise LowbitError(EINVAL, "copy_f32 needs two float32 tensors of equal size")
    _check(lib().lowbit_copy_f32(_dev(x, "x"), _dev(y, "y"), x.numel(), _stream(x)),
           "lowbit_copy_f32")
    return y


def add_inplace_f32(x: torch.Tensor, y: torch.Tensor) -> torch.Tensor:
    """y += x in place (float32), with the error-feedback compress's access
    pattern (bandwidth reference for that kernel, not a codec step)."""
    if x.dtype != torch.float32 or y.dtype != torch.float32 or y.numel() != x.numel():
        raise LowbitError(EINVAL, "add_inplace_f32 needs two float32 tensors of equal size")
    _check(lib().lowbit_add_inplace_f32(_dev(x, "x"), _dev(y, "y"), x.numel(), _stream(y)),
           "lowbit_add_inplace_f32")
    return y


def xor_streams(streams: Sequence[torch.Tensor], out: torch.Tensor) -> torch.Tensor:
    """out = XOR of the int32 streams, read with the local reduce's access
    pattern (bandwidth reference for the reduce, not a codec step)."""
    P = len(streams)
    n = out.numel()
    if out.dtype != torch.int32 or any(t.dtype != torch.int32 or t.numel() != n for t in streams):
        raise LowbitError(EINVAL, "xor_streams needs int32 tensors of equal size")
    if not 1 <= P <= 16:
        raise LowbitError(EINVAL, "xor_streams needs 1 to 16 streams")
    sp = (ctypes.c_void_p * P)(*[_dev(t, "stream") for t in streams])
    _check(lib().lowbit_xor_streams_u32(ctypes.cast(sp, ctypes.c_void_p), P, n, _dev(out, "out"),
                                        _stream(out)), "lowbit_xor_streams_u32")
    return out


def fold_f32(x: torch.Tensor, bitwidth: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Compress-volume bandwidth reference (not a codec step): reads the
    float32 x, writes num_words(x.numel(), bitwidth) int32 words of XOR folds."""
    if x.dtype != torch.float32:
        raise LowbitError(EINVAL, "fold_f32 needs a float32 tensor")
    n = x.numel()
    nw = num_words(n, bitwidth)
    if out is None:
        out = torch.empty(nw, dtype=torch.int32, device=x.device)
    elif out.dtype != torch.int32 or out.numel() < nw:
        raise LowbitError(EINVAL, f"out must be int32 with >= {nw} words")
    _check(lib().lowbit_fold_f32(_dev(x, "x"), n, int(bitwidth), _dev(out, "out"), _stream(x)),
           "lowbit_fold_f32")
    return out


def stream_probe(op: int, dst: torch.Tensor, src: Optional[torch.Tensor] = None, value: int = 0,
                 waves: int = 0, nontemporal: bool = True) -> torch.Tensor:
    """Memory-system probe (not a codec step), on int32 tensors viewed as
    32-bit words: PROBE_READ writes dst[t] = XOR of trip t (1024 words) of
    src, PROBE_WRITE dst[i] = i ^ value, PROBE_COPY dst = src.  waves = 0:
    one trip per wave; > 0: a persistent grid of that many waves."""
    nwords = src.numel() if op != PROBE_WRITE else dst.numel()
    for t, name in ((dst, "dst"), (src, "src")):
        if t is not None and t.dtype != torch.int32:
            raise LowbitError(EINVAL, f"{name} must be int32")
    if op == PROBE_READ and dst.numel() < nwords // 1024:
        raise LowbitError(EINVAL, "dst too small")
    if op == PROBE_COPY and dst.numel() < nwords:
        raise LowbitError(EINVAL, "dst too small")
    sp = _dev(src, "src") if src is not None else None
    _check(lib().lowbit_stream_probe_u32(int(op), sp, _dev(dst, "dst"), nwords,
                                         int(value) & 0xFFFFFFFF, int(waves), int(bool(nontemporal)),
                                         _stream(dst)), "lowbit_stream_probe_u32")
    return dst


# ------------------------------------------------ training-step operators --
# Plain calls outside torch's autograd, each with its gradient as a call of its own.
_U64 = 2 ** 64 - 1
_NORMS = {"rms": 0, "layer": 1}


def _opt(t: Optional[torch.Tensor], what: str) -> Optional[int]:
    return None if t is None else _dev(t, what)


def _out_like(t: torch.Tensor, out: Optional[torch.Tensor], what: str) -> torch.Tensor:
    if out is None:
        return torch.empty_like(t)
    if out.dtype != t.dtype or out.numel() != t.numel() or out.device != t.device:
        raise LowbitError(EINVAL, f"{what} must match the input in dtype, size and device")
    return out


def _outside_autograd(name: str) -> None:
    """For inputs that require a gradient: where torch would record a call, says that this one
    is not."""
    if torch.is_grad_enabled():
        warnings.warn(f"{name} is not recorded for torch's backward pass: no gradient reaches its "
                      f"inputs through its outputs.  Take it from {name}_backward (and call under "
                      "torch.no_grad(), which also silences this)", stacklevel=3)


def _scratch(nbytes: int, like: torch.Tensor, workspace: Optional[torch.Tensor], what: str):
    """The workspace given, or one of nbytes from torch's allocator."""
    if nbytes < 0:
        raise LowbitError(EINVAL, what)
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    if workspace.dtype != torch.uint8 or workspace.numel() < nbytes \
            or workspace.device != like.device:
        raise LowbitError(EINVAL, f"workspace must be uint8 with >= {nbytes} elements")
    return workspace


def dropout(x: torch.Tensor, p: float, seed: int, residual: Optional[torch.Tensor] = None,
            index_offset: int = 0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """residual + D(x) (or D(x)) of float32 or bfloat16 tensors: elements are
    dropped with probability p, rounded to a multiple of 2^-16, by a mask that
    seed alone fixes and that is never stored; the others are divided by 1 - p.

    index_offset (a multiple of 8): the mask's index of element 0, for a tensor
    that is a piece of a larger one.  `out` may be x or residual."""
    if x.requires_grad or (residual is not None and residual.requires_grad):
        _outside_autograd("dropout")
    if residual is not None and (residual.dtype != x.dtype or residual.numel() != x.numel()
                                 or residual.device != x.device):
        raise LowbitError(EINVAL, "residual must match x in dtype, size and device")
    dt = _dtype_code(x)
    out = _out_like(x, out, "out")
    _check(lib().lowbit_dropout(_dev(x, "x"), _opt(residual, "residual"), dt, x.numel(), p,
                                int(seed) & _U64, int(index_offset), _dev(out, "out"), _stream(x)),
           "lowbit_dropout")
    return out


def dropout_backward(dy: torch.Tensor, p: float, seed: int, index_offset: int = 0,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of `dropout` by x, with its p, seed and index_offset: D(dy).
    (The residual's gradient is dy.)  `out` may be dy."""
    dt = _dtype_code(dy)
    out = _out_like(dy, out, "out")
    _check(lib().lowbit_dropout_backward(_dev(dy, "dy"), dt, dy.numel(), p, int(seed) & _U64,
                                         int(index_offset), _dev(out, "out"), _stream(dy)),
           "lowbit_dropout_backward")
    return out


class BlockJoin(NamedTuple):
    """What block_join returns; stats is float32 (rows, 4)."""
    x_out: torch.Tensor
    z: torch.Tensor
    stats: torch.Tensor


class BlockJoinGrads(NamedTuple):
    """What block_join_backward returns; the parameters' gradients are float32,
    None for parameters that were not given."""
    df: torch.Tensor
    dx: torch.Tensor
    dpost_weight: Optional[torch.Tensor]
    dpost_bias: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dpre_weight: Optional[torch.Tensor]
    dpre_bias: Optional[torch.Tensor]


def _join_params(f, x, named, rows_per_gate, norm, residual_scale, eps, p, seed) -> JoinParams:
    """Checks of the tensors' types and sizes, which the C ABI cannot see."""
    if f.dim() < 1 or f.shape != x.shape:
        raise LowbitError(EINVAL, "f and x must have the same shape, (..., columns)")
    cols = f.shape[-1]
    rows = f.numel() // cols if cols else 0
    if norm not in _NORMS:
        raise LowbitError(EINVAL, "norm must be 'rms' or 'layer'")
    rows_per_gate = int(rows_per_gate)
    device = f.device
    pt = None
    for name, t in named:
        if t is None:
            continue
        if t.device != device or (pt is not None and t.dtype != pt):
            raise LowbitError(EINVAL, "weights, biases and gate must have one dtype and f's device")
        pt = t.dtype
        want = cols
        if name == "gate":
            if rows_per_gate < 1:
                raise LowbitError(EINVAL, "a gate needs rows_per_gate >= 1")
            want = -(-rows // rows_per_gate) * cols
        if t.numel() != want:
            raise LowbitError(EINVAL, f"{name} must have {want} elements")
    if x.device != device:
        raise LowbitError(EINVAL, "f and x must be on one device")
    ft = _dtype_code(f)
    # (more rows a gate than there are: one gate; as a larger number 64 bits may not hold it)
    return JoinParams(rows, cols, min(rows_per_gate, max(rows, 1)), _NORMS[norm], ft, _dtype_code(x),
                      ft if pt is None else (F32 if pt == torch.float32 else
                                             BF16 if pt == torch.bfloat16 else -1),
                      eps, residual_scale, p, int(seed) & _U64)


def block_join(f: torch.Tensor, x: torch.Tensor, post_weight: Optional[torch.Tensor] = None,
               post_bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
               rows_per_gate: int = 0, pre_weight: Optional[torch.Tensor] = None,
               pre_bias: Optional[torch.Tensor] = None, norm: str = "rms",
               residual_scale: float = 1.0, eps: float = 1e-6, p: float = 0.0, seed: int = 0,
               x_out: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None) -> BlockJoin:
    """What stands between two blocks of a residual network, in one pass:

        x_out = residual_scale * x + gate * D(norm(f) * post_weight + post_bias)
        z     = norm(x_out) * pre_weight + pre_bias

    f (..., columns): a block's output; x: the residual stream, of f's dtype or
    float32; z: the next block's input, of f's dtype.  Weights and biases
    (columns), gate (ceil(rows / rows_per_gate), columns): of f's dtype or
    float32, all the same; absent ones are 1 and 0.  norm: "rms" or "layer".
    p, seed: dropout as by `dropout`, each row beginning at an even draw.
    `x_out` may be x, `z` may be f.  stats feeds block_join_backward."""
    named = (("post_weight", post_weight), ("post_bias", post_bias), ("gate", gate),
             ("pre_weight", pre_weight), ("pre_bias", pre_bias))
    for t in (f, x, post_weight, post_bias, gate, pre_weight, pre_bias):
        if t is not None and t.requires_grad:
            _outside_autograd("block_join")
            break
    q = _join_params(f, x, named, rows_per_gate, norm, residual_scale, eps, p, seed)
    x_out = _out_like(x, x_out, "x_out")
    z = _out_like(f, z, "z")
    stats = torch.empty(q.rows, 4, dtype=torch.float32, device=f.device)
    _check(lib().lowbit_block_join(_dev(f, "f"), _dev(x, "x"), *[_opt(t, n) for n, t in named], q,
                                   _dev(x_out, "x_out"), _dev(z, "z"), _dev(stats, "stats"),
                                   _stream(f)), "lowbit_block_join")
    return BlockJoin(x_out, z, stats)


def block_join_backward(dx_out: torch.Tensor, dz: torch.Tensor, f: torch.Tensor,
                        x_out: torch.Tensor, stats: torch.Tensor,
                        post_weight: Optional[torch.Tensor] = None,
                        post_bias: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None, rows_per_gate: int = 0,
                        pre_weight: Optional[torch.Tensor] = None,
                        pre_bias: Optional[torch.Tensor] = None, norm: str = "rms",
                        residual_scale: float = 1.0, eps: float = 1e-6, p: float = 0.0,
                        seed: int = 0, df: Optional[torch.Tensor] = None,
                        dx: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None) -> BlockJoinGrads:
    """Gradients of `block_join` from those of x_out and z, with the forward
    call's f, x_out, stats and options.  `df` may be dz, `dx` may be dx_out."""
    named = (("post_weight", post_weight), ("post_bias", post_bias), ("gate", gate),
             ("pre_weight", pre_weight), ("pre_bias", pre_bias))
    q = _join_params(f, x_out, named, rows_per_gate, norm, residual_scale, eps, p, seed)
    for t, like, what in ((dx_out, x_out, "dx_out"), (dz, f, "dz")):
        if t.dtype != like.dtype or t.numel() != like.numel() or t.device != f.device:
            raise LowbitError(EINVAL, f"{what} does not match the forward call")
    if stats.dtype != torch.float32 or stats.numel() != 4 * q.rows or stats.device != f.device:
        raise LowbitError(EINVAL, "stats must be the forward call's")
    df = _out_like(f, df, "df")
    dx = _out_like(x_out, dx, "dx")
    grads = [None if t is None else torch.empty(t.shape, dtype=torch.float32, device=f.device)
             for _, t in named]
    L = lib()
    nbytes = L.lowbit_block_join_backward_workspace(q)
    if nbytes < 0 and q.cols > 16384:
        raise LowbitError(EUNSUPPORTED, "block_join_backward: more than 16384 columns")
    ws = _scratch(nbytes, f, workspace, "block_join_backward")
    _check(L.lowbit_block_join_backward(
        _dev(dx_out, "dx_out"), _dev(dz, "dz"), _dev(f, "f"), _dev(x_out, "x_out"),
        _dev(stats, "stats"), *[_opt(t, n) for n, t in named[:4]], q, _dev(df, "df"),
        _dev(dx, "dx"), *[None if g is None else g.data_ptr() for g in grads],
        _dev(ws, "workspace"), ws.numel(), _stream(f)), "lowbit_block_join_backward")
    return BlockJoinGrads(df, dx, *grads)


class LinearXent(NamedTuple):
    """What linear_xent returns: float32, one value for each row."""
    loss: torch.Tensor
    lse: torch.Tensor


class LinearXentGrads(NamedTuple):
    """What linear_xent_backward returns; None for what was not asked for."""
    dx: Optional[torch.Tensor]
    dw: Optional[torch.Tensor]


def _xent_params(x, w, targets, ignore_index) -> XentParams:
    if w.dim() != 2 or x.dim() < 1 or x.shape[-1] != w.shape[1]:
        raise LowbitError(EINVAL, "x must be (..., hidden) and w (vocab, hidden)")
    vocab, hidden = w.shape
    rows = x.numel() // hidden if hidden else 0
    if w.dtype != x.dtype or w.device != x.device or targets.device != x.device:
        raise LowbitError(EINVAL, "x and w must match in dtype, x, w and targets in device")
    if targets.dtype != torch.int64 or targets.numel() != rows:
        raise LowbitError(EINVAL, "targets must be int64, one for each row of x")
    return XentParams(rows, vocab, hidden, int(ignore_index), _dtype_code(x))


def linear_xent(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                workspace: Optional[torch.Tensor] = None) -> LinearXent:
    """Softmax cross entropy of the logits x w^T, which are not kept:
    lse = logsumexp of a row's logits, loss = lse - the target's logit, each
    float32 and of targets' shape; 0 where targets is ignore_index, NaN where
    a target lies outside the vocabulary.

    x (..., hidden), w (vocab, hidden): float32 or bfloat16; targets: int64.
    Mean loss: loss.sum() / (targets != ignore_index).sum()."""
    if x.requires_grad or w.requires_grad:
        _outside_autograd("linear_xent")
    q = _xent_params(x, w, targets, ignore_index)
    L = lib()
    ws = _scratch(L.lowbit_linear_xent_workspace(q, 0), x, workspace, "linear_xent")
    loss = torch.empty(targets.shape, dtype=torch.float32, device=x.device)
    lse = torch.empty_like(loss)
    _check(L.lowbit_linear_xent(_dev(x, "x"), _dev(w, "w"), _dev(targets, "targets"), q,
                                loss.data_ptr(), lse.data_ptr(), _dev(ws, "workspace"), ws.numel(),
                                _stream(x)), "lowbit_linear_xent")
    return LinearXent(loss, lse)


def linear_xent_backward(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor,
                         lse: torch.Tensor, dloss: torch.Tensor,
                         dlse: Optional[torch.Tensor] = None, ignore_index: int = -100,
                         dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                         need_dx: bool = True, need_dw: bool = True,
                         workspace: Optional[torch.Tensor] = None) -> LinearXentGrads:
    """Gradients of `linear_xent` by x and w, from its lse and the gradients of
    loss and (where the whole loss uses it) of lse, float32 for each row."""
    q = _xent_params(x, w, targets, ignore_index)
    for t, what in ((lse, "lse"), (dloss, "dloss"), (dlse, "dlse")):
        if t is not None and (t.dtype != torch.float32 or t.numel() != q.rows
                              or t.device != x.device):
            raise LowbitError(EINVAL, f"{what} must be float32, one for each row of x")
    dx = _out_like(x, dx, "dx") if need_dx else None
    dw = _out_like(w, dw, "dw") if need_dw else None
    L = lib()
    ws = _scratch(L.lowbit_linear_xent_workspace(q, 1), x, workspace, "linear_xent_backward")
    _check(L.lowbit_linear_xent_backward(
        _dev(x, "x"), _dev(w, "w"), _dev(targets, "targets"), _dev(lse, "lse"),
        _dev(dloss, "dloss"), _opt(dlse, "dlse"), q, _opt(dx, "dx"), _opt(dw, "dw"),
        _dev(ws, "workspace"), ws.numel(), _stream(x)), "lowbit_linear_xent_backward")
    return LinearXentGrads(dx, dw)
