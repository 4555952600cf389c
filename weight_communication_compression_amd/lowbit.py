"""Thin ctypes binding of liblowbit (the C ABI in ``include/lowbit.h`` and, for
the training-step operators, ``include/lowbit_train.h``).

Argument marshalling only: every step runs in the gfx950 HIP kernels behind the
C ABI.  torch is used for device memory (tensors) and for
the current HIP stream.  A call goes to the device of its tensors, whatever the
current one is, on the current stream there.  If the library is missing or a call fails, a
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
    "rotary_frequencies", "rotary", "rotary_backward", "RotaryParams", "attention",
    "attention_backward", "Attention", "AttentionGrads", "AttentionParams", "orthogonalize",
    "OrthogonalizeParams",
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


def _strides_of(*names):
    """lowbit_strides, one after the other (flat: nested structures take a microsecond each)"""
    return [(f"{n}_{w}", ctypes.c_int64) for n in names for w in ("row", "head")]


class RotaryParams(ctypes.Structure):
    """lowbit_rotary_params"""
    _fields_ = [("rows", ctypes.c_int64), ("rows_per_sequence", ctypes.c_int64),
                *_strides_of("x", "y"), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("type", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class AttentionParams(ctypes.Structure):
    """lowbit_attention_params"""
    _fields_ = [("q_rows", ctypes.c_int64), ("k_rows", ctypes.c_int64), ("window", ctypes.c_int64),
                ("sequences", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("type", ctypes.c_int32), ("causal", ctypes.c_int32), ("scale", ctypes.c_float),
                ("softcap", ctypes.c_float),
                *_strides_of("q", "k", "v", "out", "dout", "dq", "dk", "dv")]


class OrthogonalizeParams(ctypes.Structure):
    """lowbit_orthogonalize_params"""
    _fields_ = [("batch", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("type", ctypes.c_int32), ("steps", ctypes.c_int32), ("a", ctypes.c_float),
                ("b", ctypes.c_float), ("c", ctypes.c_float), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float)]


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
        RP, AP = ctypes.POINTER(RotaryParams), ctypes.POINTER(AttentionParams)
        OP = ctypes.POINTER(OrthogonalizeParams)
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
            "lowbit_rotary_frequencies": (ctypes.c_int, [i32, f64, i32, f64, i64, f64, f64, P, P]),
            "lowbit_rotary": (ctypes.c_int, [P, P, P, RP, P, P]),
            "lowbit_rotary_backward": (ctypes.c_int, [P, P, P, RP, P, P]),
            "lowbit_attention_workspace": (i64, [AP, i32]),
            "lowbit_attention": (ctypes.c_int, [P] * 7 + [AP] + [P] * 3 + [i64, P]),
            "lowbit_attention_backward": (ctypes.c_int, [P] * 10 + [AP] + [P] * 4 + [i64, P]),
            "lowbit_orthogonalize_workspace": (i64, [OP]),
            "lowbit_orthogonalize": (ctypes.c_int, [P, OP, P, P, i64, P]),
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


# The current device, and its current stream's handle without the Stream object around it (0.15
# instead of 2 us a call); torch versions without these take the long way.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _qp(bitwidth, block_size, stochastic=False, seed=0, index_offset=0, hints=0) -> QParams:
    return QParams(int(bitwidth), int(block_size), int(bool(stochastic)), int(hints),
                   int(seed) & (2 ** 64 - 1), int(index_offset))


def _check(status: int, what: str) -> None:
    if status != OK:
        raise LowbitError(status, what)


def _launch(fn, like: torch.Tensor, *args) -> None:
    """fn(*args, stream) on like's device, with the current stream there.  (A kernel goes to the
    current device, where the stream of another one, or its default stream, would be a wrong one.)"""
    device = like.get_device()
    if device == _current_device():
        status = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(device))
    if status != OK:
        raise LowbitError(status, fn.__name__)


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
    _launch(lib().lowbit_quantize_pack, x, _dev(x, "x"), _dtype_code(x), n, ctypes.byref(qp),
            _dev(codes, "codes"), _dev(scales, "scales"))
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
    _launch(lib().lowbit_unpack_dequant, codes, _dev(codes, "codes"), _dev(scales, "scales"), n,
            ctypes.byref(qp), _dev(out, "out"))
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
    _launch(lib().lowbit_hadamard_quantize_pack, x, _dev(x, "x"), _dtype_code(x), n,
            ctypes.byref(qp), _dev(codes, "codes"), _dev(scales, "scales"))
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
    _launch(lib().lowbit_hadamard_unpack_dequant, codes, _dev(codes, "codes"),
            _dev(scales, "scales"), n, ctypes.byref(qp), _dev(out, "out"))
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
    _launch(lib().lowbit_ef_compress, g, _dev(g, "g"), _dtype_code(g), _dev(residual, "residual"),
            n, ctypes.byref(qp), _dev(codes, "codes"), _dev(scales, "scales"))
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
    _launch(lib().lowbit_ef21_compress, g, _dev(g, "g"), _dtype_code(g), _dev(state, "state"), n,
            ctypes.byref(qp), _dev(codes, "codes"), _dev(scales, "scales"))
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
            _dev(out_sum, "out_sum") if out_sum is not None else None)
    head = (ctypes.cast(cp, ctypes.c_void_p), ctypes.cast(sp, ctypes.c_void_p), P, n,
            ctypes.byref(qi), ctypes.byref(qo))
    if residual is None:
        _launch(lib().lowbit_reduce_requant, like, *head, *tail)
    else:
        if residual.dtype != torch.float32 or residual.numel() != n:
            raise LowbitError(EINVAL, "residual must be float32 with n elements")
        _launch(lib().lowbit_reduce_requant_ef, like, *head, _dev(residual, "residual"), *tail)
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
    _launch(lib().lowbit_wdiff_compress, w_new, _dev(w_new, "w_new"), _dev(w_old, "w_old"),
            _dtype_code(w_new), n, ctypes.byref(qp), _dev(codes, "codes"), _dev(scales, "scales"))
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
    _launch(lib().lowbit_wdiff_apply, w_old, _dev(w_old, "w_old"), _dev(codes, "codes"),
            _dev(scales, "scales"), n, ctypes.byref(qp), _dev(out, "out"), _dtype_code(w_old))
    return out


def copy_f32(x: torch.Tensor, y: torch.Tensor) -> torch.Tensor:
    """Plain float32 copy kernel (bandwidth reference, not a codec step)."""
    if x.dtype != torch.float32 or y.dtype != torch.float32 or y.numel() != x.numel():
        raise LowbitError(EINVAL, "copy_f32 needs two float32 tensors of equal size")
    _launch(lib().lowbit_copy_f32, x, _dev(x, "x"), _dev(y, "y"), x.numel())
    return y


def add_inplace_f32(x: torch.Tensor, y: torch.Tensor) -> torch.Tensor:
    """y += x in place (float32), with the error-feedback compress's access
    pattern (bandwidth reference for that kernel, not a codec step)."""
    if x.dtype != torch.float32 or y.dtype != torch.float32 or y.numel() != x.numel():
        raise LowbitError(EINVAL, "add_inplace_f32 needs two float32 tensors of equal size")
    _launch(lib().lowbit_add_inplace_f32, y, _dev(x, "x"), _dev(y, "y"), x.numel())
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
    _launch(lib().lowbit_xor_streams_u32, out, ctypes.cast(sp, ctypes.c_void_p), P, n,
            _dev(out, "out"))
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
    _launch(lib().lowbit_fold_f32, x, _dev(x, "x"), n, int(bitwidth), _dev(out, "out"))
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
    _launch(lib().lowbit_stream_probe_u32, dst, int(op), sp, _dev(dst, "dst"), nwords,
            int(value) & 0xFFFFFFFF, int(waves), int(bool(nontemporal)))
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
    _launch(lib().lowbit_dropout, x, _dev(x, "x"), _opt(residual, "residual"), dt, x.numel(), p,
            int(seed) & _U64, int(index_offset), _dev(out, "out"))
    return out


def dropout_backward(dy: torch.Tensor, p: float, seed: int, index_offset: int = 0,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of `dropout` by x, with its p, seed and index_offset: D(dy).
    (The residual's gradient is dy.)  `out` may be dy."""
    dt = _dtype_code(dy)
    out = _out_like(dy, out, "out")
    _launch(lib().lowbit_dropout_backward, dy, _dev(dy, "dy"), dt, dy.numel(), p, int(seed) & _U64,
            int(index_offset), _dev(out, "out"))
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
    _launch(lib().lowbit_block_join, f, _dev(f, "f"), _dev(x, "x"), *[_opt(t, n) for n, t in named],
            q, _dev(x_out, "x_out"), _dev(z, "z"), _dev(stats, "stats"))
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
    _launch(L.lowbit_block_join_backward, f, _dev(dx_out, "dx_out"), _dev(dz, "dz"), _dev(f, "f"),
            _dev(x_out, "x_out"), _dev(stats, "stats"), *[_opt(t, n) for n, t in named[:4]], q,
            _dev(df, "df"), _dev(dx, "dx"), *[None if g is None else g.data_ptr() for g in grads],
            _dev(ws, "workspace"), ws.numel())
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
    _launch(L.lowbit_linear_xent, x, _dev(x, "x"), _dev(w, "w"), _dev(targets, "targets"), q,
            loss.data_ptr(), lse.data_ptr(), _dev(ws, "workspace"), ws.numel())
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
    _launch(L.lowbit_linear_xent_backward, x, _dev(x, "x"), _dev(w, "w"), _dev(targets, "targets"),
            _dev(lse, "lse"), _dev(dloss, "dloss"), _opt(dlse, "dlse"), q, _opt(dx, "dx"),
            _opt(dw, "dw"), _dev(ws, "workspace"), ws.numel())
    return LinearXentGrads(dx, dw)


def _at_most(n, most: int) -> int:
    """n for a field of the C ABI, which would keep the low bits of what does not fit: larger ones
    as `most`, negative ones as -1."""
    return max(-1, min(int(n), most))


_SCALINGS = {None: 0, "linear": 1, "base": 2, "parts": 3}
_LAYOUTS = {"half": 0, "interleaved": 1}


def rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: Optional[str] = None,
                       factor: float = 1.0, original_length: int = 0, slow_turns: float = 1.0,
                       fast_turns: float = 32.0):
    """The rot_dim / 2 frequencies of rotary positions in radians a position (a float64 CPU
    tensor; `rotary` takes it on the GPU), and the scale that goes with them.

    scaling: how a context `factor` times as long is reached: None; "linear": every frequency
    divided by factor; "base": a larger base, which divides the slowest by it and keeps the
    fastest; "parts": pairs that turn at most slow_turns times over original_length positions
    divided, those of at least fast_turns kept, and scale = 0.1 ln(factor) + 1."""
    if scaling not in _SCALINGS:
        raise LowbitError(EINVAL, "scaling must be None, 'linear', 'base' or 'parts'")
    if not 2 <= rot_dim <= 65536:
        raise LowbitError(EINVAL, "rot_dim must be even, 2 to 65536")
    freqs = torch.empty(rot_dim // 2, dtype=torch.float64)
    scale = ctypes.c_float()
    _check(lib().lowbit_rotary_frequencies(int(rot_dim), base, _SCALINGS[scaling], factor,
                                           _at_most(original_length, 2 ** 63 - 1), slow_turns, fast_turns,
                                           freqs.data_ptr(), ctypes.byref(scale)),
           "lowbit_rotary_frequencies")
    return freqs, scale.value


def _gpu(t: torch.Tensor, what: str) -> int:
    if not t.is_cuda:
        raise LowbitError(EINVAL, f"{what} must be a GPU tensor")
    return t.data_ptr()


def _heads(t: torch.Tensor, what: str):
    """Rows, and the steps from row to row and from head to head, of (..., heads, head_dim): one
    step for all leading dimensions, dense heads.  (A step of a dimension of one element is of no
    account.)"""
    size, step = t.shape, t.stride()
    if len(size) < 2:
        raise LowbitError(EINVAL, f"{what} must be (..., heads, head_dim)")
    heads, dim = size[-2], size[-1]
    if dim > 1 and step[-1] != 1:
        raise LowbitError(EINVAL, f"{what}: the elements of a head must be dense")
    if len(size) == 3:
        rows, row = size[0], step[0]
    else:
        rows, row = 1, 0
        for n, s in zip(size[-3::-1], step[-3::-1]):
            if n != 1:
                if rows == 1:
                    row = s
                elif s != row * rows and t.numel():
                    raise LowbitError(EINVAL, f"{what}: the leading dimensions must have one step")
                rows *= n
    return rows, row if rows > 1 else heads * dim, step[-2] if heads > 1 else dim


def _rotary(fn, x, freqs, positions, rows_per_sequence, layout, scale, out, what):
    if layout not in _LAYOUTS:
        raise LowbitError(EINVAL, "layout must be 'half' or 'interleaved'")
    rows, x_row, x_head = _heads(x, what)
    device = x.device
    if freqs.dtype != torch.float64 or freqs.device != device:
        raise LowbitError(EINVAL, "freqs must be float64 on the device of the tensor to turn")
    if positions is not None and (positions.dtype != torch.int64 or positions.numel() != rows
                                  or positions.device != device):
        raise LowbitError(EINVAL, "positions must be int64, one for each row")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=device)
        y_row, y_head = x.shape[-2] * x.shape[-1], x.shape[-1]
    else:
        if out.shape != x.shape or out.dtype != x.dtype or out.device != device:
            raise LowbitError(EINVAL, "out must match the input in shape, dtype and device")
        _, y_row, y_head = _heads(out, "out")
    p = RotaryParams(rows, _at_most(rows_per_sequence, max(rows, 1)) or max(rows, 1), x_row, x_head, y_row, y_head,
                     x.shape[-2], x.shape[-1], 2 * freqs.numel(), _LAYOUTS[layout],
                     _dtype_code(x), scale)
    _launch(fn, x, _gpu(x, what), _dev(freqs, "freqs"),
            None if positions is None else _dev(positions, "positions"), p, out.data_ptr())
    return out


def rotary(x: torch.Tensor, freqs: torch.Tensor, positions: Optional[torch.Tensor] = None,
           rows_per_sequence: int = 0, layout: str = "half", scale: float = 1.0,
           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotary positions of x (..., heads, head_dim), float32 or bfloat16: the first 2 len(freqs)
    elements of a head in pairs, (i, i + len(freqs)) for layout "half", (2 i, 2 i + 1) for
    "interleaved", turned by position * freqs[i] and multiplied by scale; the others copied.

    x may be a view, as of the heads of a packed projection, whose leading dimensions have one
    step.  freqs, scale: of `rotary_frequencies`, freqs on x's device.  positions: int64, one
    for each row; without them rows are counted from 0, anew after every rows_per_sequence
    (0: never).  `out` may be x."""
    if x.requires_grad:
        _outside_autograd("rotary")
    return _rotary(lib().lowbit_rotary, x, freqs, positions, rows_per_sequence, layout, scale, out,
                   "x")


def rotary_backward(dy: torch.Tensor, freqs: torch.Tensor,
                    positions: Optional[torch.Tensor] = None, rows_per_sequence: int = 0,
                    layout: str = "half", scale: float = 1.0,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of `rotary` by x, with its options.  `out` may be dy."""
    return _rotary(lib().lowbit_rotary_backward, dy, freqs, positions, rows_per_sequence, layout,
                   scale, out, "dy")


class Attention(NamedTuple):
    """What attention returns; lse is float32 (query heads, query rows)."""
    out: torch.Tensor
    lse: torch.Tensor


class AttentionGrads(NamedTuple):
    """What attention_backward returns."""
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor


def _offset_count(t, device, what):
    """How many sequences the offsets are of."""
    if t.dtype != torch.int32 or t.dim() != 1 or t.numel() < 1 or t.device != device:
        raise LowbitError(EINVAL, f"{what} must be int32 offsets, one more than sequences")
    return t.numel() - 1


def _attention_params(q, k, v, q_begin, k_begin, scale, causal, window, prefix, softcap, slopes):
    """Checks of the tensors' types and sizes, which the C ABI cannot see."""
    device, dtype, size, k_size = q.device, q.dtype, q.shape, k.shape
    if k.dtype != dtype or v.dtype != dtype or k.device != device or v.device != device:
        raise LowbitError(EINVAL, "q, k and v must match in dtype and device")
    n = len(size)
    if n not in (3, 4) or len(k_size) != n or k_size != v.shape:
        raise LowbitError(EINVAL, "q, k and v must be (rows, heads, head_dim), or (batch, length, "
                                  "heads, head_dim) for sequences of equal lengths")
    d = size[-1]
    if d != k_size[-1] or d < 1:
        raise LowbitError(EINVAL, "q, k and v must have one head_dim, a multiple of 8 up to 128")
    if size[-2] < 1 or k_size[-2] < 1 or size[-2] % k_size[-2]:
        raise LowbitError(EINVAL, "k's heads must divide q's")
    sequences = 1
    if n == 4:
        if q_begin is not None or k_begin is not None:
            raise LowbitError(EINVAL, "offsets go with (rows, heads, head_dim)")
        if k_size[0] != size[0]:
            raise LowbitError(EINVAL, "q and k must have one batch")
        sequences = size[0]
    if q_begin is not None:
        sequences = _offset_count(q_begin, device, "q_begin")
    if k_begin is not None:
        count = _offset_count(k_begin, device, "k_begin")
        if q_begin is not None and count != sequences:
            raise LowbitError(EINVAL, "q_begin and k_begin must have the same length")
        sequences = count
    if prefix is not None and (prefix.dtype != torch.int32 or prefix.numel() != sequences
                               or prefix.device != device):
        raise LowbitError(EINVAL, "prefix must be int32, one for each sequence")
    if slopes is not None and (slopes.dtype != torch.float32 or slopes.numel() != size[-2]
                               or slopes.device != device):
        raise LowbitError(EINVAL, "slopes must be float32, one for each head of q")
    q_rows, q_row, q_head = _heads(q, "q")
    k_rows, k_row, k_head = _heads(k, "k")
    _, v_row, v_head = _heads(v, "v")
    # (a window beyond 64 bits hides nothing either)
    return AttentionParams(q_rows, k_rows, _at_most(window, 1 << 40), sequences,
                           size[-2], k_size[-2], d, _dtype_code(q), 1 if causal else 0,
                           d ** -0.5 if scale is None else scale, softcap,
                           q_row, q_head, k_row, k_head, v_row, v_head)


def _attention_scratch(L, p, backward, like, workspace, what):
    """The workspace, which the caller holds until its kernels are enqueued (torch then keeps the
    memory for what comes behind them on the stream), its pointer and size."""
    nbytes = L.lowbit_attention_workspace(p, backward)
    if nbytes < 0 and p.head_dim % 8 == 0 and p.head_dim > 128:
        raise LowbitError(EUNSUPPORTED, f"{what}: head_dim above 128")
    if nbytes == 0 and workspace is None:
        return None, None, 0
    ws = _scratch(nbytes, like, workspace, what)
    return ws, _dev(ws, "workspace"), ws.numel()


def _attention_out(t, like, what):
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device:
        raise LowbitError(EINVAL, f"{what} must match in shape, dtype and device")


def _attention_grad(t, like, what):
    """The gradient's tensor and its steps."""
    if t is None:
        size = like.shape
        return torch.empty(size, dtype=like.dtype, device=like.device), size[-2] * size[-1], size[-1]
    _attention_out(t, like, what)
    _, row, head = _heads(t, what)
    return t, row, head


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
              q_begin: Optional[torch.Tensor] = None, k_begin: Optional[torch.Tensor] = None,
              scale: Optional[float] = None, causal: bool = True, window: int = 0,
              prefix: Optional[torch.Tensor] = None, softcap: float = 0.0,
              slopes: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None) -> Attention:
    """Softmax attention within each sequence of packed rows.

    q (rows, heads, head_dim), k and v (key rows, key-value heads, head_dim), float32 or
    bfloat16, head_dim a multiple of 8 up to 128; key-value heads divide q's and are shared by
    consecutive ones.  They may be views with dense heads, as of a packed projection.  q_begin,
    k_begin: int32 offsets of the sequences (one more than there are); k_begin None: the same.
    Without offsets: one sequence, or for 4-dimensional tensors one for each of the batch.

    With Lq queries and Lk keys query i of a sequence stands at position i + Lk - Lq and sees
    key j if  j < prefix[s]  or  (not causal or j <= position) and (window == 0 or
    |position - j| < window).  Scores are softcap * tanh(scale q.k / softcap) (softcap 0: scale
    q.k; scale None: head_dim ** -0.5) minus slopes[head] * |position - j|.  A query that sees
    nothing gives 0 and lse -infinity.  Rows outside all sequences are left as they were: in
    `out` and lse that are allocated here whatever the memory held."""
    if q.requires_grad or k.requires_grad or v.requires_grad:
        _outside_autograd("attention")
    p = _attention_params(q, k, v, q_begin, k_begin, scale, causal, window, prefix, softcap, slopes)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        p.out_row, p.out_head = p.q_heads * p.head_dim, p.head_dim
    else:
        _attention_out(out, q, "out")
        _, p.out_row, p.out_head = _heads(out, "out")
    lse = torch.empty(p.q_heads, p.q_rows, dtype=torch.float32, device=q.device)
    L = lib()
    ws, at, nbytes = _attention_scratch(L, p, 0, q, workspace, "attention")
    # (all are on q's device)
    _launch(L.lowbit_attention, q, _gpu(q, "q"), k.data_ptr(), v.data_ptr(),
            _opt(q_begin, "q_begin"), _opt(k_begin, "k_begin"), _opt(prefix, "prefix"),
            _opt(slopes, "slopes"), p, out.data_ptr(), lse.data_ptr(), at, nbytes)
    return Attention(out, lse)


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       out: torch.Tensor, lse: torch.Tensor,
                       q_begin: Optional[torch.Tensor] = None,
                       k_begin: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                       causal: bool = True, window: int = 0,
                       prefix: Optional[torch.Tensor] = None, softcap: float = 0.0,
                       slopes: Optional[torch.Tensor] = None, dq: Optional[torch.Tensor] = None,
                       dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> AttentionGrads:
    """Gradients of `attention` by q, k and v from that of out, with the forward call's out, lse
    and options.  dq, dk, dv may be views, as of a packed projection's gradient; rows outside all
    sequences are left as they were."""
    p = _attention_params(q, k, v, q_begin, k_begin, scale, causal, window, prefix, softcap, slopes)
    for t, what in ((dout, "dout"), (out, "out")):
        _attention_out(t, q, what)
    if lse.dtype != torch.float32 or lse.numel() != p.q_heads * p.q_rows or lse.device != q.device:
        raise LowbitError(EINVAL, "lse must be the forward call's")
    _, p.out_row, p.out_head = _heads(out, "out")
    _, p.dout_row, p.dout_head = _heads(dout, "dout")
    dq, p.dq_row, p.dq_head = _attention_grad(dq, q, "dq")
    dk, p.dk_row, p.dk_head = _attention_grad(dk, k, "dk")
    dv, p.dv_row, p.dv_head = _attention_grad(dv, v, "dv")
    L = lib()
    ws, at, nbytes = _attention_scratch(L, p, 1, q, workspace, "attention_backward")
    _launch(L.lowbit_attention_backward, q, dout.data_ptr(), _gpu(q, "q"), k.data_ptr(),
            v.data_ptr(), out.data_ptr(), _dev(lse, "lse"), _opt(q_begin, "q_begin"),
            _opt(k_begin, "k_begin"), _opt(prefix, "prefix"), _opt(slopes, "slopes"), p,
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), at, nbytes)
    return AttentionGrads(dq, dk, dv)


def orthogonalize(g: torch.Tensor, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315),
                  eps: float = 1e-7, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Newton-Schulz iteration on the matrices g (..., rows, columns), float32 or bfloat16:

        X = g / (||g||_F + eps);  steps times  A = X X^T,  X = a X + (b A + c A A) X

    (of the transpose where there are more rows than columns); scale X as bfloat16.  With the
    default coefficients five steps bring all but the smallest singular values to between 0.7
    and 1.2.  `out` may be a bfloat16 g."""
    if g.requires_grad:
        _outside_autograd("orthogonalize")
    if g.dim() < 2:
        raise LowbitError(EINVAL, "g must be (..., rows, columns)")
    a, b, c = coefficients
    rows, cols = g.shape[-2:]
    p = OrthogonalizeParams(g.numel() // (rows * cols) if rows and cols else 0, max(rows, 1),
                            max(cols, 1), _dtype_code(g), _at_most(steps, 65), a, b, c, eps, scale)
    if out is None:
        out = torch.empty(g.shape, dtype=torch.bfloat16, device=g.device)
    elif out.dtype != torch.bfloat16 or out.shape != g.shape or out.device != g.device:
        raise LowbitError(EINVAL, "out must be bfloat16, of g's shape and device")
    L = lib()
    ws = _scratch(L.lowbit_orthogonalize_workspace(p), g, workspace, "orthogonalize")
    _launch(L.lowbit_orthogonalize, g, _dev(g, "g"), p, _dev(out, "out"), _dev(ws, "workspace"),
            ws.numel())
    return out
