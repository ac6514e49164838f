"""Torch-facing binding of libsixbit: argument marshalling only.

Every function here allocates its output tensors with torch (device memory),
passes raw pointers and the current CUDA stream to the C ABI, and raises
``SixbitError`` on a non-zero status.  All arithmetic runs in the library's
CUDA kernels; there is no CPU path.
"""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple

import torch

from . import abi
from .abi import (EPI_GELU, EPI_NONE, EPI_RESIDUAL, MAX_ADAPTERS, MAX_EXPERTS, MAX_GROUPS, MAX_RANK, MAX_TOP_K,  # noqa: F401
                  MODE_BF16, MODE_INT8, MODE_NVFP4, MODE_SKIP, QGEMV_MAX_ROWS, SCORE_SIGMOID, SCORE_SOFTMAX, DitBlocks, PolicyCfg, PolicyState, QAct, Stats, Weights, check, lib)

_lib = lib()


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def fp4_scale_bytes(rows: int, k: int) -> int:
    return int(_lib.sixbit_fp4_scale_bytes(rows, k))


def stats_scratch_bytes(n: int) -> int:
    return int(_lib.sixbit_stats_scratch_bytes(n))


def launch_count() -> int:
    return int(_lib.sixbit_launch_count())


def qgemm_workspace_bytes(n: int, k: int) -> int:
    return int(_lib.sixbit_qgemm_workspace_bytes(n, k))


_workspaces = {}  # device -> its buffers, the largest last


def workspace(n: int, k: int, device) -> torch.Tensor:
    """A device buffer of at least qgemm_workspace_bytes(n, k) bytes, shared by every call on `device`
    that passes none of its own (calls that share it must be ordered, e.g. on one stream).  A buffer that a
    larger one replaces is kept: a captured graph goes on writing to the address it was captured with."""
    dev = torch.device(device)
    need = qgemm_workspace_bytes(n, k)
    bufs = _workspaces.setdefault(dev, [])
    if not bufs or bufs[-1].numel() < need:
        bufs.append(torch.empty(need, dtype=torch.uint8, device=dev))
    return bufs[-1]


class QActTensors:
    """Device buffers of one quantized activation tensor [M, K]."""

    fp4_codes = fp4_scales = tensor_amax = tensor_scale = i8_codes = row_scale = rotated = None

    def __init__(self, m: int, k: int, device="cuda", nvfp4=True, int8=True, rotated=False):
        self.m, self.k = m, k
        dev = torch.device(device)
        u8, f32 = torch.uint8, torch.float32
        self.fp4_codes = torch.empty((m, k // 2), dtype=u8, device=dev) if nvfp4 else None
        self.fp4_scales = torch.zeros(fp4_scale_bytes(m, k), dtype=u8, device=dev) if nvfp4 else None
        self.tensor_amax = torch.zeros(1, dtype=f32, device=dev) if nvfp4 else None
        self.tensor_scale = torch.zeros(1, dtype=f32, device=dev) if nvfp4 else None
        self.i8_codes = torch.empty((m, k), dtype=torch.int8, device=dev) if int8 else None
        self.row_scale = torch.empty(m, dtype=f32, device=dev) if int8 else None
        self.rotated = torch.empty((m, k), dtype=f32, device=dev) if rotated else None

    def c(self) -> QAct:
        return QAct(*[_p(getattr(self, f)) for f, _ in QAct._fields_])


class PackedWeights:
    """Device buffers of one packed linear layer W [N, K]."""

    def __init__(self, n: int, k: int, device="cuda"):
        self.n, self.k = n, k
        dev = torch.device(device)
        self.fp4_codes = torch.empty((n, k // 2), dtype=torch.uint8, device=dev)
        self.fp4_scales = torch.zeros(fp4_scale_bytes(n, k), dtype=torch.uint8, device=dev)
        self.fp4_amax = torch.zeros(1, dtype=torch.float32, device=dev)
        self.fp4_tensor_scale = torch.zeros(1, dtype=torch.float32, device=dev)
        self.i4_codes = torch.empty((n, k // 2), dtype=torch.uint8, device=dev)
        self.i4_scales = torch.empty((k // 128, n), dtype=torch.float32, device=dev)
        self.bf16_w = torch.empty((n, k), dtype=torch.bfloat16, device=dev)

    def c(self) -> Weights:
        return Weights(*[_p(getattr(self, f)) for f, _ in Weights._fields_])


def pack_weights(w: torch.Tensor, had_block: int, out: PackedWeights | None = None, stream=None) -> PackedWeights:
    assert w.dtype == torch.float32 and w.is_contiguous()
    n, k = w.shape
    out = out or PackedWeights(n, k, w.device)
    cw = out.c()
    check(_lib.sixbit_pack_weights(_p(w), n, k, had_block, C.byref(cw), None, _stream(stream)), "pack_weights")
    return out


def hadamard_quant(x: torch.Tensor, had_block: int, mode: int, out: QActTensors | None = None, mode_dev=None,
                   tamax=None, stream=None) -> QActTensors:
    assert x.dtype == torch.bfloat16 and x.is_contiguous()
    m, k = x.shape
    out = out or QActTensors(m, k, x.device)
    ca = out.c()
    check(_lib.sixbit_hadamard_quant(_p(x), m, k, had_block, mode, _p(mode_dev), _p(tamax), C.byref(ca), None,
                                     _stream(stream)), "hadamard_quant")
    return out


def qgemm(a: QActTensors | None, x_bf16, w: PackedWeights, mode: int, epilogue: int = EPI_NONE, residual=None,
          out=None, out_f32: bool = False, acc_dbg=None, mode_dev=None, err=None, stream=None, m: int | None = None,
          ws=None):
    """ws: the INT8 kind's workspace (qgemm_workspace_bytes); by default the device's shared one."""
    n, k = w.n, w.k
    if ws is None and (mode == MODE_INT8 or mode_dev is not None):
        ws = workspace(n, k, w.bf16_w.device)
    m = m if m is not None else (a.m if a is not None else x_bf16.shape[0])
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32 if out_f32 else torch.bfloat16, device=w.bf16_w.device)
    ca = a.c() if a is not None else None
    cw = w.c()
    y = out if out.dtype == torch.bfloat16 else None
    yf = out if out.dtype == torch.float32 else None
    check(_lib.sixbit_qgemm(C.byref(ca) if ca is not None else None, _p(x_bf16), C.byref(cw), m, n, k, mode,
                            _p(mode_dev), epilogue, _p(residual), _p(y), _p(yf), _p(acc_dbg), _p(ws), _p(err),
                            _stream(stream)), "qgemm")
    return out


def qgemm_rotamax(a: QActTensors, w: PackedWeights, had_block: int, amax_out: torch.Tensor, epilogue: int = EPI_NONE,
                  residual=None, out=None, mode_dev=None, err=None, stream=None, m: int | None = None):
    """NVFP4 qgemm whose epilogue also writes the rotated amax of its bf16 output to amax_out."""
    n, k = w.n, w.k
    m = m if m is not None else a.m
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=w.bf16_w.device)
    ca, cw = a.c(), w.c()
    check(_lib.sixbit_qgemm_rotamax(C.byref(ca), C.byref(cw), m, n, k, _p(mode_dev), epilogue, _p(residual), _p(out),
                                    had_block, _p(amax_out), _p(err), _stream(stream)), "qgemm_rotamax")
    return out


def qgemm_blockstats(a: QActTensors | None, x_bf16, w: PackedWeights, mode: int, residual, out, delta_cache,
                     parts, mode_dev=None, err=None, stream=None, m: int | None = None, ws=None):
    """qgemm with the RESIDUAL epilogue that also updates delta_cache (Delta_prev -> Delta) and writes
    the block statistics' partial rows to parts (blockstats_parts_bytes(); fold with block_stats_parts
    or dit_block_end_parts)."""
    n, k = w.n, w.k
    if ws is None and (mode == MODE_INT8 or mode_dev is not None):
        ws = workspace(n, k, w.bf16_w.device)
    m = m if m is not None else (a.m if a is not None else x_bf16.shape[0])
    ca = a.c() if a is not None else None
    cw = w.c()
    check(_lib.sixbit_qgemm_blockstats(C.byref(ca) if ca is not None else None, _p(x_bf16), C.byref(cw), m, n, k,
                                       mode, _p(mode_dev), _p(residual), _p(out), _p(delta_cache), _p(parts), _p(ws),
                                       _p(err), _stream(stream)), "qgemm_blockstats")
    return out


def blockstats_parts_bytes() -> int:
    return int(_lib.sixbit_blockstats_parts_bytes())


def new_blockstats_parts(device="cuda") -> torch.Tensor:
    return torch.zeros(blockstats_parts_bytes(), dtype=torch.uint8, device=device)


def block_stats_parts(parts: torch.Tensor, n: int, stats: torch.Tensor, stream=None):
    check(_lib.sixbit_block_stats_parts(_p(parts), n, _p(stats), None, _stream(stream)), "block_stats_parts")
    return stats


def tensor_stats(x: torch.Tensor, out: torch.Tensor, scratch: torch.Tensor, stream=None) -> torch.Tensor:
    check(_lib.sixbit_tensor_stats(_p(x), x.numel(), _p(out), _p(scratch), None, _stream(stream)), "tensor_stats")
    return out


def block_stats(x_in, x_out, delta_cache, stats: torch.Tensor, scratch: torch.Tensor, mode_dev=None, stream=None):
    check(_lib.sixbit_block_stats(_p(x_in), _p(x_out), _p(delta_cache), x_in.numel(), _p(mode_dev), _p(stats),
                                  _p(scratch), None, _stream(stream)), "block_stats")
    return stats


def block_stats_noalloc(x_in, x_out, delta_cache, stats: torch.Tensor, mode_dev=None, stream=None):
    """sixbit_block_stats without caller scratch (the library's fixed array is used).

    For callers that cannot allocate device memory for scratch; calls must not
    overlap on the GPU, since they share that array.
    """
    check(_lib.sixbit_block_stats_noalloc(_p(x_in), _p(x_out), _p(delta_cache), x_in.numel(), _p(mode_dev),
                                          _p(stats), None, _stream(stream)), "block_stats_noalloc")
    return stats


def skip_apply(x_in, delta_cache, x_out, stats: torch.Tensor, scratch: torch.Tensor, mode_dev=None, stream=None):
    check(_lib.sixbit_skip_apply(_p(x_in), _p(delta_cache), _p(x_out), x_in.numel(), _p(mode_dev), _p(stats),
                                 _p(scratch), None, _stream(stream)), "skip_apply")
    return x_out


DELTA_BF16, DELTA_MXFP8 = 0, 1
MX_BLOCK = 32


def mxfp8_cache(n: int, device, blocks: int | None = None):
    """A zeroed MXFP8 Delta cache of n elements (per block when `blocks` is given): (codes, scales) uint8."""
    assert n % MX_BLOCK == 0
    lead = () if blocks is None else (blocks,)
    return (torch.zeros(lead + (n,), dtype=torch.uint8, device=device),
            torch.zeros(lead + (n // MX_BLOCK,), dtype=torch.uint8, device=device))


def block_stats_mxfp8(x_in, x_out, codes, scales, stats: torch.Tensor, scratch: torch.Tensor, mode_dev=None,
                      stream=None):
    """sixbit_block_stats_mxfp8: the Delta cache in MXFP8 (codes [n] uint8, scales [n / 32] uint8)."""
    n = x_in.numel()
    assert codes.dtype == torch.uint8 and codes.numel() == n and scales.numel() == n // MX_BLOCK
    check(_lib.sixbit_block_stats_mxfp8(_p(x_in), _p(x_out), _p(codes), _p(scales), n, _p(mode_dev), _p(stats),
                                        _p(scratch), None, _stream(stream)), "block_stats_mxfp8")
    return stats


def skip_apply_mxfp8(x_in, codes, scales, x_out, stats: torch.Tensor, scratch: torch.Tensor, mode_dev=None,
                     stream=None):
    n = x_in.numel()
    assert codes.dtype == torch.uint8 and codes.numel() == n and scales.numel() == n // MX_BLOCK
    check(_lib.sixbit_skip_apply_mxfp8(_p(x_in), _p(codes), _p(scales), _p(x_out), n, _p(mode_dev), _p(stats),
                                       _p(scratch), None, _stream(stream)), "skip_apply_mxfp8")
    return x_out


# ---- a feed-forward layer around the W4A8 products --------------------------
# These check their tensors (type, shape, density, device) before the pointers
# leave Python, and raise ValueError.  A call of a single token takes a few
# microseconds on the GPU, so they do little else: addresses go to ctypes as
# plain integers and the stream's handle is asked for directly.

_BF16, _F32, _I8, _I32, _U8 = torch.bfloat16, torch.float32, torch.int8, torch.int32, torch.uint8
_current_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _ptr(t, name: str, dtype, shape, dev: int) -> int:
    """t's address after checking that it is a dense tensor of this type and shape on GPU `dev`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: a dense {dtype} {tuple(shape)} tensor on GPU {dev} expected, got {t.dtype} "
                     f"{tuple(t.shape)}, strides {t.stride()}, on {t.device}")


def _word(t, name: str, dev: int):
    if t is None:
        return None
    if t.dtype is not _I32 or t.numel() < 1 or t.get_device() != dev:
        raise ValueError(f"{name}: an int32 word on GPU {dev} expected")
    return t.data_ptr()


def _stream_on(dev: int, stream) -> int:
    """The handle of `stream` (None: the current one) after checking that it and the calling thread are on GPU `dev`:
    the library launches on the current device."""
    if _current_device() != dev:
        raise ValueError(f"the tensors are on GPU {dev}, the current device is {_current_device()}")
    if stream is None:
        return _current_raw_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the tensors are on GPU {dev}, the stream on {stream.device_index}")
    return stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """An uninitialised tensor allocated on `stream` (None: the current one)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def int8_act(codes: torch.Tensor, row_scale: torch.Tensor) -> QActTensors:
    """INT8 activations that already exist: codes int8 [M, K], row_scale float32 [M]."""
    a = QActTensors.__new__(QActTensors)
    a.m, a.k = codes.shape
    a.i8_codes, a.row_scale = codes, row_scale
    return a


class Int4Weights:
    """The INT4 form alone of one layer (codes [N, K/2] uint8, scales [K/128, N] float32) or of E experts
    (codes [E, N, K/2], scales [E, K/128, N]): what qgemv and qgemm_grouped read, 0.53 bytes a weight."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        self.i4_codes, self.i4_scales = codes, scales
        shape = codes.shape
        self.n, self.k = shape[-2], 2 * shape[-1]
        self.experts = shape[0] if len(shape) == 3 else None


def pack_experts(w: torch.Tensor, had_block: int, stream=None) -> Int4Weights:
    """Experts' weights [E, N, K] float32, each packed by pack_weights, INT4 form kept."""
    if w.dim() != 3:
        raise ValueError(f"w: [E, N, K] expected, got {tuple(w.shape)}")
    if w.dtype is not _F32 or not w.is_contiguous() or w.get_device() < 0:
        raise ValueError(f"w: dense float32 on the GPU expected, got {w.dtype}, strides {w.stride()}, on {w.device}")
    e, n, k = w.shape
    with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(w.device)):
        codes = torch.empty((e, n, k // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((e, k // 128, n), dtype=torch.float32, device=w.device)
        one = PackedWeights(n, k, w.device)
        for i in range(e):
            pack_weights(w[i], had_block, one)
            codes[i].copy_(one.i4_codes)
            scales[i].copy_(one.i4_scales)
    return Int4Weights(codes, scales)


def add_rmsnorm_quant(x: torch.Tensor, residual: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                      eps: float = 1e-6, had_block: int = 0, out: QActTensors | None = None, sum_out=None,
                      mode_dev=None, stream=None):
    """h = x + residual, RMS norm times weight, rotation by had_block (0: none), INT8 codes and row scales.

    x, residual: bf16 [M, K]; weight: float32 [K].  Returns (activations, h): the QActTensors that qgemv,
    qgemm_grouped and qgemm read, and bf16(h) (in sum_out, which may be x or residual; x itself when there
    is no residual)."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x: [M, K] expected, got {tuple(shape)}")
    m, k = shape
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"x must be on the GPU, not on {x.device}")
    st = _stream_on(dev, stream)
    px = _ptr(x, "x", _BF16, shape, dev)
    pw = None if weight is None else _ptr(weight, "weight", _F32, (k,), dev)
    pr = ps = None
    if residual is not None:
        pr = _ptr(residual, "residual", _BF16, shape, dev)
        if sum_out is None:
            sum_out = _empty(shape, _BF16, x.device, stream)
            ps = sum_out.data_ptr()
        else:
            ps = _ptr(sum_out, "sum_out", _BF16, shape, dev)
    elif sum_out is not None:
        raise ValueError("sum_out without a residual")
    if out is None:
        device = x.device
        codes, scale = _empty(shape, _I8, device, stream), _empty((m,), _F32, device, stream)
        out = int8_act(codes, scale)
        pc, pscale = codes.data_ptr(), scale.data_ptr()
    else:
        pc, pscale = (_ptr(out.i8_codes, "out.i8_codes", _I8, shape, dev),
                      _ptr(out.row_scale, "out.row_scale", _F32, (m,), dev))
    status = _lib.sixbit_add_rmsnorm_quant(px, pr, pw, m, k, eps, had_block,
                                           None if mode_dev is None else _word(mode_dev, "mode_dev", dev), ps,
                                           C.byref(QAct(None, None, None, None, pc, pscale, None)), None, st)
    if status:
        check(status, "add_rmsnorm_quant")
    return out, (x if residual is None else sum_out)


def _w4a8(a, w, experts, offsets, epilogue, residual, out, out_f32, mode_dev, err, stream, ws):
    """qgemv (experts None) and qgemm_grouped: checks, the output, the call."""
    codes = a.i8_codes
    if codes is None or codes.dim() != 2:
        raise ValueError("INT8 activations [M, K] expected")
    shape = codes.shape
    m, k = shape
    n = w.n
    if w.k != k:
        raise ValueError(f"activations have {k} inputs, the weights {w.k}")
    dev = codes.get_device()
    if dev < 0:
        raise ValueError(f"i8_codes must be on the GPU, not on {codes.device}")
    st = _stream_on(dev, stream)
    if experts is None:
        shape4, shapes = (n, k // 2), (k // 128, n)
    else:
        shape4, shapes = (experts, n, k // 2), (experts, k // 128, n)
    ca = QAct(None, None, None, None, _ptr(codes, "i8_codes", _I8, shape, dev),
              _ptr(a.row_scale, "row_scale", _F32, (m,), dev), None)
    cw = Weights(None, None, None, None, _ptr(w.i4_codes, "i4_codes", _U8, shape4, dev),
                 _ptr(w.i4_scales, "i4_scales", _F32, shapes, dev), None)
    py = pf = pr = None
    if out is None:
        out = _empty((m, n), _F32 if out_f32 else _BF16, codes.device, stream)
        if out_f32:
            pf = out.data_ptr()
        else:
            py = out.data_ptr()
    elif out.dtype is _F32:
        pf = _ptr(out, "out", _F32, (m, n), dev)
    else:
        py = _ptr(out, "out", _BF16, (m, n), dev)
    if residual is not None:
        if epilogue != EPI_RESIDUAL:
            raise ValueError("a residual without the residual epilogue")
        pr = _ptr(residual, "residual", _BF16, (m, n), dev)
    pm = None if mode_dev is None else _word(mode_dev, "mode_dev", dev)
    pe = None if err is None else _word(err, "err", dev)
    if experts is None:
        status = _lib.sixbit_qgemv(C.byref(ca), C.byref(cw), m, n, k, pm, epilogue, pr, py, pf, pe, st)
        if status:
            check(status, "qgemv")
        return out
    po = _ptr(offsets, "offsets", _I32, (experts + 1,), dev)
    need = 2 * m * k + m * (k // 128) * 4  # sixbit_qgemm_grouped_workspace_bytes
    if ws is None:
        ws = _empty((need,), _U8, out.device, stream)
    elif ws.get_device() != dev or not ws.is_contiguous() or ws.numel() * ws.element_size() < need:
        raise ValueError(f"ws: {need} dense bytes on GPU {dev} expected")
    status = _lib.sixbit_qgemm_grouped(C.byref(ca), C.byref(cw), po, experts, m, n, k, pm, epilogue, pr, py, pf,
                                       ws.data_ptr(), pe, st)
    if status:
        check(status, "qgemm_grouped")
    return out


def qgemv(a: QActTensors, w, epilogue: int = EPI_NONE, residual=None, out=None, out_f32: bool = False, mode_dev=None,
          err=None, stream=None):
    """The W4A8 product of 1 to QGEMV_MAX_ROWS rows (sixbit_qgemv).  w: PackedWeights or Int4Weights.  Returns
    out: bf16 [M, N], or float32 with out_f32 or a float32 `out`."""
    return _w4a8(a, w, None, None, epilogue, residual, out, out_f32, mode_dev, err, stream, None)


def qgemm_grouped_workspace_bytes(m: int, k: int) -> int:
    return int(_lib.sixbit_qgemm_grouped_workspace_bytes(m, k))


def qgemm_grouped(a: QActTensors, w: Int4Weights, offsets: torch.Tensor, epilogue: int = EPI_NONE, residual=None,
                  out=None, out_f32: bool = False, mode_dev=None, err=None, stream=None, ws=None):
    """The W4A8 product grouped by expert (sixbit_qgemm_grouped): rows offsets[e] .. offsets[e + 1] - 1 of `a`
    times expert e's weight.  offsets: int32 [E + 1] on the GPU; it is not read on the host.  Rows of `out`
    outside every expert's range are left as they are.  ws: qgemm_grouped_workspace_bytes(M, K) bytes (uint8),
    allocated for the call by default."""
    experts = getattr(w, "experts", None)
    if experts is None:
        raise ValueError("experts' weights expected (Int4Weights with [E, N, K/2] codes)")
    return _w4a8(a, w, experts, offsets, epilogue, residual, out, out_f32, mode_dev, err, stream, ws)


# ---- what stands around those products --------------------------------------

_route_workspace_bytes, _lowrank_workspace_bytes = _lib.sixbit_moe_route_workspace_bytes, _lib.sixbit_lowrank_workspace_bytes


def _gpu(t, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be on the GPU, not on {t.device}")
    return dev


def gated_rmsnorm_quant(x: torch.Tensor, residual: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                        post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                        scale: torch.Tensor | None = None, shift: torch.Tensor | None = None,
                        segment: torch.Tensor | None = None, residual_scale: float = 1.0, eps: float = 1e-6,
                        had_block: int = 0, quantize: bool = True, out=None, sum_out=None, mode_dev=None, err=None,
                        stream=None):
    """h = residual_scale residual + gate u, u = x or (with post_weight) its RMS norm times post_weight; then
    y = norm(h) weight (1 + scale) + shift, rotation by had_block (0: none), INT8 codes and row scales
    (sixbit_gated_rmsnorm_quant); with quantize=False bf16 y instead (had_block 0).

    x, residual: bf16 [M, K]; weight, post_weight: float32 [K]; gate, scale, shift: float32 [K], or [S, K] for S
    segments of rows: segment int32 [M] names each row's, by default they are S equal runs of rows.  Returns (result,
    h): QActTensors or bf16 [M, K] (in `out`), and bf16(h) (in sum_out, which may be x or residual)."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x: [M, K] expected, got {tuple(shape)}")
    m, k = shape
    dev = _gpu(x, "x")
    st = _stream_on(dev, stream)
    px = _ptr(x, "x", _BF16, shape, dev)
    pr = None if residual is None else _ptr(residual, "residual", _BF16, shape, dev)
    pw = None if weight is None else _ptr(weight, "weight", _F32, (k,), dev)
    pp = None if post_weight is None else _ptr(post_weight, "post_weight", _F32, (k,), dev)
    s, mods = None, [None, None, None]
    for i, v in enumerate((gate, scale, shift)):
        if v is not None:
            if s is None:
                s = v.shape[0] if v.dim() == 2 else 1
            mods[i] = _ptr(v, ("gate", "scale", "shift")[i], _F32, (s, k) if v.dim() == 2 else (k,), dev)
            if v.dim() != 2 and s != 1:
                raise ValueError(f"gate, scale and shift of {s} segments or of one")
    pseg = None
    if segment is not None:
        pseg = _ptr(segment, "segment", _I32, (m,), dev)
        if s is None:
            pseg = None  # (nothing is modulated)
    elif s is not None and s > 1 and m % s:
        raise ValueError(f"{m} rows are not {s} equal segments: segment expected")
    if sum_out is None:
        sum_out = _empty(shape, _BF16, x.device, stream)
        ps = sum_out.data_ptr()
    else:
        ps = _ptr(sum_out, "sum_out", _BF16, shape, dev)
    py = None
    qa = None
    if not quantize:
        if out is None:
            out = _empty(shape, _BF16, x.device, stream)
            py = out.data_ptr()
        else:
            py = _ptr(out, "out", _BF16, shape, dev)
    elif out is None:
        codes, rs = _empty(shape, _I8, x.device, stream), _empty((m,), _F32, x.device, stream)
        out = int8_act(codes, rs)
        qa = QAct(None, None, None, None, codes.data_ptr(), rs.data_ptr(), None)
    else:
        qa = QAct(None, None, None, None, _ptr(out.i8_codes, "out.i8_codes", _I8, shape, dev),
                  _ptr(out.row_scale, "out.row_scale", _F32, (m,), dev), None)
    if m == 0:
        return out, sum_out
    status = _lib.sixbit_gated_rmsnorm_quant(px, pr, residual_scale, pw, pp, mods[0], mods[1], mods[2], pseg,
                                             s if s is not None else 1, m, k, eps, had_block,
                                             None if mode_dev is None else _word(mode_dev, "mode_dev", dev), ps, py,
                                             None if qa is None else C.byref(qa),
                                             None if err is None else _word(err, "err", dev), st)
    if status:
        check(status, "gated_rmsnorm_quant")
    return out, sum_out


class Routing(NamedTuple):
    """moe_route's result: each token's experts int32 [T, k] and weights float32 [T, k], the row of each choice int32
    [T, k] in the order that qgemm_grouped takes, the token of each row int32 [T k], and the experts' offsets int32
    [E + 1]."""
    experts: torch.Tensor
    weights: torch.Tensor
    rows: torch.Tensor
    token: torch.Tensor
    offsets: torch.Tensor


def moe_route(logits: torch.Tensor, top_k: int, score: int = SCORE_SOFTMAX, bias: torch.Tensor | None = None,
              groups: int = 1, top_groups: int = 1, group_best: int = 2, renormalize: bool = True, scale: float = 1.0,
              out: Routing | None = None, stream=None, ws=None) -> Routing:
    """Routing of T tokens to top_k of E experts (sixbit_moe_route).

    logits: float32 or bf16 [T, E].  score: SCORE_SOFTMAX or SCORE_SIGMOID; bias: float32 [E], added for the choice and
    not to the weights.  With groups > 1 only experts of the top_groups groups are chosen, by the sum of a group's
    group_best (1 or 2) largest keys.  Equal keys go to the lower number.  The weights are the chosen experts' scores,
    divided by their sum (renormalize), times scale.  out: an earlier result of these sizes to write into; ws:
    moe_route_workspace_bytes(T, E) bytes, allocated for the call by default."""
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError(f"logits: [T, E] expected, got {tuple(shape)}")
    t, e = shape
    dev = _gpu(logits, "logits")
    st = _stream_on(dev, stream)
    if not 1 <= top_k <= min(MAX_TOP_K, e):
        raise ValueError(f"1 <= top_k <= {min(MAX_TOP_K, e)} expected, got {top_k}")
    pl = ph = None
    if logits.dtype is _BF16:
        ph = _ptr(logits, "logits", _BF16, shape, dev)
    else:
        pl = _ptr(logits, "logits", _F32, shape, dev)
    pb = None if bias is None else _ptr(bias, "bias", _F32, (e,), dev)
    tk = (t, top_k)
    if out is None:
        # (tensors of their own: views into one allocation take twice the time on the host)
        device = logits.device
        out = experts, weights, rows, token, offsets = Routing(
            _empty(tk, _I32, device, stream), _empty(tk, _F32, device, stream), _empty(tk, _I32, device, stream),
            _empty((t * top_k,), _I32, device, stream), _empty((e + 1,), _I32, device, stream))
        pe, pw, pr, pt, po = (experts.data_ptr(), weights.data_ptr(), rows.data_ptr(), token.data_ptr(), offsets.data_ptr())
    else:
        pe, pw, pr = (_ptr(out.experts, "experts", _I32, tk, dev), _ptr(out.weights, "weights", _F32, tk, dev),
                      _ptr(out.rows, "rows", _I32, tk, dev))
        pt, po = _ptr(out.token, "token", _I32, (t * top_k,), dev), _ptr(out.offsets, "offsets", _I32, (e + 1,), dev)
    need = _route_workspace_bytes(t, e)
    if ws is None:
        if need:
            ws = _empty((need,), _U8, logits.device, stream)
    elif ws.get_device() != dev or not ws.is_contiguous() or ws.numel() * ws.element_size() < need:
        raise ValueError(f"ws: {need} dense bytes on GPU {dev} expected")
    status = _lib.sixbit_moe_route(pl, ph, pb, t, e, top_k, score, groups, top_groups, group_best, renormalize, scale,
                                   pe, pw, pr, pt, po, None if ws is None else ws.data_ptr(), st)
    if status:
        check(status, "moe_route")
    return out


def moe_route_workspace_bytes(t: int, e: int) -> int:
    return int(_route_workspace_bytes(t, e))


def moe_combine(d: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor, out=None, out_f32: bool = False, err=None,
                stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] d[rows[t, j]] in FP32 (sixbit_moe_combine).  d: float32 or bf16 [R, H]; rows: int32
    [T, k] (-1: none); weights: float32 [T, k].  Returns bf16 [T, H], or float32 with out_f32 or a float32 `out`."""
    if d.dim() != 2 or rows.dim() != 2:
        raise ValueError(f"d [R, H] and rows [T, k] expected, got {tuple(d.shape)} and {tuple(rows.shape)}")
    r, h = d.shape
    t, k = shape = rows.shape
    dev = _gpu(d, "d")
    st = _stream_on(dev, stream)
    pd = pf = None
    if d.dtype is _F32:
        pf = _ptr(d, "d", _F32, d.shape, dev)
    else:
        pd = _ptr(d, "d", _BF16, d.shape, dev)
    pr, pw = _ptr(rows, "rows", _I32, shape, dev), _ptr(weights, "weights", _F32, shape, dev)
    py = pyf = None
    if out is None:
        out = _empty((t, h), _F32 if out_f32 else _BF16, d.device, stream)
        if out_f32:
            pyf = out.data_ptr()
        else:
            py = out.data_ptr()
    elif out.dtype is _F32:
        pyf = _ptr(out, "out", _F32, (t, h), dev)
    else:
        py = _ptr(out, "out", _BF16, (t, h), dev)
    status = _lib.sixbit_moe_combine(pd, pf, pr, pw, t, k, r, h, py, pyf,
                                     None if err is None else _word(err, "err", dev), st)
    if status:
        check(status, "moe_combine")
    return out


class LowRank:
    """L adapters of one projection [N, K]: a bf16 [L, R, K], b bf16 [L, N, R], alpha float32 [L] or None (1).  R is a
    multiple of 16 up to MAX_RANK.  Beside INT8 codes, a is in the codes' rotated basis (pack_lowrank)."""

    def __init__(self, a: torch.Tensor, b: torch.Tensor, alpha: torch.Tensor | None = None):
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise ValueError(f"a [L, R, K] and b [L, N, R] expected, got {tuple(a.shape)} and {tuple(b.shape)}")
        self.a, self.b, self.alpha = a, b, alpha
        self.count, self.rank, self.k = a.shape
        self.n = b.shape[1]


def pack_lowrank(a: torch.Tensor, b: torch.Tensor, alpha: torch.Tensor | None, had_block: int, stream=None) -> LowRank:
    """Adapters as they were trained (a bf16 [L, R, K], b bf16 [L, N, R], any R up to MAX_RANK) for a projection whose
    activations are rotated by had_block (0: not rotated): a is rotated in FP32 and rounded to bf16, the ranks are
    padded with zeros to a multiple of 16."""
    if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
        raise ValueError(f"a [L, R, K] and b [L, N, R] expected, got {tuple(a.shape)} and {tuple(b.shape)}")
    count, rank, k = a.shape
    n = b.shape[1]
    dev = _gpu(a, "a")
    _ptr(a, "a", _BF16, a.shape, dev)
    _ptr(b, "b", _BF16, b.shape, dev)
    if not 1 <= rank <= MAX_RANK:
        raise ValueError(f"1 <= R <= {MAX_RANK} expected, got {rank}")
    st = _stream_on(dev, stream)
    padded = (rank + 15) // 16 * 16
    with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(a.device)):
        pa = torch.zeros((count, padded, k), dtype=_BF16, device=a.device)
        pb = torch.zeros((count, n, padded), dtype=_BF16, device=a.device)
        pb[:, :, :rank] = b
        if had_block:
            rows = a.view(count * rank, k)
            q = QActTensors(count * rank, k, a.device, nvfp4=False, rotated=True)
            ca = q.c()
            check(_lib.sixbit_hadamard_quant(_p(rows), count * rank, k, had_block, MODE_INT8, None, None, C.byref(ca),
                                             None, C.c_void_p(st)), "pack_lowrank")
            pa[:, :rank] = q.rotated.view(count, rank, k)
        else:
            pa[:, :rank] = a
    return LowRank(pa, pb, alpha)


def lowrank_add(x, w: LowRank, ids: torch.Tensor, base: torch.Tensor | None = None, epilogue: int = EPI_NONE,
                residual=None, out=None, out_f32: bool = False, mode_dev=None, err=None, stream=None, ws=None):
    """out[m] = epilogue(base[m] + alpha[l] B_l (A_l x[m])), l = ids[m] (sixbit_lowrank_add).

    x: INT8 QActTensors or bf16 [M, K]; ids: int32 [M] on the GPU, -1 for rows without an adapter; base: the shared
    projection's result, float32 or bf16 [M, N], or None.  `out` may be base or residual.  ws:
    lowrank_workspace_bytes(M, R) bytes, allocated for the call by default.  Returns bf16 [M, N], or float32 with
    out_f32 or a float32 `out`."""
    if isinstance(x, torch.Tensor):
        dev = _gpu(x, "x")
        shape, device = x.shape, x.device
        if len(shape) != 2:
            raise ValueError(f"x: [M, K] expected, got {tuple(shape)}")
        ca, px = None, _ptr(x, "x", _BF16, shape, dev)
    else:
        codes = x.i8_codes
        if codes is None or codes.dim() != 2:
            raise ValueError("INT8 activations [M, K] expected")
        dev = _gpu(codes, "i8_codes")
        shape, device, px = codes.shape, codes.device, None
        ca = C.byref(QAct(None, None, None, None, _ptr(codes, "i8_codes", _I8, shape, dev),
                          _ptr(x.row_scale, "row_scale", _F32, (shape[0],), dev), None))
    m, k = shape
    n, r, count = w.n, w.rank, w.count
    if w.k != k:
        raise ValueError(f"activations have {k} inputs, the adapters {w.k}")
    st = _stream_on(dev, stream)
    pa, pb = _ptr(w.a, "a", _BF16, (count, r, k), dev), _ptr(w.b, "b", _BF16, (count, n, r), dev)
    pal = None if w.alpha is None else _ptr(w.alpha, "alpha", _F32, (count,), dev)
    pi = _ptr(ids, "ids", _I32, (m,), dev)
    p0 = p0f = py = pf = pr = None
    if base is not None:
        if base.dtype is _F32:
            p0f = _ptr(base, "base", _F32, (m, n), dev)
        else:
            p0 = _ptr(base, "base", _BF16, (m, n), dev)
    if out is None:
        out = _empty((m, n), _F32 if out_f32 else _BF16, device, stream)
        if out_f32:
            pf = out.data_ptr()
        else:
            py = out.data_ptr()
    elif out.dtype is _F32:
        pf = _ptr(out, "out", _F32, (m, n), dev)
    else:
        py = _ptr(out, "out", _BF16, (m, n), dev)
    if residual is not None:
        if epilogue != EPI_RESIDUAL:
            raise ValueError("a residual without the residual epilogue")
        pr = _ptr(residual, "residual", _BF16, (m, n), dev)
    need = _lowrank_workspace_bytes(m, r)
    if ws is None:
        if need:
            ws = _empty((need,), _U8, device, stream)
    elif ws.get_device() != dev or not ws.is_contiguous() or ws.numel() * ws.element_size() < need:
        raise ValueError(f"ws: {need} dense bytes on GPU {dev} expected")
    status = _lib.sixbit_lowrank_add(ca, px, pa, pb, pal, pi, count, m, n, k, r, p0, p0f,
                                     None if mode_dev is None else _word(mode_dev, "mode_dev", dev), epilogue, pr, py,
                                     pf, None if ws is None else ws.data_ptr(), None if err is None else _word(err, "err", dev), st)
    if status:
        check(status, "lowrank_add")
    return out


def lowrank_workspace_bytes(m: int, r: int) -> int:
    return int(_lowrank_workspace_bytes(m, r))


def check_err(err: torch.Tensor, what: str, stream=None) -> None:
    """Waits for `stream` (None: the current one), clears the error word and raises SixbitError with what the calls that
    were given it recorded there (sixbit_check)."""
    dev = err.get_device()
    check(_lib.sixbit_check(_word(err, "err", dev), _stream_on(dev, stream)), what)


def policy_cfg(gamma_thr=0.1, cos_thr=0.99, err_cap=0.05, pdr_ratio=30.0, near_rel=1e-6, refresh_bf16=False):
    return PolicyCfg(gamma_thr, cos_thr, err_cap, pdr_ratio, near_rel, int(refresh_bf16), 0)


def policy_step(cfg: PolicyCfg, state: torch.Tensor, last_stats: torch.Tensor, in_stats: torch.Tensor,
                mode_word: torch.Tensor, stream=None):
    check(_lib.sixbit_policy_step(C.byref(cfg), _p(state), _p(last_stats), _p(in_stats), _p(mode_word), None,
                                  _stream(stream)), "policy_step")
    return mode_word


def policy_cfgs_tensor(cfgs, device="cuda") -> torch.Tensor:
    """Per-block thresholds as the device array sixbit_dit_blocks.block_cfg points to."""
    raw = b"".join(bytes(c) for c in cfgs)
    return torch.frombuffer(bytearray(raw), dtype=torch.uint8).to(device)


def dit_blocks(states, stats, modes, run_len, in_stats0, x0, buf0, buf1, deltas, conds=None,
               delta_scales=None, block_cfg=None) -> DitBlocks:
    """The sixbit_dit_blocks record of a stack of residual blocks (device tensors; deltas [L, ...];
    run_len: int32 [L], zeroed; conds: int64 [L] graph condition handles, or None).  The Delta
    cache is bf16 (deltas bf16 [L, n]) or, with delta_scales, MXFP8 (deltas uint8 [L, n] E4M3
    codes, delta_scales uint8 [L, n / 32] E8M0 codes).  block_cfg: the policy_cfgs_tensor of L
    per-block thresholds, or None."""
    L = states.shape[0]
    n = x0.numel()
    assert stats.shape[0] == L and modes.numel() == L and run_len.numel() == L and deltas.shape[0] == L
    assert run_len.dtype == torch.int32 and run_len.is_contiguous() and deltas.numel() == L * n
    assert in_stats0.dtype == torch.float64 and in_stats0.numel() >= 4
    assert conds is None or (conds.dtype == torch.int64 and conds.numel() == L)
    if delta_scales is None:
        assert deltas.dtype == torch.bfloat16
        fmt = DELTA_BF16
    else:
        assert deltas.dtype == torch.uint8 and delta_scales.dtype == torch.uint8
        assert delta_scales.is_contiguous() and delta_scales.numel() == L * (n // MX_BLOCK)
        fmt = DELTA_MXFP8
    assert block_cfg is None or (block_cfg.dtype == torch.uint8 and block_cfg.numel() == L * C.sizeof(PolicyCfg))
    return DitBlocks(_p(states), _p(stats), _p(modes), _p(in_stats0), _p(x0),
                     (C.c_void_p * 2)(buf0.data_ptr(), buf1.data_ptr()), _p(deltas), _p(delta_scales), _p(run_len),
                     _p(conds), _p(block_cfg), n, L, fmt)


def dit_begin(cfg: PolicyCfg, blocks: DitBlocks, scratch: torch.Tensor, err=None, stream=None):
    """sixbit_dit_begin: statistics of the step input, then block 0's decision."""
    check(_lib.sixbit_dit_begin(C.byref(cfg), C.byref(blocks), _p(scratch), _p(err), _stream(stream)), "dit_begin")


def dit_block_end_parts(cfg: PolicyCfg, blocks: DitBlocks, l: int, parts: torch.Tensor, err=None, stream=None):
    """sixbit_dit_block_end_parts: fold the statistics block l's down projection wrote to parts, then
    block l+1's decision (nothing when block l skipped)."""
    check(_lib.sixbit_dit_block_end_parts(C.byref(cfg), C.byref(blocks), l, _p(parts), _p(err), _stream(stream)),
          "dit_block_end_parts")


def dit_block_end(cfg: PolicyCfg, blocks: DitBlocks, l: int, scratch: torch.Tensor, err=None, stream=None):
    """sixbit_dit_block_end: block l's statistics and Delta update (if it computed), then block l+1's decision."""
    check(_lib.sixbit_dit_block_end(C.byref(cfg), C.byref(blocks), l, _p(scratch), _p(err), _stream(stream)),
          "dit_block_end")


def dit_skip_run(cfg: PolicyCfg, blocks: DitBlocks, l: int, scratch: torch.Tensor, err=None, stream=None):
    """sixbit_dit_skip_run: the run of skips block l starts (if any), then the decisions up to its end + 1."""
    check(_lib.sixbit_dit_skip_run(C.byref(cfg), C.byref(blocks), l, _p(scratch), _p(err), _stream(stream)),
          "dit_skip_run")


def graph_cond_create(stream, nbranches: int) -> int:
    """A conditional handle in the graph `stream` is capturing (default value: no body)."""
    h = C.c_uint64()
    check(_lib.sixbit_graph_cond_create(C.c_void_p(stream.cuda_stream), nbranches, C.byref(h)), "graph_cond_create")
    return int(h.value)


class GraphSwitch:
    """A device-selected branch in the CUDA graph being captured on `stream` (sixbit_graph_switch_*).

    Body i runs when the low byte of mode_word equals first_mode + i.  Use
    ``with sw.branch(i):`` to capture body i: inside it the current torch
    stream is `body_stream`, which is capturing into that body.
    """

    def __init__(self, stream, body_stream, mode_word: torch.Tensor | None, first_mode: int, nbranches: int,
                 cond: int | None = None):
        """With cond (a handle from graph_cond_create, set by a kernel already captured) no selector is added."""
        self.h = C.c_void_p()
        self.body_stream = body_stream
        if cond is not None:
            check(_lib.sixbit_graph_switch_begin_cond(C.c_void_p(stream.cuda_stream),
                                                      C.c_void_p(body_stream.cuda_stream), cond, nbranches,
                                                      C.byref(self.h)), "graph_switch_begin_cond")
        else:
            check(_lib.sixbit_graph_switch_begin(C.c_void_p(stream.cuda_stream),
                                                 C.c_void_p(body_stream.cuda_stream), _p(mode_word), first_mode,
                                                 nbranches, C.byref(self.h)), "graph_switch_begin")

    def branch(self, i: int):
        sw = self

        class _Branch:
            def __enter__(self):
                s = C.c_void_p()
                check(_lib.sixbit_graph_branch_begin(sw.h, i, C.byref(s)), "graph_branch_begin")
                self.ctx = torch.cuda.stream(sw.body_stream)
                self.ctx.__enter__()
                return sw.body_stream

            def __exit__(self, *exc):
                self.ctx.__exit__(*exc)
                check(_lib.sixbit_graph_branch_end(sw.h), "graph_branch_end")
                return False

        return _Branch()

    def close(self):
        check(_lib.sixbit_graph_switch_end(self.h), "graph_switch_end")


def new_stats(device="cuda", count: int = 1) -> torch.Tensor:
    """Zeroed device storage for `count` sixbit_stats records (float64 x 8 each)."""
    return torch.zeros((count, 8), dtype=torch.float64, device=device)


def new_policy_state(device="cuda", count: int = 1) -> torch.Tensor:
    """Zeroed device storage for `count` sixbit_policy_state records (80 bytes each)."""
    assert C.sizeof(PolicyState) == 80
    return torch.zeros((count, 80), dtype=torch.uint8, device=device)


def decode_state(raw: torch.Tensor) -> PolicyState:
    b = bytes(raw.cpu().numpy().tobytes())
    return PolicyState.from_buffer_copy(b)


def new_scratch(n: int, device="cuda") -> torch.Tensor:
    """Zeroed scratch for the statistics kernels (its counter must start at zero)."""
    return torch.zeros(stats_scratch_bytes(n), dtype=torch.uint8, device=device)
