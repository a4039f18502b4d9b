"""ctypes binding of libsdverify.so: argument marshalling only.

Every step of the verify path runs in the library's HIP kernels; this module
checks tensor dtypes, devices and shapes, allocates outputs with torch when
the caller does not pass them, and forwards raw device pointers plus the
current HIP stream. There is no fallback: if the shared library is missing,
importing this module raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsdverify.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")

_lib = ctypes.CDLL(LIB_PATH)

_i32, _i64, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_sz, _vp = ctypes.c_size_t, ctypes.c_void_p
_SIGS = {
    "sd_abi_version": (_i32, []),
    "sd_status_string": (ctypes.c_char_p, [_i32]),
    "sd_verify_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "sd_accept_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "sd_workspace_init": (_i32, [_vp, _sz, _vp]),
    "sd_device_flags": (_i32, [_vp, _vp, ctypes.POINTER(ctypes.c_uint32), _i32]),
    "sd_truncate_by_confidence": (_i32, [_vp, _i32, _i32, _f32, _vp, _vp, _vp]),
    "sd_schedule_prefix": (_i32, [_vp, _vp, _i32, _i32, _vp, _i32, _i32, _vp, _vp, _vp]),
    "sd_w12_encode": (_i32, [_vp, _i32, _i32, _vp, _vp, _vp, _vp]),
    "sd_verify_logits_w12": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _f32, _vp, _vp,
                                    _vp, _sz, _vp]),
    "sd_verify_contraction_w12": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _f32, _vp, _vp,
                                         _sz, _vp]),
    "sd_verify_greedy_w12": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp,
                                    _vp, _vp, _sz, _vp]),
    "sd_verify_logits": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _f32, _vp, _vp,
                                _vp, _sz, _vp]),
    "sd_lm_head_block_bytes": (_sz, [_i32, _i32]),
    "sd_lm_head_block": (_i32, [_vp, _i32, _i32, _vp, _sz, _vp]),
    "sd_verify_logits_blocked": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _f32, _vp,
                                        _vp, _vp, _sz, _vp]),
    "sd_verify_contraction_blocked": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _f32, _vp,
                                             _vp, _sz, _vp]),
    "sd_verify_greedy_blocked": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp,
                                        _vp, _vp, _vp, _sz, _vp]),
    "sd_verify_contraction": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _sz,
                                     _vp]),
    "sd_verify_greedy": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                _vp, _sz, _vp]),
    "sd_verify_greedy_noalloc": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp,
                                        _vp, _vp, _vp, _vp]),
    "sd_accept_greedy": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp]),
    "sd_accept_rejection": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _f32,
                                   _vp, _vp, _vp, _vp, _sz, _vp]),
    "sd_accept_rejection_ex": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                                      _f32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sd_verify_rejection": (_i32, [_vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                                   _i32, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _sz,
                                   _vp]),
    "sd_mxfp4_columns": (_i32, [_i32]),
    "sd_mxfp4_quantize": (_i32, [_vp, _i32, _i32, _i32, _i64, _vp, _vp, _vp]),
    "sd_mxfp4_dequantize": (_i32, [_vp, _vp, _i32, _i32, _vp, _i32, _i64, _vp]),
    "sd_mxfp4_head_bytes": (_sz, [_i32, _i32]),
    "sd_mxfp4_head": (_i32, [_vp, _vp, _i32, _i32, _vp, _sz, _vp]),
    "sd_mxfp4_logits_workspace_bytes": (_sz, [_i32, _i32]),
    "sd_mxfp4_logits": (_i32, [_vp, _i32, _i32, _i32, _i64, _vp, _i32, _vp, _i32, _i64, _vp, _sz,
                               _vp]),
    "sd_sample_workspace_bytes": (_sz, [_i32, _i32]),
    "sd_sample": (_i32, [_vp, _i32, _i64, _i32, _i32, _vp, _vp, _i32, _vp, _i64, _vp, _vp, _vp,
                         _sz, _vp]),
    "sd_accept_filtered_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "sd_accept_filtered": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp,
                                  _vp, _vp, _vp, _sz, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)

# Layout of sd_row_stats (32 bytes).
ROW_STATS_DTYPE = np.dtype([("argmax", "<i4"), ("top1", "<f4"), ("top2", "<f4"), ("pos", "<i4"),
                            ("lse", "<f8"), ("z_draft", "<f8")])
assert ROW_STATS_DTYPE.itemsize == 32

FLAG_VERIFY_LEN, FLAG_ROW_OFFSETS, FLAG_NO_RESIDUAL, FLAG_WAIT = 1, 2, 4, 8
FLAG_SAMPLING, FLAG_EMPTY_ROW = 16, 32
LM_HEAD_ROWS, LM_HEAD_BLOCKED, LM_HEAD_W12 = 0, 1, 2


class SdError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {_lib.sd_status_string(status).decode()} (status {status})")
        self.status = status


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise SdError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        # The current stream's handle without a Stream object around it: 0.3 us, not 3.
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t: torch.Tensor, name: str, dtype, shape=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def abi_version() -> int:
    return int(_lib.sd_abi_version())


def verify_workspace_bytes(B: int, gamma: int, d: int, V: int) -> int:
    return int(_lib.sd_verify_workspace_bytes(B, gamma, d, V))


def accept_workspace_bytes(B: int, gamma: int, V: int) -> int:
    return int(_lib.sd_accept_workspace_bytes(B, gamma, V))


def new_workspace(nbytes: int, device, stream=None) -> torch.Tensor:
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    _check("sd_workspace_init", _lib.sd_workspace_init(_ptr(ws), ws.numel(), _stream(stream)))
    return ws


def device_flags(workspace: torch.Tensor, clear: bool = True, stream=None) -> int:
    out = ctypes.c_uint32(0)
    _check("sd_device_flags", _lib.sd_device_flags(_ptr(workspace), _stream(stream),
                                                   ctypes.byref(out), int(clear)))
    return int(out.value)


def new_stats(B: int, gamma: int, device) -> torch.Tensor:
    """Device buffer for B * (gamma + 1) sd_row_stats records (viewed as int64 [rows][4])."""
    return torch.empty((B * (gamma + 1), 4), dtype=torch.int64, device=device)


def stats_to_numpy(stats: torch.Tensor) -> np.ndarray:
    """Host copy of a stats buffer as a structured array with the sd_row_stats fields."""
    return stats.detach().cpu().numpy().view(ROW_STATS_DTYPE).reshape(-1)


# ------------------------------------------------------------------ entry points

def sd_truncate_by_confidence(conf: torch.Tensor, threshold: float,
                              verify_len: Optional[torch.Tensor] = None,
                              row_offsets: Optional[torch.Tensor] = None, stream=None):
    _need(conf, "conf", torch.float32)
    B, g = conf.shape
    if verify_len is None:
        verify_len = torch.empty(B, dtype=torch.int32, device=conf.device)
    if row_offsets is None:
        row_offsets = torch.empty(B + 1, dtype=torch.int32, device=conf.device)
    _need(verify_len, "verify_len", torch.int32, (B,))
    _need(row_offsets, "row_offsets", torch.int32, (B + 1,))
    _check("sd_truncate_by_confidence",
           _lib.sd_truncate_by_confidence(_ptr(conf), B, g, float(threshold), _ptr(verify_len),
                                          _ptr(row_offsets), _stream(stream)))
    return verify_len, row_offsets


SCHED_EARLY_STOP, SCHED_TOP_K = 0, 1
SCHED_MAX_CANDIDATES = 16384


def sd_schedule_prefix(conf: torch.Tensor, sps: torch.Tensor, mode: int = SCHED_EARLY_STOP,
                       conf_stale: Optional[torch.Tensor] = None,
                       verify_len: Optional[torch.Tensor] = None,
                       row_offsets: Optional[torch.Tensor] = None, stream=None):
    """Hardware-aware prefix scheduler; same outputs as sd_truncate_by_confidence."""
    _need(conf, "conf", torch.float32)
    R, g = conf.shape
    _need(sps, "sps", torch.float32)
    if conf_stale is not None:
        _need(conf_stale, "conf_stale", torch.float32, (R, g))
    if verify_len is None:
        verify_len = torch.empty(R, dtype=torch.int32, device=conf.device)
    if row_offsets is None:
        row_offsets = torch.empty(R + 1, dtype=torch.int32, device=conf.device)
    _need(verify_len, "verify_len", torch.int32, (R,))
    _need(row_offsets, "row_offsets", torch.int32, (R + 1,))
    _check("sd_schedule_prefix",
           _lib.sd_schedule_prefix(_ptr(conf), _ptr(conf_stale), R, g, _ptr(sps), sps.numel(),
                                   int(mode), _ptr(verify_len), _ptr(row_offsets),
                                   _stream(stream)))
    return verify_len, row_offsets


def profile_sps(R: int, gamma: int, lm_head: torch.Tensor, temperature: float = 0.0,
                breakpoints: Optional[Sequence[int]] = None, repeats: int = 10,
                stream=None) -> torch.Tensor:
    """Steps-per-second table SPS(B), B = 0 .. R * (gamma + 1), of this library's own verify
    call (sd_verify_logits) for R requests with gamma drafts each.

    The verify cost is a staircase in the number of rows B (the contraction works on
    row tiles), so it is timed at the top of each stair -- every multiple of 256 rows
    and the full capacity, by default -- and every B takes the rate of the first timed
    point at or above it. Returns fp32 [R * (gamma + 1) + 1] on lm_head's device.
    """
    _need(lm_head, "lm_head", torch.bfloat16)
    V, d = lm_head.shape
    dev = lm_head.device
    cap = R * (gamma + 1)
    if breakpoints is None:
        breakpoints = sorted({min(cap, max(R, 256 * i)) for i in range(1, cap // 256 + 1)} | {cap})
    breakpoints = sorted({int(b) for b in breakpoints if R <= int(b) <= cap} | {cap})
    gen = torch.Generator(device="cpu").manual_seed(1234)
    hidden = (torch.randn((R, gamma + 1, d), generator=gen) / 4).to(torch.bfloat16).to(dev)
    drafts = torch.randint(0, V, (R, gamma), generator=gen, dtype=torch.int32).to(dev)
    stats = new_stats(R, gamma, dev)
    logits = (torch.empty((cap, V), dtype=torch.float32, device=dev) if temperature > 0
              else None)
    ws = new_workspace(verify_workspace_bytes(R, gamma, d, V), dev, stream)
    st = torch.cuda.Stream(device=dev) if stream is None else stream
    times = []
    for rows in breakpoints:
        extra = rows - R
        L = [min(gamma, max(0, extra - gamma * r)) for r in range(R)]
        offs = [0]
        for x in L:
            offs.append(offs[-1] + x + 1)
        vl = torch.tensor(L, dtype=torch.int32, device=dev)
        ro = torch.tensor(offs, dtype=torch.int32, device=dev)
        with torch.cuda.stream(st):
            for _ in range(2):
                sd_verify_logits(hidden, lm_head, drafts, vl, ro, temperature, logits, stats, ws,
                                 stream=st)
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record(st)
            for _ in range(repeats):
                sd_verify_logits(hidden, lm_head, drafts, vl, ro, temperature, logits, stats, ws,
                                 stream=st)
            e1.record(st)
        e1.synchronize()
        times.append(e0.elapsed_time(e1) / repeats)
    sps = torch.empty(cap + 1, dtype=torch.float32)
    i = 0
    for B in range(cap + 1):
        while breakpoints[i] < B:
            i += 1
        sps[B] = 1e3 / times[i]
    return sps.to(dev)


class _SdW12(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("corr", ctypes.c_void_p), ("cap", ctypes.c_int32),
                ("b2", ctypes.c_int32)]


def w12_encode(W_bits: np.ndarray):
    """Host W12 encoding of a bf16 LM head (uint16 bit patterns [V][d]) by the library's
    sd_w12_encode: returns (codes uint8 [V/64][d/128][64][16][12] (region-blocked),
    corr uint32 [V/64][d/128][cap], cap, b2, V)."""
    W_bits = np.ascontiguousarray(W_bits, dtype=np.uint16)
    V, d = W_bits.shape
    cap, b2 = ctypes.c_int32(0), ctypes.c_int32(0)
    _check("sd_w12_encode", _lib.sd_w12_encode(W_bits.ctypes.data, V, d, None, None,
                                               ctypes.byref(cap), ctypes.byref(b2)))
    codes = np.empty(((V + 63) // 64, d // 128, 64, 16, 12), dtype=np.uint8)
    corr = np.empty(((V + 63) // 64, d // 128, cap.value), dtype=np.uint32)
    _check("sd_w12_encode", _lib.sd_w12_encode(W_bits.ctypes.data, V, d, codes.ctypes.data,
                                               corr.ctypes.data, ctypes.byref(cap),
                                               ctypes.byref(b2)))
    return codes, corr, int(cap.value), int(b2.value), V


class _Handle:
    """Attributes that are fixed once made: calls read device memory at the addresses and sizes
    that were checked then."""

    def __setattr__(self, name, value):
        if "_made" in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name} is fixed: write into its tensors, "
                                 "or make another")
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        raise AttributeError(f"{type(self).__name__}.{name} is fixed")


class W12Weights:
    """A W12 LM head in device memory: 12-byte groups, correction slots, window start.
    Pass it as `lm_head` to sd_verify_logits / sd_verify_greedy / VerifyRound."""

    def __init__(self, codes: np.ndarray, corr: np.ndarray, cap: int, b2: int, V: int,
                 device="cuda"):
        self.V, self.d = int(V), codes.shape[1] * 128
        self.cap, self.b2 = int(cap), int(b2)
        self.codes = torch.from_numpy(np.ascontiguousarray(codes)).to(device)
        self.corr = torch.from_numpy(np.ascontiguousarray(corr).view(np.int32)).to(device)
        self.shape = (self.V, self.d)
        self.nbytes = self.codes.numel() + 4 * self.corr.numel()

    @classmethod
    def from_bf16(cls, W_bits: np.ndarray, device="cuda") -> "W12Weights":
        return cls(*w12_encode(W_bits), device=device)

    def descriptor(self):
        # From the tensors as they are: a kept address would outlive one that is replaced.
        return ctypes.byref(_SdW12(self.codes.data_ptr(), self.corr.data_ptr(), self.cap, self.b2))


def sd_verify_logits_w12(hidden, lm_head: W12Weights, *args, **kwargs):
    return sd_verify_logits(hidden, lm_head, *args, **kwargs)


def sd_verify_contraction_w12(hidden, lm_head: W12Weights, *args, **kwargs):
    return sd_verify_contraction(hidden, lm_head, *args, **kwargs)


def sd_verify_greedy_w12(hidden, lm_head: W12Weights, *args, **kwargs):
    return sd_verify_greedy(hidden, lm_head, *args, **kwargs)


class BlockedWeights:
    """A bf16 LM head re-laid once into slab blocks (sd_lm_head_block) so the streaming
    contraction reads each stage as one contiguous 16 KB block. Same values as the
    [V][d] tensor; pass it as `lm_head` to sd_verify_logits / sd_verify_greedy /
    VerifyRound (the streaming regime: d % 128 == 0, B * (gamma + 1) <= 64)."""

    def __init__(self, lm_head: torch.Tensor, stream=None):
        _need(lm_head, "lm_head", torch.bfloat16)
        V, d = lm_head.shape
        nbytes = int(_lib.sd_lm_head_block_bytes(V, d))
        if nbytes == 0:
            raise ValueError(f"no blocked layout for a [{V}][{d}] LM head (d % 128 != 0)")
        self.V, self.d, self.shape, self.nbytes = int(V), int(d), (int(V), int(d)), nbytes
        self.buf = torch.empty(nbytes // 2, dtype=torch.bfloat16, device=lm_head.device)
        _check("sd_lm_head_block", _lib.sd_lm_head_block(_ptr(lm_head), V, d, _ptr(self.buf),
                                                         nbytes, _stream(stream)))


def _lm_head(lm_head, d):
    """(pointer or descriptor, V, entry-point suffix) of a bf16 LM head tensor,
    W12Weights or BlockedWeights."""
    if isinstance(lm_head, (W12Weights, BlockedWeights)):
        if lm_head.d != d:
            raise ValueError("lm_head must be [V][d] with the hidden size of `hidden`")
        if isinstance(lm_head, W12Weights):
            return lm_head.descriptor(), lm_head.V, "_w12"
        return _ptr(lm_head.buf), lm_head.V, "_blocked"
    _need(lm_head, "lm_head", torch.bfloat16)
    if lm_head.shape[1] != d:
        raise ValueError("lm_head must be [V][d] with the hidden size of `hidden`")
    return _ptr(lm_head), lm_head.shape[0], ""


def sd_verify_logits(hidden: torch.Tensor, lm_head: torch.Tensor,
                     draft_tokens: Optional[torch.Tensor] = None,
                     verify_len: Optional[torch.Tensor] = None,
                     row_offsets: Optional[torch.Tensor] = None, temperature: float = 0.0,
                     logits: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Returns (logits or None, stats). Pass logits=True to have one allocated.
    lm_head: bf16 [V][d] tensor, W12Weights (then sd_verify_logits_w12 runs) or
    BlockedWeights (sd_verify_logits_blocked)."""
    _need(hidden, "hidden", torch.bfloat16)
    B, g1, d = hidden.shape
    g = g1 - 1
    head, V, fmt = _lm_head(lm_head, d)
    dev = hidden.device
    if draft_tokens is not None:
        _need(draft_tokens, "draft_tokens", torch.int32, (B, g))
    if verify_len is not None:
        _need(verify_len, "verify_len", torch.int32, (B,))
    if row_offsets is not None:
        _need(row_offsets, "row_offsets", torch.int32, (B + 1,))
    if logits is True:
        logits = torch.empty((B * g1, V), dtype=torch.float32, device=dev)
    if logits is not None:
        _need(logits, "logits", torch.float32, (B * g1, V))
    if stats is None:
        stats = new_stats(B, g, dev)
    _need(stats, "stats", torch.int64, (B * g1, 4))
    if workspace is None:
        workspace = new_workspace(verify_workspace_bytes(B, g, d, V), dev, stream)
    name = "sd_verify_logits" + fmt
    _check(name, getattr(_lib, name)(_ptr(hidden), head, _ptr(draft_tokens), _ptr(verify_len),
                                     _ptr(row_offsets), B, g, d, V, float(temperature),
                                     _ptr(logits), _ptr(stats), _ptr(workspace),
                                     workspace.numel(), _stream(stream)))
    return logits, stats


def sd_verify_contraction(hidden: torch.Tensor, lm_head: torch.Tensor,
                          verify_len: Optional[torch.Tensor] = None,
                          row_offsets: Optional[torch.Tensor] = None, temperature: float = 0.0,
                          logits: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """The contraction stage alone (logits and workspace partials, no row statistics).
    lm_head: bf16 [V][d] tensor, W12Weights (then sd_verify_contraction_w12 runs) or
    BlockedWeights (sd_verify_contraction_blocked)."""
    _need(hidden, "hidden", torch.bfloat16)
    B, g1, d = hidden.shape
    head, V, fmt = _lm_head(lm_head, d)
    if logits is not None:
        _need(logits, "logits", torch.float32, (B * g1, V))
    if workspace is None:
        workspace = new_workspace(verify_workspace_bytes(B, g1 - 1, d, V), hidden.device, stream)
    name = "sd_verify_contraction" + fmt
    _check(name, getattr(_lib, name)(_ptr(hidden), head, _ptr(verify_len), _ptr(row_offsets), B,
                                     g1 - 1, d, V, float(temperature), _ptr(logits),
                                     _ptr(workspace), workspace.numel(), _stream(stream)))
    return logits


def sd_verify_greedy(hidden: torch.Tensor, lm_head: torch.Tensor, draft_tokens: torch.Tensor,
                     verify_len: Optional[torch.Tensor] = None,
                     row_offsets: Optional[torch.Tensor] = None,
                     stats: Optional[torch.Tensor] = None,
                     accept_len: Optional[torch.Tensor] = None,
                     next_token: Optional[torch.Tensor] = None,
                     counters: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Greedy verify in one call: returns (stats, accept_len, next_token).
    lm_head: bf16 [V][d] tensor, W12Weights (then sd_verify_greedy_w12 runs) or
    BlockedWeights (sd_verify_greedy_blocked)."""
    _need(hidden, "hidden", torch.bfloat16)
    B, g1, d = hidden.shape
    g = g1 - 1
    head, V, fmt = _lm_head(lm_head, d)
    dev = hidden.device
    _need(draft_tokens, "draft_tokens", torch.int32, (B, g))
    if verify_len is not None:
        _need(verify_len, "verify_len", torch.int32, (B,))
    if row_offsets is not None:
        _need(row_offsets, "row_offsets", torch.int32, (B + 1,))
    stats = new_stats(B, g, dev) if stats is None else stats
    _need(stats, "stats", torch.int64, (B * g1, 4))
    accept_len = torch.empty(B, dtype=torch.int32, device=dev) if accept_len is None else accept_len
    next_token = torch.empty(B, dtype=torch.int32, device=dev) if next_token is None else next_token
    _need(accept_len, "accept_len", torch.int32, (B,))
    _need(next_token, "next_token", torch.int32, (B,))
    if counters is not None:
        _need(counters, "counters", torch.int64, (2,))
    if workspace is None:
        workspace = new_workspace(verify_workspace_bytes(B, g, d, V), dev, stream)
    name = "sd_verify_greedy" + fmt
    _check(name, getattr(_lib, name)(_ptr(hidden), head, _ptr(draft_tokens), _ptr(verify_len),
                                     _ptr(row_offsets), B, g, d, V, _ptr(stats), _ptr(accept_len),
                                     _ptr(next_token), _ptr(counters), _ptr(workspace),
                                     workspace.numel(), _stream(stream)))
    return stats, accept_len, next_token


NOALLOC_SCRATCH_BYTES = 16 << 20


def sd_verify_greedy_noalloc(hidden: torch.Tensor, lm_head: torch.Tensor,
                             draft_tokens: torch.Tensor, verify_len: Optional[torch.Tensor] = None,
                             row_offsets: Optional[torch.Tensor] = None,
                             stats: torch.Tensor = None, accept_len: torch.Tensor = None,
                             next_token: torch.Tensor = None,
                             counters: Optional[torch.Tensor] = None,
                             flags: Optional[torch.Tensor] = None, stream=None):
    """sd_verify_greedy with the library's own per-GPU scratch instead of a workspace.
    The caller passes every output (stats, accept_len, next_token; counters and the
    uint32 flag word optional), so the call allocates nothing; bf16 [V][d] LM head."""
    _need(hidden, "hidden", torch.bfloat16)
    B, g1, d = hidden.shape
    g = g1 - 1
    _need(lm_head, "lm_head", torch.bfloat16)
    V = lm_head.shape[0]
    _need(lm_head, "lm_head", torch.bfloat16, (V, d))
    _need(draft_tokens, "draft_tokens", torch.int32, (B, g))
    if verify_len is not None:
        _need(verify_len, "verify_len", torch.int32, (B,))
    if row_offsets is not None:
        _need(row_offsets, "row_offsets", torch.int32, (B + 1,))
    if stats is None or accept_len is None or next_token is None:
        raise ValueError("sd_verify_greedy_noalloc: pass stats, accept_len and next_token")
    _need(stats, "stats", torch.int64, (B * g1, 4))
    _need(accept_len, "accept_len", torch.int32, (B,))
    _need(next_token, "next_token", torch.int32, (B,))
    if counters is not None:
        _need(counters, "counters", torch.int64, (2,))
    if flags is not None:
        _need(flags, "flags", torch.int32, (1,))
    _check("sd_verify_greedy_noalloc",
           _lib.sd_verify_greedy_noalloc(_ptr(hidden), _ptr(lm_head), _ptr(draft_tokens),
                                         _ptr(verify_len), _ptr(row_offsets), B, g, d, V,
                                         _ptr(stats), _ptr(accept_len), _ptr(next_token),
                                         _ptr(counters), _ptr(flags), _stream(stream)))
    return stats, accept_len, next_token


def sd_accept_greedy(stats: torch.Tensor, draft_tokens: torch.Tensor,
                     verify_len: Optional[torch.Tensor] = None,
                     row_offsets: Optional[torch.Tensor] = None,
                     accept_len: Optional[torch.Tensor] = None,
                     next_token: Optional[torch.Tensor] = None,
                     counters: Optional[torch.Tensor] = None, stream=None):
    _need(draft_tokens, "draft_tokens", torch.int32)
    B, g = draft_tokens.shape
    dev = draft_tokens.device
    _need(stats, "stats", torch.int64, (B * (g + 1), 4))
    accept_len = torch.empty(B, dtype=torch.int32, device=dev) if accept_len is None else accept_len
    next_token = torch.empty(B, dtype=torch.int32, device=dev) if next_token is None else next_token
    _need(accept_len, "accept_len", torch.int32, (B,))
    _need(next_token, "next_token", torch.int32, (B,))
    if counters is not None:
        _need(counters, "counters", torch.int64, (2,))
    _check("sd_accept_greedy",
           _lib.sd_accept_greedy(_ptr(stats), _ptr(draft_tokens), _ptr(verify_len),
                                 _ptr(row_offsets), B, g, _ptr(accept_len), _ptr(next_token),
                                 _ptr(counters), _stream(stream)))
    return accept_len, next_token


def sd_accept_rejection(logits: torch.Tensor, stats: torch.Tensor, draft_logits: torch.Tensor,
                        draft_tokens: torch.Tensor, verify_len: Optional[torch.Tensor],
                        row_offsets: Optional[torch.Tensor], u_accept: torch.Tensor,
                        u_resample: torch.Tensor, temperature: float,
                        accept_len: Optional[torch.Tensor] = None,
                        next_token: Optional[torch.Tensor] = None,
                        counters: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    accept_len, next_token, _ = _accept_rejection(
        "sd_accept_rejection", logits, stats, draft_logits, draft_tokens, verify_len, row_offsets,
        u_accept, u_resample, temperature, accept_len, next_token, counters, None, workspace,
        stream)
    return accept_len, next_token


def sd_accept_rejection_ex(logits: torch.Tensor, stats: torch.Tensor, draft_logits: torch.Tensor,
                           draft_tokens: torch.Tensor, verify_len: Optional[torch.Tensor],
                           row_offsets: Optional[torch.Tensor], u_accept: torch.Tensor,
                           u_resample: torch.Tensor, temperature: float,
                           accept_len: Optional[torch.Tensor] = None,
                           next_token: Optional[torch.Tensor] = None,
                           counters: Optional[torch.Tensor] = None,
                           accept_rate: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """sd_accept_rejection plus accept_rate float64 [B][gamma] (allocated when None)."""
    B, g = draft_tokens.shape
    if accept_rate is None:
        accept_rate = torch.empty((B, g), dtype=torch.float64, device=draft_tokens.device)
    return _accept_rejection("sd_accept_rejection_ex", logits, stats, draft_logits, draft_tokens,
                             verify_len, row_offsets, u_accept, u_resample, temperature,
                             accept_len, next_token, counters, accept_rate, workspace, stream)


def _accept_rejection(name, logits, stats, draft_logits, draft_tokens, verify_len, row_offsets,
                      u_accept, u_resample, temperature, accept_len, next_token, counters,
                      accept_rate, workspace, stream):
    _need(draft_tokens, "draft_tokens", torch.int32)
    B, g = draft_tokens.shape
    dev = draft_tokens.device
    _need(draft_logits, "draft_logits", torch.bfloat16)
    V = draft_logits.shape[2]
    _need(draft_logits, "draft_logits", torch.bfloat16, (B, g, V))
    _need(logits, "logits", torch.float32, (B * (g + 1), V))
    _need(stats, "stats", torch.int64, (B * (g + 1), 4))
    _need(u_accept, "u_accept", torch.float32, (B, g))
    _need(u_resample, "u_resample", torch.float32, (B, g + 1))
    accept_len = torch.empty(B, dtype=torch.int32, device=dev) if accept_len is None else accept_len
    next_token = torch.empty(B, dtype=torch.int32, device=dev) if next_token is None else next_token
    if counters is not None:
        _need(counters, "counters", torch.int64, (2,))
    if workspace is None:
        workspace = new_workspace(accept_workspace_bytes(B, g, V), dev, stream)
    args = [_ptr(logits), _ptr(stats), _ptr(draft_logits), _ptr(draft_tokens), _ptr(verify_len),
            _ptr(row_offsets), _ptr(u_accept), _ptr(u_resample), B, g, V, float(temperature),
            _ptr(accept_len), _ptr(next_token), _ptr(counters)]
    if name == "sd_accept_rejection_ex":
        _need(accept_rate, "accept_rate", torch.float64, (B, g))
        args.append(_ptr(accept_rate))
    args += [_ptr(workspace), workspace.numel(), _stream(stream)]
    _check(name, getattr(_lib, name)(*args))
    return accept_len, next_token, accept_rate


def sd_verify_rejection(hidden: torch.Tensor, lm_head, draft_tokens: torch.Tensor,
                        draft_logits: torch.Tensor, verify_len: Optional[torch.Tensor],
                        row_offsets: Optional[torch.Tensor], u_accept: torch.Tensor,
                        u_resample: torch.Tensor, temperature: float,
                        logits: Optional[torch.Tensor] = None,
                        stats: Optional[torch.Tensor] = None,
                        accept_len: Optional[torch.Tensor] = None,
                        next_token: Optional[torch.Tensor] = None,
                        counters: Optional[torch.Tensor] = None,
                        accept_rate: Optional[torch.Tensor] = None,
                        ws_verify: Optional[torch.Tensor] = None,
                        ws_accept: Optional[torch.Tensor] = None, stream=None):
    """Rejection verify in one call: returns (logits, stats, accept_len, next_token).
    lm_head: bf16 [V][d] tensor, BlockedWeights or W12Weights; accept_rate float64
    [B][gamma] or None (not computed)."""
    _need(hidden, "hidden", torch.bfloat16)
    B, g1, d = hidden.shape
    g = g1 - 1
    head, V, fmt = _lm_head(lm_head, d)
    layout = {"": LM_HEAD_ROWS, "_blocked": LM_HEAD_BLOCKED, "_w12": LM_HEAD_W12}[fmt]
    dev = hidden.device
    _need(draft_tokens, "draft_tokens", torch.int32, (B, g))
    _need(draft_logits, "draft_logits", torch.bfloat16, (B, g, V))
    if verify_len is not None:
        _need(verify_len, "verify_len", torch.int32, (B,))
    if row_offsets is not None:
        _need(row_offsets, "row_offsets", torch.int32, (B + 1,))
    _need(u_accept, "u_accept", torch.float32, (B, g))
    _need(u_resample, "u_resample", torch.float32, (B, g1))
    if logits is None:
        logits = torch.empty((B * g1, V), dtype=torch.float32, device=dev)
    _need(logits, "logits", torch.float32, (B * g1, V))
    if stats is None:
        stats = new_stats(B, g, dev)
    _need(stats, "stats", torch.int64, (B * g1, 4))
    accept_len = torch.empty(B, dtype=torch.int32, device=dev) if accept_len is None else accept_len
    next_token = torch.empty(B, dtype=torch.int32, device=dev) if next_token is None else next_token
    _need(accept_len, "accept_len", torch.int32, (B,))
    _need(next_token, "next_token", torch.int32, (B,))
    if counters is not None:
        _need(counters, "counters", torch.int64, (2,))
    if accept_rate is not None:
        _need(accept_rate, "accept_rate", torch.float64, (B, g))
    if ws_verify is None:
        ws_verify = new_workspace(verify_workspace_bytes(B, g, d, V), dev, stream)
    if ws_accept is None:
        ws_accept = new_workspace(accept_workspace_bytes(B, g, V), dev, stream)
    _check("sd_verify_rejection", _lib.sd_verify_rejection(
        _ptr(hidden), head, layout, _ptr(draft_logits), _ptr(draft_tokens), _ptr(verify_len),
        _ptr(row_offsets), _ptr(u_accept), _ptr(u_resample), B, g, d, V, float(temperature),
        _ptr(logits), _ptr(stats), _ptr(accept_len), _ptr(next_token), _ptr(counters),
        _ptr(accept_rate), _ptr(ws_verify), ws_verify.numel(), _ptr(ws_accept),
        ws_accept.numel(), _stream(stream)))
    return logits, stats, accept_len, next_token


# --------------------------------------------------------------- MXFP4 and sampling

_F32_MAX = torch.finfo(torch.float32).max
_TYPE_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _rows(t: torch.Tensor, name: str, dtype=None) -> None:
    """A device matrix of an element type the library takes, with contiguous rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _TYPE_CODES or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be {dtype or 'float32, bfloat16 or float16'}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2 or t.shape[0] < 1 or t.shape[1] < 1:
        raise ValueError(f"{name} must be a matrix, got shape {tuple(t.shape)}")
    if t.stride(1) != 1 and t.shape[1] > 1 or t.stride(0) < t.shape[1] and t.shape[0] > 1:
        raise ValueError(f"{name} must have contiguous, separate rows, got strides {t.stride()}")


def _row_stride(t: torch.Tensor) -> int:
    return max(t.stride(0), t.shape[1])


def _same_device(dev: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != dev and t.device is not None:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _call(name: str, dev: torch.device, stream, *args) -> None:
    """The entry point on dev's current stream (or `stream`), with dev current."""
    if dev.index == torch.cuda.current_device():
        _check(name, getattr(_lib, name)(*args, _stream(stream)))
        return
    with torch.cuda.device(dev):
        _check(name, getattr(_lib, name)(*args, _stream(stream)))


def _current(stream, dev: torch.device):
    """`stream` as torch's current stream, or the one that is."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(handle, device=dev)
    return torch.cuda.stream(stream)


def _empty(shape, dtype, dev: torch.device, stream) -> torch.Tensor:
    """Memory for a call on `stream`: taken on that stream, so that neither an earlier user of
    it is still at work nor a later one begins before the call is over."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with _current(stream, dev):
        return torch.empty(shape, dtype=dtype, device=dev)


def _workspace(nbytes: int, dev: torch.device, stream) -> torch.Tensor:
    ws = _empty(max(nbytes, 256), torch.uint8, dev, stream)
    _call("sd_workspace_init", dev, stream, _ptr(ws), ws.numel())
    return ws


def mxfp4_columns(d: int) -> int:
    """Stored columns of an MXFP4 row: d rounded up to a multiple of 128."""
    kp = int(_lib.sd_mxfp4_columns(d))
    if kp == 0:
        raise ValueError(f"MXFP4 rows need a positive multiple of 8 columns, got {d}")
    return kp


def mxfp4_logits_workspace_bytes(rows: int, d: int) -> int:
    return int(_lib.sd_mxfp4_logits_workspace_bytes(rows, d))


def sample_workspace_bytes(rows: int, V: int) -> int:
    return int(_lib.sd_sample_workspace_bytes(rows, V))


def accept_filtered_workspace_bytes(B: int, gamma: int, V: int) -> int:
    return int(_lib.sd_accept_filtered_workspace_bytes(B, gamma, V))


def sd_mxfp4_quantize(x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                      scales: Optional[torch.Tensor] = None, stream=None):
    """MXFP4 form of the rows of x (float32, bfloat16 or float16, any row stride): returns
    (codes uint8 [rows][kp / 2], scales uint8 [rows][kp / 32]), kp = mxfp4_columns(d)."""
    _rows(x, "x")
    rows, d = x.shape
    kp = mxfp4_columns(d)
    dev = x.device
    if codes is None:
        codes = _empty((rows, kp // 2), torch.uint8, dev, stream)
    else:
        _need(codes, "codes", torch.uint8, (rows, kp // 2))
        _same_device(dev, codes=codes)
    if scales is None:
        scales = _empty((rows, kp // 32), torch.uint8, dev, stream)
    else:
        _need(scales, "scales", torch.uint8, (rows, kp // 32))
        _same_device(dev, scales=scales)
    _call("sd_mxfp4_quantize", dev, stream, _ptr(x), _TYPE_CODES[x.dtype], rows, d,
          _row_stride(x), _ptr(codes), _ptr(scales))
    return codes, scales


def sd_mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, d: int,
                        dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """The values that MXFP4 rows stand for, [rows][d] of `dtype` (or into out)."""
    kp = mxfp4_columns(d)
    _need(codes, "codes", torch.uint8)
    rows = codes.shape[0]
    _need(codes, "codes", torch.uint8, (rows, kp // 2))
    _need(scales, "scales", torch.uint8, (rows, kp // 32))
    if out is None:
        if dtype not in _TYPE_CODES:
            raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
        out = _empty((rows, d), dtype, codes.device, stream)
    else:
        _rows(out, "out")
        if tuple(out.shape) != (rows, d):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(rows, d)}")
    _same_device(codes.device, scales=scales, out=out)
    _call("sd_mxfp4_dequantize", codes.device, stream, _ptr(codes), _ptr(scales), rows, d,
          _ptr(out), _TYPE_CODES[out.dtype], _row_stride(out))
    return out


class Mxfp4Weights(_Handle):
    """An MXFP4 LM head in the form sd_mxfp4_logits reads (sd_mxfp4_head), made once from codes
    uint8 [V][kp / 2] and scales uint8 [V][kp / 32], kp = mxfp4_columns(d), or from rows
    without the padding, [V][d / 2] and [V][d / 32] for d a multiple of 32."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, d: int, stream=None):
        kp = mxfp4_columns(d)
        _need(codes, "codes", torch.uint8)
        _need(scales, "scales", torch.uint8)
        V = codes.shape[0]
        if d % 32 == 0 and kp != d and tuple(codes.shape) == (V, d // 2):
            _need(scales, "scales", torch.uint8, (V, d // 32))
            with _current(stream, codes.device):
                codes = torch.nn.functional.pad(codes, (0, (kp - d) // 2))
                scales = torch.nn.functional.pad(scales, (0, (kp - d) // 32))
        _need(codes, "codes", torch.uint8, (V, kp // 2))
        _need(scales, "scales", torch.uint8, (V, kp // 32))
        _same_device(codes.device, scales=scales)
        nbytes = int(_lib.sd_mxfp4_head_bytes(V, d))
        if nbytes == 0:
            raise ValueError(f"no MXFP4 LM head of [{V}][{d}]")
        self.V, self.d, self.shape, self.device = int(V), int(d), (int(V), int(d)), codes.device
        self.nbytes = nbytes
        self.buf = _empty(nbytes, torch.uint8, codes.device, stream)
        _call("sd_mxfp4_head", codes.device, stream, _ptr(codes), _ptr(scales), self.V, self.d,
              _ptr(self.buf), nbytes)
        self._made = True

    @classmethod
    def from_tensor(cls, lm_head: torch.Tensor, stream=None) -> "Mxfp4Weights":
        """Quantise a [V][d] LM head (float32, bfloat16 or float16)."""
        return cls(*sd_mxfp4_quantize(lm_head, stream=stream), lm_head.shape[1], stream=stream)


def sd_mxfp4_logits(hidden: torch.Tensor, lm_head: Mxfp4Weights,
                    logits: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float32,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Logits [M][V] of hidden rows [M][d] (float32, bfloat16 or float16, any row stride)
    under an MXFP4 LM head, as `dtype` or into `logits` (any row stride)."""
    _rows(hidden, "hidden")
    if not isinstance(lm_head, Mxfp4Weights):
        raise TypeError("lm_head must be Mxfp4Weights")
    M, d = hidden.shape
    if d != lm_head.d:
        raise ValueError("lm_head must be [V][d] with the hidden size of `hidden`")
    dev = hidden.device
    if logits is None:
        if dtype not in _TYPE_CODES:
            raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
        logits = _empty((M, lm_head.V), dtype, dev, stream)
    else:
        _rows(logits, "logits")
        if tuple(logits.shape) != (M, lm_head.V):
            raise ValueError(f"logits has shape {tuple(logits.shape)}, expected {(M, lm_head.V)}")
    if workspace is None:
        workspace = _workspace(mxfp4_logits_workspace_bytes(M, d), dev, stream)
    _same_device(dev, lm_head=lm_head, logits=logits, workspace=workspace)
    _call("sd_mxfp4_logits", dev, stream, _ptr(hidden), _TYPE_CODES[hidden.dtype], M, d,
          _row_stride(hidden), _ptr(lm_head.buf), lm_head.V, _ptr(logits), _TYPE_CODES[logits.dtype],
          _row_stride(logits), _ptr(workspace), workspace.numel())
    return logits


class _SdSampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p),
                ("top_p", ctypes.c_void_p), ("min_p", ctypes.c_void_p)]


class SamplingParams(_Handle):
    """Sampling settings of n requests in device memory, for sd_sample, sd_accept_filtered and
    VerifyRound. Each of temperature (default 1; 0 is greedy), top_k (< 1: off), top_p
    (>= 1: off) and min_p (<= 0: off) is None (its filter is off), one number for every
    request, a sequence of n numbers, or a device tensor of n values that is used as it is
    (float32; int32 for top_k), so that writing to it changes later calls. The attributes
    themselves are fixed: calls read the tensors at the addresses they were made with."""

    def __init__(self, temperature=None, top_k=None, top_p=None, min_p=None,
                 n: Optional[int] = None, device="cuda"):
        given = dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
        for name, v in given.items():
            if v is None or isinstance(v, (int, float)):
                continue
            size = v.numel() if isinstance(v, torch.Tensor) else len(v)
            if isinstance(v, torch.Tensor):
                device = v.device if v.is_cuda else device
            if n is None:
                n = size
            if size != n or size < 1:
                raise ValueError(f"{name} has {size} values, expected {n}")
        self.n = 1 if n is None else int(n)
        if self.n < 1:
            raise ValueError("sampling settings need at least one request")
        self.device = torch.device(device)
        for name, v in given.items():
            setattr(self, name, self._array(name, v))
        # Without any array the settings are those of no device in particular.
        self.device = next((t.device for t in self._arrays() if t is not None), None)
        _same_device(self.device, **{k: getattr(self, k) for k in given})
        self._desc = _SdSampling(*[None if t is None else t.data_ptr() for t in self._arrays()])
        self._ref = ctypes.byref(self._desc)
        self._made = True

    def _arrays(self):
        return (self.temperature, self.top_k, self.top_p, self.min_p)

    def _array(self, name, v):
        if v is None:
            return None
        dtype = torch.int32 if name == "top_k" else torch.float32
        if isinstance(v, torch.Tensor) and v.is_cuda:
            _need(v, name, dtype, (self.n,))
            return v
        if isinstance(v, torch.Tensor):
            v = v.tolist()
        v = [v] * self.n if isinstance(v, (int, float)) else list(v)
        for x in v:
            if name == "top_k":
                if not -2**31 <= x < 2**31 or int(x) != x:
                    raise ValueError(f"top_k must be whole 32-bit numbers, got {x}")
            elif x != x or (name == "temperature" and not 0 <= x <= _F32_MAX):
                raise ValueError(f"{name} cannot be {x}")
        return torch.tensor([int(x) if name == "top_k" else float(x) for x in v], dtype=dtype,
                            device=self.device)


def _vector(t: torch.Tensor, name: str, dtype, n: int) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor of {dtype}")
    if tuple(t.shape) != (n,) or (n > 1 and t.stride(0) < 1):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, stride {t.stride()}, expected {(n,)}")


def sd_sample(logits: torch.Tensor, u: torch.Tensor, params: SamplingParams,
              tokens: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None,
              logprob: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              stream=None):
    """One token per row of logits [R][V] (float32, bfloat16 or float16, any row stride) under
    `params` (of R requests, or of R / k: then k rows in turn share an entry), from the
    uniforms u float32 [R]. Returns (tokens int32 [R], kept int32 [R], logprob float32 [R]);
    a tokens tensor passed in may have any stride (a column of draft tokens)."""
    _rows(logits, "logits")
    R, V = logits.shape
    dev = logits.device
    _need(u, "u", torch.float32, (R,))
    if not isinstance(params, SamplingParams):
        raise TypeError("params must be SamplingParams")
    if R % params.n != 0:
        raise ValueError(f"{R} rows cannot share the settings of {params.n} requests")
    if tokens is None:
        tokens = _empty(R, torch.int32, dev, stream)
    else:
        _vector(tokens, "tokens", torch.int32, R)
    if kept is None:
        kept = _empty(R, torch.int32, dev, stream)
    else:
        _need(kept, "kept", torch.int32, (R,))
    if logprob is None:
        logprob = _empty(R, torch.float32, dev, stream)
    else:
        _need(logprob, "logprob", torch.float32, (R,))
    if workspace is None:
        workspace = _workspace(sample_workspace_bytes(R, V), dev, stream)
    _same_device(dev, u=u, params=params, tokens=tokens, kept=kept, logprob=logprob,
                 workspace=workspace)
    _call("sd_sample", dev, stream, _ptr(logits), _TYPE_CODES[logits.dtype], _row_stride(logits), R,
          V, _ptr(u), params._ref, R // params.n, _ptr(tokens), max(1, tokens.stride(0)),
          _ptr(kept), _ptr(logprob), _ptr(workspace), workspace.numel())
    return tokens, kept, logprob


def sd_accept_filtered(logits: torch.Tensor, draft_logits: torch.Tensor,
                       draft_tokens: torch.Tensor, verify_len: Optional[torch.Tensor],
                       row_offsets: Optional[torch.Tensor], u_accept: torch.Tensor,
                       u_resample: torch.Tensor, params: SamplingParams,
                       accept_len: Optional[torch.Tensor] = None,
                       next_token: Optional[torch.Tensor] = None,
                       counters: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None):
    """Rejection acceptance when target and drafter are both sampled under `params` (of B
    requests): returns (accept_len, next_token). Other arguments as for sd_accept_rejection."""
    _need(draft_tokens, "draft_tokens", torch.int32)
    B, g = draft_tokens.shape
    dev = draft_tokens.device
    _need(draft_logits, "draft_logits", torch.bfloat16)
    V = draft_logits.shape[2]
    _need(draft_logits, "draft_logits", torch.bfloat16, (B, g, V))
    _need(logits, "logits", torch.float32, (B * (g + 1), V))
    if verify_len is not None:
        _need(verify_len, "verify_len", torch.int32, (B,))
    if row_offsets is not None:
        _need(row_offsets, "row_offsets", torch.int32, (B + 1,))
    _need(u_accept, "u_accept", torch.float32, (B, g))
    _need(u_resample, "u_resample", torch.float32, (B, g + 1))
    if not isinstance(params, SamplingParams):
        raise TypeError("params must be SamplingParams")
    if params.n != B:
        raise ValueError(f"params holds the settings of {params.n} requests, expected {B}")
    accept_len = _empty(B, torch.int32, dev, stream) if accept_len is None else accept_len
    next_token = _empty(B, torch.int32, dev, stream) if next_token is None else next_token
    _need(accept_len, "accept_len", torch.int32, (B,))
    _need(next_token, "next_token", torch.int32, (B,))
    if counters is not None:
        _need(counters, "counters", torch.int64, (2,))
    if workspace is None:
        workspace = _workspace(accept_filtered_workspace_bytes(B, g, V), dev, stream)
    _same_device(dev, logits=logits, draft_logits=draft_logits, verify_len=verify_len,
                 row_offsets=row_offsets, u_accept=u_accept, u_resample=u_resample, params=params,
                 accept_len=accept_len, next_token=next_token, counters=counters,
                 workspace=workspace)
    _call("sd_accept_filtered", dev, stream, _ptr(logits), _ptr(draft_logits), _ptr(draft_tokens),
          _ptr(verify_len), _ptr(row_offsets), _ptr(u_accept), _ptr(u_resample), params._ref, B, g,
          V, _ptr(accept_len), _ptr(next_token), _ptr(counters), _ptr(workspace),
          workspace.numel())
    return accept_len, next_token


# --------------------------------------------------------------- a whole round

class VerifyRound:
    """Buffers for repeated verify rounds of one shape; each run() enqueues the whole path.

    truncate -> verify logits -> accept (greedy when temperature == 0, else rejection),
    all on one stream with no host synchronisation. The verify and accept steps run
    through sd_verify_greedy at temperature 0 and sd_verify_rejection otherwise (fewer
    launches, for every LM-head format); fused=False keeps the separate sd_verify_logits
    + sd_accept_* calls. With `sampling` (SamplingParams of B requests) the accept step is
    sd_accept_filtered under those settings, after sd_verify_logits at `temperature`.
    """

    def __init__(self, B: int, gamma: int, d: int, V: int, temperature: float,
                 truncate: bool, threshold: float = 0.3, device="cuda", stream=None,
                 fused: bool = True, accept_rate: bool = False, scheduler: Optional[int] = None,
                 sps: Optional[torch.Tensor] = None,
                 sampling: Optional[SamplingParams] = None):
        self.B, self.gamma, self.d, self.V = B, gamma, d, V
        self.sampling = sampling
        if sampling is not None and (not isinstance(sampling, SamplingParams) or sampling.n != B):
            raise ValueError("sampling must be SamplingParams of B requests")
        if sampling is not None and accept_rate:
            raise ValueError("the acceptance rate is not computed under sampling filters")
        # With a scheduler mode (SCHED_EARLY_STOP / SCHED_TOP_K) and an SPS table, the
        # prefix scheduler replaces the confidence threshold.
        self.scheduler, self.sps = scheduler, sps
        if scheduler is not None and (not truncate or sps is None):
            raise ValueError("a scheduler needs truncate=True and an SPS table")
        self.fused = fused
        self.T, self.truncate, self.threshold = float(temperature), truncate, float(threshold)
        dev = torch.device(device)
        rows = B * (gamma + 1)
        self.verify_len = torch.empty(B, dtype=torch.int32, device=dev) if truncate else None
        self.row_offsets = torch.empty(B + 1, dtype=torch.int32, device=dev) if truncate else None
        self.stats = new_stats(B, gamma, dev)
        self.logits = (torch.empty((rows, V), dtype=torch.float32, device=dev)
                       if self.T > 0 or sampling is not None else None)
        self.accept_len = torch.empty(B, dtype=torch.int32, device=dev)
        self.next_token = torch.empty(B, dtype=torch.int32, device=dev)
        self.counters = torch.zeros(2, dtype=torch.int64, device=dev)
        self.ws_verify = new_workspace(verify_workspace_bytes(B, gamma, d, V), dev, stream)
        self.ws_accept = (new_workspace(accept_filtered_workspace_bytes(B, gamma, V), dev, stream)
                          if sampling is not None else
                          new_workspace(accept_workspace_bytes(B, gamma, V), dev, stream)
                          if self.T > 0 else None)
        # Analytic acceptance rate per verified draft position (rejection rounds only).
        self.accept_rate = (torch.empty((B, gamma), dtype=torch.float64, device=dev)
                            if accept_rate and self.T > 0 else None)

    def run(self, hidden, lm_head, draft_tokens, conf=None, draft_logits=None, u_accept=None,
            u_resample=None, stream=None, conf_stale=None):
        if self.truncate and self.scheduler is not None:
            sd_schedule_prefix(conf, self.sps, self.scheduler,
                               conf_stale if self.scheduler == SCHED_TOP_K else None,
                               self.verify_len, self.row_offsets, stream=stream)
        elif self.truncate:
            sd_truncate_by_confidence(conf, self.threshold, self.verify_len, self.row_offsets,
                                      stream=stream)
        if self.sampling is not None:
            sd_verify_logits(hidden, lm_head, draft_tokens, self.verify_len, self.row_offsets,
                             self.T, self.logits, self.stats, self.ws_verify, stream=stream)
            sd_accept_filtered(self.logits, draft_logits, draft_tokens, self.verify_len,
                               self.row_offsets, u_accept, u_resample, self.sampling,
                               self.accept_len, self.next_token, self.counters, self.ws_accept,
                               stream=stream)
            return self.accept_len, self.next_token
        if self.T == 0 and self.fused:
            sd_verify_greedy(hidden, lm_head, draft_tokens, self.verify_len, self.row_offsets,
                             self.stats, self.accept_len, self.next_token, self.counters,
                             self.ws_verify, stream=stream)
            return self.accept_len, self.next_token
        if self.T > 0 and self.fused:
            sd_verify_rejection(hidden, lm_head, draft_tokens, draft_logits, self.verify_len,
                                self.row_offsets, u_accept, u_resample, self.T, self.logits,
                                self.stats, self.accept_len, self.next_token, self.counters,
                                self.accept_rate, self.ws_verify, self.ws_accept, stream=stream)
            return self.accept_len, self.next_token
        sd_verify_logits(hidden, lm_head, draft_tokens, self.verify_len, self.row_offsets,
                         self.T, self.logits, self.stats, self.ws_verify, stream=stream)
        if self.T > 0 and self.accept_rate is not None:
            sd_accept_rejection_ex(self.logits, self.stats, draft_logits, draft_tokens,
                                   self.verify_len, self.row_offsets, u_accept, u_resample,
                                   self.T, self.accept_len, self.next_token, self.counters,
                                   self.accept_rate, self.ws_accept, stream=stream)
        elif self.T > 0:
            sd_accept_rejection(self.logits, self.stats, draft_logits, draft_tokens,
                                self.verify_len, self.row_offsets, u_accept, u_resample, self.T,
                                self.accept_len, self.next_token, self.counters, self.ws_accept,
                                stream=stream)
        else:
            sd_accept_greedy(self.stats, draft_tokens, self.verify_len, self.row_offsets,
                             self.accept_len, self.next_token, self.counters, stream=stream)
        return self.accept_len, self.next_token
