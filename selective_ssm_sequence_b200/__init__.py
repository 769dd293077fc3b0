"""Thin Python binding of libhm.so, the HedgeMamba mixer-scan library for B200.

Argument marshalling only: every function here fills the C structs declared
in ``include/hm.h`` from torch tensors (device memory and streams come from
PyTorch) and calls the C entry point of the same name.  All arithmetic runs
in the library's CUDA kernels; there is no CPU or PyTorch fallback, and
importing this package fails loudly if the built library is missing.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhm.so")

HM_OK, HM_ERR_INVALID_ARG, HM_ERR_UNSUPPORTED, HM_ERR_CUDA, HM_ERR_TIMEOUT, HM_ERR_DEVICE = range(6)
HM_F32, HM_BF16 = 0, 1
HM_FLAG_DT_SCALED_INPUT, HM_FLAG_PER_FEATURE_DECAY, HM_FLAG_ROPE = 1, 2, 4
HM_INPUT_PLAIN, HM_INPUT_STEP, HM_INPUT_UNIT = 0, 1, 2
HM_NORM_RMS, HM_NORM_LAYER = 0, 1
HM_ROTARY_HALF, HM_ROTARY_INTERLEAVED = 0, 1
HM_ROTARY_PLAIN, HM_ROTARY_LINEAR, HM_ROTARY_NTK, HM_ROTARY_BY_PARTS = 0, 1, 2, 3

if not os.path.exists(LIB_PATH):
    raise ImportError("libhm.so is not built (%s); run __graft_entry__.build() or "
                      "python selective_ssm_sequence_b200/_build.py" % LIB_PATH)

lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_SZ = ctypes.c_size_t


class ScanArgs(ctypes.Structure):
    """Mirror of hm_scan_args."""
    _fields_ = [("B", _I64), ("L", _I64), ("H", _I), ("d", _I), ("p", _I), ("dv", _I),
                ("io_dtype", _I), ("q", _P), ("k", _P), ("v", _P), ("W_q", _P), ("W_k", _P),
                ("w_head_stride", _I64), ("b_q", _P), ("b_k", _P), ("dt", _P), ("A_log", _P),
                ("S0", _P), ("z0", _P), ("o", _P), ("S_out", _P), ("z_out", _P),
                ("workspace", _P), ("workspace_bytes", _SZ), ("flags", ctypes.c_uint),
                ("log_decay_out", _P), ("rope_base", ctypes.c_double), ("pos0", _I64)]


class ScanBwdArgs(ctypes.Structure):
    """Mirror of hm_scan_bwd_args."""
    _fields_ = [("B", _I64), ("L", _I64), ("H", _I), ("d", _I), ("p", _I), ("dv", _I), ("io_dtype", _I),
                ("q", _P), ("k", _P), ("v", _P), ("W_q", _P), ("W_k", _P), ("dt", _P), ("A_log", _P),
                ("S0", _P), ("z0", _P), ("dout", _P), ("grad_q", _P), ("grad_k", _P), ("grad_v", _P),
                ("grad_W_q", _P), ("grad_W_k", _P), ("grad_dt", _P), ("grad_A_log", _P), ("grad_S0", _P),
                ("grad_z0", _P), ("workspace", _P), ("workspace_bytes", _SZ)]


class CombineArgs(ctypes.Structure):
    """Mirror of hm_combine_args."""
    _fields_ = [("n_parts", _I64), ("BH", _I64), ("F", _I), ("dv", _I), ("per_feature", _I),
                ("parts", _P), ("part_len", _I64), ("S0", _P), ("z0", _P), ("only_part", _I64),
                ("S_start", _P), ("z_start", _P), ("S_end", _P), ("z_end", _P)]


class DecodeArgs(ctypes.Structure):
    """Mirror of hm_decode_args."""
    _fields_ = [("B", _I64), ("H", _I), ("d", _I), ("p", _I), ("dv", _I), ("io_dtype", _I),
                ("q", _P), ("k", _P), ("v", _P), ("W_q", _P), ("W_k", _P),
                ("w_head_stride", _I64), ("b_q", _P), ("b_k", _P), ("dt", _P), ("A_log", _P),
                ("S", _P), ("z", _P), ("o", _P), ("workspace", _P), ("workspace_bytes", _SZ),
                ("flags", ctypes.c_uint), ("rope_base", ctypes.c_double), ("positions", _P)]


class MixerArgs(ctypes.Structure):
    """Mirror of hm_mixer_args."""
    _fields_ = [("B", _I64), ("L", _I64), ("d_model", _I), ("H", _I), ("E", _I), ("p", _I),
                ("conv_k", _I), ("x", _P), ("W_q", _P), ("W_k", _P), ("W_v", _P), ("W_g", _P),
                ("W_dt", _P), ("b_dt", _P), ("b_g", _P), ("conv_w", _P), ("conv_b", _P),
                ("W_hq", _P), ("W_hk", _P), ("A_log", _P), ("W_o", _P), ("out", _P)]


class BlockArgs(ctypes.Structure):
    """Mirror of hm_block_args."""
    _fields_ = [("mixer", MixerArgs), ("ln1_w", _P), ("ln1_b", _P), ("ln2_w", _P), ("ln2_b", _P),
                ("eps", ctypes.c_float), ("d_ff", _I), ("W_fc1", _P), ("b_fc1", _P), ("W_fc2", _P),
                ("b_fc2", _P)]


class GatedScanArgs(ctypes.Structure):
    """Mirror of hm_gated_scan_args."""
    _fields_ = [("B", _I64), ("L", _I64), ("D", _I64), ("io_dtype", _I), ("input_scale", _I), ("x", _P), ("dt", _P),
                ("y", _P), ("x_stride_b", _I64), ("x_stride_t", _I64), ("dt_stride_b", _I64), ("dt_stride_t", _I64),
                ("y_stride_b", _I64), ("y_stride_t", _I64), ("A_log", _P), ("dt_bias", _P), ("h0", _P),
                ("lengths", _P), ("h_out", _P), ("states", _P), ("states_bytes", _SZ)]


class GatedScanBwdArgs(ctypes.Structure):
    """Mirror of hm_gated_scan_bwd_args."""
    _fields_ = [("B", _I64), ("L", _I64), ("D", _I64), ("io_dtype", _I), ("input_scale", _I), ("x", _P), ("dt", _P),
                ("dy", _P), ("dx", _P), ("ddt", _P), ("x_stride_b", _I64), ("x_stride_t", _I64),
                ("dt_stride_b", _I64), ("dt_stride_t", _I64), ("dy_stride_b", _I64), ("dy_stride_t", _I64),
                ("dx_stride_b", _I64), ("dx_stride_t", _I64), ("ddt_stride_b", _I64), ("ddt_stride_t", _I64),
                ("A_log", _P), ("dt_bias", _P), ("lengths", _P), ("states", _P), ("states_bytes", _SZ),
                ("dh_out", _P), ("dA_log", _P), ("d_dt_bias", _P), ("dh0", _P), ("workspace", _P),
                ("workspace_bytes", _SZ)]


class GatedStepArgs(ctypes.Structure):
    """Mirror of hm_gated_step_args."""
    _fields_ = [("B", _I64), ("D", _I64), ("io_dtype", _I), ("input_scale", _I), ("x", _P), ("dt", _P), ("y", _P),
                ("x_stride", _I64), ("dt_stride", _I64), ("y_stride", _I64), ("A_log", _P), ("dt_bias", _P),
                ("h", _P), ("h_out", _P)]


class NormGateArgs(ctypes.Structure):
    """Mirror of hm_norm_gate_args."""
    _fields_ = [("rows", _I64), ("D", _I64), ("io_dtype", _I), ("norm", _I), ("post", _I), ("eps", ctypes.c_float),
                ("alpha", ctypes.c_float), ("y", _P), ("gate", _P), ("r", _P), ("r_out", _P), ("xn", _P),
                ("y_stride", _I64), ("gate_stride", _I64), ("r_stride", _I64), ("r_out_stride", _I64),
                ("xn_stride", _I64), ("scale", _P), ("post_w", _P), ("post_b", _P), ("pre_w", _P), ("pre_b", _P)]


class NormGateBwdArgs(ctypes.Structure):
    """Mirror of hm_norm_gate_bwd_args."""
    _fields_ = [("rows", _I64), ("D", _I64), ("io_dtype", _I), ("norm", _I), ("post", _I), ("eps", ctypes.c_float),
                ("alpha", ctypes.c_float), ("y", _P), ("gate", _P), ("r_out", _P), ("dr_out", _P), ("dxn", _P),
                ("dy", _P), ("dgate", _P), ("dr", _P), ("y_stride", _I64), ("gate_stride", _I64),
                ("r_out_stride", _I64), ("dr_out_stride", _I64), ("dxn_stride", _I64), ("dy_stride", _I64),
                ("dgate_stride", _I64), ("dr_stride", _I64), ("scale", _P), ("post_w", _P), ("post_b", _P),
                ("pre_w", _P), ("dscale", _P), ("dpost_w", _P), ("dpost_b", _P), ("dpre_w", _P), ("dpre_b", _P),
                ("workspace", _P), ("workspace_bytes", _SZ)]


class RotaryArgs(ctypes.Structure):
    """Mirror of hm_rotary_args."""
    _fields_ = [("B", _I64), ("L", _I64), ("Hq", _I), ("Hk", _I), ("d", _I), ("rot", _I), ("io_dtype", _I),
                ("layout", _I), ("scaling", _I), ("transpose", _I), ("q", _P), ("k", _P), ("q_out", _P),
                ("k_out", _P), ("q_stride_b", _I64), ("q_stride_t", _I64), ("q_stride_h", _I64),
                ("k_stride_b", _I64), ("k_stride_t", _I64), ("k_stride_h", _I64), ("q_out_stride_b", _I64),
                ("q_out_stride_t", _I64), ("q_out_stride_h", _I64), ("k_out_stride_b", _I64),
                ("k_out_stride_t", _I64), ("k_out_stride_h", _I64), ("positions", _P), ("pos_stride_b", _I64),
                ("pos_stride_t", _I64), ("pos0", _I64), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("orig_len", ctypes.c_double), ("beta_slow", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("mscale", ctypes.c_double)]


lib.hm_status_string.restype = ctypes.c_char_p
lib.hm_status_string.argtypes = [_I]
lib.hm_last_error_detail.restype = ctypes.c_char_p
lib.hm_last_error_detail.argtypes = []
lib.hm_version.restype = ctypes.c_char_p
lib.hm_featmap.restype = _I
lib.hm_featmap.argtypes = [_P, _I, _I64, _I, _I, _I, _P, _I64, _P, _P, _I, _P]
lib.hm_scan_workspace_size.restype = _SZ
lib.hm_scan_workspace_size.argtypes = [ctypes.POINTER(ScanArgs)]
lib.hm_scan_chunked_fwd.restype = _I
lib.hm_scan_chunked_fwd.argtypes = [ctypes.POINTER(ScanArgs), _P]
lib.hm_decode_workspace_size.restype = _SZ
lib.hm_decode_workspace_size.argtypes = [ctypes.POINTER(DecodeArgs)]
lib.hm_step_decode.restype = _I
lib.hm_step_decode.argtypes = [ctypes.POINTER(DecodeArgs), _P]
lib.hm_step_decode_noalloc.restype = _I
lib.hm_step_decode_noalloc.argtypes = [ctypes.POINTER(DecodeArgs), _P]
lib.hm_mixer_workspace_size.restype = _SZ
lib.hm_mixer_workspace_size.argtypes = [ctypes.POINTER(MixerArgs)]
lib.hm_mixer_fwd.restype = _I
lib.hm_mixer_fwd.argtypes = [ctypes.POINTER(MixerArgs), _P, _SZ, _P]
lib.hm_block_workspace_size.restype = _SZ
lib.hm_block_workspace_size.argtypes = [ctypes.POINTER(BlockArgs)]
lib.hm_block_fwd.restype = _I
lib.hm_block_fwd.argtypes = [ctypes.POINTER(BlockArgs), _P, _SZ, _P]
lib.hm_scan_bwd_workspace_size.restype = _SZ
lib.hm_scan_bwd_workspace_size.argtypes = [ctypes.POINTER(ScanBwdArgs)]
lib.hm_scan_bwd.restype = _I
lib.hm_scan_bwd.argtypes = [ctypes.POINTER(ScanBwdArgs), _P]
lib.hm_scan_combine.restype = _I
lib.hm_scan_combine.argtypes = [ctypes.POINTER(CombineArgs), _P]
for _name, _cls in (("hm_gated_scan_fwd", GatedScanArgs), ("hm_gated_scan_bwd", GatedScanBwdArgs),
                    ("hm_gated_scan_step", GatedStepArgs), ("hm_norm_gate_fwd", NormGateArgs),
                    ("hm_norm_gate_bwd", NormGateBwdArgs), ("hm_rotary", RotaryArgs)):
    getattr(lib, _name).restype = _I
    getattr(lib, _name).argtypes = [ctypes.POINTER(_cls), _P]
for _name, _cls in (("hm_gated_scan_states_size", GatedScanArgs),
                    ("hm_gated_scan_bwd_workspace_size", GatedScanBwdArgs),
                    ("hm_norm_gate_bwd_workspace_size", NormGateBwdArgs)):
    getattr(lib, _name).restype = _SZ
    getattr(lib, _name).argtypes = [ctypes.POINTER(_cls)]
lib.hm_launch_count.restype = ctypes.c_uint64
lib.hm_launch_count.argtypes = []
lib.hm_get_device_error.restype = _I
lib.hm_get_device_error.argtypes = [_P]
lib.hm_selftest_wait_timeout.restype = _I
lib.hm_selftest_wait_timeout.argtypes = [ctypes.c_uint32, _P]

EXPORTED = ("hm_status_string", "hm_last_error_detail", "hm_version", "hm_featmap",
            "hm_scan_workspace_size", "hm_scan_chunked_fwd", "hm_decode_workspace_size",
            "hm_step_decode", "hm_mixer_workspace_size", "hm_mixer_fwd", "hm_get_device_error",
            "hm_launch_count", "hm_step_decode_noalloc", "hm_selftest_wait_timeout", "hm_scan_combine",
            "hm_scan_bwd_workspace_size", "hm_scan_bwd", "hm_block_workspace_size", "hm_block_fwd",
            "hm_gated_scan_states_size", "hm_gated_scan_fwd", "hm_gated_scan_bwd_workspace_size",
            "hm_gated_scan_bwd", "hm_gated_scan_step", "hm_norm_gate_fwd", "hm_norm_gate_bwd_workspace_size",
            "hm_norm_gate_bwd", "hm_rotary")


class HMError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = lib.hm_last_error_detail().decode()
        msg = "%s: %s" % (where, lib.hm_status_string(status).decode())
        if detail:
            msg += " (%s)" % detail
        super().__init__(msg)


def _check(status: int, where: str) -> None:
    if status != HM_OK:
        raise HMError(status, where)


# ---------------------------------------------------------------- marshalling helpers

def _ptr(t) -> Optional[int]:
    """Device address of a tensor (or an int address, or None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _dtype_code(t) -> int:
    torch = _need_torch()
    if t.dtype is torch.bfloat16:
        return HM_BF16
    if t.dtype is torch.float32:
        return HM_F32
    raise TypeError("unsupported dtype %s (float32 or bfloat16)" % t.dtype)


_torch = None


def _need_torch():
    """The torch module, imported at the first call that handles tensors."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


class _NoFiller:
    """Gives up on every call, as the native filler does on calls that it does not know."""

    def __getattr__(self, name):
        return lambda *args: None


_native = None


def _filler():
    """The native argument filler, built beside libhm.so (imported after torch, whose libraries it
    uses).  It saves the helpers time and nothing else: without it they fill their structs in Python."""
    global _native
    if _native is None:
        _need_torch()
        try:
            from . import _marshal as mod
            from ._build import marshal_tag
            if getattr(mod, "built_for", None) != marshal_tag():
                raise ImportError("built for another torch or Python")
        except ImportError as e:
            import warnings
            warnings.warn("_marshal.so cannot be used (%s): calls of a few rows take some microseconds longer; run "
                          "__graft_entry__.build() or python selective_ssm_sequence_b200/_build.py" % e,
                          RuntimeWarning, stacklevel=3)
            mod = _NoFiller()
        _native = mod
    return _native


def _stream(stream) -> Optional[int]:
    if stream is None:
        torch = _need_torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # the address without a Stream object
        if raw is not None and torch.cuda.is_initialized():
            return raw(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _require_cuda(*ts) -> None:
    for t in ts:
        if t is not None and not isinstance(t, int) and not t.is_cuda:
            raise ValueError("libhm works on device memory; got a CPU tensor")


# ---------------------------------------------------------------- entry points

def hm_version() -> str:
    return lib.hm_version().decode()


def hm_featmap(x, W, phi, H: int = 1, bias=None, w_head_stride: int = 0, stream=None) -> None:
    """phi = softmax([W x + b, -(W x + b)]) row-wise.  x: [..., d] (row r is
    head r mod H); W: [p, d] (or per-head, with w_head_stride); phi: [..., 2p]."""
    _require_cuda(x, W, phi, bias)
    d = x.shape[-1]
    p = W.shape[-2]
    rows = x.numel() // d
    st = lib.hm_featmap(_ptr(x), _dtype_code(x), rows, int(H), d, p, _ptr(W), int(w_head_stride),
                        _ptr(bias), _ptr(phi), _dtype_code(phi), _stream(stream))
    _check(st, "hm_featmap")


def scan_args(q, k, v, o, W_q=None, W_k=None, dt=None, A_log=None, S0=None, z0=None,
              S_out=None, z_out=None, b_q=None, b_k=None, w_head_stride: int = 0,
              workspace=None, flags: int = 0, log_decay_out=None, rope_base: float = 0.0,
              pos0: int = 0) -> ScanArgs:
    """Fill an hm_scan_args from tensors (q, k: [B, L, H, d]; v, o: [B, L, H, dv]).
    o = None (with S_out) makes a state-only call; q may then be None too."""
    B, L, H, d = k.shape
    dv = v.shape[-1]
    a = ScanArgs()
    a.B, a.L, a.H, a.d, a.dv = B, L, H, d, dv
    a.p = W_q.shape[-2] if W_q is not None else 0
    a.io_dtype = _dtype_code(k)
    a.q, a.k, a.v, a.o = _ptr(q), _ptr(k), _ptr(v), _ptr(o)
    a.W_q, a.W_k, a.w_head_stride = _ptr(W_q), _ptr(W_k), int(w_head_stride)
    a.b_q, a.b_k = _ptr(b_q), _ptr(b_k)
    a.dt, a.A_log = _ptr(dt), _ptr(A_log)
    a.S0, a.z0, a.S_out, a.z_out = _ptr(S0), _ptr(z0), _ptr(S_out), _ptr(z_out)
    a.flags = int(flags)
    a.log_decay_out = _ptr(log_decay_out)
    a.rope_base, a.pos0 = float(rope_base), int(pos0)
    if workspace is not None:
        a.workspace = _ptr(workspace)
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    # the struct holds raw addresses: keep the tensors alive as long as it lives
    a._refs = (q, k, v, o, W_q, W_k, dt, A_log, S0, z0, S_out, z_out, b_q, b_k, workspace, log_decay_out)
    return a


def hm_scan_workspace_size(args: ScanArgs) -> int:
    return int(lib.hm_scan_workspace_size(ctypes.byref(args)))


def hm_scan_chunked_fwd(args: ScanArgs, stream=None) -> None:
    _check(lib.hm_scan_chunked_fwd(ctypes.byref(args), _stream(stream)), "hm_scan_chunked_fwd")


def scan_bwd_args(q, k, v, dout, grad_q, grad_k, grad_v, W_q=None, W_k=None, grad_W_q=None,
                  grad_W_k=None, dt=None, A_log=None, grad_dt=None, grad_A_log=None, S0=None, z0=None,
                  grad_S0=None, grad_z0=None, workspace=None) -> ScanBwdArgs:
    """Fill an hm_scan_bwd_args (forward inputs, dout [B, L, H, dv] and the fp32
    gradient buffers)."""
    B, L, H, d = q.shape
    a = ScanBwdArgs()
    a.B, a.L, a.H, a.d, a.dv = B, L, H, d, v.shape[-1]
    a.p = W_q.shape[-2] if W_q is not None else 0
    a.io_dtype = _dtype_code(q)
    a.q, a.k, a.v, a.dout = _ptr(q), _ptr(k), _ptr(v), _ptr(dout)
    a.W_q, a.W_k, a.dt, a.A_log, a.S0, a.z0 = map(_ptr, (W_q, W_k, dt, A_log, S0, z0))
    a.grad_q, a.grad_k, a.grad_v = _ptr(grad_q), _ptr(grad_k), _ptr(grad_v)
    a.grad_W_q, a.grad_W_k, a.grad_dt, a.grad_A_log = map(_ptr, (grad_W_q, grad_W_k, grad_dt, grad_A_log))
    a.grad_S0, a.grad_z0 = _ptr(grad_S0), _ptr(grad_z0)
    if workspace is not None:
        a.workspace = _ptr(workspace)
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    a._refs = (q, k, v, dout, grad_q, grad_k, grad_v, W_q, W_k, grad_W_q, grad_W_k, dt, A_log, grad_dt,
               grad_A_log, S0, z0, grad_S0, grad_z0, workspace)
    return a


def hm_scan_bwd_workspace_size(args: ScanBwdArgs) -> int:
    return int(lib.hm_scan_bwd_workspace_size(ctypes.byref(args)))


def hm_scan_bwd(args: ScanBwdArgs, stream=None) -> None:
    _check(lib.hm_scan_bwd(ctypes.byref(args), _stream(stream)), "hm_scan_bwd")


def combine_args(parts, n_parts: int, BH: int, F: int, dv: int, part_len: int, S_start, z_start,
                 per_feature: bool = False, S0=None, z0=None, only_part: int = -1, S_end=None,
                 z_end=None) -> CombineArgs:
    """Fill an hm_combine_args: `parts` holds n_parts records of part_len fp32
    values, each [log_decay (padded to 4) | S | z] of one sequence segment."""
    a = CombineArgs()
    a.n_parts, a.BH, a.F, a.dv, a.per_feature = int(n_parts), int(BH), int(F), int(dv), int(per_feature)
    a.parts, a.part_len = _ptr(parts), int(part_len)
    a.S0, a.z0, a.only_part = _ptr(S0), _ptr(z0), int(only_part)
    a.S_start, a.z_start, a.S_end, a.z_end = _ptr(S_start), _ptr(z_start), _ptr(S_end), _ptr(z_end)
    a._refs = (parts, S0, z0, S_start, z_start, S_end, z_end)
    return a


def hm_scan_combine(args: CombineArgs, stream=None) -> None:
    _check(lib.hm_scan_combine(ctypes.byref(args), _stream(stream)), "hm_scan_combine")


def combine_record_len(BH: int, F: int, dv: int, per_feature: bool = False) -> int:
    """fp32 values of one [log_decay | S | z] record (the log-decay part padded to 4)."""
    nl = BH * F if per_feature else BH
    return (nl + 3) // 4 * 4 + BH * F * dv + BH * F


def decode_args(q, k, v, o, S, z, W_q=None, W_k=None, dt=None, A_log=None, b_q=None, b_k=None,
                w_head_stride: int = 0, workspace=None, flags: int = 0, rope_base: float = 0.0,
                positions=None) -> DecodeArgs:
    """Fill an hm_decode_args (q, k: [B, H, d]; v, o: [B, H, dv]; S: [B, H, F, dv])."""
    B, H, d = q.shape
    a = DecodeArgs()
    a.B, a.H, a.d, a.dv = B, H, d, v.shape[-1]
    a.p = W_q.shape[-2] if W_q is not None else 0
    a.io_dtype = _dtype_code(q)
    a.q, a.k, a.v, a.o = _ptr(q), _ptr(k), _ptr(v), _ptr(o)
    a.W_q, a.W_k, a.w_head_stride = _ptr(W_q), _ptr(W_k), int(w_head_stride)
    a.b_q, a.b_k = _ptr(b_q), _ptr(b_k)
    a.dt, a.A_log = _ptr(dt), _ptr(A_log)
    a.S, a.z = _ptr(S), _ptr(z)
    a.flags = int(flags)
    a.rope_base, a.positions = float(rope_base), _ptr(positions)
    if workspace is not None:
        a.workspace = _ptr(workspace)
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    a._refs = (q, k, v, o, S, z, W_q, W_k, dt, A_log, b_q, b_k, workspace, positions)
    return a


def hm_decode_workspace_size(args: DecodeArgs) -> int:
    return int(lib.hm_decode_workspace_size(ctypes.byref(args)))


def hm_step_decode(args: DecodeArgs, stream=None) -> None:
    _check(lib.hm_step_decode(ctypes.byref(args), _stream(stream)), "hm_step_decode")


def hm_step_decode_noalloc(args: DecodeArgs, stream=None) -> None:
    """hm_step_decode without a caller-provided workspace: for callers that
    cannot allocate device memory.  The feature vectors use a fixed 4 MiB
    device array inside the library (B * H * F <= 524288 when W_q is given);
    calls that overlap on the GPU share that array and must be serialised."""
    _check(lib.hm_step_decode_noalloc(ctypes.byref(args), _stream(stream)), "hm_step_decode_noalloc")


def mixer_args(x, out, W_q, W_k, W_v, W_g, W_dt, conv_w, W_hq, W_hk, A_log, W_o, n_heads: int,
               conv_b=None, b_g=None, b_dt=None) -> MixerArgs:
    """Fill an hm_mixer_args (x, out: [B, L, D]; W_*: [E, D]; conv_w: [3, E, K])."""
    B, L, D = x.shape
    a = MixerArgs()
    a.B, a.L, a.d_model, a.H, a.E = B, L, D, int(n_heads), W_q.shape[0]
    a.p = W_hq.shape[0]
    a.conv_k = conv_w.shape[-1]
    a.x, a.out = _ptr(x), _ptr(out)
    a.W_q, a.W_k, a.W_v, a.W_g, a.W_dt, a.W_o = map(_ptr, (W_q, W_k, W_v, W_g, W_dt, W_o))
    a.b_dt, a.b_g = _ptr(b_dt), _ptr(b_g)
    a.conv_w, a.conv_b = _ptr(conv_w), _ptr(conv_b)
    a.W_hq, a.W_hk, a.A_log = _ptr(W_hq), _ptr(W_hk), _ptr(A_log)
    a._refs = (x, out, W_q, W_k, W_v, W_g, W_dt, conv_w, W_hq, W_hk, A_log, W_o, conv_b, b_g, b_dt)
    return a


def hm_mixer_workspace_size(args: MixerArgs) -> int:
    return int(lib.hm_mixer_workspace_size(ctypes.byref(args)))


def hm_mixer_fwd(args: MixerArgs, workspace, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib.hm_mixer_fwd(ctypes.byref(args), _ptr(workspace), nbytes, _stream(stream)),
           "hm_mixer_fwd")


def block_args(x, out, mixer: dict, ln1_w, ln1_b, ln2_w, ln2_b, W_fc1, b_fc1, W_fc2, b_fc2, n_heads: int,
               eps: float = 1e-5) -> BlockArgs:
    """Fill an hm_block_args: ``mixer`` holds the mixer_args keywords other
    than x, out and n_heads; x, out: [B, L, D]; W_fc1: [d_ff, D]; W_fc2: [D, d_ff]."""
    a = BlockArgs()
    m = mixer_args(x, out, n_heads=n_heads, **mixer)
    a.mixer = m
    a.ln1_w, a.ln1_b, a.ln2_w, a.ln2_b = map(_ptr, (ln1_w, ln1_b, ln2_w, ln2_b))
    a.eps = float(eps)
    a.d_ff = W_fc1.shape[0]
    a.W_fc1, a.b_fc1, a.W_fc2, a.b_fc2 = map(_ptr, (W_fc1, b_fc1, W_fc2, b_fc2))
    a._refs = (m._refs, ln1_w, ln1_b, ln2_w, ln2_b, W_fc1, b_fc1, W_fc2, b_fc2)
    return a


def hm_block_workspace_size(args: BlockArgs) -> int:
    return int(lib.hm_block_workspace_size(ctypes.byref(args)))


def hm_block_fwd(args: BlockArgs, workspace, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib.hm_block_fwd(ctypes.byref(args), _ptr(workspace), nbytes, _stream(stream)), "hm_block_fwd")


# ---- the operators around the mixer: gated recurrence, seam between blocks, rotary positions.
# Their helpers check what the C side cannot see (shapes, dtypes, devices) and raise ValueError.
# A decode loop calls them for every token, so the native module _marshal fills the struct in the
# common case; where it gives up (None), the checks below say what is wrong with which tensor, or
# fill the struct themselves.

def _io(who: str, shape, like, **ts):
    """Each given tensor has `like`'s dtype, this shape and contiguous elements in its last axis."""
    for name, t in ts.items():
        if t is None:
            continue
        if t.shape != shape:
            raise ValueError("%s: %s has shape %s, not %s" % (who, name, tuple(t.shape), tuple(shape)))
        if t.dtype != like.dtype:
            raise ValueError("%s: %s is %s, not %s" % (who, name, t.dtype, like.dtype))
        if t.stride(-1) != 1 and t.shape[-1] > 1 and t.numel() > 0:
            raise ValueError("%s: the last axis of %s is not contiguous" % (who, name))


def _dense(who: str, shape, dtype, **ts):
    """Each given tensor is dense, of this shape and dtype."""
    for name, t in ts.items():
        if t is None:
            continue
        if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
            raise ValueError("%s: %s must be a contiguous %s tensor of shape %s, got %s %s" % (
                who, name, dtype, tuple(shape), t.dtype, tuple(t.shape)))


def _buffer(who: str, **ts) -> None:
    """Each given byte buffer is dense: its size is that of the memory behind it."""
    for name, t in ts.items():
        if t is not None and not t.is_contiguous():
            raise ValueError("%s: %s must be contiguous, got strides %s" % (who, name, tuple(t.stride())))


def _one_device(who: str, *ts) -> None:
    """All tensors on the current CUDA device: the kernels run there, on its stream."""
    torch = _need_torch()
    dev = -1
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("libhm works on device memory; got a CPU tensor")
        if dev < 0:
            dev = torch.cuda.current_device()
        if t.get_device() != dev:
            raise ValueError("%s: a tensor is on cuda:%d, the current device is cuda:%d" % (who, t.get_device(), dev))


def gated_scan_args(x, dt, y, A_log, dt_bias=None, h0=None, h_out=None, lengths=None, input_scale: int = 0,
                    states=None) -> GatedScanArgs:
    """Fill an hm_gated_scan_args (x, dt, y: [B, L, D], channels contiguous; h0,
    h_out: [B, D] fp32; lengths: [B] int32; A_log, dt_bias: [D] fp32)."""
    refs = (x, dt, y, A_log, dt_bias, h0, h_out, lengths, states)
    raw = _filler().gated_scan(*refs, input_scale)
    if raw is not None:
        a = GatedScanArgs.from_buffer_copy(raw)
        a._refs = refs
        return a
    who = "gated_scan_args"
    torch = _need_torch()
    B, L, D = x.shape
    _io(who, x.shape, x, x=x, dt=dt, y=y)
    _dense(who, (D,), torch.float32, A_log=A_log, dt_bias=dt_bias)
    _dense(who, (B, D), torch.float32, h0=h0, h_out=h_out)
    _dense(who, (B,), torch.int32, lengths=lengths)
    _buffer(who, states=states)
    _one_device(who, *refs)
    xs, ds, ys = x.stride(), dt.stride(), y.stride() if y is not None else (0, 0)
    a = GatedScanArgs(B, L, D, _dtype_code(x), int(input_scale), _ptr(x), _ptr(dt), _ptr(y), xs[0], xs[1], ds[0],
                      ds[1], ys[0], ys[1], _ptr(A_log), _ptr(dt_bias), _ptr(h0), _ptr(lengths), _ptr(h_out),
                      _ptr(states), states.numel() * states.element_size() if states is not None else 0)
    a._refs = refs
    return a


def hm_gated_scan_states_size(args: GatedScanArgs) -> int:
    return int(lib.hm_gated_scan_states_size(ctypes.byref(args)))


def hm_gated_scan_fwd(args: GatedScanArgs, stream=None) -> None:
    _check(lib.hm_gated_scan_fwd(ctypes.byref(args), _stream(stream)), "hm_gated_scan_fwd")


def gated_scan_bwd_args(x, dt, dy, dx, ddt, A_log, dA_log, states, dt_bias=None, d_dt_bias=None, dh_out=None,
                        dh0=None, lengths=None, input_scale: int = 0, workspace=None) -> GatedScanBwdArgs:
    """Fill an hm_gated_scan_bwd_args (the forward's inputs and its `states`;
    dy, dx, ddt: [B, L, D]; dh_out, dh0: [B, D] fp32; dA_log, d_dt_bias: [D] fp32)."""
    refs = (x, dt, dy, dx, ddt, A_log, dA_log, states, dt_bias, d_dt_bias, dh_out, dh0, lengths)
    raw = _filler().gated_scan_bwd(*refs, input_scale, workspace)
    if raw is not None:
        a = GatedScanBwdArgs.from_buffer_copy(raw)
        a._refs = refs, workspace
        return a
    who = "gated_scan_bwd_args"
    torch = _need_torch()
    B, L, D = x.shape
    _io(who, x.shape, x, x=x, dt=dt, dy=dy, dx=dx, ddt=ddt)
    _dense(who, (D,), torch.float32, A_log=A_log, dt_bias=dt_bias, dA_log=dA_log, d_dt_bias=d_dt_bias)
    _dense(who, (B, D), torch.float32, dh_out=dh_out, dh0=dh0)
    _dense(who, (B,), torch.int32, lengths=lengths)
    _buffer(who, states=states, workspace=workspace)
    _one_device(who, *refs, workspace)
    s = [v for t in (x, dt, dy, dx, ddt) for v in t.stride()[:2]]
    a = GatedScanBwdArgs(B, L, D, _dtype_code(x), int(input_scale), _ptr(x), _ptr(dt), _ptr(dy), _ptr(dx), _ptr(ddt),
                         *s, _ptr(A_log), _ptr(dt_bias), _ptr(lengths), _ptr(states),
                         states.numel() * states.element_size() if states is not None else 0, _ptr(dh_out),
                         _ptr(dA_log), _ptr(d_dt_bias), _ptr(dh0), _ptr(workspace),
                         workspace.numel() * workspace.element_size() if workspace is not None else 0)
    a._refs = refs, workspace
    return a


def hm_gated_scan_bwd_workspace_size(args: GatedScanBwdArgs) -> int:
    return int(lib.hm_gated_scan_bwd_workspace_size(ctypes.byref(args)))


def hm_gated_scan_bwd(args: GatedScanBwdArgs, stream=None) -> None:
    _check(lib.hm_gated_scan_bwd(ctypes.byref(args), _stream(stream)), "hm_gated_scan_bwd")


def gated_step_args(x, dt, y, h, h_out, A_log, dt_bias=None, input_scale: int = 0) -> GatedStepArgs:
    """Fill an hm_gated_step_args (x, dt, y: [B, D]; h, h_out: [B, D] fp32, may be one tensor)."""
    refs = (x, dt, y, h, h_out, A_log, dt_bias)
    raw = _filler().gated_step(*refs, input_scale)
    if raw is not None:
        a = GatedStepArgs.from_buffer_copy(raw)
        a._refs = refs
        return a
    who = "gated_step_args"
    torch = _need_torch()
    B, D = x.shape
    _io(who, x.shape, x, x=x, dt=dt, y=y)
    _dense(who, (D,), torch.float32, A_log=A_log, dt_bias=dt_bias)
    _dense(who, (B, D), torch.float32, h=h, h_out=h_out)
    _one_device(who, *refs)
    a = GatedStepArgs(B, D, _dtype_code(x), int(input_scale), x.data_ptr(), dt.data_ptr(), y.data_ptr(), x.stride(0),
                      dt.stride(0), y.stride(0), A_log.data_ptr(), _ptr(dt_bias), h.data_ptr(), h_out.data_ptr())
    a._refs = refs
    return a


def hm_gated_scan_step(args: GatedStepArgs, stream=None) -> None:
    _check(lib.hm_gated_scan_step(ctypes.byref(args), _stream(stream)), "hm_gated_scan_step")


def _row_stride(t) -> int:
    """Elements between the rows of [..., D], whose leading axes must be dense over one another.
    A broadcast axis (stride 0) is refused: its rows are one row, and a single stride that
    stands for the other axes would count past the tensor's end."""
    if t is None:
        return 0
    if t.dim() == 2:
        return t.stride()[0]
    if t.numel() == 0:
        return t.shape[-1]
    step = want = None
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if st == 0:
            raise ValueError("a tensor of shape %s with strides %s repeats its rows along an axis: pass a dense "
                             "copy (.contiguous())" % (tuple(t.shape), tuple(t.stride())))
        if step is None:
            step = want = st
        elif st != want:
            raise ValueError("rows of a tensor with strides %s are not equally spaced" % (tuple(t.stride()),))
        want *= n
    return t.shape[-1] if step is None else step


def norm_gate_args(y, r, r_out, xn, gate=None, norm: int = 0, post: bool = True, eps: float = 1e-5,
                   alpha: float = 1.0, scale=None, post_w=None, post_b=None, pre_w=None, pre_b=None) -> NormGateArgs:
    """Fill an hm_norm_gate_args (y, gate, r, r_out, xn: [..., D], equally spaced rows, no
    broadcast axes; parameters: [D] fp32)."""
    refs = (y, r, r_out, xn, gate)
    par = (scale, post_w, post_b, pre_w, pre_b)
    raw = _filler().norm_gate(*refs, norm, post, eps, alpha, *par)
    if raw is not None:
        a = NormGateArgs.from_buffer_copy(raw)
        a._refs = refs, par
        return a
    who = "norm_gate_args"
    torch = _need_torch()
    D = y.shape[-1]
    _io(who, y.shape, y, y=y, gate=gate, r=r, r_out=r_out, xn=xn)
    _dense(who, (D,), torch.float32, scale=scale, post_w=post_w, post_b=post_b, pre_w=pre_w, pre_b=pre_b)
    _one_device(who, *refs, *par)
    st = [_row_stride(t) for t in (y, gate, r, r_out, xn)]
    a = NormGateArgs(y.numel() // D if D else 0, D, _dtype_code(y), int(norm), int(post), eps, alpha, _ptr(y),
                     _ptr(gate), _ptr(r), _ptr(r_out), _ptr(xn), *st, _ptr(scale), _ptr(post_w), _ptr(post_b), _ptr(pre_w),
                     _ptr(pre_b))
    a._refs = refs, par
    return a


def hm_norm_gate_fwd(args: NormGateArgs, stream=None) -> None:
    _check(lib.hm_norm_gate_fwd(ctypes.byref(args), _stream(stream)), "hm_norm_gate_fwd")


def norm_gate_bwd_args(y, r_out, dr_out, dxn, dy, dr, gate=None, dgate=None, norm: int = 0, post: bool = True,
                       eps: float = 1e-5, alpha: float = 1.0, scale=None, post_w=None, post_b=None, pre_w=None,
                       dscale=None, dpost_w=None, dpost_b=None, dpre_w=None, dpre_b=None,
                       workspace=None) -> NormGateBwdArgs:
    """Fill an hm_norm_gate_bwd_args (y, gate and the forward's r_out, the gradients of its
    outputs, the gradient buffers; rows [..., D] of one dtype, equally spaced, no broadcast axes;
    parameters and theirs [D] fp32)."""
    refs = (y, r_out, dr_out, dxn, dy, dr, gate, dgate)
    par = (scale, post_w, post_b, pre_w, dscale, dpost_w, dpost_b, dpre_w, dpre_b, workspace)
    raw = _filler().norm_gate_bwd(*refs, norm, post, eps, alpha, *par)
    if raw is not None:
        a = NormGateBwdArgs.from_buffer_copy(raw)
        a._refs = refs, par
        return a
    torch = _need_torch()
    who = "norm_gate_bwd_args"
    D = y.shape[-1]
    _io(who, y.shape, y, y=y, gate=gate, r_out=r_out, dr_out=dr_out, dxn=dxn, dy=dy, dgate=dgate, dr=dr)
    _dense(who, (D,), torch.float32, scale=scale, post_w=post_w, post_b=post_b, pre_w=pre_w, dscale=dscale,
           dpost_w=dpost_w, dpost_b=dpost_b, dpre_w=dpre_w, dpre_b=dpre_b)
    _buffer(who, workspace=workspace)
    _one_device(who, *refs, *par)
    a = NormGateBwdArgs(y.numel() // D if D else 0, D, _dtype_code(y), int(norm), int(post), eps, alpha, _ptr(y),
                        _ptr(gate), _ptr(r_out), _ptr(dr_out), _ptr(dxn), _ptr(dy), _ptr(dgate), _ptr(dr),
                        _row_stride(y), _row_stride(gate), _row_stride(r_out), _row_stride(dr_out), _row_stride(dxn),
                        _row_stride(dy), _row_stride(dgate), _row_stride(dr), _ptr(scale), _ptr(post_w),
                        _ptr(post_b), _ptr(pre_w), _ptr(dscale), _ptr(dpost_w), _ptr(dpost_b), _ptr(dpre_w),
                        _ptr(dpre_b), _ptr(workspace),
                        workspace.numel() * workspace.element_size() if workspace is not None else 0)
    a._refs = refs, par
    return a


def hm_norm_gate_bwd_workspace_size(args: NormGateBwdArgs) -> int:
    return int(lib.hm_norm_gate_bwd_workspace_size(ctypes.byref(args)))


def hm_norm_gate_bwd(args: NormGateBwdArgs, stream=None) -> None:
    _check(lib.hm_norm_gate_bwd(ctypes.byref(args), _stream(stream)), "hm_norm_gate_bwd")


def rotary_args(q, k, q_out, k_out, rot: int = 0, base: float = 10000.0, layout: int = 0, scaling: int = 0,
                factor: float = 1.0, orig_len: float = 0.0, beta_slow: float = 1.0, beta_fast: float = 32.0,
                mscale: float = 1.0, transpose: bool = False, positions=None, pos0: int = 0) -> RotaryArgs:
    """Fill an hm_rotary_args (q, q_out: [B, L, Hq, d]; k, k_out: [B, L, Hk, d] or None; rot = 0
    turns whole heads; positions: int64 [B, L], or [1, L] / [B, 1] shared along an axis of their own)."""
    refs = (q, k, q_out, k_out, positions)
    raw = _filler().rotary(q, k, q_out, k_out, rot, base, layout, scaling, factor, orig_len, beta_slow, beta_fast,
                            mscale, transpose, positions, pos0)
    if raw is not None:
        a = RotaryArgs.from_buffer_copy(raw)
        a._refs = refs
        return a
    who = "rotary_args"
    torch = _need_torch()
    B, L, Hq, d = q.shape
    Hk = 0
    qs, os = q.stride(), q_out.stride()
    ks = ko = (0, 0, 0, 1)
    if (k is None) != (k_out is None):
        raise ValueError("%s: k and k_out come together" % who)
    pb = pt = 0
    if positions is not None:
        if positions.dtype is not torch.int64 or positions.dim() != 2 or positions.shape[0] not in (1, B) \
                or positions.shape[1] not in (1, L):
            raise ValueError("%s: positions must be int64 [B or 1, L or 1]" % who)
        pb = 0 if positions.shape[0] == 1 else positions.stride(0)
        pt = 0 if positions.shape[1] == 1 else positions.stride(1)
    _io(who, q.shape, q, q=q, q_out=q_out)
    if k is not None:
        Hk = k.shape[2]
        ks, ko = k.stride(), k_out.stride()
        _io(who, (B, L, Hk, d), q, k=k, k_out=k_out)
    _one_device(who, *refs)
    a = RotaryArgs(B, L, Hq, Hk, d, int(rot) or d, _dtype_code(q), int(layout), int(scaling), int(transpose), _ptr(q),
                   _ptr(k), _ptr(q_out), _ptr(k_out), qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], os[0], os[1], os[2],
                   ko[0], ko[1], ko[2], _ptr(positions), pb, pt, int(pos0), base, factor, orig_len, beta_slow,
                   beta_fast, mscale)
    a._refs = refs
    return a


def hm_rotary(args: RotaryArgs, stream=None) -> None:
    _check(lib.hm_rotary(ctypes.byref(args), _stream(stream)), "hm_rotary")


def hm_launch_count() -> int:
    """Kernels enqueued by libhm.so in this process so far."""
    return int(lib.hm_launch_count())


def hm_get_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word status."""
    return int(lib.hm_get_device_error(_stream(stream)))


def hm_selftest_wait_timeout(polls: int, stream=None) -> None:
    """Enqueue the bounded-wait self-test (records HM_ERR_TIMEOUT on the device)."""
    _check(lib.hm_selftest_wait_timeout(int(polls), _stream(stream)), "hm_selftest_wait_timeout")


def alloc_workspace(nbytes: int, device=None):
    """A 256-byte-aligned device byte buffer of at least nbytes (torch allocation)."""
    torch = _need_torch()
    if device is None and torch.cuda.is_initialized():
        buf = _filler().alloc(nbytes)
        if buf is not None:
            return buf
    n = max(int(nbytes), 1) + 256
    buf = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    off = (-buf.data_ptr()) % 256
    return buf[off:off + max(int(nbytes), 1)]
