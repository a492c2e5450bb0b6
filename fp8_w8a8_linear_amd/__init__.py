"""Python binding of libnhm, the FP8 W8A8 NemotronH Mamba2 mixer for MI355X (gfx950).

Argument marshalling only: every computation runs in the HIP kernels of
``libnhm.so`` behind the C ABI declared in ``include/nhm.h``. torch supplies
device memory and the current stream. Importing this module fails loudly when
the library has not been built; there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os

__all__ = ["lib", "LIB_PATH", "NhmError", "Geometry", "Layout", "WsLayout", "Fp8Weight", "MixerParams",
           "GEOMETRY", "mixer_layout", "quantize_static", "fp8_linear", "fp8_linear_workspace_bytes",
           "decode_ws_layout", "prefill_ws_layout", "mixer_decode", "mixer_prefill", "NHM_BF16", "NHM_E4M3",
           "NHM_F32", "fp8_dequant_channel_bf16", "mixer_decode_noalloc", "mixer_decode_q",
           "dispatch_counters", "Lora", "fp8_linear_lora", "fp8_linear_lora_workspace_bytes", "beam_select",
           "beam_select_workspace_bytes", "beam_reorder", "BatchPlan", "batch_plan", "mixer_decode_lora",
           "mixer_prefill_lora", "decode_lora_ws_layout", "prefill_lora_ws_layout"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnhm.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python fp8_w8a8_linear_amd/build.py` "
                      "(or __graft_entry__.build()); this package has no non-HIP fallback")
lib = C.CDLL(LIB_PATH)

NHM_BF16, NHM_E4M3, NHM_F32 = 0, 1, 2
_STATUS = {0: "NHM_OK", 1: "NHM_ERR_NULL", 2: "NHM_ERR_SHAPE", 3: "NHM_ERR_ALIGN", 4: "NHM_ERR_UNSUPPORTED",
           5: "NHM_ERR_WORKSPACE", 6: "NHM_ERR_HIP"}


class NhmError(RuntimeError):
    def __init__(self, status, detail):
        super().__init__(f"{_STATUS.get(status, status)}: {detail}")
        self.status = status


class Geometry(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("n_heads", C.c_int32), ("head_dim", C.c_int32), ("d_state", C.c_int32),
                ("n_groups", C.c_int32), ("conv_width", C.c_int32), ("rms_eps", C.c_float)]


class Layout(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "d_inner", "conv_dim", "d_in_proj", "z_off", "z_width", "xbc_off", "xbc_width", "dt_off", "dt_width",
        "x_off", "x_width", "b_off", "b_width", "c_off", "c_width", "heads_per_group", "norm_group")]


class WsLayout(C.Structure):
    _fields_ = [(n, C.c_size_t) for n in ("total", "q_in", "zxbcdt", "xbc_conv", "y", "norm", "q_out")]


class _DispatchCounter(C.Structure):
    _fields_ = [("kernel", C.c_char_p), ("launches", C.c_uint64), ("rows", C.c_uint64)]


class _Fp8Weight(C.Structure):
    _fields_ = [("w", C.c_void_p), ("w_scale", C.c_void_p), ("a_scale", C.c_void_p), ("n", C.c_int64),
                ("k", C.c_int64), ("w_scale_per_tensor", C.c_int32)]


class _MixerParams(C.Structure):
    _fields_ = [("g", Geometry), ("in_proj", _Fp8Weight), ("out_proj", _Fp8Weight), ("conv_w", C.c_void_p),
                ("conv_b", C.c_void_p), ("norm_w", C.c_void_p), ("A_log", C.c_void_p), ("D", C.c_void_p),
                ("dt_bias", C.c_void_p)]


class _Lora(C.Structure):
    _fields_ = [("a", C.c_void_p), ("b", C.c_void_p), ("scale", C.c_void_p), ("n_adapters", C.c_int32),
                ("rank", C.c_int32)]


class _StatePool(C.Structure):
    _fields_ = [("ssm", C.c_void_p), ("conv", C.c_void_p)]


_p, _i32, _i64, _sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
_SIGS = {
    "nhm_status_str": (C.c_char_p, [C.c_int]),
    "nhm_last_error": (C.c_char_p, []),
    "nhm_build_arch": (C.c_char_p, []),
    "nhm_mixer_layout": (C.c_int, [C.POINTER(Geometry), C.POINTER(Layout)]),
    "nhm_fp8_quantize_static": (C.c_int, [_p, _i64, _i64, _i64, _p, _p, _i64, _p]),
    "nhm_fp8_linear_workspace_bytes": (_sz, [_i64, _i64, _i64, C.c_int]),
    "nhm_fp8_dequant_channel_bf16": (C.c_int, [_p, _p, _i64, _i64, _i64, _p, _i64, _p]),
    "nhm_fp8_linear": (C.c_int, [_p, C.c_int, _i64, _i64, C.POINTER(_Fp8Weight), _p, _i64, _p, _sz, _p]),
    "nhm_fp8_linear_ex": (C.c_int, [_p, C.c_int, _i64, _i64, C.POINTER(_Fp8Weight), _p, C.c_int, _i64, _p, _sz, _p]),
    "nhm_fp8_linear_exact": (C.c_int, [_p, C.c_int, _i64, _i64, C.POINTER(_Fp8Weight), _p, C.c_int, _i64, _p, _sz,
                                       _p]),
    "nhm_mixer_decode_ws_layout": (C.c_int, [C.POINTER(Geometry), _i32, C.POINTER(WsLayout)]),
    "nhm_mixer_prefill_ws_layout": (C.c_int, [C.POINTER(Geometry), _i64, _i32, _i32, C.POINTER(WsLayout)]),
    "nhm_mixer_decode": (C.c_int, [C.POINTER(_MixerParams), _p, _i32, _p, _p, _p, _i32, _p, _p, _sz, _p]),
    "nhm_mixer_prefill": (C.c_int, [C.POINTER(_MixerParams), _p, _i64, _p, _i32, _p, _p, _i32, _p, _p, _i32, _p,
                                    _p, _sz, _p]),
    "nhm_mixer_decode_ex": (C.c_int, [C.POINTER(_MixerParams), _p, _i32, _p, _p, C.c_int, _p, _i32, _p, _p, _sz,
                                      _p]),
    "nhm_dispatch_counters": (C.c_int32, [C.POINTER(_DispatchCounter), C.c_int32, C.c_int32]),
    "nhm_mixer_decode_q": (C.c_int, [C.POINTER(_MixerParams), _p, _p, _i32, _p, _p, C.c_int, _p, _i32, _p, _p, _p,
                                     _p, _sz, _p]),
    "nhm_mixer_decode_noalloc": (C.c_int, [C.POINTER(_MixerParams), _p, _i32, _p, _p, C.c_int, _p, _i32, _p, _p]),
    "nhm_mixer_prefill_ex": (C.c_int, [C.POINTER(_MixerParams), _p, _i64, _p, _i32, _p, _p, _i32, _p, C.c_int, _p,
                                       _i32, _p, _p, _sz, _p]),
    "nhm_fp8_linear_lora_workspace_bytes": (_sz, [_i64, _i64, _i64, C.c_int, _i32]),
    "nhm_fp8_linear_lora": (C.c_int, [_p, C.c_int, _i64, _i64, C.POINTER(_Fp8Weight), C.POINTER(_Lora), _p, _p, C.c_int,
                                      _i64, _i32, _p, _sz, _p]),
    "nhm_mixer_decode_lora_ws_layout": (C.c_int, [C.POINTER(Geometry), _i32, _i32, C.POINTER(WsLayout)]),
    "nhm_mixer_prefill_lora_ws_layout": (C.c_int, [C.POINTER(Geometry), _i64, _i32, _i32, _i32, C.POINTER(WsLayout)]),
    "nhm_mixer_decode_lora": (C.c_int, [C.POINTER(_MixerParams), C.POINTER(_Lora), C.POINTER(_Lora), _p, _p, _i32, _p, _p,
                                        C.c_int, _p, _i32, _p, _p, _sz, _p]),
    "nhm_mixer_prefill_lora": (C.c_int, [C.POINTER(_MixerParams), C.POINTER(_Lora), C.POINTER(_Lora), _p, _p, _i64, _p,
                                         _i32, _p, _p, _i32, _p, C.c_int, _p, _i32, _p, _p, _sz, _p]),
    "nhm_beam_select_workspace_bytes": (_sz, [_i64, _i32, _i64, _i32]),
    "nhm_beam_select": (C.c_int, [_p, C.c_int, _i64, _i64, _i32, _i64, _p, _p, _i32, _i32, _p, _p, _p, _p, _sz, _p]),
    "nhm_beam_reorder": (C.c_int, [C.POINTER(Geometry), _p, _p, _i64, _i32, C.POINTER(_StatePool), _i32, C.c_int, _i32,
                                   _p, _p]),
    "nhm_batch_plan": (C.c_int, [_p, _p, _p, _i32, _i64, _p, _p, _p, _p, _p, _p]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.restype, _f.argtypes = _res, _args


def _check(status):
    if status != 0:
        raise NhmError(status, lib.nhm_last_error().decode())


GEOMETRY = dict(hidden=2688, n_heads=64, head_dim=64, d_state=128, n_groups=8, conv_width=4, rms_eps=1e-5)


def _geom(g):
    return Geometry(**g) if isinstance(g, dict) else g


def mixer_layout(g=GEOMETRY):
    out = Layout()
    _check(lib.nhm_mixer_layout(C.byref(_geom(g)), C.byref(out)))
    return {n: getattr(out, n) for n, _ in Layout._fields_}


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _dev_tensor(x, name):
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return x


def _empty(shape, dtype, dev, stream, kept=True):
    """Memory that a call on `stream` (None: the current one) writes, taken under that stream, so that no earlier tenant's
    work is still in it and none gets it while the call runs. kept: it goes to the caller, who may use it on the current
    stream too."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if kept:
        t.record_stream(torch.cuda.current_stream(dev))
    return t


class Fp8Weight:
    """One FP8 W8A8 projection on the device: e4m3 codes [n, k] (uint8), f32 weight scale [n] (per
    output channel) or [1] (per tensor), f32 a_scale [1]."""

    def __init__(self, w, w_scale, a_scale):
        self.w = _dev_tensor(w, "w")
        self.w_scale = _dev_tensor(w_scale, "w_scale")
        self.a_scale = _dev_tensor(a_scale, "a_scale")
        self.n, self.k = int(w.shape[0]), int(w.shape[1])
        ns = int(self.w_scale.numel())
        if ns not in (1, self.n):
            raise ValueError(f"w_scale has {ns} entries: {self.n} (per channel) or 1 (per tensor)")
        self.per_tensor = ns == 1 and self.n != 1
        self._s = _Fp8Weight(self.w.data_ptr(), self.w_scale.data_ptr(), self.a_scale.data_ptr(), self.n, self.k,
                             1 if self.per_tensor else 0)

    @property
    def struct(self):
        return self._s


class MixerParams:
    """All parameters of one mixer block as device tensors (bf16 as int16/uint16 bit patterns)."""

    def __init__(self, in_proj: Fp8Weight, out_proj: Fp8Weight, conv_w, conv_b, norm_w, A_log, D, dt_bias,
                 g=GEOMETRY):
        self.in_proj, self.out_proj = in_proj, out_proj
        self.tensors = dict(conv_w=_dev_tensor(conv_w, "conv_w"), conv_b=_dev_tensor(conv_b, "conv_b"),
                            norm_w=_dev_tensor(norm_w, "norm_w"), A_log=_dev_tensor(A_log, "A_log"),
                            D=_dev_tensor(D, "D"), dt_bias=_dev_tensor(dt_bias, "dt_bias"))
        self.geometry = dict(g)
        t = self.tensors
        self._s = _MixerParams(_geom(g), in_proj.struct, out_proj.struct, t["conv_w"].data_ptr(),
                               t["conv_b"].data_ptr(), t["norm_w"].data_ptr(), t["A_log"].data_ptr(),
                               t["D"].data_ptr(), t["dt_bias"].data_ptr())

    @property
    def struct(self):
        return self._s


def quantize_static(x, scale, q=None, stream=None):
    """e4m3 codes of a bf16 [rows, cols] tensor (given as int16/uint16/bfloat16) with a device f32 scale [1]."""
    import torch
    x = _dev_tensor(x, "x")
    rows, cols = (x.shape[0], x.shape[1]) if x.dim() == 2 else (1, x.numel())
    if q is None:
        q = _empty((rows, cols), torch.uint8, x.device, stream)
    _check(lib.nhm_fp8_quantize_static(_ptr(x), rows, cols, cols, _ptr(scale), _ptr(q), cols, _stream(stream)))
    return q


def fp8_linear_workspace_bytes(m, n, k, a_type):
    return int(lib.nhm_fp8_linear_workspace_bytes(m, n, k, a_type))


def fp8_linear(a, weight: Fp8Weight, out=None, ws=None, a_type=None, stream=None, out_type=None, exact=False):
    """[m, n] = W8A8(a [m, k], weight). a: bf16 bits (int16/uint16/bfloat16) or e4m3 codes (uint8).

    The output is bf16 bits (int16) unless out_type is NHM_F32 (or out is a float32 tensor).
    exact=True calls nhm_fp8_linear_exact (every product summed in f32 on every path)."""
    import torch
    a = _dev_tensor(a, "a")
    if a_type is None:
        a_type = NHM_E4M3 if a.dtype == torch.uint8 else NHM_BF16
    if out_type is None:
        out_type = NHM_F32 if out is not None and out.dtype == torch.float32 else NHM_BF16
    m = int(a.shape[0])
    if out is None:
        out = _empty((m, weight.n), torch.float32 if out_type == NHM_F32 else torch.int16, a.device, stream)
    need = fp8_linear_workspace_bytes(m, weight.n, weight.k, a_type)
    if ws is None and need > 0:
        ws = _empty(need, torch.uint8, a.device, stream, kept=False)
    fn = lib.nhm_fp8_linear_exact if exact else lib.nhm_fp8_linear_ex
    _check(fn(_ptr(a), a_type, m, a.shape[1], C.byref(weight.struct), _ptr(out), out_type, out.shape[1], _ptr(ws),
              0 if ws is None else ws.numel(), _stream(stream)))
    return out


def fp8_dequant_channel_bf16(w, w_scale, out=None, stream=None):
    """bf16 [n, k] = bf16(val(w) * w_scale[row]) of an e4m3 weight [n, k] (uint8)."""
    import torch
    w = _dev_tensor(w, "w")
    n, k = int(w.shape[0]), int(w.shape[1])
    if out is None:
        out = _empty((n, k), torch.int16, w.device, stream)
    _check(lib.nhm_fp8_dequant_channel_bf16(_ptr(w), _ptr(w_scale), n, k, w.stride(0), _ptr(out), out.stride(0),
                                            _stream(stream)))
    return out


def decode_ws_layout(batch, g=GEOMETRY):
    out = WsLayout()
    _check(lib.nhm_mixer_decode_ws_layout(C.byref(_geom(g)), batch, C.byref(out)))
    return {n: int(getattr(out, n)) for n, _ in WsLayout._fields_}


def prefill_ws_layout(n_tokens, n_seqs, chunk=128, g=GEOMETRY):
    out = WsLayout()
    _check(lib.nhm_mixer_prefill_ws_layout(C.byref(_geom(g)), n_tokens, n_seqs, chunk, C.byref(out)))
    return {n: int(getattr(out, n)) for n, _ in WsLayout._fields_}


def _ssm_type(pool):
    """NHM_F32 for a float32 state pool, NHM_BF16 for bf16 bits (int16/uint16) or bfloat16."""
    import torch
    if pool.dtype == torch.float32:
        return NHM_F32
    if pool.dtype in (torch.int16, torch.uint16, torch.bfloat16):
        return NHM_BF16
    raise TypeError(f"SSM state pool of dtype {pool.dtype}: float32 or bf16 bits")


def mixer_decode(params: MixerParams, hidden, slot_idx, ssm_pool, conv_pool, out, ws, stream=None):
    """One decode token per sequence; pools updated in place (f32 or bf16 state pool).
    ws: uint8 device tensor of the layout size."""
    batch = int(hidden.shape[0])
    _check(lib.nhm_mixer_decode_ex(C.byref(params.struct), _ptr(hidden), batch, _ptr(slot_idx), _ptr(ssm_pool),
                                   _ssm_type(ssm_pool), _ptr(conv_pool), int(ssm_pool.shape[0]), _ptr(out), _ptr(ws),
                                   ws.numel(), _stream(stream)))
    return out


def dispatch_counters(reset=False):
    """{kernel: (launches, rows)} of every kernel launched since the last reset (host-side
    counters; a launch captured into a graph counts once). reset=True zeroes them after reading."""
    n = int(lib.nhm_dispatch_counters(None, 0, 0))
    arr = (_DispatchCounter * n)()
    lib.nhm_dispatch_counters(arr, n, 1 if reset else 0)
    return {c.kernel.decode(): (int(c.launches), int(c.rows)) for c in arr if c.launches}


def mixer_decode_q(params: MixerParams, hidden, slot_idx, ssm_pool, conv_pool, out, ws, hidden_q=None, out_q=None,
                   out_q_scale=None, stream=None):
    """mixer_decode with a pre-quantized input (hidden_q: e4m3 codes under in_proj's a_scale; hidden
    may then be None) and/or the output's codes (out_q under out_q_scale, a device f32 [1])."""
    src = hidden if hidden is not None else hidden_q
    batch = int(src.shape[0])
    _check(lib.nhm_mixer_decode_q(C.byref(params.struct), _ptr(hidden), _ptr(hidden_q), batch, _ptr(slot_idx),
                                  _ptr(ssm_pool), _ssm_type(ssm_pool), _ptr(conv_pool), int(ssm_pool.shape[0]),
                                  _ptr(out), _ptr(out_q), _ptr(out_q_scale), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def mixer_decode_noalloc(params: MixerParams, hidden, slot_idx, ssm_pool, conv_pool, out, stream=None):
    """mixer_decode with the library's per-device scratch instead of a workspace (nothing is
    allocated by the call; calls that overlap on one GPU race)."""
    batch = int(hidden.shape[0])
    _check(lib.nhm_mixer_decode_noalloc(C.byref(params.struct), _ptr(hidden), batch, _ptr(slot_idx), _ptr(ssm_pool),
                                        _ssm_type(ssm_pool), _ptr(conv_pool), int(ssm_pool.shape[0]), _ptr(out),
                                        _stream(stream)))
    return out


def mixer_prefill(params: MixerParams, hidden, cu_seqlens, slot_idx, has_initial, ssm_pool, conv_pool, out, ws,
                  chunk=128, stream=None):
    """Varlen prefill of packed sequences; pools updated in place (f32 or bf16 state pool).
    ws: uint8 device tensor of the layout size."""
    n_tokens = int(hidden.shape[0])
    n_seqs = int(slot_idx.shape[0])
    _check(lib.nhm_mixer_prefill_ex(C.byref(params.struct), _ptr(hidden), n_tokens, _ptr(cu_seqlens), n_seqs,
                                    _ptr(slot_idx), _ptr(has_initial), chunk, _ptr(ssm_pool), _ssm_type(ssm_pool),
                                    _ptr(conv_pool), int(ssm_pool.shape[0]), _ptr(out), _ptr(ws), ws.numel(),
                                    _stream(stream)))
    return out


# ---- serving operators (include/nhm_serving.h)

def _on(dev, shapes):
    """Checks (tensor, name, dtypes, shape) entries: contiguous, on `dev`, of one of the dtypes and of the shape
    (None: not checked). Optional tensors may be None."""
    import torch
    index = dev.index
    for t, name, dtypes, shape in shapes:
        if t is None or (isinstance(t, torch.Tensor) and t.get_device() == index and t.is_contiguous()
                         and t.dtype in dtypes and (shape is None or t.shape == shape)):
            continue
        _dev_tensor(t, name)
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, not on {dev}")
        if t.dtype not in dtypes:
            raise TypeError(f"{name} of dtype {t.dtype}: expected {' or '.join(str(d) for d in dtypes)}")
        raise ValueError(f"{name} of shape {tuple(t.shape)}: expected {shape}")


def _call(dev, stream, fn, *args):
    """One library call on `stream` (default: the current stream of `dev`) with `dev` current."""
    import torch
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev.index)     # torch.cuda.current_stream(dev) builds an object: 1.8 us
    elif stream.device != dev:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {dev}")
    else:
        handle = stream.cuda_stream
    if torch.cuda.current_device() == dev.index:
        _check(fn(*args, handle))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, handle))


def _bf16_types():
    import torch
    return (torch.bfloat16, torch.int16, torch.uint16)


def _workspace(ws, need, dev, stream):
    import torch
    if ws is None:
        return _empty(max(need, 1), torch.uint8, dev, stream, kept=False)
    _on(dev, [(ws, "ws", (torch.uint8,), None)])
    return ws


class Lora:
    """The low-rank adapters of one projection [n, k] on the device: a [n_adapters, rank, k] and b
    [n_adapters, n, rank] as bf16 (bits or bfloat16), scale f32 [n_adapters] or None (1)."""

    def __init__(self, a, b, scale=None):
        import torch
        if a.dim() != 3 or b.dim() != 3 or b.shape[0] != a.shape[0] or b.shape[2] != a.shape[1]:
            raise ValueError(f"a {tuple(a.shape)} and b {tuple(b.shape)}: expected [e, rank, k] and [e, n, rank]")
        self.n_adapters, self.rank, self.k = (int(v) for v in a.shape)
        self.n = int(b.shape[1])
        _on(a.device, [(a, "a", _bf16_types(), None), (b, "b", _bf16_types(), None),
                       (scale, "scale", (torch.float32,), (self.n_adapters,))])
        self.a, self.b, self.scale = a, b, scale
        self._s = _Lora(a.data_ptr(), b.data_ptr(), None if scale is None else scale.data_ptr(), self.n_adapters, self.rank)

    @property
    def struct(self):
        return self._s


def fp8_linear_lora_workspace_bytes(m, n, k, a_type, rank):
    return int(lib.nhm_fp8_linear_lora_workspace_bytes(m, n, k, a_type, rank))


def fp8_linear_lora(a, weight: Fp8Weight, lora: Lora, row_adapter, out=None, ws=None, out_type=None, exact=False,
                    stream=None):
    """[m, n] = W8A8(a [m, k], weight) + each row's adapter (row_adapter int32 [m]; a value outside
    [0, lora.n_adapters): none). a: bf16 (bits or bfloat16) or e4m3 codes (uint8).

    The output is bf16 bits (int16) unless out_type is NHM_F32 (or out is a float32 tensor)."""
    import torch
    dev = a.device
    _on(dev, [(a, "a", _bf16_types() + (torch.uint8,), None), (row_adapter, "row_adapter", (torch.int32,), (a.shape[0],)),
              (weight.w, "weight", (weight.w.dtype,), None), (lora.a, "lora", (lora.a.dtype,), None)])
    a_type = NHM_E4M3 if a.dtype == torch.uint8 else NHM_BF16
    if out_type is None:
        out_type = NHM_F32 if out is not None and out.dtype == torch.float32 else NHM_BF16
    m = int(a.shape[0])
    if a.dim() != 2 or a.shape[1] != weight.k:
        raise ValueError(f"a of shape {tuple(a.shape)}: expected [m, {weight.k}]")
    if (lora.n, lora.k) != (weight.n, weight.k):
        raise ValueError(f"adapters of a [{lora.n}, {lora.k}] projection beside a [{weight.n}, {weight.k}] weight")
    if out is None:
        out = _empty((m, weight.n), torch.float32 if out_type == NHM_F32 else torch.int16, dev, stream)
    else:
        _on(dev, [(out, "out", (torch.float32,) if out_type == NHM_F32 else _bf16_types(), (m, weight.n))])
    ws = _workspace(ws, 0 if ws is not None else fp8_linear_lora_workspace_bytes(m, weight.n, weight.k, a_type, lora.rank),
                    dev, stream)
    _call(dev, stream, lib.nhm_fp8_linear_lora, a.data_ptr(), a_type, m, weight.k, C.byref(weight.struct),
          C.byref(lora.struct), row_adapter.data_ptr(), out.data_ptr(), out_type, weight.n, 1 if exact else 0,
          ws.data_ptr(), ws.numel())
    return out


def decode_lora_ws_layout(batch, rank, g=GEOMETRY):
    out = WsLayout()
    _check(lib.nhm_mixer_decode_lora_ws_layout(C.byref(_geom(g)), batch, rank, C.byref(out)))
    return {n: int(getattr(out, n)) for n, _ in WsLayout._fields_}


def prefill_lora_ws_layout(n_tokens, n_seqs, rank, chunk=128, g=GEOMETRY):
    out = WsLayout()
    _check(lib.nhm_mixer_prefill_lora_ws_layout(C.byref(_geom(g)), n_tokens, n_seqs, chunk, rank, C.byref(out)))
    return {n: int(getattr(out, n)) for n, _ in WsLayout._fields_}


def _pool_rows(geom, ssm_pool, conv_pool, what):
    """The rows (slots) of a layer's pools, which must hold equally many of the geometry's states and windows."""
    rows = int(ssm_pool.shape[0])
    row = geom.n_heads * geom.head_dim * geom.d_state
    win = (geom.conv_width - 1) * (geom.n_heads * geom.head_dim + 2 * geom.n_groups * geom.d_state)
    if ssm_pool.numel() != rows * row or conv_pool.numel() != rows * win:
        raise ValueError(f"{what}: pools of shapes {tuple(ssm_pool.shape)} and {tuple(conv_pool.shape)} do not hold {rows} rows")
    return rows


def _mixer_lora(params, lora_in, lora_out, row_adapter, hidden, slot_idx, ssm_pool, conv_pool, out, ws):
    """Checks a mixer call with adapters; the C arguments of the two sets and the row map."""
    import torch
    dev, shape = _dev_tensor(hidden, "hidden").device, (hidden.shape[0], params.geometry["hidden"])
    for lo, w, name in ((lora_in, params.in_proj, "lora_in"), (lora_out, params.out_proj, "lora_out")):
        if lo is not None and (lo.n, lo.k) != (w.n, w.k):
            raise ValueError(f"{name} is for a [{lo.n}, {lo.k}] projection, the block's is [{w.n}, {w.k}]")
        if lo is not None and lo.a.device != dev:
            raise ValueError(f"{name} is on {lo.a.device}, not on {dev}")
    _on(dev, [(hidden, "hidden", _bf16_types(), shape), (out, "out", _bf16_types(), shape),
              (row_adapter, "row_adapter", (torch.int32,), (shape[0],)), (slot_idx, "slot_idx", (torch.int32,), None),
              (ssm_pool, "ssm_pool", _bf16_types() + (torch.float32,), None), (conv_pool, "conv_pool", _bf16_types(), None),
              (ws, "ws", (torch.uint8,), None)])
    _pool_rows(_geom(params.geometry), ssm_pool, conv_pool, "the mixer")
    ref = lambda lo: None if lo is None else C.byref(lo.struct)  # noqa: E731
    return ref(lora_in), ref(lora_out), None if row_adapter is None else row_adapter.data_ptr()


def mixer_decode_lora(params: MixerParams, lora_in, lora_out, row_adapter, hidden, slot_idx, ssm_pool, conv_pool, out, ws,
                      stream=None):
    """mixer_decode with adapters beside in_proj and out_proj (Lora or None each); row_adapter int32 [batch].
    ws: uint8 device tensor of the decode_lora_ws_layout size (for the larger rank)."""
    dev = hidden.device
    args = _mixer_lora(params, lora_in, lora_out, row_adapter, hidden, slot_idx, ssm_pool, conv_pool, out, ws)
    if slot_idx.shape != (hidden.shape[0],):
        raise ValueError(f"slot_idx of shape {tuple(slot_idx.shape)}: expected one slot per row")
    _call(dev, stream, lib.nhm_mixer_decode_lora, C.byref(params.struct), *args, hidden.data_ptr(), int(hidden.shape[0]),
          slot_idx.data_ptr(), ssm_pool.data_ptr(), _ssm_type(ssm_pool), conv_pool.data_ptr(), int(ssm_pool.shape[0]),
          out.data_ptr(), ws.data_ptr(), ws.numel())
    return out


def mixer_prefill_lora(params: MixerParams, lora_in, lora_out, row_adapter, hidden, cu_seqlens, slot_idx, has_initial,
                       ssm_pool, conv_pool, out, ws, chunk=128, stream=None):
    """mixer_prefill with adapters beside in_proj and out_proj (Lora or None each); row_adapter int32 [n_tokens]
    (BatchPlan.token_adapter). ws: uint8 device tensor of the prefill_lora_ws_layout size (for the larger rank)."""
    dev = hidden.device
    args = _mixer_lora(params, lora_in, lora_out, row_adapter, hidden, slot_idx, ssm_pool, conv_pool, out, ws)
    import torch
    n = int(slot_idx.shape[0])
    _on(dev, [(cu_seqlens, "cu_seqlens", (torch.int32,), (n + 1,)), (has_initial, "has_initial", (torch.int32,), (n,))])
    _call(dev, stream, lib.nhm_mixer_prefill_lora, C.byref(params.struct), *args, hidden.data_ptr(), int(hidden.shape[0]),
          cu_seqlens.data_ptr(), int(slot_idx.shape[0]), slot_idx.data_ptr(), has_initial.data_ptr(), chunk,
          ssm_pool.data_ptr(), _ssm_type(ssm_pool), conv_pool.data_ptr(), int(ssm_pool.shape[0]), out.data_ptr(),
          ws.data_ptr(), ws.numel())
    return out


def beam_select_workspace_bytes(n_groups, n_beams, vocab, n_cand):
    return int(lib.nhm_beam_select_workspace_bytes(n_groups, n_beams, vocab, n_cand))


def beam_select(logits, cum, n_cand, finished=None, eos=0, scores=None, parents=None, tokens=None, ws=None, stream=None):
    """(scores f32, parents int32, tokens int32), each [groups, n_cand]: the n_cand best continuations of each
    group's beams, best first. logits: bf16 (bits or bfloat16) or float32 [groups * beams, vocab] (or [groups, beams,
    vocab]); cum: float32 [groups, beams]; finished: int32 [groups, beams], non-zero for beams that go on by eos alone."""
    import torch
    dev = logits.device
    if cum.dim() != 2:
        raise ValueError(f"cum of shape {tuple(cum.shape)}: expected [groups, beams]")
    G, K = (int(v) for v in cum.shape)
    V = int(logits.shape[-1])
    if logits.numel() != G * K * V:
        raise ValueError(f"logits of shape {tuple(logits.shape)}: expected [{G} * {K}, vocab]")
    i32, f32 = (torch.int32,), (torch.float32,)
    _on(dev, [(logits, "logits", _bf16_types() + f32, None), (cum, "cum", f32, None), (finished, "finished", i32, (G, K)),
              (scores, "scores", f32, (G, n_cand)), (parents, "parents", i32, (G, n_cand)),
              (tokens, "tokens", i32, (G, n_cand))])
    if scores is None:
        scores = _empty((G, n_cand), torch.float32, dev, stream)
    if parents is None:
        parents = _empty((G, n_cand), torch.int32, dev, stream)
    if tokens is None:
        tokens = _empty((G, n_cand), torch.int32, dev, stream)
    ws = _workspace(ws, 0 if ws is not None else beam_select_workspace_bytes(G, K, V, n_cand), dev, stream)
    _call(dev, stream, lib.nhm_beam_select, logits.data_ptr(), NHM_F32 if logits.dtype == torch.float32 else NHM_BF16, V,
          G, K, V, cum.data_ptr(), None if finished is None else finished.data_ptr(), int(eos), n_cand,
          scores.data_ptr(), parents.data_ptr(), tokens.data_ptr(), ws.data_ptr(), ws.numel())
    return scores, parents, tokens


def beam_reorder(parents, slots, ssm_pools, conv_pools, new_slots=None, g=GEOMETRY, stream=None):
    """The slots of each group's beams after a selection (int32 [groups, beams]); the states of beams that share a
    parent are copied between the pools' rows in place. parents, slots: int32 [groups, beams]; ssm_pools, conv_pools:
    one tensor per layer, as mixer_decode takes them."""
    import torch
    dev = parents.device
    ssm_pools, conv_pools = list(ssm_pools), list(conv_pools)
    if len(ssm_pools) != len(conv_pools) or not ssm_pools:
        raise ValueError(f"{len(ssm_pools)} SSM pools and {len(conv_pools)} conv pools: one of each per layer")
    if parents.dim() != 2:
        raise ValueError(f"parents of shape {tuple(parents.shape)}: expected [groups, beams]")
    geom = _geom(g)
    st = _ssm_type(ssm_pools[0])
    st_types, bf16 = (ssm_pools[0].dtype,), _bf16_types()
    S = int(ssm_pools[0].shape[0])
    for i, (sp, cp) in enumerate(zip(ssm_pools, conv_pools)):
        _on(dev, ((sp, "an SSM pool", st_types, None), (cp, "a conv pool", bf16, None)))
        if _pool_rows(geom, sp, cp, "a layer") != S:
            raise ValueError(f"layer {i}: pools of {int(sp.shape[0])} rows, the first layer's hold {S}")
    i32, shape = (torch.int32,), tuple(parents.shape)
    _on(dev, [(parents, "parents", i32, None), (slots, "slots", i32, shape), (new_slots, "new_slots", i32, shape)])
    if new_slots is None:
        new_slots = _empty(shape, torch.int32, dev, stream)
    arr = (_StatePool * len(ssm_pools))(*[(sp.data_ptr(), cp.data_ptr()) for sp, cp in zip(ssm_pools, conv_pools)])
    _call(dev, stream, lib.nhm_beam_reorder, C.byref(geom), parents.data_ptr(), slots.data_ptr(), shape[0], shape[1], arr,
          len(arr), st, S, new_slots.data_ptr())
    return new_slots


class BatchPlan:
    """The index tensors of a packed batch of up to n_tokens tokens in n_seqs sequences (int32, filled by
    batch_plan): cu_seqlens [n_seqs + 1], has_initial [n_seqs], and per token token_seq, token_pos, token_adapter."""

    def __init__(self, n_seqs, n_tokens, device="cuda"):
        import torch
        self.n_seqs, self.n_tokens = int(n_seqs), int(n_tokens)
        new = lambda n: torch.empty(n, dtype=torch.int32, device=device)  # noqa: E731
        self.cu_seqlens, self.has_initial = new(self.n_seqs + 1), new(self.n_seqs)
        self.token_seq, self.token_pos, self.token_adapter = new(self.n_tokens), new(self.n_tokens), new(self.n_tokens)


def batch_plan(lengths, plan: BatchPlan, past=None, adapters=None, stream=None):
    """Fills plan from lengths int32 [n_seqs] (this batch's tokens of each sequence), past (tokens its state holds
    already) and adapters (its adapter), both int32 [n_seqs] or None. Returns plan."""
    import torch
    dev, n = lengths.device, (plan.n_seqs,)
    i32 = (torch.int32,)
    _on(dev, [(lengths, "lengths", i32, n), (past, "past", i32, n), (adapters, "adapters", i32, n),
              (plan.cu_seqlens, "plan", i32, None)])
    opt = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _call(dev, stream, lib.nhm_batch_plan, lengths.data_ptr(), opt(past), opt(adapters), plan.n_seqs, plan.n_tokens,
          plan.cu_seqlens.data_ptr(), plan.has_initial.data_ptr(), plan.token_seq.data_ptr(), plan.token_pos.data_ptr(),
          plan.token_adapter.data_ptr())
    return plan
