"""ctypes binding of libmq.so (C ABI in include/mq.h).

Argument marshalling only: every step of the quantizer and the GEMM runs in
the CUDA kernels of libmq.so.  There is no CPU fallback; if the library has
not been built or the current device is not a B200 (sm_100a), calls raise.

The functions keep the C names.  They take torch CUDA tensors (for device
memory) and enqueue on the current torch stream unless `stream` is given.
With MQ_DEBUG=1 in the environment the debug build (libmq_debug.so, every
index-computed access and TMA coordinate bounds-checked) is loaded instead.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmq_debug.so" if os.environ.get("MQ_DEBUG") == "1" else "libmq.so")

MQ_OK = 0
MQ_ERR_TIMEOUT = -7

_lib = None


class MQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib().mq_status_string(status).decode()} ({status})")


def lib() -> ctypes.CDLL:
    """Load libmq.so (built by ``python -m nvfp4_w4a4_quantized_03_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m nvfp4_w4a4_quantized_03_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        L.mq_status_string.argtypes = [ctypes.c_int]
        L.mq_status_string.restype = ctypes.c_char_p
        for name in ("mq_nvfp4_codes_bytes", "mq_nvfp4_scales_bytes", "mq_linear_w4a4_workspace_bytes"):
            getattr(L, name).argtypes = [i64, i64]
            getattr(L, name).restype = sz
        L.mq_workspace_bytes.argtypes = []
        L.mq_workspace_bytes.restype = sz
        L.mq_tensor_scale.argtypes = [vp, i64, vp, vp, sz, vp]
        L.mq_tensor_amax.argtypes = [vp, i64, vp, vp, sz, vp]
        L.mq_alpha_from_amax.argtypes = [vp, vp, vp]
        L.mq_nvfp4_quantize.argtypes = [vp, i64, i64, vp, vp, vp, vp]
        L.mq_nvfp4_gemm.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, sz, vp]
        L.mq_linear_w4a4.argtypes = [vp, i64, i64, vp, vp, vp, i64, vp, vp, sz, vp]
        L.mq_read_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int32)]
        L.mq_nvfp4_gemm_swiglu.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, sz, vp]
        L.mq_mlp_w4a4_workspace_bytes.argtypes = [i64, i64, i64]
        L.mq_mlp_w4a4_workspace_bytes.restype = sz
        L.mq_mlp_w4a4.argtypes = [vp, i64, i64, vp, vp, vp, i64, vp, vp, vp, i64, vp, vp, sz, vp]
        i32, cache, batch = ctypes.c_int32, vp, vp
        L.mq_linear_w4a16.argtypes = [vp, i64, i64, vp, vp, vp, i64, vp, vp]
        L.mq_rope_kv_append.argtypes = [vp, i64, i64, i32, vp, i64, i32, i32, cache, batch, vp, vp, sz, vp]
        L.mq_kv_attention_workspace_bytes.argtypes = [i32, i32, i32, i32, i64, i64]
        L.mq_kv_attention_workspace_bytes.restype = sz
        L.mq_kv_attention.argtypes = [vp, i64, i64, i32, cache, batch, i64, i64, ctypes.c_float, vp, vp, sz, vp]
        L.mq_is_debug_build.argtypes = []
        L.mq_debug_bounds_hits.argtypes = [ctypes.POINTER(ctypes.c_int64)]
        L.mq_set_switch.argtypes = [ctypes.c_int, ctypes.c_int]
        L.mq_get_switch.argtypes = [ctypes.c_int]
        L.mq_debug_noalloc_fill_header.argtypes = [ctypes.c_uint32, vp]
        for name in ("mq_tensor_scale", "mq_tensor_amax", "mq_alpha_from_amax", "mq_nvfp4_quantize",
                     "mq_nvfp4_gemm", "mq_linear_w4a4", "mq_read_status", "mq_nvfp4_gemm_swiglu",
                     "mq_mlp_w4a4", "mq_linear_w4a16", "mq_rope_kv_append", "mq_kv_attention", "mq_is_debug_build", "mq_debug_bounds_hits", "mq_set_switch",
                     "mq_get_switch", "mq_debug_noalloc_fill_header"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _torch_stream(stream, device) -> torch.cuda.Stream:
    """A stream or its address as torch's stream (address 0: the default one,
    which ExternalStream would take for a new stream)."""
    if hasattr(stream, "cuda_stream"):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)


def _check(status: int, what: str):
    if status != MQ_OK:
        raise MQError(status, what)


# -- selectable alternatives (MQ_SWITCH_* in mq.h) -------------------------

SWITCHES = {"linear_path": 0, "gemm_form": 1, "gemm_decode": 2, "decode_split": 3, "gemm_stages": 4,
            "gemm_group_m": 5, "pdl": 6}
LINEAR_PATHS = {"onepass": 0, "split": 1, "ingemm": 2}


def _switch_id(name) -> int:
    return name if isinstance(name, int) else SWITCHES[name]


def mq_set_switch(name, value: int) -> None:
    """Set a process-wide switch by name (SWITCHES) or MQ_SWITCH_* number;
    the linear path also takes its name (LINEAR_PATHS)."""
    if name == "linear_path" and isinstance(value, str):
        value = LINEAR_PATHS[value]
    _check(lib().mq_set_switch(_switch_id(name), int(value)), f"mq_set_switch({name}, {value})")


def mq_get_switch(name) -> int:
    v = int(lib().mq_get_switch(_switch_id(name)))
    if v < 0:
        raise MQError(v, f"mq_get_switch({name})")
    return v


class switch:
    """Context manager: `with mq.switch(gemm_form=2): ...` sets switches for
    the block and puts the previous values back afterwards."""

    def __init__(self, **values):
        self.values = values
        self.saved = {}

    def __enter__(self):
        for name, v in self.values.items():
            self.saved[name] = mq_get_switch(name)
            mq_set_switch(name, v)
        return self

    def __exit__(self, *exc):
        for name, v in self.saved.items():
            mq_set_switch(name, v)
        return False


# -- sizes ------------------------------------------------------------------

def mq_nvfp4_codes_bytes(rows: int, K: int) -> int:
    return int(lib().mq_nvfp4_codes_bytes(rows, K))


def mq_nvfp4_scales_bytes(rows: int, K: int) -> int:
    return int(lib().mq_nvfp4_scales_bytes(rows, K))


def mq_workspace_bytes() -> int:
    return int(lib().mq_workspace_bytes())


def mq_linear_w4a4_workspace_bytes(M: int, K: int) -> int:
    return int(lib().mq_linear_w4a4_workspace_bytes(M, K))


# -- calls ------------------------------------------------------------------

def mq_tensor_scale(x: torch.Tensor, alpha: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    assert x.dtype == torch.bfloat16 and alpha.dtype == torch.float32
    _check(lib().mq_tensor_scale(_ptr(x), x.numel(), _ptr(alpha), _ptr(ws), ws.numel() * ws.element_size(),
                                 _stream(stream)), "mq_tensor_scale")


def mq_tensor_amax(x: torch.Tensor, amax: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    assert x.dtype == torch.bfloat16 and amax.dtype == torch.float32
    _check(lib().mq_tensor_amax(_ptr(x), x.numel(), _ptr(amax), _ptr(ws), ws.numel() * ws.element_size(),
                                _stream(stream)), "mq_tensor_amax")


def mq_alpha_from_amax(amax: torch.Tensor, alpha: torch.Tensor, stream=None) -> None:
    assert amax.dtype == torch.float32 and alpha.dtype == torch.float32
    _check(lib().mq_alpha_from_amax(_ptr(amax), _ptr(alpha), _stream(stream)), "mq_alpha_from_amax")


def mq_nvfp4_quantize(x: torch.Tensor, alpha: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                      stream=None) -> None:
    assert x.dtype == torch.bfloat16 and x.dim() == 2
    rows, K = x.shape
    assert codes.numel() * codes.element_size() >= mq_nvfp4_codes_bytes(rows, K)
    assert scales.numel() * scales.element_size() >= mq_nvfp4_scales_bytes(rows, K)
    _check(lib().mq_nvfp4_quantize(_ptr(x), rows, K, _ptr(alpha), _ptr(codes), _ptr(scales), _stream(stream)),
           "mq_nvfp4_quantize")


def mq_nvfp4_gemm(a_codes, a_scales, alpha_a, b_codes, b_scales, alpha_b, M: int, N: int, K: int,
                  y: torch.Tensor, ws: torch.Tensor | None = None, stream=None) -> None:
    assert y.dtype == torch.bfloat16 and y.numel() >= M * N
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().mq_nvfp4_gemm(_ptr(a_codes), _ptr(a_scales), _ptr(alpha_a), _ptr(b_codes), _ptr(b_scales),
                               _ptr(alpha_b), M, N, K, _ptr(y), _ptr(ws), ws_bytes, _stream(stream)),
           "mq_nvfp4_gemm")


def mq_linear_w4a4(x: torch.Tensor, w_codes, w_scales, alpha_w, N: int, y: torch.Tensor, ws: torch.Tensor,
                   stream=None) -> None:
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and y.dtype == torch.bfloat16
    M, K = x.shape
    assert y.numel() >= M * N
    _check(lib().mq_linear_w4a4(_ptr(x), M, K, _ptr(w_codes), _ptr(w_scales), _ptr(alpha_w), N, _ptr(y),
                                _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), "mq_linear_w4a4")


def mq_nvfp4_gemm_swiglu(a_codes, a_scales, alpha_a, b_codes, b_scales, alpha_b, M: int, inter: int, K: int,
                         h: torch.Tensor, h_amax: torch.Tensor, ws: torch.Tensor | None = None, stream=None) -> None:
    assert h.dtype == torch.bfloat16 and h.numel() >= M * inter and h_amax.dtype == torch.float32
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().mq_nvfp4_gemm_swiglu(_ptr(a_codes), _ptr(a_scales), _ptr(alpha_a), _ptr(b_codes), _ptr(b_scales),
                                      _ptr(alpha_b), M, inter, K, _ptr(h), _ptr(h_amax), _ptr(ws), ws_bytes,
                                      _stream(stream)), "mq_nvfp4_gemm_swiglu")


def mq_mlp_w4a4_workspace_bytes(M: int, K: int, inter: int) -> int:
    return int(lib().mq_mlp_w4a4_workspace_bytes(M, K, inter))


def mq_mlp_w4a4(x: torch.Tensor, wgu_codes, wgu_scales, alpha_gu, inter: int, wd_codes, wd_scales, alpha_d,
                N: int, y: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and y.dtype == torch.bfloat16
    M, K = x.shape
    assert y.numel() >= M * N
    _check(lib().mq_mlp_w4a4(_ptr(x), M, K, _ptr(wgu_codes), _ptr(wgu_scales), _ptr(alpha_gu), inter,
                             _ptr(wd_codes), _ptr(wd_scales), _ptr(alpha_d), N, _ptr(y), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "mq_mlp_w4a4")


# The kernels of a decode step run for a few microseconds, so the checks and the
# marshalling of its calls are native (csrc/mq_torch.cpp); arguments that it
# refuses raise ValueError before the library sees them.

_calls = None


def _load_calls():
    global _calls
    if _calls is None:
        path = os.path.join(_HERE, "_mq_torch.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m nvfp4_w4a4_quantized_03_b200.build`")
        from . import _mq_torch
        L = lib()
        _mq_torch.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                         for f in (L.mq_linear_w4a16, L.mq_rope_kv_append, L.mq_kv_attention)))
        _calls = _mq_torch
    return _calls


def mq_linear_w4a16(x: torch.Tensor, w_codes, w_scales, alpha_w, N: int, y: torch.Tensor, stream=None) -> None:
    """y = x W^T, x bf16 [M, K] with M <= 64, W quantized."""
    status = (_calls or _load_calls()).linear(x, w_codes, w_scales, alpha_w, N, y, stream)
    if status:
        raise MQError(status, "mq_linear_w4a16")


def mq_rope_kv_append(qkv: torch.Tensor, rope, cu_rows, lens, page_table, k_codes, v_codes, k_scales, v_scales,
                      q_out: torch.Tensor, ws: torch.Tensor | None = None, rot_dim: int | None = None,
                      interleaved: bool = False, stream=None) -> None:
    """Rotates Q and K of qkv [T, (q heads + 2 kv heads) head_dim] into q_out
    [T, q heads, head_dim] and, with V, into the cache (k_codes, v_codes
    [pages, kv heads, page size, head_dim], scales [pages, kv heads]).  rope:
    [positions, rot_dim] float32 (rope_table), None for rot_dim = 0."""
    status = (_calls or _load_calls()).append(qkv, rope, cu_rows, lens, page_table, k_codes, v_codes, k_scales, v_scales,
                                              q_out, ws, rot_dim, interleaved, stream)
    if status:
        raise MQError(status, "mq_rope_kv_append")


def mq_kv_attention_workspace_bytes(batch: int, q_heads: int, kv_heads: int, head_dim: int, max_q: int,
                                    max_len: int) -> int:
    return int(lib().mq_kv_attention_workspace_bytes(batch, q_heads, kv_heads, head_dim, max_q, max_len))


def mq_kv_attention(q: torch.Tensor, cu_rows, lens, page_table, k_codes, v_codes, k_scales, v_scales,
                    out: torch.Tensor, ws: torch.Tensor, max_q: int, max_len: int, scale: float,
                    stream=None) -> None:
    """Causal attention of q [T, q heads, head_dim] (rows may be apart, e.g. a
    slice of a wider tensor) over the cache, into out of the same shape."""
    status = (_calls or _load_calls()).attention(q, cu_rows, lens, page_table, k_codes, v_codes, k_scales, v_scales, out, ws,
                                                 max_q, max_len, scale, stream)
    if status:
        raise MQError(status, "mq_kv_attention")


def mq_is_debug_build() -> bool:
    return bool(lib().mq_is_debug_build())


def mq_debug_bounds_hits() -> int:
    """Failed bounds checks since the previous call (synchronizes the device;
    always 0 in the release build)."""
    out = ctypes.c_int64(0)
    _check(lib().mq_debug_bounds_hits(ctypes.byref(out)), "mq_debug_bounds_hits")
    return int(out.value)


def mq_read_status(ws: torch.Tensor, stream=None) -> int:
    out = ctypes.c_int32(0)
    _check(lib().mq_read_status(_ptr(ws), _stream(stream), ctypes.byref(out)), "mq_read_status")
    return int(out.value)


# -- conveniences (allocation through torch, then the calls above) ----------

class QuantizedTensor:
    """NVFP4 tensor [rows, K]: packed codes, MMA-ordered scales, alpha (device)."""

    def __init__(self, rows: int, K: int, device):
        self.rows, self.K = rows, K
        self.codes = torch.empty(mq_nvfp4_codes_bytes(rows, K), dtype=torch.uint8, device=device)
        self.scales = torch.empty(mq_nvfp4_scales_bytes(rows, K), dtype=torch.uint8, device=device)
        self.alpha = torch.empty(1, dtype=torch.float32, device=device)


def workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-filled workspace buffer (the calls keep its counters at zero)."""
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


class _Workspaces:
    """The workspaces of one object's calls: one per stream, made and zero-filled
    on it, so that calls on several streams may overlap; and one per stream of a
    graph capture, which no other call uses, so that graphs may overlap with one
    another and with later calls."""

    def __init__(self, keep: bool = False):
        self.by_place, self.last = {}, None
        self.sizes, self.nbytes = None, 0
        # workspaces that were too small for a later call: those that a graph holds, and all if
        # they are to be kept.  Each is at least half as large again as the one before, so those
        # of a place are together at most twice the newest.
        self.keep, self.replaced = keep, []

    def of(self, bytes_of, sizes, device, stream=None) -> torch.Tensor:
        """get() of the bytes of a call of these sizes (asking the library takes a
        microsecond, and calls of the same sizes follow one another)."""
        if sizes != self.sizes:
            self.sizes, self.nbytes = sizes, bytes_of(*sizes)
        return self.get(self.nbytes, device, stream)

    def get(self, nbytes: int, device, stream=None) -> torch.Tensor:
        if not isinstance(device, torch.device):
            device = torch.device(device)
        place = (_calls or _load_calls()).place(stream, device)
        ws = self.by_place.get(place)
        if ws is None or ws.numel() < nbytes:
            if ws is not None and (self.keep or place[2]):
                self.replaced.append(ws)
                nbytes = max(nbytes, ws.numel() * 3 // 2)
            if place[2]:
                ws = self._outside_the_capture(nbytes, place)
            else:
                with torch.cuda.stream(None if stream is None else _torch_stream(stream, device)):
                    ws = workspace(nbytes, device)
            self.by_place[place] = ws
        self.last = ws
        return ws

    @staticmethod
    def _outside_the_capture(nbytes: int, place) -> torch.Tensor:
        """Zero-filled now, on a stream that is in no capture: a fill in the graph
        would run at every replay, and not before the first."""
        device, relaxed = torch.device("cuda", place[0]), 2              # cudaStreamCaptureModeRelaxed
        mode = _calls.capture_mode(relaxed)
        try:
            for _ in range(64):                      # torch hands out the streams of a pool in turn
                side = torch.cuda.Stream(device)
                if not _calls.place(side, device)[2]:
                    break
            else:
                raise RuntimeError("no stream outside the capture")
            with torch.cuda.stream(side):
                ws = workspace(nbytes, device)
            side.synchronize()
        finally:
            _calls.capture_mode(mode)
        return ws


class _HasWorkspaces:
    """`_ws`: the last call's workspace; setting it to None lets all go."""

    _keep_workspaces = False

    def __init__(self):
        self._spaces = _Workspaces(self._keep_workspaces)

    @property
    def _ws(self):
        return self._spaces.last

    @_ws.setter
    def _ws(self, ws):
        assert ws is None
        self._spaces = _Workspaces(self._keep_workspaces)


def _output(out, shape, device, stream) -> torch.Tensor:
    """`out`, or a new tensor: of the call's stream, since memory that the current
    one gave back may still be in use there, and not handed out again before
    what the current one holds when it is let go."""
    if out is not None:
        return out
    if stream is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        out = torch.empty(shape, dtype=torch.bfloat16, device=device)
    out.record_stream(torch.cuda.current_stream(device))
    return out


def quantize(x: torch.Tensor, ws: torch.Tensor | None = None, stream=None) -> QuantizedTensor:
    """alpha_x of x, then its NVFP4 codes and scales (e.g. offline weight quantization)."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream, x.device)):
            q = quantize(x, ws)
        for t in (q.codes, q.scales, q.alpha):
            t.record_stream(torch.cuda.current_stream(x.device))
        return q
    rows, K = x.shape
    q = QuantizedTensor(rows, K, x.device)
    if ws is None:
        ws = workspace(mq_workspace_bytes(), x.device)
    mq_tensor_scale(x, q.alpha, ws)
    mq_nvfp4_quantize(x, q.alpha, q.codes, q.scales)
    return q


class LinearW4A4(_HasWorkspaces):
    """A linear layer y = x W^T on the FP4 prefill path: W quantized once at
    construction, x quantized per call inside mq_linear_w4a4.  Calls on
    different streams may overlap."""

    def __init__(self, weight: torch.Tensor):
        super().__init__()
        assert weight.dtype == torch.bfloat16 and weight.is_cuda
        self.N, self.K = weight.shape
        self.w = quantize(weight.contiguous())

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        M, K = x.shape
        assert K == self.K
        ws = self._spaces.of(mq_linear_w4a4_workspace_bytes, (M, K), x.device, stream)
        out = _output(out, (M, self.N), x.device, stream)
        mq_linear_w4a4(x, self.w.codes, self.w.scales, self.w.alpha, self.N, out, ws, stream)
        return out


class MLPW4A4(_HasWorkspaces):
    """A decoder MLP on the FP4 prefill path: y = (SwiGLU(x Wg^T, x Wu^T)) Wd^T
    with both linears W4A4.  The gate and up weights are quantized as one
    [2 inter, K] tensor (gate rows first), the down weight [N, inter] on its
    own, once at construction; x and H are quantized per call.  Calls on
    different streams may overlap."""

    def __init__(self, w_gate_up: torch.Tensor, w_down: torch.Tensor):
        super().__init__()
        assert w_gate_up.dtype == torch.bfloat16 and w_down.dtype == torch.bfloat16
        two_inter, self.K = w_gate_up.shape
        self.inter = two_inter // 2
        self.N = w_down.shape[0]
        assert two_inter == 2 * self.inter and w_down.shape[1] == self.inter
        self.wgu = quantize(w_gate_up.contiguous())
        self.wd = quantize(w_down.contiguous())

    def workspace(self, M: int, device, stream=None) -> torch.Tensor:
        return self._spaces.of(mq_mlp_w4a4_workspace_bytes, (M, self.K, self.inter), device, stream)

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        M, K = x.shape
        assert K == self.K
        ws = self.workspace(M, x.device, stream)
        out = _output(out, (M, self.N), x.device, stream)
        mq_mlp_w4a4(x, self.wgu.codes, self.wgu.scales, self.wgu.alpha, self.inter, self.wd.codes, self.wd.scales,
                    self.wd.alpha, self.N, out, ws, stream)
        return out

    def h_view(self, M: int) -> torch.Tensor:
        """H [M, inter] as the last call left it in the workspace."""
        off = mq_linear_w4a4_workspace_bytes(M, self.K)
        return self._ws[off:off + M * self.inter * 2].view(torch.bfloat16).view(M, self.inter)


class LinearW4A16:
    """A linear layer y = x W^T whose activation stays in bf16 (decode steps of
    at most 64 rows): W in NVFP4, quantized here or shared with a LinearW4A4."""

    def __init__(self, weight):
        if isinstance(weight, LinearW4A4):
            weight = weight.w
        if not isinstance(weight, QuantizedTensor):
            assert weight.dtype == torch.bfloat16 and weight.is_cuda
            weight = quantize(weight.contiguous())
        self.w, self.N, self.K = weight, weight.rows, weight.K

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        M, K = x.shape
        assert K == self.K
        out = _output(out, (M, self.N), x.device, stream)
        mq_linear_w4a16(x, self.w.codes, self.w.scales, self.w.alpha, self.N, out, stream)
        return out


def rope_table(positions: int, rot_dim: int, theta: float = 10000.0, scaling: dict | None = None,
               device="cuda") -> torch.Tensor:
    """[positions, rot_dim] float32: cos, then sin, of position * f_j, f_j =
    theta^(-2 j / rot_dim), j < rot_dim / 2, with angles in 64 bits.

    scaling, for contexts longer than a model was trained on:
      {"kind": "linear", "factor": s}   f_j / s
      {"kind": "yarn", "factor": s, "original": L, "beta_fast": 32, "beta_slow": 1}
          f_j / s for pairs that turn less than beta_slow times within L
          positions, f_j for those that turn more than beta_fast times, a
          linear blend over j between, and cos and sin times 0.1 ln(s) + 1
          (Peng et al., "YaRN: Efficient Context Window Extension of Large
          Language Models", 2023, section 3)."""
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim: a positive even number expected")
    j = torch.arange(rot_dim // 2, dtype=torch.float64)
    f, size = theta ** (-2.0 * j / rot_dim), 1.0
    if scaling is not None:
        kind, s = scaling["kind"], float(scaling["factor"])
        if kind == "linear":
            f = f / s
        elif kind == "yarn":
            # the pair that turns `beta` times within L positions: f L = 2 pi beta
            at = [rot_dim * math.log(scaling["original"] / (2 * math.pi * scaling.get(name, beta))) / (2 * math.log(theta))
                  for name, beta in (("beta_fast", 32.0), ("beta_slow", 1.0))]
            low, high = max(0, math.floor(at[0])), min(rot_dim - 1, math.ceil(at[1]))
            ramp = ((j - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
            f = f / s * ramp + f * (1.0 - ramp)
            size = 0.1 * math.log(s) + 1.0 if s > 1.0 else 1.0
        else:
            raise ValueError(f"scaling: kind 'linear' or 'yarn' expected, got {kind!r}")
    f = f.to(device)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * f
    return (torch.cat([angle.cos(), angle.sin()], 1) * size).float()


class PagedKVCache:
    """A pool of E4M3 pages (mq_kv_cache): k, v [pages, kv heads, page size,
    head_dim], one power-of-two scale per (page, kv head).  Which page holds
    what is the caller's page table."""

    def __init__(self, num_pages: int, page_size: int, kv_heads: int, head_dim: int, device):
        shape = (num_pages, kv_heads, page_size, head_dim)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in "kv")
        self.k_scale, self.v_scale = (torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in "kv")
        self.page_size, self.kv_heads, self.head_dim = page_size, kv_heads, head_dim

    def tensors(self):
        return self.k, self.v, self.k_scale, self.v_scale


class AttentionW4A4(_HasWorkspaces):
    """The attention block of a decoder layer, from its input to its O linear:
    QKV linear, rotary positions, append to the paged cache, attention, O
    linear.  The weights are NVFP4; `precise` says whether the linears quantize
    their activation (prefill, LinearW4A4) or not (decode, LinearW4A16, at most
    64 rows).

    w_qkv [(q heads + 2 kv heads) head_dim, hidden] (q, k, v rows in this
    order), w_o [hidden, q heads * head_dim]; rope: rope_table(...).  Calls on
    different streams and replays of captured ones, with caches of their own,
    may overlap; a capture's workspaces live as long as the block."""

    _keep_workspaces = True

    def __init__(self, w_qkv: torch.Tensor, w_o: torch.Tensor, q_heads: int, kv_heads: int, head_dim: int,
                 rope: torch.Tensor, interleaved: bool = False):
        super().__init__()
        assert w_qkv.shape[0] == (q_heads + 2 * kv_heads) * head_dim and w_o.shape[1] == q_heads * head_dim
        self.qkv, self.o = LinearW4A4(w_qkv), LinearW4A4(w_o)
        self.qkv_precise, self.o_precise = LinearW4A16(self.qkv), LinearW4A16(self.o)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.rope, self.interleaved = rope, interleaved

    @property
    def _kept(self):
        return self._spaces.replaced

    def workspace(self, batch: int, max_q: int, max_len: int, device) -> torch.Tensor:
        return self._spaces.of(mq_kv_attention_workspace_bytes,
                               (batch, self.q_heads, self.kv_heads, self.head_dim, max_q, max_len), device)

    def __call__(self, x: torch.Tensor, cache: PagedKVCache, cu_rows, lens, page_table, max_q: int, max_len: int,
                 precise: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x [T, hidden]: the new tokens of the batch (mq_kv_batch of mq.h);
        no sequence has more than max_q of them, or more than max_len tokens, or
        more than the rotary table has positions.
        Rows that no sequence owns, and those of a sequence that has more, come
        out undefined (zero from the quantizing linears) and leave the others
        as they are, but for one thing: the QKV linear's tensor scale is taken
        over all rows of x, so padding rows should be zeros.  On another stream than
        the current one the call is what it is under torch.cuda.stream(stream):
        its intermediate tensors, workspaces and output belong to that stream."""
        if stream is not None:
            with torch.cuda.stream(_torch_stream(stream, x.device)):
                return self(x, cache, cu_rows, lens, page_table, max_q, max_len, precise, out)
        T = x.shape[0]
        if self.rope is not None:
            # the append leaves the rows of positions behind the table's: so does the attention
            max_len = min(max_len, self.rope.size(0))
        ws = self.workspace(page_table.shape[0], max_q, max_len, x.device)
        q = torch.empty(T, self.q_heads, self.head_dim, dtype=torch.bfloat16, device=x.device)
        # the quantizing O linear takes one tensor scale over all rows, those too
        # that the attention does not write
        attended = torch.empty_like(q) if precise else torch.zeros_like(q)
        qkv = (self.qkv_precise if precise else self.qkv)(x)
        mq_rope_kv_append(qkv, self.rope, cu_rows, lens, page_table, *cache.tensors(), q, ws,
                          interleaved=self.interleaved)
        mq_kv_attention(q, cu_rows, lens, page_table, *cache.tensors(), attended, ws, max_q, max_len,
                        self.head_dim ** -0.5)
        return (self.o_precise if precise else self.o)(attended.view(T, -1), out)

    def status(self, stream=None) -> int:
        """The workspaces' status words (mq_read_status), the first that is not
        MQ_OK: MQ_ERR_INVALID_ARG when a length, position or page number was
        outside the tables, MQ_ERR_TIMEOUT when a wait in a kernel of the
        attention or of a quantizing linear ran out.  Of calls on other streams than `stream` it sees
        what has ended, or what `stream` waits for."""
        for spaces in (self._spaces, self.qkv._spaces, self.o._spaces):
            for ws in [*spaces.by_place.values(), *spaces.replaced]:
                status = mq_read_status(ws, stream)
                if status != MQ_OK:
                    return status
        return MQ_OK


# -- the allocation-free variant (library-owned scratch) ---------------------

MQ_NOALLOC_SCRATCH_BYTES = 64 << 20


def mq_linear_w4a4_noalloc(x: torch.Tensor, w_codes, w_scales, alpha_w, N: int, y: torch.Tensor,
                           stream=None) -> None:
    """mq_linear_w4a4 without a workspace, for callers that cannot allocate:
    the library's static 64 MiB scratch is used (shared by every call on a
    device, so calls must not overlap on the GPU)."""
    f = lib().mq_linear_w4a4_noalloc
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    f.argtypes = [vp, i64, i64, vp, vp, vp, i64, vp, vp]
    f.restype = ctypes.c_int
    M, K = x.shape
    _check(f(_ptr(x), M, K, _ptr(w_codes), _ptr(w_scales), _ptr(alpha_w), N, _ptr(y), _stream(stream)),
           "mq_linear_w4a4_noalloc")
