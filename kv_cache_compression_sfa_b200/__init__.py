"""Python binding of the SFA C ABI (``include/sfa.h``).

Argument marshalling only: every step of the operator runs in the CUDA
library ``libsfa.so`` built from ``csrc/``.  PyTorch supplies device memory
and streams.  There is no CPU fallback: if the library is missing the calls
raise.

The functions keep the C names (``sfa_init``, ``sfa_prefill``,
``sfa_decode_step``, ``sfa_state_reset``, ...).  ``SfaOperator`` bundles a
handle with its state and workspace buffers for convenience.

Sources (web pages):
  [P1] "Signal Field Attention (SFA)：8KB代码实现4.16倍推理加速与248倍内存压缩"
  [P2] "Signal Field Attention (SFA)" (project README page)
  [P3] "Dalin Soma SFA基于信号场注意力机制的神经网络推理加速框架"
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsfa.so")

SFA_OK = 0
SFA_ERR_INVALID_ARG = -1
SFA_ERR_UNSUPPORTED = -2
SFA_ERR_ALIGNMENT = -3
SFA_ERR_STATE_MISMATCH = -4
SFA_ERR_CUDA = -5
SFA_ERR_DEVICE_TIMEOUT = -6
SFA_ERR_WORKSPACE = -7

SFA_F32 = 0
SFA_BF16 = 1

SFA_OUT_F32 = 0       # out fp32 = x + enhancement (default)
SFA_OUT_BF16 = 1      # out bf16 = x + enhancement
SFA_OUT_ADD_F32 = 2   # out fp32 += enhancement (out holds the caller's attention output)
SFA_OUT_ADD_BF16 = 3  # out bf16 += enhancement

SFA_ROPE_HALF = 0     # rotation pairs (x[j], x[j + dims/2])
SFA_ROPE_PAIRS = 1    # rotation pairs (x[2j], x[2j + 1])
SFA_TREE_MAX = 1024   # most nodes of a drafted tree

EXPORTED = (
    "sfa_config_default", "sfa_config_validate", "sfa_state_layout_for", "sfa_init",
    "sfa_destroy", "sfa_state_bytes", "sfa_prefill_workspace_bytes", "sfa_state_reset",
    "sfa_prefill", "sfa_decode_step", "sfa_check_device_status", "sfa_status_string",
    "sfa_abi_version", "sfa_debug_set_wait_limit", "sfa_debug_set_paths", "sfa_prefill_static_ws",
    "sfa_prefill_layers_workspace_bytes", "sfa_prefill_layers", "sfa_decode_step_ex",
    "sfa_set_decode_input_prefetch", "sfa_prefill_ragged", "sfa_set_output_mode",
    "sfa_tree_plan", "sfa_kv_append", "sfa_kv_attend_workspace_bytes", "sfa_kv_attend",
    "sfa_kv_accept",
)


class SfaError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {sfa_status_string(code)} ({code})" if what else
                         f"{sfa_status_string(code)} ({code})")


class sfa_config(ctypes.Structure):
    _fields_ = [
        ("n_layers", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("window_k", ctypes.c_int), ("gamma_far", ctypes.c_float),
        ("alpha_far", ctypes.c_float), ("ring_size", ctypes.c_int), ("ema_gamma", ctypes.c_float),
        ("n_slots", ctypes.c_int), ("temperature", ctypes.c_float), ("clip_eps", ctypes.c_float),
        ("alpha_base", ctypes.c_float), ("cross_decay", ctypes.c_float),
        ("in_dtype", ctypes.c_int), ("slots", ctypes.c_void_p),
    ]


class sfa_state_layout(ctypes.Structure):
    _fields_ = [(name, ctypes.c_size_t) for name in (
        "header_bytes", "stream_stride", "total_bytes", "off_pos", "off_win_k", "off_win_v",
        "off_far", "off_field", "off_ring_sum", "off_ring")]


class sfa_kv_cache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("n_pages", ctypes.c_longlong), ("page_size", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("page_table", ctypes.c_void_p)]


class sfa_rope(ctypes.Structure):
    _fields_ = [("style", ctypes.c_int), ("dims", ctypes.c_int), ("base", ctypes.c_double),
                ("inv_freq", ctypes.POINTER(ctypes.c_double))]


_lock = threading.Lock()
_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Loads libsfa.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                f"SFA CUDA library not found at {path}; build it with "
                "`python kv_cache_compression_sfa_b200/build.py` or __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        vp, i, ll, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
        P = ctypes.POINTER
        sigs = {
            "sfa_config_default": (None, [P(sfa_config)]),
            "sfa_config_validate": (i, [P(sfa_config)]),
            "sfa_state_layout_for": (i, [P(sfa_config), i, P(sfa_state_layout)]),
            "sfa_init": (i, [P(sfa_config), P(vp)]),
            "sfa_destroy": (i, [vp]),
            "sfa_state_bytes": (sz, [vp, i]),
            "sfa_prefill_workspace_bytes": (sz, [vp, i, ll]),
            "sfa_state_reset": (i, [vp, vp, i, vp]),
            "sfa_prefill": (i, [vp, vp, vp, vp, ll, i, vp, vp, vp, sz, vp]),
            "sfa_decode_step": (i, [vp, vp, vp, vp, i, vp, vp, vp]),
            "sfa_check_device_status": (i, [vp, vp]),
            "sfa_status_string": (ctypes.c_char_p, [i]),
            "sfa_abi_version": (i, []),
            "sfa_debug_set_wait_limit": (i, [vp, ctypes.c_uint, ll]),
            "sfa_debug_set_paths": (i, [vp, i, i]),
            "sfa_prefill_static_ws": (i, [vp, vp, vp, vp, ll, i, vp, vp, vp]),
            "sfa_prefill_layers_workspace_bytes": (sz, [vp, i, i, ll]),
            "sfa_prefill_layers": (i, [vp, i, i, vp, vp, vp, ll, i, vp, vp, vp, sz, vp]),
            "sfa_decode_step_ex": (i, [vp, i, i, vp, i, vp, vp, vp, i, vp, vp, vp]),
            "sfa_set_decode_input_prefetch": (i, [vp, i]),
            "sfa_prefill_ragged": (i, [vp, vp, vp, vp, ll, vp, i, vp, vp, vp, sz, vp]),
            "sfa_set_output_mode": (i, [vp, i]),
            "sfa_tree_plan": (i, [vp, vp, i, vp, vp, i, vp, vp, vp]),
            "sfa_kv_append": (i, [vp, P(sfa_kv_cache), i, i, vp, vp, vp, i, vp, vp, vp,
                                  P(sfa_rope), i, vp, vp, vp]),
            "sfa_kv_attend_workspace_bytes": (sz, [vp, i]),
            "sfa_kv_attend": (i, [vp, P(sfa_kv_cache), i, i, vp, i, vp, vp, vp, i, vp, vp, sz, vp]),
            "sfa_kv_accept": (i, [vp, P(sfa_kv_cache), i, i, vp, i, vp, vp, i, vp]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


# --------------------------------------------------------------- host-only


@dataclass
class SfaConfig:
    """Python view of ``sfa_config``; defaults are the pages' SFA_Config."""

    n_layers: int
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    window_k: int = 16
    gamma_far: float = 0.9
    alpha_far: float = 0.1
    ring_size: int = 16
    ema_gamma: float = 0.98
    n_slots: int = 64
    temperature: float = 0.07
    clip_eps: float = 0.5
    alpha_base: float = 0.1
    cross_decay: float = 0.8
    in_dtype: int = SFA_BF16

    @property
    def hidden(self) -> int:
        return self.n_q_heads * self.head_dim

    @property
    def torch_dtype(self) -> torch.dtype:
        return torch.float32 if self.in_dtype == SFA_F32 else torch.bfloat16

    def to_c(self, slots_ptr: int = 0) -> sfa_config:
        c = sfa_config()
        for f, _ in sfa_config._fields_:
            if f != "slots":
                setattr(c, f, getattr(self, f))
        c.slots = slots_ptr
        return c


def sfa_config_default() -> sfa_config:
    c = sfa_config()
    load_library().sfa_config_default(ctypes.byref(c))
    return c


def sfa_config_validate(cfg: sfa_config) -> int:
    return int(load_library().sfa_config_validate(ctypes.byref(cfg)))


def sfa_state_layout_for(cfg: sfa_config, batch: int) -> sfa_state_layout:
    lay = sfa_state_layout()
    rc = load_library().sfa_state_layout_for(ctypes.byref(cfg), batch, ctypes.byref(lay))
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_state_layout_for")
    return lay


def sfa_status_string(code: int) -> str:
    return load_library().sfa_status_string(int(code)).decode()


def sfa_abi_version() -> int:
    return int(load_library().sfa_abi_version())


# --------------------------------------------------------------- device


def _stream_ptr(stream) -> int:
    if stream is None:
        # the current stream's handle without a Stream object, where torch has it
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return int(raw(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _stream_object(stream, device) -> torch.cuda.Stream:
    """The Stream of a call's `stream`: a Stream, or a handle as an integer."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    ptr = _stream_ptr(stream)
    return torch.cuda.ExternalStream(ptr, device=device) if ptr else torch.cuda.default_stream(device)


def _hand_over(t: torch.Tensor, stream) -> None:
    """Makes a tensor that is new on its device's current stream fit for use on
    `stream`: the call comes after the memory's earlier use (and a fill), and the
    allocator gives it to others only after the call."""
    if stream is not None:
        stream = _stream_object(stream, t.device)
        stream.wait_stream(torch.cuda.current_stream(t.device))
        t.record_stream(stream)


def _empty_on(stream, nbytes: int, device) -> torch.Tensor:
    """Uninitialised bytes from the pool of the call's stream: free again for
    work behind the call, and in a torch.cuda.graph capture memory of the graph."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(_stream_object(stream, device)):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _capturing(stream, device) -> bool:
    """Whether a graph is being captured on the call's stream."""
    if device.type != "cuda":
        return False
    if stream is None and device.index in (None, torch.cuda.current_device()):
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(device), torch.cuda.stream(None if stream is None else _stream_object(stream, device)):
        return torch.cuda.is_current_stream_capturing()


def _is_cuda_tensor(t) -> bool:
    return isinstance(t, torch.Tensor) and t.is_cuda


def _dev(t: torch.Tensor, name: str, dtype=None, min_numel: int = 0) -> int:
    if not _is_cuda_tensor(t):
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.numel() < min_numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {min_numel}")
    return t.data_ptr()


class Handle:
    """An initialised sfa_handle and the configuration it was built from."""

    def __init__(self, ptr: int, cfg: SfaConfig):
        self.ptr = ptr
        self.cfg = cfg
        self.out_mode = SFA_OUT_F32

    @property
    def out_dtype(self) -> torch.dtype:
        """dtype of `out` in the handle's output mode."""
        return torch.bfloat16 if self.out_mode in (SFA_OUT_BF16, SFA_OUT_ADD_BF16) else torch.float32

    def __del__(self):
        if getattr(self, "ptr", None):
            try:
                load_library().sfa_destroy(self.ptr)
            except Exception:
                pass
            self.ptr = None


def sfa_init(cfg: SfaConfig, slots: torch.Tensor) -> Handle:
    L, P, H = cfg.n_layers, cfg.n_slots, cfg.hidden
    _dev(slots, "slots", torch.float32, L * P * H)
    c = cfg.to_c(slots.data_ptr())
    h = ctypes.c_void_p()
    rc = load_library().sfa_init(ctypes.byref(c), ctypes.byref(h))
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_init")
    return Handle(h.value, cfg)


def sfa_destroy(h: Handle) -> None:
    if h.ptr:
        rc = load_library().sfa_destroy(h.ptr)
        h.ptr = None
        if rc != SFA_OK:
            raise SfaError(rc, "sfa_destroy")


def sfa_state_bytes(h: Handle, batch: int) -> int:
    return int(load_library().sfa_state_bytes(h.ptr, batch))


def sfa_prefill_workspace_bytes(h: Handle, batch: int, n: int) -> int:
    return int(load_library().sfa_prefill_workspace_bytes(h.ptr, batch, n))


def sfa_state_reset(h: Handle, state: torch.Tensor, batch: int, stream=None) -> None:
    _dev(state, "state", torch.uint8, sfa_state_bytes(h, batch))
    rc = load_library().sfa_state_reset(h.ptr, state.data_ptr(), batch, _stream_ptr(stream))
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_state_reset")


def _qkv_checks(h: Handle, q, k, v, tokens: int, batch: int, layers: Optional[int] = None):
    c = h.cfg
    rows = (c.n_layers if layers is None else layers) * batch * tokens
    return (_dev(q, "q", c.torch_dtype, rows * c.n_q_heads * c.head_dim),
            _dev(k, "k", c.torch_dtype, rows * c.n_kv_heads * c.head_dim),
            _dev(v, "v", c.torch_dtype, rows * c.n_kv_heads * c.head_dim))


def sfa_prefill(h: Handle, q, k, v, n: int, batch: int, state: torch.Tensor, out: torch.Tensor,
                workspace: Optional[torch.Tensor], stream=None) -> None:
    if n == 0:
        return
    qp, kp, vp = _qkv_checks(h, q, k, v, n, batch)
    sp = _dev(state, "state", torch.uint8, sfa_state_bytes(h, batch))
    op = _dev(out, "out", h.out_dtype, h.cfg.n_layers * batch * n * h.cfg.hidden)
    need = sfa_prefill_workspace_bytes(h, batch, n)
    if workspace is None or workspace.numel() < need:
        raise SfaError(SFA_ERR_WORKSPACE, "sfa_prefill")
    wp = _dev(workspace, "workspace", torch.uint8)
    rc = load_library().sfa_prefill(h.ptr, qp, kp, vp, n, batch, sp, op, wp,
                                    workspace.numel(), _stream_ptr(stream))
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_prefill")


def sfa_prefill_ragged(h: Handle, q, k, v, n_max: int, lens: torch.Tensor, batch: int,
                       state: torch.Tensor, out: torch.Tensor, workspace: Optional[torch.Tensor],
                       stream=None) -> None:
    """sfa_prefill where sequence b folds in lens[b] (device int32) tokens of
    its rows 0 .. lens[b]-1 of the n_max-row inputs; out rows past lens[b]
    are left as they were."""
    if n_max == 0:
        return
    qp, kp, vp = _qkv_checks(h, q, k, v, n_max, batch)
    sp = _dev(state, "state", torch.uint8, sfa_state_bytes(h, batch))
    op = _dev(out, "out", h.out_dtype, h.cfg.n_layers * batch * n_max * h.cfg.hidden)
    lp = _dev(lens, "lens", torch.int32, batch)
    need = sfa_prefill_workspace_bytes(h, batch, n_max)
    if workspace is None or workspace.numel() < need:
        raise SfaError(SFA_ERR_WORKSPACE, "sfa_prefill_ragged")
    wp = _dev(workspace, "workspace", torch.uint8)
    rc = load_library().sfa_prefill_ragged(h.ptr, qp, kp, vp, n_max, lp, batch, sp, op, wp,
                                           workspace.numel(), _stream_ptr(stream))
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_prefill_ragged")


def sfa_prefill_layers_workspace_bytes(h: Handle, layer_count: int, batch: int, n: int) -> int:
    return int(load_library().sfa_prefill_layers_workspace_bytes(h.ptr, layer_count, batch, n))


def sfa_prefill_layers(h: Handle, layer_begin: int, layer_count: int, q, k, v, n: int,
                       batch: int, state: torch.Tensor, out: torch.Tensor,
                       workspace: Optional[torch.Tensor], stream=None) -> None:
    """sfa_prefill for layers layer_begin .. layer_begin+layer_count-1 only;
    q/k/v/out hold those layers alone."""
    if n == 0:
        return
    qp, kp, vp = _qkv_checks(h, q, k, v, n, batch, layer_count)
    sp = _dev(state, "state", torch.uint8, sfa_state_bytes(h, batch))
    op = _dev(out, "out", h.out_dtype, layer_count * batch * n * h.cfg.hidden)
    need = sfa_prefill_layers_workspace_bytes(h, layer_count, batch, n)
    if workspace is None or workspace.numel() < need:
        raise SfaError(SFA_ERR_WORKSPACE, "sfa_prefill_layers")
    wp = _dev(workspace, "workspace", torch.uint8)
    rc = load_library().sfa_prefill_layers(h.ptr, layer_begin, layer_count, qp, kp, vp, n, batch,
                                           sp, op, wp, workspace.numel(), _stream_ptr(stream))
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_prefill_layers")


def sfa_decode_step_ex(h: Handle, layer_begin: int, layer_count: int,
                       seq_ids: Optional[torch.Tensor], q, k, v, batch: int,
                       state: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """sfa_decode_step for a layer range and (optionally) a device int32
    tensor of distinct sequence indices; q/k/v/out rows follow seq_ids."""
    n_seq = batch if seq_ids is None else int(seq_ids.numel())
    qp, kp, vp = _qkv_checks(h, q, k, v, 1, n_seq, layer_count)
    sp = _dev(state, "state", torch.uint8, sfa_state_bytes(h, batch))
    op = _dev(out, "out", h.out_dtype, layer_count * n_seq * h.cfg.hidden)
    ip = None if seq_ids is None else _dev(seq_ids, "seq_ids", torch.int32, n_seq)
    rc = load_library().sfa_decode_step_ex(h.ptr, layer_begin, layer_count, ip, n_seq, qp, kp, vp,
                                           batch, sp, op, _stream_ptr(stream))
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_decode_step_ex")


SFA_STATIC_WORKSPACE_BYTES = 16 << 20


def sfa_prefill_static_ws(h: Handle, q, k, v, n: int, batch: int, state: torch.Tensor,
                          out: torch.Tensor, stream=None) -> None:
    """sfa_prefill on the library's fixed device scratch (no workspace
    argument, nothing allocated); see include/sfa.h for the limits."""
    if n == 0:
        return
    qp, kp, vp = _qkv_checks(h, q, k, v, n, batch)
    sp = _dev(state, "state", torch.uint8, sfa_state_bytes(h, batch))
    op = _dev(out, "out", h.out_dtype, h.cfg.n_layers * batch * n * h.cfg.hidden)
    rc = load_library().sfa_prefill_static_ws(h.ptr, qp, kp, vp, n, batch, sp, op,
                                              _stream_ptr(stream))
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_prefill_static_ws")


def sfa_decode_step(h: Handle, q, k, v, batch: int, state: torch.Tensor, out: torch.Tensor,
                    stream=None) -> None:
    """One token per sequence, all layers.  q, k and v are read once the
    previous kernel on the stream has finished, unless the handle's input
    prefetch is on (sfa_set_decode_input_prefetch)."""
    qp, kp, vp = _qkv_checks(h, q, k, v, 1, batch)
    sp = _dev(state, "state", torch.uint8, sfa_state_bytes(h, batch))
    op = _dev(out, "out", h.out_dtype, h.cfg.n_layers * batch * h.cfg.hidden)
    rc = load_library().sfa_decode_step(h.ptr, qp, kp, vp, batch, sp, op, _stream_ptr(stream))
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_decode_step")


def sfa_set_decode_input_prefetch(h: Handle, enable: bool) -> None:
    """Declare (True) that every later decode call's q, k and v are complete
    when the call is enqueued and that nothing still running on the stream
    writes them; the decode kernel then fetches them before the previous
    kernel on the stream has finished.  False (the default) fetches them
    after it.  Results are identical either way."""
    rc = load_library().sfa_set_decode_input_prefetch(h.ptr, 1 if enable else 0)
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_set_decode_input_prefetch")


def sfa_set_output_mode(h: Handle, mode: int) -> None:
    """What later compute calls write into out: SFA_OUT_F32 / SFA_OUT_BF16
    (x + enhancement) or SFA_OUT_ADD_F32 / SFA_OUT_ADD_BF16 (out, holding
    the caller's attention output, plus the enhancement in place)."""
    rc = load_library().sfa_set_output_mode(h.ptr, int(mode))
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_set_output_mode")
    h.out_mode = int(mode)


def sfa_check_device_status(h: Handle, stream=None) -> int:
    return int(load_library().sfa_check_device_status(h.ptr, _stream_ptr(stream)))


def sfa_debug_set_wait_limit(h: Handle, spin_limit: int = 0, withhold_tile: int = -1) -> None:
    """Test hook of the bounded waits.  Prefill: the pool CTA of tile
    `withhold_tile` (tile * streams + stream) waits on a barrier that nothing
    completes, giving up after `spin_limit` polls (0: default); -1 disables.
    Paged attention in bf16: a role of every CTA begins with such a wait (0, 4
    softmax, 8 keys, 9 products, 10 values), and its others give up as early."""
    rc = load_library().sfa_debug_set_wait_limit(h.ptr, spin_limit, withhold_tile)
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_debug_set_wait_limit")


def sfa_debug_set_paths(h: Handle, decode_tile: int = -1, prefill_near=3) -> None:
    """Test hook that pins the kernel variants: decode_tile -1 (by batch
    size), 0 (per-sequence kernel) or 1 (batch-tiled kernel); prefill near
    field, where the tensor cores apply, 3 by call size (the default; also
    True), 2 fused with the pool scores, 1 tensor cores with a separate pool
    kernel, 0 CUDA cores (also False)."""
    mode = {True: 3, False: 0}[prefill_near] if isinstance(prefill_near, bool) else int(prefill_near)
    rc = load_library().sfa_debug_set_paths(h.ptr, int(decode_tile), mode)
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_debug_set_paths")


class SfaOperator:
    """A handle plus the device buffers one batch of sequences needs.

    ``prefill(q, k, v)`` takes [L, B, n, heads, d] tensors and returns
    out [L, B, n, hidden] fp32; ``decode(q, k, v)`` takes [L, B, heads, d]
    and returns [L, B, hidden].
    """

    def __init__(self, cfg: SfaConfig, slots: torch.Tensor, batch: int,
                 max_prefill: int = 0, device=None):
        self.cfg = cfg
        self.batch = batch
        self.device = torch.device(device or slots.device)
        self.handle = sfa_init(cfg, slots)
        self._state_bytes = sfa_state_bytes(self.handle, batch)
        self.state = torch.empty(self._state_bytes, dtype=torch.uint8, device=self.device)
        # Per-call constants of decode(), which a serving loop calls once per
        # token: the C entry point, the element counts and the input dtype.
        rows = cfg.n_layers * batch
        self._dec_numel = (rows * cfg.n_q_heads * cfg.head_dim, rows * cfg.n_kv_heads * cfg.head_dim,
                           rows * cfg.hidden)
        self._in_dtype = cfg.torch_dtype
        self._decode_fn = load_library().sfa_decode_step
        self.workspace, self._workspace_on, self._in_graph, self._kept = None, None, False, []
        if max_prefill > 0:
            self._ensure_workspace(max_prefill)
        self.reset()

    def _grow_workspace(self, need: int, stream=None):
        """A workspace of at least `need` bytes; one serves all calls, which the
        operator's state puts in order.  It is marked as used on every stream but
        the one whose pool it came from, so that a buffer that a larger one replaces
        goes back behind all calls; one that a graph has captured is kept as long as
        the operator."""
        on = _stream_ptr(stream)
        if self.workspace is None or self.workspace.numel() < need:
            if self._in_graph:
                self._kept.append(self.workspace)
            self.workspace, self._in_graph = _empty_on(stream, need, self.device), False
            self._workspace_on = on
        elif on != self._workspace_on:
            self.workspace.record_stream(torch.cuda.current_stream(self.device) if stream is None
                                         else _stream_object(stream, self.device))
        self._in_graph = self._in_graph or _capturing(stream, self.device)

    def _ensure_workspace(self, n: int, stream=None):
        self._grow_workspace(sfa_prefill_workspace_bytes(self.handle, self.batch, n), stream)

    def reset(self, stream=None):
        sfa_state_reset(self.handle, self.state, self.batch, stream)

    def set_output_mode(self, mode: int) -> None:
        sfa_set_output_mode(self.handle, mode)

    def _new_out(self, shape, stream=None, fill: Optional[float] = None):
        """A result buffer allocated (and filled) on the current stream and
        handed over to the call's."""
        if self.handle.out_mode in (SFA_OUT_ADD_F32, SFA_OUT_ADD_BF16):
            raise ValueError("the add output modes need out: it holds the attention output")
        out = torch.empty(shape, dtype=self.handle.out_dtype, device=self.device)
        if fill is not None:
            out.fill_(fill)
        _hand_over(out, stream)
        return out

    def prefill(self, q, k, v, out: Optional[torch.Tensor] = None, stream=None):
        n = q.shape[2]
        c = self.cfg
        if out is None:
            out = self._new_out((c.n_layers, self.batch, n, c.hidden), stream)
        if n > 0:
            self._ensure_workspace(n, stream)
            sfa_prefill(self.handle, q, k, v, n, self.batch, self.state, out, self.workspace,
                        stream)
        return out

    def prefill_ragged(self, q, k, v, lens: torch.Tensor, out: Optional[torch.Tensor] = None,
                       stream=None):
        """Prefill where sequence b takes lens[b] (device int32) of the n_max
        rows of q, k, v ([L, B, n_max, heads, d]); out rows past lens[b] keep
        their contents (a new out starts as NaN there)."""
        n = q.shape[2]
        c = self.cfg
        if out is None:
            out = self._new_out((c.n_layers, self.batch, n, c.hidden), stream, fill=float("nan"))
        if n > 0:
            self._ensure_workspace(n, stream)
            sfa_prefill_ragged(self.handle, q, k, v, n, lens, self.batch, self.state, out,
                               self.workspace, stream)
        return out

    def decode(self, q, k, v, out: Optional[torch.Tensor] = None, stream=None):
        """One token per sequence, all layers: the checks and the call of
        sfa_decode_step, with the per-operator constants looked up once."""
        if out is None:
            c = self.cfg
            out = self._new_out((c.n_layers, self.batch, c.hidden), stream)
        nq, nkv, nout = self._dec_numel
        dt = self._in_dtype
        rc = self._decode_fn(self.handle.ptr, _dev(q, "q", dt, nq), _dev(k, "k", dt, nkv),
                             _dev(v, "v", dt, nkv),
                             self.batch, _dev(self.state, "state", torch.uint8, self._state_bytes),
                             _dev(out, "out", self.handle.out_dtype, nout), _stream_ptr(stream))
        if rc != SFA_OK:
            raise SfaError(rc, "sfa_decode_step")
        return out

    def prefill_layers(self, layer_begin: int, q, k, v, out: Optional[torch.Tensor] = None,
                       stream=None):
        """Prefill of layers layer_begin .. layer_begin + q.shape[0] - 1."""
        lc, n = q.shape[0], q.shape[2]
        if out is None:
            out = self._new_out((lc, self.batch, n, self.cfg.hidden), stream)
        if n > 0:
            self._grow_workspace(sfa_prefill_layers_workspace_bytes(self.handle, lc, self.batch, n),
                                 stream)
            sfa_prefill_layers(self.handle, layer_begin, lc, q, k, v, n, self.batch, self.state,
                               out, self.workspace, stream)
        return out

    def decode_ex(self, layer_begin: int, q, k, v, seq_ids: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, stream=None):
        """Decode of layers layer_begin .. layer_begin + q.shape[0] - 1 for the
        sequences in seq_ids (int32, on the device; None = all)."""
        lc, ns = q.shape[0], q.shape[1]
        if out is None:
            out = self._new_out((lc, ns, self.cfg.hidden), stream)
        sfa_decode_step_ex(self.handle, layer_begin, lc, seq_ids, q, k, v, self.batch,
                           self.state, out, stream)
        return out

    def check(self, stream=None) -> int:
        return sfa_check_device_status(self.handle, stream)

    def layout(self) -> sfa_state_layout:
        return sfa_state_layout_for(_layout_cfg(self.cfg), self.batch)


# ------------------------------------------------------ paged key/value cache


def _load_fast():
    """The per-step calls without ctypes, or None where they are not built, or
    for another torch (whose tensors they would misread): the Python checks
    below serve then."""
    try:
        from . import _fast
        from .build import fast_stamp
        return _fast if _fast.built_for == fast_stamp() else None
    except (ImportError, AttributeError):
        return None


_fast = _load_fast()


def _address(fn) -> int:
    return ctypes.cast(fn, ctypes.c_void_p).value


class SfaRope:
    """Position rotation of sfa_kv_append (``sfa_rope``): the first ``dims``
    elements of a head (0: all), in ``style`` SFA_ROPE_HALF or SFA_ROPE_PAIRS,
    pair j turning by base ** (-2j/dims) or inv_freq[j] per position."""

    def __init__(self, base: float = 10000.0, style: int = SFA_ROPE_HALF, dims: int = 0,
                 inv_freq=None):
        self.base, self.style, self.dims = float(base), int(style), int(dims)
        self.inv_freq = None if inv_freq is None else [float(f) for f in inv_freq]
        if self.inv_freq is not None and self.dims and len(self.inv_freq) < self.dims // 2:
            raise ValueError(f"inv_freq has {len(self.inv_freq)} values, needs {self.dims // 2}")
        self._arr = (None if self.inv_freq is None
                     else (ctypes.c_double * len(self.inv_freq))(*self.inv_freq))
        self.c = sfa_rope(self.style, self.dims, self.base, self._arr)
        self.ref = ctypes.byref(self.c)
        self.address = ctypes.addressof(self.c)

    def check(self, head_dim: int) -> None:
        if self.inv_freq is None:
            return
        need = (self.dims or head_dim) // 2
        if len(self.inv_freq) < need:
            raise ValueError(f"inv_freq has {len(self.inv_freq)} values, needs {need}")


def _need(t, name: str, dtype, shape, index: int) -> int:
    """Pointer of a contiguous CUDA tensor of exactly this dtype and shape on
    device `index`.  One test in the usual case: these calls run once per layer
    and step, where a microsecond of checks is a microsecond of the step."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == index and t.is_contiguous() and _is_cuda_tensor(t)):
        return t.data_ptr()
    _dev(t, name, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, needs {tuple(shape)}")
    raise ValueError(f"{name} is on device {t.get_device()}, not on {index}")


def _call_on(index: int, stream, fn, *args) -> int:
    """fn(*args, stream) with device `index` current; stream None is that
    device's current stream."""
    if index < 0 or index == torch.cuda.current_device():
        return fn(*args, _stream_ptr(stream))
    with torch.cuda.device(index):
        return fn(*args, _stream_ptr(stream))


def sfa_tree_plan(h: Handle, parents: torch.Tensor, ctx_lens: torch.Tensor,
                  lens: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                  mask: Optional[torch.Tensor] = None, stream=None):
    """Positions [B, n] and ancestor masks [B, n, (n + 31) // 32] (int32) of the
    drafted trees parents [B, n] (int32, -1: no parent, else below the node's
    own index).  Returns (positions, mask); given tensors are written in
    place, and rows past lens keep what they held (new ones start as zero)."""
    if not isinstance(parents, torch.Tensor) or parents.dim() != 2:
        raise ValueError("parents must be a [batch, n] tensor")
    B, n = parents.shape
    dev, i32 = parents.get_device(), torch.int32
    words = (n + 31) // 32
    if positions is None:
        positions = _zeros_for((B, n), i32, parents.device, stream)
    if mask is None:
        mask = _zeros_for((B, n, words), i32, parents.device, stream)
    if _fast is not None and parents.is_cuda:
        rc = _fast.plan(_plan_address(), h.ptr, parents, ctx_lens, lens, positions, mask,
                        None if stream is None else _stream_ptr(stream))
        if rc == SFA_OK:
            return positions, mask
        if rc is not None:
            raise SfaError(rc, "sfa_tree_plan")
    rc = _call_on(dev, stream, load_library().sfa_tree_plan, h.ptr,
                  _need(parents, "parents", i32, (B, n), dev), n,
                  None if lens is None else _need(lens, "lens", i32, (B,), dev),
                  _need(ctx_lens, "ctx_lens", i32, (B,), dev), B,
                  _need(positions, "positions", i32, (B, n), dev),
                  _need(mask, "mask", i32, (B, n, words), dev))
    if rc != SFA_OK:
        raise SfaError(rc, "sfa_tree_plan")
    return positions, mask


_plan_addr = None


def _plan_address() -> int:
    global _plan_addr
    if _plan_addr is None:
        _plan_addr = _address(load_library().sfa_tree_plan)
    return _plan_addr


def _zeros_for(shape, dtype, device, stream):
    t = torch.zeros(shape, dtype=dtype, device=device)
    _hand_over(t, stream)
    return t


def sfa_kv_attend_workspace_bytes(h: Handle, n_max: int) -> int:
    return int(load_library().sfa_kv_attend_workspace_bytes(h.ptr, n_max))


class SfaPagedCache:
    """A paged key/value cache of the handle's layers: k_pages and v_pages
    [L, n_pages, n_kv, page_size, d] in the handle's input dtype and page_table
    [batch, max_pages] int32.  The tensors stay the caller's: a table changed in
    place is seen by the next call.

    ``append``, ``attend`` and ``accept`` are sfa_kv_append, sfa_kv_attend and
    sfa_kv_accept for layers layer_begin .. layer_begin + q.shape[0] - 1; q is
    [layers, B, n, n_q, d], ctx_lens and lens [B] int32 on the device.  attend
    takes its workspace from torch's allocator for the length of the call, in a
    torch.cuda.graph capture from the graph's pool; a ``workspace`` that is given
    serves one call at a time (host threads and graphs that share one take turns)."""

    def __init__(self, handle: Handle, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 page_table: torch.Tensor):
        c = handle.cfg
        self.handle = handle
        if k_pages.dim() != 5 or page_table.dim() != 2:
            raise ValueError("k_pages must be [L, n_pages, n_kv, page_size, d] and page_table [batch, max_pages]")
        self.device, dev = k_pages.device, k_pages.get_device()
        self.n_pages, self.page_size = k_pages.shape[1], k_pages.shape[3]
        self.batch, self.max_pages = page_table.shape
        shape = (c.n_layers, self.n_pages, c.n_kv_heads, self.page_size, c.head_dim)
        kp = _need(k_pages, "k_pages", c.torch_dtype, shape, dev)
        vp = _need(v_pages, "v_pages", c.torch_dtype, shape, dev)
        tp = _need(page_table, "page_table", torch.int32, page_table.shape, dev)
        self.k_pages, self.v_pages, self.page_table = k_pages, v_pages, page_table
        self.c = sfa_kv_cache(kp, vp, self.n_pages, self.page_size, self.max_pages, tp)
        # what the calls, made once per layer and step, look up
        self._ref = ctypes.byref(self.c)
        self._index, self._dtype, self._lens_shape = dev, c.torch_dtype, (self.batch,)
        self._q_tail, self._kv_tail = (c.n_q_heads, c.head_dim), (c.n_kv_heads, c.head_dim)
        lib = load_library()
        self._append_fn, self._attend_fn, self._accept_fn = lib.sfa_kv_append, lib.sfa_kv_attend, lib.sfa_kv_accept
        self._spec = None
        if _fast is not None and dev >= 0:
            self._spec = _fast.spec(_address(lib.sfa_kv_append), _address(lib.sfa_kv_attend), _address(lib.sfa_kv_accept),
                                    _address(lib.sfa_kv_attend_workspace_bytes), ctypes.addressof(self.c), dev, c.in_dtype == SFA_BF16, self.batch, *self._q_tail[:1],
                                    *self._kv_tail)

    def _len_ptr(self, t, name: str) -> Optional[int]:
        return None if t is None else _need(t, name, torch.int32, self._lens_shape, self._index)

    def append(self, layer_begin: int, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
               ctx_lens: torch.Tensor, lens: Optional[torch.Tensor] = None,
               positions: Optional[torch.Tensor] = None, rope: Optional[SfaRope] = None,
               q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
               stream=None):
        """Rotated keys and values of the new tokens into their pages; returns
        (q_out, k_out), the rotated queries (a new tensor unless given; None
        without q) and keys (None unless given)."""
        if q is not None and q_out is None:
            _need(q, "q", self._dtype, q.shape, self._index)
            q_out = _zeros_for(q.shape, self._dtype, self.device, stream)
        if self._spec is not None:
            if rope is not None:
                rope.check(self._kv_tail[1])
            rc = _fast.append(self._spec, self.handle.ptr, layer_begin, q, k, v, ctx_lens, lens, positions,
                              None if rope is None else rope.address, q_out, k_out,
                              None if stream is None else _stream_ptr(stream))
            if rc == SFA_OK:
                return q_out, k_out
            if rc is not None:
                raise SfaError(rc, "sfa_kv_append")
        if k.dim() != 5:
            raise ValueError("k must be [layers, batch, n, n_kv, d]")
        dev, dt, B = self._index, self._dtype, self.batch
        Lc, n = k.shape[0], k.shape[2]
        rows = (Lc, B, n)
        kv, qs = rows + self._kv_tail, rows + self._q_tail
        qp = qo = ko = None
        if q is not None:
            qp = _need(q, "q", dt, qs, dev)
            qo = _need(q_out, "q_out", dt, qs, dev)
        elif q_out is not None:
            raise ValueError("q_out needs q")
        if k_out is not None:
            ko = _need(k_out, "k_out", dt, kv, dev)
        rp = None
        if rope is not None:
            rope.check(self._kv_tail[1])
            rp = rope.ref
        rc = _call_on(dev, stream, self._append_fn, self.handle.ptr, self._ref, layer_begin, Lc, qp,
                      _need(k, "k", dt, kv, dev), _need(v, "v", dt, kv, dev), n,
                      self._len_ptr(lens, "lens"), _need(ctx_lens, "ctx_lens", torch.int32, (B,), dev),
                      None if positions is None else _need(positions, "positions", torch.int32, (B, n), dev),
                      rp, B, qo, ko)
        if rc != SFA_OK:
            raise SfaError(rc, "sfa_kv_append")
        return q_out, k_out

    def attend(self, layer_begin: int, q: torch.Tensor, ctx_lens: torch.Tensor,
               lens: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
        """Attention of the new tokens (appended before) over the cache:
        out [layers, B, n, hidden] in the input dtype.  mask [B, n, words] as of
        sfa_tree_plan, or None: every new token sees those before it.  Rows past
        lens keep what out held (a new out is zero there)."""
        if out is None:
            if q.dim() != 5:
                raise ValueError("q must be [layers, batch, n, n_q, d]")
            _need(q, "q", self._dtype, q.shape, self._index)
            out = _zeros_for(q.shape[:3] + (self._q_tail[0] * self._q_tail[1],), self._dtype, self.device, stream)
        if self._spec is not None and q.dim() == 5 and q.shape[2] > 0:
            rc = _fast.attend(self._spec, self.handle.ptr, layer_begin, q, ctx_lens, lens, mask, out, workspace,
                              None if stream is None else _stream_ptr(stream))
            if rc == SFA_OK:
                return out
            if rc is not None:
                raise SfaError(rc, "sfa_kv_attend")
        if q.dim() != 5:
            raise ValueError("q must be [layers, batch, n, n_q, d]")
        dev, dt, B = self._index, self._dtype, self.batch
        Lc, n = q.shape[0], q.shape[2]
        rows = (Lc, B, n)
        qp = _need(q, "q", dt, rows + self._q_tail, dev)
        cp = _need(ctx_lens, "ctx_lens", torch.int32, self._lens_shape, dev)
        mp = None if mask is None else _need(mask, "mask", torch.int32, (B, n, (n + 31) // 32), dev)
        hidden = self._q_tail[0] * self._q_tail[1]
        op = _need(out, "out", dt, rows + (hidden,), dev)
        if n == 0:
            return out
        if workspace is None:
            workspace = _empty_on(stream, sfa_kv_attend_workspace_bytes(self.handle, n), self.device)
        size = workspace.numel()
        rc = _call_on(dev, stream, self._attend_fn, self.handle.ptr, self._ref, layer_begin, Lc, qp, n,
                      self._len_ptr(lens, "lens"), cp, mp, B, op,
                      _need(workspace, "workspace", torch.uint8, (size,), dev), size)
        if rc != SFA_OK:
            raise SfaError(rc, "sfa_kv_attend")
        return out

    def accept(self, layer_begin: int, layer_count: int, path: torch.Tensor, n_accept: torch.Tensor,
               ctx_lens: torch.Tensor, stream=None) -> None:
        """The keys and values of nodes path[b, :n_accept[b]] ([B, n] and [B]
        int32, rising node indices) moved up behind the context; the caller
        then adds n_accept to ctx_lens."""
        if self._spec is not None:
            rc = _fast.accept(self._spec, self.handle.ptr, layer_begin, layer_count, path, n_accept, ctx_lens,
                              None if stream is None else _stream_ptr(stream))
            if rc == SFA_OK:
                return
            if rc is not None:
                raise SfaError(rc, "sfa_kv_accept")
        if path.dim() != 2:
            raise ValueError("path must be [batch, n]")
        dev, B, n = self._index, self.batch, path.shape[1]
        rc = _call_on(dev, stream, self._accept_fn, self.handle.ptr, self._ref, layer_begin, layer_count,
                      _need(path, "path", torch.int32, (B, n), dev), n,
                      _need(n_accept, "n_accept", torch.int32, (B,), dev),
                      _need(ctx_lens, "ctx_lens", torch.int32, (B,), dev), B)
        if rc != SFA_OK:
            raise SfaError(rc, "sfa_kv_accept")


def _layout_cfg(cfg: SfaConfig) -> sfa_config:
    # Layout arithmetic needs a non-null, aligned slots pointer only for the
    # validity check; 16 is a stand-in address that is never dereferenced.
    return cfg.to_c(16)


def read_state(op: SfaOperator) -> dict:
    """Copies the state of every stream to host tensors (for tests/inspection):
    pos [L,B], win_k/win_v [L,B,k,n_kv,d], far [L,B,n_kv,d], field, ring_sum
    [L,B,H], ring [L,B,16,H]."""
    c = op.cfg
    lay = sfa_state_layout_for(_layout_cfg(c), op.batch)
    raw = op.state.cpu()
    L, B = c.n_layers, op.batch
    body = raw[lay.header_bytes: lay.header_bytes + L * B * lay.stream_stride]
    body = body.view(L, B, lay.stream_stride)
    esz = 4 if c.in_dtype == SFA_F32 else 2
    wdt = torch.float32 if c.in_dtype == SFA_F32 else torch.bfloat16
    K, nkv, d, H = c.window_k, c.n_kv_heads, c.head_dim, c.hidden

    def grab(off, nbytes, dtype, shape):
        return body[:, :, off: off + nbytes].contiguous().view(dtype).view(L, B, *shape)

    return {
        "pos": grab(lay.off_pos, 8, torch.int64, ()),
        "win_k": grab(lay.off_win_k, K * nkv * d * esz, wdt, (K, nkv, d)),
        "win_v": grab(lay.off_win_v, K * nkv * d * esz, wdt, (K, nkv, d)),
        "far": grab(lay.off_far, nkv * d * 4, torch.float32, (nkv, d)),
        "field": grab(lay.off_field, H * 4, torch.float32, (H,)),
        "ring_sum": grab(lay.off_ring_sum, H * 4, torch.float32, (H,)),
        "ring": grab(lay.off_ring, 16 * H * 4, torch.float32, (16, H)),
    }


# The C names, on a cache: sfa_kv_append(cache, layer_begin, q, k, v, ...) and so on.
sfa_kv_append = SfaPagedCache.append
sfa_kv_attend = SfaPagedCache.attend
sfa_kv_accept = SfaPagedCache.accept
