"""GB300-native 4-bit mixture-of-experts FFN layer.

Python binding of libmoe.so: every entry point of include/moe.h under the same
name, doing argument marshalling only. All of the layer's work runs in the
library's CUDA kernels; torch is used for device memory and streams. There is
no fallback: if the library is missing, calls raise.

The layer follows "Optimizing on-device inference for Apple Silicon"
(Perplexity, 2026): 4-bit groupwise-affine experts (64 weights per bf16
scale/bias group), top-8-of-256 routing plus one shared expert, SwiGLU.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmoe.so")

MOE_OK = 0
MOE_ERR_ARG = 1
MOE_ERR_SHAPE = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE_TIMEOUT = 5
MOE_ERR_DEVICE_CHECK = 6

MOE_OPT_GEMV_MAX_ROWS = 1
MOE_OPT_FORCE_PATH = 2
MOE_OPT_KERNEL_TIMING = 3
MOE_OPT_GEMM_IMPL = 4
MOE_OPT_TEST_WAIT_CYCLES = 5
MOE_OPT_BLOCK_M = 6
MOE_OPT_DECODE_FUSED = 7
MOE_OPT_CHUNK_TOKENS = 8
MOE_OPT_HOST_SYNC_ROUTING = 9

PATH_AUTO, PATH_GEMV, PATH_GEMM = 0, 1, 2
GEMM_TENSOR_CORE, GEMM_CUDA_CORE, GEMM_TENSOR_CORE_SMEM = 0, 1, 2


class moe_qmatrix(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p)]


class moe_weights(ctypes.Structure):
    _fields_ = [("D", ctypes.c_int), ("E", ctypes.c_int), ("k", ctypes.c_int), ("I", ctypes.c_int),
                ("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("gate", moe_qmatrix), ("up", moe_qmatrix), ("down", moe_qmatrix),
                ("s_gate", moe_qmatrix), ("s_up", moe_qmatrix), ("s_down", moe_qmatrix)]


class moe_route_view(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("block_m", ctypes.c_int), ("max_blocks", ctypes.c_int),
                ("logits", ctypes.c_void_p), ("topk_idx", ctypes.c_void_p), ("topk_w", ctypes.c_void_p),
                ("count", ctypes.c_void_p), ("off", ctypes.c_void_p), ("perm", ctypes.c_void_p),
                ("inv", ctypes.c_void_p), ("blocks", ctypes.c_void_p), ("n_blocks", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("y_acc", ctypes.c_void_p)]


class moe_kv_cache(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("k_biases", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("v_biases", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class moe_kv_batch(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int), ("n_tokens", ctypes.c_int), ("max_new", ctypes.c_int),
                ("max_kv", ctypes.c_int), ("q_off", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int)]


class moe_attention(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int), ("window", ctypes.c_int), ("sinks", ctypes.c_int),
                ("scale", ctypes.c_float)]


# name -> (restype, argtypes), mirroring include/moe.h
_VP, _CI, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_W = ctypes.POINTER(moe_weights)
_KC, _KB, _AT = ctypes.POINTER(moe_kv_cache), ctypes.POINTER(moe_kv_batch), ctypes.POINTER(moe_attention)
_LL = ctypes.c_longlong
SIGNATURES = {
    "moe_workspace_size": (_SZ, [_W, _CI]),
    "moe_layer_forward": (_CI, [_W, _VP, _CI, _VP, _VP, _SZ, _VP]),
    "moe_layer_forward_static": (_CI, [_W, _VP, _CI, _VP, _VP]),
    "moe_get_device_status_static": (_CI, [_VP]),
    "moe_host_staging_size": (_SZ, [_W, _CI]),
    "moe_layer_forward_host": (_CI, [_W, _VP, _CI, _VP, _VP, _SZ, _VP]),
    "moe_route": (_CI, [_W, _VP, _CI, _VP, _SZ, _VP, ctypes.POINTER(moe_route_view)]),
    "moe_workspace_view": (_CI, [_W, _CI, _VP, _SZ, ctypes.POINTER(moe_route_view)]),
    "moe_get_device_status": (_CI, [_VP, _VP]),
    "moe_set_option": (_CI, [_CI, _CI]),
    "moe_get_option": (_CI, [_CI]),
    "moe_kernel_times": (_CI, [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float),
                               ctypes.POINTER(ctypes.c_int), _CI, ctypes.POINTER(ctypes.c_int)]),
    "moe_debug_dequant": (_CI, [ctypes.POINTER(moe_qmatrix), _CI, _CI, _CI, _VP, _VP]),
    "moe_expanded_weights_bytes": (_SZ, [_W]),
    "moe_layer_forward_expanded": (_CI, [_W, _VP, _CI, _VP, _VP, _SZ, _VP, _SZ, _VP]),
    "moe_kv_append": (_CI, [_KC, _KB, _VP, _LL, _VP, _LL, _VP]),
    "moe_kv_read": (_CI, [_KC, _KB, _VP, _VP, _VP]),
    "moe_attention_workspace_size": (_SZ, [_KC, _KB, _AT]),
    "moe_attention_forward": (_CI, [_KC, _KB, _AT, _VP, _LL, _VP, _VP, _VP, _SZ, _VP]),
    "moe_last_launch_count": (_CI, []),
    "moe_status_string": (ctypes.c_char_p, [_CI]),
}

_lib = None


def lib():
    """The loaded CUDA library. Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built ({LIB_PATH}); run bit_moe_expert_routing_gb300.build.build()")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(l, name)
            f.restype, f.argtypes = res, args
        _lib = l
    return _lib


class MoEError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {moe_status_string(status)} ({status})")


def _check(status: int, what: str) -> None:
    if status != MOE_OK:
        raise MoEError(status, what)


# --- the C entry points, same names --------------------------------------------------------

def moe_workspace_size(w: moe_weights, T: int) -> int:
    return lib().moe_workspace_size(ctypes.byref(w), T)


def moe_host_staging_size(w: moe_weights, T: int) -> int:
    return lib().moe_host_staging_size(ctypes.byref(w), T)


def moe_layer_forward(w, x_ptr, T, y_ptr, ws_ptr, ws_bytes, stream) -> int:
    return lib().moe_layer_forward(ctypes.byref(w), x_ptr, T, y_ptr, ws_ptr, ws_bytes, stream)


def moe_layer_forward_static(w, x_ptr, T, y_ptr, stream) -> int:
    """The layer with the library's fixed device scratch array as its
    workspace, for callers that cannot allocate device memory (include/moe.h
    says which)."""
    return lib().moe_layer_forward_static(ctypes.byref(w), x_ptr, T, y_ptr, stream)


def moe_get_device_status_static(stream) -> int:
    return lib().moe_get_device_status_static(stream)


def moe_expanded_weights_bytes(w: moe_weights) -> int:
    return lib().moe_expanded_weights_bytes(ctypes.byref(w))


def moe_layer_forward_expanded(w, x_ptr, T, y_ptr, ws_ptr, ws_bytes, wbuf_ptr, wbuf_bytes, stream) -> int:
    """The unfused form: a separate pass expands the selected experts'
    weights to bf16 in wbuf, then the GEMMs read them."""
    return lib().moe_layer_forward_expanded(ctypes.byref(w), x_ptr, T, y_ptr, ws_ptr, ws_bytes, wbuf_ptr, wbuf_bytes,
                                            stream)


def moe_layer_forward_host(w, x_host_ptr, T, y_host_ptr, ws_ptr, ws_bytes, stream) -> int:
    return lib().moe_layer_forward_host(ctypes.byref(w), x_host_ptr, T, y_host_ptr, ws_ptr, ws_bytes, stream)


def moe_route(w, x_ptr, T, ws_ptr, ws_bytes, stream, view: moe_route_view | None = None) -> int:
    return lib().moe_route(ctypes.byref(w), x_ptr, T, ws_ptr, ws_bytes, stream,
                           ctypes.byref(view) if view is not None else None)


def moe_workspace_view(w, T, ws_ptr, ws_bytes, view: moe_route_view) -> int:
    return lib().moe_workspace_view(ctypes.byref(w), T, ws_ptr, ws_bytes, ctypes.byref(view))


def moe_get_device_status(ws_ptr, stream) -> int:
    return lib().moe_get_device_status(ws_ptr, stream)


def moe_set_option(option: int, value: int) -> int:
    return lib().moe_set_option(option, value)


def moe_get_option(option: int) -> int:
    return lib().moe_get_option(option)


def moe_kernel_times(max_entries: int = 32) -> dict[str, tuple[float, int]]:
    """{kernel name: (total ms, launches)} since the previous call."""
    names = (ctypes.c_char_p * max_entries)()
    ms = (ctypes.c_float * max_entries)()
    cnt = (ctypes.c_int * max_entries)()
    n = ctypes.c_int(0)
    _check(lib().moe_kernel_times(names, ms, cnt, max_entries, ctypes.byref(n)), "moe_kernel_times")
    return {names[i].decode(): (ms[i], cnt[i]) for i in range(n.value)}


def moe_debug_dequant(m: moe_qmatrix, expert, rows, K, out_ptr, stream) -> int:
    return lib().moe_debug_dequant(ctypes.byref(m), expert, rows, K, out_ptr, stream)


def moe_kv_append(cache, batch, k_ptr, k_stride, v_ptr, v_stride, stream) -> int:
    return lib().moe_kv_append(ctypes.byref(cache), ctypes.byref(batch), k_ptr, k_stride, v_ptr, v_stride, stream)


def moe_kv_read(cache, batch, k_ptr, v_ptr, stream) -> int:
    return lib().moe_kv_read(ctypes.byref(cache), ctypes.byref(batch), k_ptr, v_ptr, stream)


def moe_attention_workspace_size(cache, batch, attn: moe_attention) -> int:
    return lib().moe_attention_workspace_size(ctypes.byref(cache), ctypes.byref(batch), ctypes.byref(attn))


def moe_attention_forward(cache, batch, attn, q_ptr, q_stride, out_ptr, lse_ptr, ws_ptr, ws_bytes, stream) -> int:
    return lib().moe_attention_forward(ctypes.byref(cache), ctypes.byref(batch), ctypes.byref(attn), q_ptr, q_stride,
                                       out_ptr, lse_ptr, ws_ptr, ws_bytes, stream)


def moe_last_launch_count() -> int:
    return lib().moe_last_launch_count()


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


# --- torch helpers (allocation and streams only) ----------------------------------------

def _stream_ptr(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


class DeviceLayer:
    """A layer's packed weights resident in device memory (torch tensors) and
    the moe_weights struct that points at them. `layer` is anything with the
    fields of synth.Layer (numpy arrays; bf16 as uint16 bit patterns)."""

    def __init__(self, layer, device="cuda"):
        import numpy as np
        import torch

        self.D, self.E, self.k, self.I = layer.D, layer.E, layer.k, layer.I
        self._t = []

        def up(arr, dtype):
            a = np.ascontiguousarray(arr)
            t = torch.from_numpy(a.view({np.uint32: np.int32, np.uint16: np.int16}.get(a.dtype.type, a.dtype)))
            t = t.to(device)
            self._t.append(t)
            return t

        def qm(m):
            c, s, b = up(m.codes, None), up(m.scales, None), up(m.biases, None)
            return moe_qmatrix(c.data_ptr(), s.data_ptr(), b.data_ptr())

        self.router_w = up(layer.router_w.astype(np.float32), None)
        self.router_bias = None if layer.router_bias is None else up(layer.router_bias.astype(np.float32), None)
        self.w = moe_weights(layer.D, layer.E, layer.k, layer.I, self.router_w.data_ptr(),
                             None if self.router_bias is None else self.router_bias.data_ptr(),
                             qm(layer.gate), qm(layer.up), qm(layer.down),
                             qm(layer.s_gate), qm(layer.s_up), qm(layer.s_down))

    def workspace_bytes(self, T: int, host_staging: bool = False) -> int:
        """Device bytes of the workspace for T tokens (one pass of at most the chunk size)."""
        n = moe_workspace_size(self.w, T)
        if n == 0:
            raise MoEError(MOE_ERR_ARG, "moe_workspace_size")
        return n + (moe_host_staging_size(self.w, T) if host_staging else 0)

    def workspace(self, T: int, host_staging: bool = False):
        import torch
        return torch.empty(self.workspace_bytes(T, host_staging), dtype=torch.uint8, device=self._t[0].device)

    def forward(self, x, y=None, workspace=None, stream=None):
        """x: bf16 [T, D] on the device. Returns y: bf16 [T, D]."""
        import torch
        T = x.shape[0]
        assert x.dtype == torch.bfloat16 and x.is_contiguous() and x.shape[1] == self.D
        if y is None:
            y = torch.empty_like(x)
        if workspace is None:
            workspace = self.workspace(T)
        _check(moe_layer_forward(self.w, x.data_ptr(), T, y.data_ptr(), workspace.data_ptr(),
                                 workspace.numel(), _stream_ptr(stream)), "moe_layer_forward")
        return y

    def route(self, x, workspace, stream=None) -> moe_route_view:
        v = moe_route_view()
        _check(moe_route(self.w, x.data_ptr(), x.shape[0], workspace.data_ptr(), workspace.numel(),
                         _stream_ptr(stream), v), "moe_route")
        return v

    def view(self, T, workspace) -> moe_route_view:
        v = moe_route_view()
        _check(moe_workspace_view(self.w, T, workspace.data_ptr(), workspace.numel(), v), "moe_workspace_view")
        return v


def ws_tensor(workspace, ptr: int, shape, dtype):
    """A torch view of the workspace array at device pointer `ptr` (from a moe_route_view)."""
    import numpy as np
    import torch
    itemsize = torch.empty((), dtype=dtype).element_size()
    n = int(np.prod(shape))
    off = int(ptr) - workspace.data_ptr()
    assert 0 <= off and off + n * itemsize <= workspace.numel() and off % itemsize == 0
    return workspace[off:off + n * itemsize].view(dtype).reshape(shape)


def _int32(**values):
    """Refuses what a C int does not hold (ctypes would cut it without a word)."""
    for name, v in values.items():
        if not -2 ** 31 <= v < 2 ** 31:
            raise ValueError(f"{name}: {v} is not a 32-bit integer")


class KVBatch:
    """The sequences of one step (moe_kv_batch): int32 device tensors `q_off`
    [n_seqs + 1], `kv_len` [n_seqs] and `block_table` [n_seqs, pages], and the
    host's bounds on them. The tensors are kept, not copied: a serving loop
    may update them in place between steps."""

    def __init__(self, q_off, kv_len, block_table, n_tokens: int, max_new: int, max_kv: int):
        import torch
        for name, t, nd in (("q_off", q_off, 1), ("kv_len", kv_len, 1), ("block_table", block_table, 2)):
            if t.dtype != torch.int32 or t.dim() != nd or t.device.type != "cuda" or (t.numel() and t.stride(-1) != 1):
                raise ValueError(f"{name}: a CUDA int32 tensor with {nd} dimension(s), last one contiguous")
            if t.device != q_off.device:
                raise ValueError("q_off, kv_len and block_table: on one device")
        _int32(n_tokens=n_tokens, max_new=max_new, max_kv=max_kv)
        n = kv_len.shape[0]
        if q_off.shape[0] != n + 1 or block_table.shape[0] != n:
            raise ValueError("q_off has n_seqs + 1 entries, kv_len and block_table n_seqs")
        # a row may be read up to its stride: take the width where rows are the tensor's own
        stride = block_table.stride(0) if n > 1 else block_table.shape[1]
        if stride != block_table.shape[1]:
            raise ValueError("block_table: contiguous")
        self._t = (q_off, kv_len, block_table)
        self.n_tokens, self.device = n_tokens, q_off.device
        self.c = moe_kv_batch(n, n_tokens, max_new, max_kv, q_off.data_ptr(), kv_len.data_ptr(),
                              block_table.data_ptr(), stride)
        self._ref = ctypes.byref(self.c)


class KVCache:
    """A 4-bit key/value cache: the arrays of moe_kv_cache as torch tensors
    (codes int32 [pages, kv heads, page size, head dim / 8]; scales and biases
    bf16 [pages, kv heads, page size, head dim / 64]) and the operations on
    it. Calls are enqueued on `stream` (the current one by default); tensors
    they make are made there, and tensors they are given must be ready there."""

    def __init__(self, k_codes, k_scales, k_biases, v_codes, v_scales, v_biases):
        import torch
        pages, heads, size, words = k_codes.shape
        for codes, scales, biases in ((k_codes, k_scales, k_biases), (v_codes, v_scales, v_biases)):
            for t, dt, n in ((codes, torch.int32, words), (scales, torch.bfloat16, words // 8),
                             (biases, torch.bfloat16, words // 8)):
                if t.shape != (pages, heads, size, n) or t.dtype != dt or not t.is_contiguous() or \
                        t.device != k_codes.device or t.device.type != "cuda":
                    raise ValueError("a cache has contiguous CUDA codes int32 [pages, kv heads, page size, head dim / 8] "
                                     "and scales, biases bf16 [pages, kv heads, page size, head dim / 64]")
        self.k_codes, self.k_scales, self.k_biases = k_codes, k_scales, k_biases
        self.v_codes, self.v_scales, self.v_biases = v_codes, v_scales, v_biases
        self.kv_heads, self.head_dim, self.device = heads, words * 8, k_codes.device
        self.status = torch.zeros(256, dtype=torch.uint8, device=k_codes.device)
        self.c = moe_kv_cache(pages, size, heads, words * 8, k_codes.data_ptr(), k_scales.data_ptr(),
                              k_biases.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(), v_biases.data_ptr(),
                              self.status.data_ptr())
        self._ref = ctypes.byref(self.c)
        self._settings = {}  # moe_attention structs by their values
        self._torch, self._bf16 = torch, torch.bfloat16  # (an import statement costs as much as a check)

    @classmethod
    def empty(cls, n_pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda"):
        import torch
        a = []
        for _ in range(2):
            a.append(torch.zeros(n_pages, kv_heads, page_size, head_dim // 8, dtype=torch.int32, device=device))
            for _ in range(2):
                a.append(torch.zeros(n_pages, kv_heads, page_size, head_dim // 64, dtype=torch.bfloat16, device=device))
        return cls(*a)

    def _stream(self, stream):
        if stream is not None:
            return stream.cuda_stream
        return self._torch._C._cuda_getCurrentRawStream(self.device.index)  # without the stream object's 2 us

    def _batch(self, batch):
        """The batch, whose pointers go to this cache's device."""
        if batch.device != self.device:
            raise ValueError("batch: on the cache's device")
        return batch._ref

    def _rows(self, name, t, n_tokens, heads):
        """Checks a [n_tokens, heads, head dim] operand; its elements between tokens."""
        d = self.head_dim
        if t.shape != (n_tokens, heads, d) or t.dtype != self._bf16 or t.device != self.device:
            raise ValueError(f"{name}: bf16 [{n_tokens}, {heads}, {d}] on the cache's device")
        s = t.stride()
        if n_tokens == 0:
            return heads * d
        if s[2] != 1 or (heads > 1 and s[1] != d):
            raise ValueError(f"{name}: the heads of a token are contiguous")
        return s[0] if n_tokens > 1 else heads * d

    def append(self, k, v, batch: KVBatch, stream=None):
        """Quantises k, v (bf16 [n_tokens, kv heads, head dim]) into the cache."""
        ks = self._rows("k", k, batch.n_tokens, self.kv_heads)
        vs = self._rows("v", v, batch.n_tokens, self.kv_heads)
        st = lib().moe_kv_append(self._ref, self._batch(batch), k.data_ptr(), ks, v.data_ptr(), vs, self._stream(stream))
        if st:
            _check(st, "moe_kv_append")

    def read(self, batch: KVBatch, stream=None):
        """The step's tokens as the cache holds them: (k, v) bf16 [n_tokens, kv heads, head dim]."""
        if stream is not None:
            with self._torch.cuda.stream(stream):
                return self.read(batch)
        b = self._batch(batch)
        shape = (batch.n_tokens, self.kv_heads, self.head_dim)
        k = self._torch.empty(shape, dtype=self._bf16, device=self.device)
        v = self._torch.empty(shape, dtype=self._bf16, device=self.device)
        st = lib().moe_kv_read(self._ref, b, k.data_ptr(), v.data_ptr(), self._stream(None))
        if st:
            _check(st, "moe_kv_read")
        return k, v

    def attention_workspace(self, heads: int, batch: KVBatch, window: int = 0, sinks: int = 0):
        """A workspace for attention() with these arguments (a larger batch's serves a smaller one)."""
        import torch
        _int32(heads=heads, window=window, sinks=sinks)
        n = moe_attention_workspace_size(self.c, batch.c, moe_attention(heads, window, sinks, 1.0))
        if n == 0:
            raise MoEError(MOE_ERR_ARG, "moe_attention_workspace_size")
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def attention(self, q, batch: KVBatch, scale: float | None = None, window: int = 0, sinks: int = 0, out=None,
                  lse: bool = False, workspace=None, stream=None):
        """Causal attention of the step's tokens over the cache: q bf16
        [n_tokens, heads, head dim] -> out (the same shape), or (out, lse) with
        lse fp32 [n_tokens, heads]. scale: 1 / sqrt(head dim) by default."""
        torch = self._torch
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.attention(q, batch, scale, window, sinks, out, lse, workspace)
        if q.dim() != 3:
            raise ValueError("q: bf16 [n_tokens, heads, head dim]")
        b = self._batch(batch)
        n, heads, _ = shape = q.shape
        qs = self._rows("q", q, batch.n_tokens, heads)
        if out is None:
            out = torch.empty_like(q) if q.is_contiguous() else torch.empty(shape, dtype=self._bf16, device=self.device)
        elif out.shape != shape or out.dtype != self._bf16 or not out.is_contiguous() or out.device != self.device:
            raise ValueError("out: contiguous, of q's shape, type and device")
        l = lp = None
        if lse:
            l = torch.empty((n, heads), dtype=torch.float32, device=self.device)
            lp = l.data_ptr()
        if workspace is None:
            workspace = self.attention_workspace(heads, batch, window, sinks)
        elif workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError("workspace: contiguous, on the cache's device")
        at = self._settings.get((heads, window, sinks, scale))
        if at is None:
            _int32(window=window, sinks=sinks)
            if len(self._settings) > 64:
                self._settings.clear()
            at = moe_attention(heads, window, sinks, self.head_dim ** -0.5 if scale is None else scale)
            self._settings[heads, window, sinks, scale] = at = ctypes.byref(at)
        st = lib().moe_attention_forward(self._ref, b, at, q.data_ptr(), qs, out.data_ptr(), lp, workspace.data_ptr(),
                                         workspace.nbytes, self._stream(None))
        if st:
            _check(st, "moe_attention_forward")
        return (out, l) if lse else out

    def check(self, stream=None):
        """Synchronises the stream and raises if a call since the last check met a device-side error."""
        _check(moe_get_device_status(ctypes.c_void_p(self.status.data_ptr()), _stream_ptr(stream)), "kv cache")
