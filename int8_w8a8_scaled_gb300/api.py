"""Python binding of the C ABI: torch tensors in, library calls out.

This layer only marshals arguments (pointers, sizes, strides, dtypes, the
current CUDA stream); every step of the computation runs in the CUDA
library.  Tensors must already live on the current CUDA device.

    scaled_quant(x, q, scale, per_token=True, dynamic=True)
    scaled_dequant(q, scale, y, per_token=False)
    scaled_mm(a_q, b_q, scale_a, scale_b, out)

Naming follows the pages: ``cutlass_scaled_mm_dq(a, b, scale_a, scale_b,
out_dtype)`` of "[Kernel] Add w8a8 CUTLASS kernels" (here the output tensor is
passed in, as in that page's C++ op) with B given as a [K, N] column-major
view, i.e. a [N, K] row-major tensor; the quantiser follows the "Scaling
semantics" section of "Enable scaled FP8 (e4m3fn) KV cache on ROCm".
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import threading

import torch

from . import _lib
from ._lib import (BF16, DYNAMIC, E4M3, FP16, FP32, INT8, INT32, PER_ROW, PER_TENSOR, STATIC,
                   MmConfig, W8A8Error, check)

__all__ = [
    "scaled_quant", "scaled_dequant", "scaled_mm", "mm_workspace_size",
    "quant_workspace_size", "pick_config", "device_status", "Workspace", "quant_scaled_mm",
    "expand_shard_scales", "requant_shards", "fp8_kv_decode_attention", "attention_workspace_size",
    "kv4_cache_shape", "kv4_cache_write", "kv4_cache_read", "build_block_tables", "kv4_attention",
    "kv4_attention_workspace_size", "verify_drafts", "fp8_kv_rotate_write", "fp8_kv_attention",
    "fp8_kv_attention_workspace_size", "fp8_kv_block_means", "fp8_kv_select_blocks",
    "fp8_kv_select_blocks_workspace_size", "fp8_kv_sparse_attention", "fp8_kv_sparse_attention_workspace_size",
    "W8A8Error", "MmConfig",
]


def _qkind(t: torch.Tensor, q_dtype=None) -> int:
    if q_dtype is not None:
        return q_dtype
    if t.dtype == torch.float8_e4m3fn:
        return E4M3
    if t.dtype == torch.int8:
        return INT8
    raise TypeError(f"quantised tensors must be float8_e4m3fn or int8 (got {t.dtype}); "
                    "pass q_dtype= for a uint8 view")


def _fkind(t: torch.Tensor, wide: bool = False) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float16:
        return FP16
    if wide and t.dtype == torch.float32:
        return FP32
    if wide and t.dtype == torch.int32:
        return INT32
    raise TypeError(f"expected bfloat16 or float16 (got {t.dtype})")


def _ld(t: torch.Tensor) -> int:
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("rows must be contiguous (stride(1) == 1)")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


@functools.lru_cache(maxsize=None)
def _gpus() -> int:
    return torch.cuda.device_count()


def _cuda(*ts) -> int:
    """The current device, where the library launches; refuses tensors that are
    not on it.  With one GPU visible every CUDA tensor is (which saves a call
    about 1 us: 11 for one short attention request, 12 with the devices looked at)."""
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")
    if _gpus() == 1:
        return 0
    devices = {t.get_device() for t in ts if t is not None}
    if len(devices) > 1:
        raise ValueError("all tensors must be on one device")
    device = torch._C._cuda_getDevice()
    if devices != {device}:
        raise ValueError(f"the tensors are on cuda:{devices.pop()}, which is not the current device")
    return device


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _stream(stream, device: int) -> int:
    """The given stream of `device`, the current one, or its current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if getattr(stream, "device_index", None) not in (None, device):
        raise ValueError("the stream belongs to another device than the tensors")
    return stream.cuda_stream


class Workspace:
    """A zero-filled device scratch buffer reused across calls on one stream.

    The arrival counters at its head (of split-K matmuls and of attention) must
    start at zero; the library leaves them at zero after each successful call, so
    the buffer only needs zeroing once, on the stream that is current where it is
    made (a larger one that a call needs: on that call's stream), and one
    Workspace serves calls of every operator that takes one.  The first call on
    another stream waits for the zeroing; what calls on several streams do with
    the buffer is for their caller to order.

    A buffer that a captured call uses is kept as long as the Workspace, so that
    the graph can be replayed after the Workspace has grown.  Make it before the
    capture and large enough: a captured call that needs more gets a buffer of
    the graph's own, which every replay zeroes.  A replay counts as calls on the
    stream that it runs on: where it may overlap others, give it a Workspace of
    its own.
    """

    def __init__(self, nbytes: int = 0, device=None):
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self._captured = []          # buffers that graphs hold the address of
        self._zero(max(nbytes, 256), torch.cuda.current_stream(self.device))

    def _zero(self, nbytes: int, stream) -> None:
        """A new buffer, zeroed on `stream`, the current one."""
        self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        self._ordered = {stream.cuda_stream}        # streams that come after the zeroing
        self._zeroed = None if _capturing() else stream.record_event()

    def ensure(self, nbytes: int, stream=None) -> "Workspace":
        """At least nbytes, for a call on `stream` (None: the current one)."""
        handle = torch._C._cuda_getCurrentRawStream(self.buf.get_device()) if stream is None else stream.cuda_stream
        capturing = handle != 0 and _capturing()    # (the legacy default stream, handle 0, cannot be captured)
        if nbytes <= self.buf.numel():
            if capturing:
                if not (self._captured and self._captured[-1] is self.buf):
                    self._captured.append(self.buf)
            elif handle not in self._ordered and self._zeroed is not None:
                with _launching_on(self.device, stream) as launch:
                    launch.wait_event(self._zeroed)
                    self.buf.record_stream(launch)
                self._ordered.add(handle)
            return self
        with _launching_on(self.device, stream) as launch:
            if _capturing():
                return Workspace(nbytes, self.device)
            self.buf.record_stream(launch)          # earlier calls there may still use it
            self._zero(nbytes, launch)
        return self

    @property
    def nbytes(self) -> int:
        return self.buf.numel()


def _capturing() -> bool:
    """Whether the current stream is being captured into a graph."""
    return torch._C._cuda_isCurrentStreamCapturing()


@contextlib.contextmanager
def _launching_on(device: torch.device, stream):
    """The given stream (None: the current one) as the current stream."""
    if stream is None:
        yield torch.cuda.current_stream(device)
    else:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
        with torch.cuda.stream(stream):
            yield stream


_ws_lock = threading.Lock()
_default_ws: dict = {}


def _default_workspace(device: int, nbytes: int, kind: str, stream, handle: int) -> Workspace:
    """Per (device, stream that the call runs on, kind) scratch, zeroed on that
    stream; the matmul's buffer is never shared with the quantiser (whose absmax
    word would land on a counter).  Scratch first made during a capture belongs to
    the graph, whose replay zeroes it, and is not kept: before that replay it
    holds anything.  stream: as given to the call, handle: what it stands for."""
    key = (kind, device, handle)
    ws = _default_ws.get(key)
    # (the legacy default stream, handle 0, cannot be captured)
    if ws is not None and ws.buf.numel() >= nbytes and (handle == 0 or not _capturing()):
        return ws
    if ws is None:
        on = torch.device("cuda", device)
        with _ws_lock, _launching_on(on, stream):
            ws = _default_ws.get(key)
            if ws is None:
                ws = Workspace(nbytes, on)
                if not _capturing():
                    _default_ws[key] = ws
                return ws
    with _ws_lock:
        return ws.ensure(nbytes, stream)


def quant_workspace_size(rows: int, cols: int, per_token: bool, dynamic: bool) -> int:
    return _lib.load().w8a8_scaled_quant_workspace_size(
        rows, cols, PER_ROW if per_token else PER_TENSOR, DYNAMIC if dynamic else STATIC)


def scaled_quant(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, per_token: bool = True,
                 dynamic: bool = True, workspace: torch.Tensor | None = None, q_dtype=None,
                 stream=None) -> None:
    """q = sat_round(x / scale); dynamic mode writes scale = absmax / 448
    (e4m3) or absmax / 127 (int8), per token (row) or per tensor."""
    device = _cuda(x, q, scale, workspace)
    handle = _stream(stream, device)
    lib = _lib.load()
    rows, cols = x.shape
    if tuple(q.shape) != (rows, cols):
        raise ValueError("q must have the shape of x")
    if scale.dtype != torch.float32 or not scale.is_contiguous():
        raise ValueError("scale must be a contiguous float32 tensor")
    need_scale = rows if per_token else 1
    if scale.numel() != need_scale:
        raise ValueError(f"scale must have {need_scale} elements")
    gran = PER_ROW if per_token else PER_TENSOR
    mode = DYNAMIC if dynamic else STATIC
    need = lib.w8a8_scaled_quant_workspace_size(rows, cols, gran, mode)
    if need and workspace is None:
        workspace = _default_workspace(device, need, "quant", stream, handle).buf
    check(lib.w8a8_scaled_quant(
        _ptr(x), _fkind(x), rows, cols, _ld(x), _ptr(q), _qkind(q, q_dtype), _ld(q),
        _ptr(scale), gran, mode, _ptr(workspace) if need else None,
        workspace.numel() if (need and workspace is not None) else 0, handle))


def scaled_dequant(q: torch.Tensor, scale: torch.Tensor, y: torch.Tensor, per_token: bool = False,
                   q_dtype=None, stream=None) -> None:
    """y = round16(decode(q) * scale)."""
    device = _cuda(q, scale, y)
    lib = _lib.load()
    rows, cols = q.shape
    if tuple(y.shape) != (rows, cols):
        raise ValueError("y must have the shape of q")
    if scale.dtype != torch.float32 or not scale.is_contiguous():
        raise ValueError("scale must be a contiguous float32 tensor")
    check(lib.w8a8_scaled_dequant(
        _ptr(q), _qkind(q, q_dtype), rows, cols, _ld(q), _ptr(scale),
        PER_ROW if per_token else PER_TENSOR, _ptr(y), _fkind(y), _ld(y), _stream(stream, device)))


def _cfg(config) -> MmConfig | None:
    if config is None:
        return None
    if isinstance(config, MmConfig):
        return config
    return MmConfig(int(config.get("swap_ab", 0)), int(config.get("block_n", 0)),
                    int(config.get("split_k", 0)), int(config.get("stages", 0)),
                    int(config.get("ctas_per_sm", 0)), int(config.get("reduce", 0)),
                    int(config.get("cta_pair", 0)))


def pick_config(M: int, N: int, K: int, q_dtype: int = E4M3) -> dict:
    c = MmConfig()
    check(_lib.load().w8a8_scaled_mm_pick_config(M, N, K, q_dtype, ctypes.byref(c)))
    return c.as_dict()


def mm_workspace_size(M: int, N: int, K: int, q_dtype: int = E4M3, config=None) -> int:
    lib = _lib.load()
    c = _cfg(config)
    if c is None:
        return lib.w8a8_scaled_mm_workspace_size(M, N, K, q_dtype)
    return lib.w8a8_scaled_mm_config_workspace_size(M, N, K, q_dtype, ctypes.byref(c))


def scaled_mm(a_q: torch.Tensor, b_q: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor,
              out: torch.Tensor, workspace: torch.Tensor | Workspace | None = None, config=None,
              q_dtype=None, stream=None) -> torch.Tensor:
    """out[m, n] = round16(sum_k a_q[m, k] b_q[n, k] * scale_a[m|0] * scale_b[n|0]).

    a_q: [M, K] e4m3 / int8, rows contiguous.  b_q: [N, K] (the [K, N]
    column-major weight), rows contiguous.  scale_a: [M] or [1] fp32,
    scale_b: [N] or [1] fp32.  out: [M, N] bf16 / fp16 (or float32 for the
    unrounded e4m3 result, int32 for the raw int8 accumulators).
    """
    device = _cuda(a_q, b_q, scale_a, scale_b, out)
    handle = _stream(stream, device)
    lib = _lib.load()
    M, K = a_q.shape
    N, K2 = b_q.shape
    if K != K2:
        raise ValueError("a_q is [M, K] and b_q is [N, K]: K must match")
    if tuple(out.shape) != (M, N):
        raise ValueError("out must be [M, N]")
    for s in (scale_a, scale_b):
        if s.dtype != torch.float32 or not s.is_contiguous():
            raise ValueError("scales must be contiguous float32 tensors")
    a_gran = PER_ROW if scale_a.numel() == M and M > 1 else PER_TENSOR
    b_gran = PER_ROW if scale_b.numel() == N and N > 1 else PER_TENSOR
    if a_gran == PER_TENSOR and scale_a.numel() != 1:
        raise ValueError("scale_a must have 1 or M elements")
    if b_gran == PER_TENSOR and scale_b.numel() != 1:
        raise ValueError("scale_b must have 1 or N elements")
    qk = _qkind(a_q, q_dtype)
    if _qkind(b_q, q_dtype) != qk:
        raise TypeError("a_q and b_q must have the same element type")
    c = _cfg(config)
    need = (lib.w8a8_scaled_mm_config_workspace_size(M, N, K, qk, ctypes.byref(c)) if c is not None
            else lib.w8a8_scaled_mm_workspace_size(M, N, K, qk))
    if isinstance(workspace, Workspace):
        workspace = workspace.ensure(need, stream).buf
    elif workspace is None and need:
        workspace = _default_workspace(device, need, "mm", stream, handle).buf
    _cuda(a_q, workspace)
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (_ptr(a_q), _ld(a_q), _ptr(b_q), _ld(b_q), _ptr(scale_a), a_gran, _ptr(scale_b), b_gran,
            _ptr(out), _ld(out), M, N, K, qk, _fkind(out, wide=True), ws_ptr, ws_bytes)
    if c is None:
        check(lib.w8a8_scaled_mm(*args, handle))
    else:
        check(lib.w8a8_scaled_mm_with_config(*args, ctypes.byref(c), handle))
    return out


def quant_scaled_mm(x: torch.Tensor, b_q: torch.Tensor, scale_b: torch.Tensor, out: torch.Tensor,
                    scale_a_out: torch.Tensor | None = None, workspace: torch.Tensor | Workspace | None = None,
                    route: str = "auto", stream=None) -> torch.Tensor:
    """Dynamic per-token quantisation of x and the scaled matmul in one call:
    the bits of ``scaled_quant(x, ..., per_token=True, dynamic=True)``
    followed by ``scaled_mm``.

    x: [M, K] bf16 / fp16, rows contiguous.  b_q: [N, K] e4m3 / int8 (the
    operand type).  scale_b: [N] or [1] fp32.  out: [M, N] bf16 / fp16 (or
    float32 with e4m3 weights).  scale_a_out: optional [M] fp32 that receives
    the per-token scales.  route: "auto", "one_kernel" (the matmul
    quantises its own activations; decode shapes only) or "two_step".
    """
    device = _cuda(x, b_q, scale_b, out)
    handle = _stream(stream, device)
    lib = _lib.load()
    M, K = x.shape
    N, K2 = b_q.shape
    if K != K2:
        raise ValueError("x is [M, K] and b_q is [N, K]: K must match")
    if tuple(out.shape) != (M, N):
        raise ValueError("out must be [M, N]")
    if scale_b.dtype != torch.float32 or not scale_b.is_contiguous():
        raise ValueError("scale_b must be a contiguous float32 tensor")
    b_gran = PER_ROW if scale_b.numel() == N and N > 1 else PER_TENSOR
    if b_gran == PER_TENSOR and scale_b.numel() != 1:
        raise ValueError("scale_b must have 1 or N elements")
    if scale_a_out is not None:
        _cuda(x, scale_a_out)
        if scale_a_out.dtype != torch.float32 or scale_a_out.numel() != M or not scale_a_out.is_contiguous():
            raise ValueError("scale_a_out must be a contiguous float32 tensor of M elements")
    qk = _qkind(b_q)
    need = lib.w8a8_quant_scaled_mm_workspace_size(M, N, K, qk)
    if isinstance(workspace, Workspace):
        workspace = workspace.ensure(need, stream).buf
    elif workspace is None and need:
        workspace = _default_workspace(device, need, "mm", stream, handle).buf
    _cuda(x, workspace)
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    check(lib.w8a8_quant_scaled_mm(_ptr(x), _fkind(x), _ld(x), _ptr(b_q), _ld(b_q), _ptr(scale_b), b_gran,
                                   _ptr(out), _ld(out), M, N, K, qk, _fkind(out, wide=True),
                                   _ptr(scale_a_out) if scale_a_out is not None else None,
                                   _lib.ROUTES[route], ws_ptr, ws_bytes, handle))
    return out


def _shard_rows(shard_rows):
    arr = (ctypes.c_int64 * len(shard_rows))(*[int(r) for r in shard_rows])
    return arr, len(shard_rows)


def expand_shard_scales(shard_scales: torch.Tensor, shard_rows, scale_b: torch.Tensor, stream=None) -> torch.Tensor:
    """scale_b[n] = shard_scales[shard of row n]: per-shard weight scales of a
    merged layer as a per-channel vector for the fused epilogue."""
    device = _cuda(shard_scales, scale_b)
    arr, n = _shard_rows(shard_rows)
    check(_lib.load().w8a8_expand_shard_scales(_ptr(shard_scales), arr, n, _ptr(scale_b), _stream(stream, device)))
    return scale_b


def requant_shards(q: torch.Tensor, shard_scales: torch.Tensor, shard_rows, q_out: torch.Tensor,
                   scale_out: torch.Tensor, q_dtype=None, stream=None) -> None:
    """Rewrite a row-sharded merged weight to one shared scale (the largest
    shard scale, written to scale_out): q' = encode(decode(q) * s_i / s_max)."""
    device = _cuda(q, shard_scales, q_out, scale_out)
    arr, n = _shard_rows(shard_rows)
    rows, cols = q.shape
    if tuple(q_out.shape) != (rows, cols):
        raise ValueError("q_out must have the shape of q")
    check(_lib.load().w8a8_requant_shards(_ptr(q), _qkind(q, q_dtype), cols, _ld(q), _ptr(shard_scales), arr, n,
                                          _ptr(q_out), _ld(q_out), _ptr(scale_out), _stream(stream, device)))


def device_status() -> int:
    """Synchronise and read/clear the device status word (1 = a bounded
    pipeline wait timed out)."""
    v = ctypes.c_int(0)
    check(_lib.load().w8a8_device_status(ctypes.byref(v)))
    return v.value


def attention_workspace_size(batch: int, num_q_heads: int, max_seq_len: int) -> int:
    return int(_lib.load().w8a8_fp8_kv_attention_workspace_size(batch, num_q_heads, max_seq_len))


def fp8_kv_decode_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            seq_lens: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                            out: torch.Tensor, sm_scale: float | None = None,
                            block_table: torch.Tensor | None = None, workspace=None, stream=None) -> None:
    """Decode attention reading an e4m3 KV cache with per-tensor scales
    ("Enable scaled FP8 (e4m3fn) KV cache on ROCm", "Scaling semantics").

    q, out: [batch, num_q_heads, 128] bf16 / fp16.  Without block_table the
    caches are [batch, max_seq_len, num_kv_heads, 128]; with block_table
    (int32 [batch, max_blocks]) they are [num_blocks, block_size,
    num_kv_heads, 128] (the paged cache).  Codes are float8_e4m3fn (or uint8
    views).  seq_lens: int32 [batch]; k_scale, v_scale: float32 [1].
    sm_scale defaults to 1/sqrt(128)."""
    device = _cuda(q, k_cache, v_cache, seq_lens, k_scale, v_scale, out)
    handle = _stream(stream, device)
    lib = _lib.load()
    if q.dim() != 3 or not q.is_contiguous() or tuple(out.shape) != tuple(q.shape) or not out.is_contiguous():
        raise ValueError("q and out must be contiguous [batch, num_q_heads, head_dim] tensors")
    batch, hq, d = q.shape
    if k_cache.dim() != 4 or tuple(k_cache.shape) != tuple(v_cache.shape):
        raise ValueError("k_cache and v_cache must be 4-d tensors of one shape")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("caches must be contiguous")
    for c in (k_cache, v_cache):
        if c.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise TypeError("caches must hold float8_e4m3fn codes (or uint8 views)")
    hkv = k_cache.shape[2]
    if k_cache.shape[3] != d:
        raise ValueError("cache head_dim must equal q's")
    if seq_lens.dtype != torch.int32 or seq_lens.numel() != batch or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous int32 tensor of batch entries")
    for s_ in (k_scale, v_scale):
        if s_.dtype != torch.float32 or s_.numel() != 1:
            raise ValueError("k_scale and v_scale must be float32 tensors of one element")
    if block_table is None:
        if k_cache.shape[0] != batch:
            raise ValueError("without a block table the caches are [batch, max_seq_len, num_kv_heads, head_dim]")
        max_seq = k_cache.shape[1]
        bt, bsz, maxb, nblk = None, 0, 0, 0
    else:
        if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != batch \
                or not block_table.is_contiguous():
            raise ValueError("block_table must be a contiguous int32 [batch, max_blocks] tensor")
        _cuda(q, block_table)
        nblk, bsz = k_cache.shape[0], k_cache.shape[1]
        maxb = block_table.shape[1]
        max_seq = maxb * bsz
        bt = _ptr(block_table)
    need = lib.w8a8_fp8_kv_attention_workspace_size(batch, hq, max_seq)
    if isinstance(workspace, Workspace):
        wbuf = workspace.ensure(need, stream).buf
    elif workspace is None:
        wbuf = _default_workspace(device, need, "attention", stream, handle).buf
    else:
        wbuf = workspace
    if workspace is not None:
        _cuda(q, wbuf)
    if sm_scale is None:
        sm_scale = 1.0 / float(d) ** 0.5
    check(lib.w8a8_fp8_kv_decode_attention(
        _ptr(q), _fkind(q), batch, hq, hkv, d, _ptr(k_cache), _ptr(v_cache), max_seq, bt, bsz, maxb, nblk,
        _ptr(seq_lens), _ptr(k_scale), _ptr(v_scale), float(sm_scale), _ptr(out), _fkind(out),
        _ptr(wbuf), wbuf.numel(), handle))


# ---------------------------------------------------------------- a serving step over a 4-bit paged KV cache


def kv4_cache_shape(num_blocks: int, num_kv_heads: int, block_size: int, head_dim: int) -> tuple:
    """Shape of a 4-bit cache, a contiguous uint8 tensor: [num_blocks,
    num_kv_heads, block_size / 16, 18 * head_dim], one record of 16 tokens'
    keys and values (codes and group scales) in the last dimension."""
    if _lib.load().w8a8_kv4_cache_bytes(num_blocks, num_kv_heads, block_size, head_dim) == 0:
        raise ValueError("block_size must be a multiple of 16, head_dim 64 or 128, counts >= 1")
    return (num_blocks, num_kv_heads, block_size // 16, 18 * head_dim)


def _kv4_cache(cache: torch.Tensor) -> tuple:
    """(num_blocks, num_kv_heads, block_size, head_dim) of a cache tensor."""
    if cache.dtype is not torch.uint8 or cache.ndim != 4 or not cache.is_contiguous():
        raise ValueError("the cache must be a contiguous uint8 CUDA tensor of kv4_cache_shape()")
    nb, h, records, nbytes = cache.shape
    if nbytes % 18:
        raise ValueError("the cache must be a contiguous uint8 CUDA tensor of kv4_cache_shape()")
    return nb, h, 16 * records, nbytes // 18


def _kv4_kind(kind: str) -> int:
    if kind not in _lib.KV4_KINDS:
        raise ValueError(f"kind must be one of {sorted(_lib.KV4_KINDS)}")
    return _lib.KV4_KINDS[kind]


def _vectors(checks, dtype) -> None:
    """Refuses what is not a contiguous tensor of `dtype` with n elements, for
    (name, tensor, n) in `checks`."""
    for name, t, n in checks:
        if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} vector of {n} entries")


def _one_scale(*ts: torch.Tensor) -> None:
    for t in ts:
        if t.dtype is not torch.float32 or t.numel() != 1:
            raise ValueError("k_scale and v_scale must be float32 tensors of one element")


def _heads(name: str, t: torch.Tensor, shape: tuple) -> tuple:
    """Token and head strides of a [tokens, heads, head_dim] tensor."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    token, head, dim = t.stride()
    if dim != 1:
        raise ValueError(f"the dims of a head of {name} must be consecutive (stride(2) == 1)")
    return token, head


def _kv4_tokens(k, v, cache, slots, k_scale, v_scale, kind) -> tuple:
    nb, h, bs, d = _kv4_cache(cache)
    if k.ndim != 3:
        raise ValueError("k and v must be [tokens, num_kv_heads, head_dim]")
    n = k.shape[0]
    shape = (n, h, d)
    ks, vs = _heads("k", k, shape), _heads("v", v, shape)
    if v.dtype is not k.dtype:
        raise TypeError("k and v must have the same element type")
    _vectors((("slots", slots, n),), torch.int64)
    _one_scale(k_scale, v_scale)
    device = _cuda(k, v, cache, slots, k_scale, v_scale)
    return nb, bs, (_fkind(k), n, h, d, *ks, *vs), _kv4_kind(kind), device


def kv4_cache_write(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor,
                    k_scale: torch.Tensor, v_scale: torch.Tensor, kind: str = "e2m1", stream=None) -> None:
    """Quantise new keys and values to 4 bits and write them at their slots.

    k, v: [tokens, num_kv_heads, head_dim] bf16 / fp16, any token and head
    strides.  cache: uint8 of kv4_cache_shape().  slots: int64 [tokens]
    (block * block_size + offset; one outside the cache is skipped).
    k_scale, v_scale: float32 [1], the tensors' scales: with absmax / (6 * 448)
    (e2m1) or absmax / (7 * 448) (int4) of the values met, no group saturates.
    kind: "e2m1" or "int4"."""
    nb, bs, sizes, kd, device = _kv4_tokens(k, v, cache, slots, k_scale, v_scale, kind)
    if sizes[1] == 0:
        return
    check(_lib.load().w8a8_kv4_cache_write(
        k.data_ptr(), v.data_ptr(), *sizes, cache.data_ptr(), nb, bs, slots.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), kd, _stream(stream, device)))


def kv4_cache_read(cache: torch.Tensor, slots: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                   k: torch.Tensor, v: torch.Tensor, kind: str = "e2m1", stream=None) -> None:
    """The values that the tokens at `slots` stand for, into k and v (bf16 /
    fp16 [tokens, num_kv_heads, head_dim]); zeros for a slot outside the
    cache.  Arguments as for kv4_cache_write."""
    nb, bs, sizes, kd, device = _kv4_tokens(k, v, cache, slots, k_scale, v_scale, kind)
    if sizes[1] == 0:
        return
    check(_lib.load().w8a8_kv4_cache_read(
        cache.data_ptr(), nb, bs, slots.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), kd, k.data_ptr(),
        v.data_ptr(), *sizes, _stream(stream, device)))


def build_block_tables(context_lens: torch.Tensor, new_lens: torch.Tensor, free_blocks: torch.Tensor,
                       free_count: torch.Tensor, block_table: torch.Tensor, block_size: int,
                       query_start: torch.Tensor, seq_lens: torch.Tensor, slots: torch.Tensor,
                       positions: torch.Tensor, free_left: torch.Tensor, free_count_out: torch.Tensor | None = None,
                       stream=None) -> None:
    """Block tables, slots and positions of a step's tokens, on the GPU.

    context_lens, new_lens: int32 [batch], the tokens each request holds and
    adds.  free_blocks: int32 ids, of which the first free_count[0] (int32
    [1]) are free; blocks are taken from the end, in request order.
    Written: the new entries of block_table (int32 [batch, max_blocks]),
    query_start (int32 [batch + 1]), seq_lens (int32 [batch]; 0 for a request
    that its table, the free list or the packed tokens have no room for), slots (int64) and
    positions (int32) of the packed tokens (-1 and 0 past the last one, -1 for
    a refused request's), free_left (int32 [1], a balance: free_count less the
    needs of all requests up to the last admitted one, refused ones among them
    included, so that it may be negative) and free_count_out (int32 [1], optional: the ids still
    free, the next call's free_count).  None of them may share memory with an
    input or with each other."""
    if block_table.dtype is not torch.int32 or block_table.ndim != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 [batch, max_blocks] CUDA tensor")
    batch, max_blocks = block_table.shape
    tokens, ids = slots.numel(), free_blocks.numel()
    _vectors((("context_lens", context_lens, batch), ("new_lens", new_lens, batch), ("free_blocks", free_blocks, ids),
              ("free_count", free_count, 1), ("query_start", query_start, batch + 1), ("seq_lens", seq_lens, batch),
              ("positions", positions, tokens), ("free_left", free_left, 1)), torch.int32)
    _vectors((("slots", slots, tokens),), torch.int64)
    if free_count_out is not None:
        _vectors((("free_count_out", free_count_out, 1),), torch.int32)
    device = _cuda(context_lens, new_lens, free_blocks, free_count, block_table, query_start, seq_lens, slots, positions,
                   free_left, free_count_out)
    check(_lib.load().w8a8_build_block_tables(
        context_lens.data_ptr(), new_lens.data_ptr(), batch, free_blocks.data_ptr(), free_count.data_ptr(), ids,
        block_table.data_ptr(), max_blocks, block_size, query_start.data_ptr(), seq_lens.data_ptr(), slots.data_ptr(),
        positions.data_ptr(), tokens, free_left.data_ptr(), _ptr(free_count_out), _stream(stream, device)))


def kv4_attention_workspace_size(batch: int, max_query_len: int, num_q_heads: int, num_kv_heads: int,
                                 head_dim: int) -> int:
    return int(_lib.load().w8a8_kv4_attention_workspace_size(batch, max_query_len, num_q_heads, num_kv_heads, head_dim))


@functools.lru_cache(maxsize=4096)
def _kv4_attention_need(device_index: int, *sizes: int) -> int:
    """The same, looked up once for a device and sizes (it depends on nothing else)."""
    return kv4_attention_workspace_size(*sizes)


def kv4_attention(q: torch.Tensor, cache: torch.Tensor, seq_lens: torch.Tensor, block_table: torch.Tensor,
                  k_scale: torch.Tensor, v_scale: torch.Tensor, out: torch.Tensor,
                  query_start: torch.Tensor | None = None, max_query_len: int = 1, sm_scale: float | None = None,
                  kind: str = "e2m1", workspace=None, stream=None) -> None:
    """Attention of new tokens over a 4-bit paged cache that holds their keys
    and values already.

    q, out: [tokens, num_q_heads, head_dim] bf16 / fp16, any token and head
    strides.  seq_lens: int32 [batch], lengths with the new tokens.
    block_table: int32 [batch, max_blocks].  query_start: int32 [batch + 1],
    the first row of each request in q, with max_query_len the most rows of
    one (or more; rows past it are not written); None: one row a request.  Row i of a request's n sees its tokens
    t <= seq_len - n + i; a row that sees none gives zeros.  sm_scale defaults
    to 1 / sqrt(head_dim).  workspace: a Workspace, or a zero-filled uint8
    tensor of kv4_attention_workspace_size(); None: the default one of the
    stream that the call runs on."""
    nb, hkv, bs, d = _kv4_cache(cache)
    shape = q.shape
    if len(shape) != 3 or shape[2] != d:
        raise ValueError("q must be [tokens, num_q_heads, head_dim] with the cache's head_dim")
    tokens, hq, _ = shape
    qs, os_ = _heads("q", q, shape), _heads("out", out, shape)
    if block_table.dtype is not torch.int32 or block_table.ndim != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 [batch, max_blocks] CUDA tensor")
    batch, max_blocks = block_table.shape
    if query_start is None:
        _vectors((("seq_lens", seq_lens, batch),), torch.int32)
    else:
        _vectors((("seq_lens", seq_lens, batch), ("query_start", query_start, batch + 1)), torch.int32)
    _one_scale(k_scale, v_scale)
    device = _cuda(q, cache, seq_lens, block_table, k_scale, v_scale, out, query_start)
    handle = _stream(stream, device)
    kd = _kv4_kind(kind)
    if tokens == 0:
        return
    need = _kv4_attention_need(device, batch, max_query_len, hq, hkv, d)
    if isinstance(workspace, Workspace):
        wbuf = workspace.ensure(need, stream).buf
    elif workspace is None:
        wbuf = _default_workspace(device, need, "kv4_attention", stream, handle).buf
    else:
        wbuf = workspace
    if workspace is not None:
        _cuda(q, wbuf)
    if sm_scale is None:
        sm_scale = 1.0 / float(d) ** 0.5
    check(_lib.load().w8a8_kv4_attention(
        q.data_ptr(), _fkind(q), tokens, hq, hkv, d, *qs, cache.data_ptr(), nb, bs, block_table.data_ptr(), max_blocks,
        seq_lens.data_ptr(), _ptr(query_start), batch, max_query_len, k_scale.data_ptr(), v_scale.data_ptr(), sm_scale, kd,
        out.data_ptr(), _fkind(out), *os_, wbuf.data_ptr(), wbuf.numel() * wbuf.element_size(), handle))


def verify_drafts(target_probs: torch.Tensor, draft_probs: torch.Tensor | None, draft_tokens: torch.Tensor,
                  draft_start: torch.Tensor, uniform: torch.Tensor, sample_uniform: torch.Tensor,
                  out_tokens: torch.Tensor, num_accepted: torch.Tensor, stream=None) -> None:
    """Accept drafted tokens against the target's probabilities, and draw the
    token after the last accepted one.

    target_probs: [rows + batch, vocab] fp32 / bf16 / fp16, rows contiguous:
    n + 1 rows for a request of n drafts.  draft_probs: [rows, vocab] of the
    same type, or None for a draft that gave its tokens alone.  draft_tokens:
    int32 [rows]; draft_start: int32 [batch + 1], the first drafted row of
    each request.  uniform: float32 [rows] and sample_uniform: float32 [batch],
    random numbers in [0, 1).  Written: out_tokens, int32 [batch,
    max_drafts + 1] (accepted tokens, the drawn one, then -1), and
    num_accepted, int32 [batch]."""
    if out_tokens.dtype is not torch.int32 or out_tokens.ndim != 2 or not out_tokens.is_contiguous():
        raise ValueError("out_tokens must be a contiguous int32 [batch, max_drafts + 1] CUDA tensor")
    batch, columns = out_tokens.shape
    rows = draft_tokens.numel()
    if target_probs.ndim != 2 or target_probs.shape[0] != rows + batch:
        raise ValueError("target_probs must be [rows + batch, vocab]")
    vocab = target_probs.shape[1]
    if draft_probs is not None:
        if draft_probs.shape != (rows, vocab):
            raise ValueError("draft_probs must be [rows, vocab]")
        if draft_probs.dtype is not target_probs.dtype:
            raise TypeError("target_probs and draft_probs must have the same element type")
    _vectors((("draft_tokens", draft_tokens, rows), ("draft_start", draft_start, batch + 1),
              ("num_accepted", num_accepted, batch)), torch.int32)
    _vectors((("uniform", uniform, rows), ("sample_uniform", sample_uniform, batch)), torch.float32)
    device = _cuda(target_probs, draft_probs, draft_tokens, draft_start, uniform, sample_uniform, out_tokens, num_accepted)
    check(_lib.load().w8a8_verify_drafts(
        target_probs.data_ptr(), _ptr(draft_probs),
        FP32 if target_probs.dtype is torch.float32 else _fkind(target_probs), vocab, _ld(target_probs),
        vocab if draft_probs is None else _ld(draft_probs), draft_tokens.data_ptr(), draft_start.data_ptr(), batch, rows,
        uniform.data_ptr(), sample_uniform.data_ptr(), out_tokens.data_ptr(), columns - 1, num_accepted.data_ptr(),
        _stream(stream, device)))


# ---------------------------------------------------------------- long contexts over the paged fp8 KV cache


def _fp8_cache(cache: torch.Tensor, name: str) -> tuple:
    """(num_blocks, block_size, num_kv_heads, head_dim) of an fp8 cache."""
    if cache.ndim != 4 or not cache.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [num_blocks, block_size, num_kv_heads, head_dim] tensor")
    if cache.dtype is not torch.float8_e4m3fn and cache.dtype is not torch.uint8:
        raise TypeError(f"{name} must hold float8_e4m3fn codes (or a uint8 view)")
    return tuple(cache.shape)


def _fp8_caches(k_cache: torch.Tensor, v_cache: torch.Tensor) -> tuple:
    shape = _fp8_cache(k_cache, "k_cache")
    if _fp8_cache(v_cache, "v_cache") != shape:
        raise ValueError("k_cache and v_cache must have one shape")
    return shape


def _paged_rows(seq_lens: torch.Tensor, block_table: torch.Tensor, query_start: torch.Tensor | None) -> tuple:
    """(batch, max_blocks) of a step's requests."""
    if block_table.dtype is not torch.int32 or block_table.ndim != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 [batch, max_blocks] CUDA tensor")
    batch, max_blocks = block_table.shape
    if query_start is None:
        _vectors((("seq_lens", seq_lens, batch),), torch.int32)
    else:
        _vectors((("seq_lens", seq_lens, batch), ("query_start", query_start, batch + 1)), torch.int32)
    return batch, max_blocks


def _scratch(workspace, need: int, kind: str, device: int, stream, handle: int, like: torch.Tensor) -> torch.Tensor:
    """A call's scratch: its caller's, or the default one of its stream."""
    if workspace is None:
        return _default_workspace(device, need, kind, stream, handle).buf
    buf = workspace.ensure(need, stream).buf if isinstance(workspace, Workspace) else workspace
    _cuda(like, buf)
    return buf


def fp8_kv_rotate_write(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, cos_sin: torch.Tensor,
                        positions: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor,
                        k_scale: torch.Tensor, v_scale: torch.Tensor, q_out: torch.Tensor | None, sections=None,
                        interleaved: bool = False, stream=None) -> None:
    """Rotate queries and keys by their positions, and write keys and values
    into the paged fp8 cache at their slots.

    q: [tokens, num_q_heads, head_dim], k, v: [tokens, num_kv_heads,
    head_dim], bf16 / fp16, any token and head strides.  cos_sin: float32
    [max_position, rot_dim], cosines of the rot_dim / 2 pairs, then sines;
    pairs are dims i and i + rot_dim / 2 of a head, with interleaved 2 i and
    2 i + 1; dims from rot_dim on stay.  positions: int32 [tokens], or
    [axes, tokens] with sections, the number of pairs that turn by each axis
    (they add up to rot_dim / 2); one outside cos_sin gives NaN.  k_cache,
    v_cache: [num_blocks, block_size, num_kv_heads, head_dim] float8_e4m3fn (or
    uint8 views).  slots: int64 [tokens] (block * block_size + offset; one
    outside the cache is skipped; no slot twice).  k_scale, v_scale: float32
    [1].  q_out: rotated queries, as q; q itself is fine.  q and q_out may be
    None."""
    nb, bs, h, d = _fp8_caches(k_cache, v_cache)
    if k.ndim != 3:
        raise ValueError("k and v must be [tokens, num_kv_heads, head_dim]")
    n = k.shape[0]
    ks, vs = _heads("k", k, (n, h, d)), _heads("v", v, (n, h, d))
    if v.dtype is not k.dtype:
        raise TypeError("q, k, v and q_out must have the same element type")
    hq, qs, os_ = 0, (0, 0), (0, 0)
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        if q.ndim != 3:
            raise ValueError("q must be [tokens, num_q_heads, head_dim]")
        hq = q.shape[1]
        qs, os_ = _heads("q", q, (n, hq, d)), _heads("q_out", q_out, (n, hq, d))
        if q.dtype is not k.dtype or q_out.dtype is not k.dtype:
            raise TypeError("q, k, v and q_out must have the same element type")
    if cos_sin.dtype is not torch.float32 or cos_sin.ndim != 2 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be a contiguous float32 [max_position, rot_dim] tensor")
    axes, counts = 1, None
    if sections is not None:
        axes = len(sections)
        if not 1 <= axes <= 4:
            raise ValueError("there are 1 to 4 sections")
        counts = (ctypes.c_int32 * axes)(*sections)
    if positions.dtype is not torch.int32 or not positions.is_contiguous() or \
            tuple(positions.shape) not in (((axes, n), (n,)) if axes == 1 else ((axes, n),)):
        raise ValueError(f"positions must be a contiguous int32 {'[tokens]' if axes == 1 else f'[{axes}, tokens]'} tensor")
    _vectors((("slots", slots, n),), torch.int64)
    _one_scale(k_scale, v_scale)
    device = _cuda(q, k, v, cos_sin, positions, k_cache, v_cache, slots, k_scale, v_scale, q_out)
    dtype = _fkind(k)
    if n == 0:
        return
    check(_lib.load().w8a8_fp8_kv_rotate_write(
        _ptr(q), k.data_ptr(), v.data_ptr(), dtype, n, hq, h, d, *qs, *ks, *vs, cos_sin.data_ptr(), *cos_sin.shape,
        positions.data_ptr(), axes, counts, int(interleaved), k_cache.data_ptr(), v_cache.data_ptr(), nb, bs, slots.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), _ptr(q_out), *os_, _stream(stream, device)))


def fp8_kv_attention_workspace_size(batch: int, max_query_len: int, num_q_heads: int, num_kv_heads: int,
                                    head_dim: int) -> int:
    return int(_lib.load().w8a8_fp8_kv_paged_attention_workspace_size(batch, max_query_len, num_q_heads, num_kv_heads, head_dim))


@functools.lru_cache(maxsize=4096)
def _fp8_attention_need(device_index: int, *sizes: int) -> int:
    """The same, looked up once for a device and sizes (it depends on nothing else)."""
    return fp8_kv_attention_workspace_size(*sizes)


def fp8_kv_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, seq_lens: torch.Tensor,
                     block_table: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, out: torch.Tensor,
                     query_start: torch.Tensor | None = None, max_query_len: int = 1, sm_scale: float | None = None,
                     workspace=None, stream=None) -> None:
    """Attention of new tokens (single ones, drafts, prompt chunks) over the
    paged fp8 cache that holds their keys and values already.

    q, out: [tokens, num_q_heads, head_dim] bf16 / fp16, any token and head
    strides; out may not share memory with q.  k_cache, v_cache:
    [num_blocks, block_size, num_kv_heads, head_dim] float8_e4m3fn (or uint8
    views), block_size a multiple of 16, head_dim 64 or 128.  seq_lens: int32
    [batch], lengths with the new tokens.  block_table: int32 [batch,
    max_blocks].  query_start: int32 [batch + 1], the first row of each request
    in q, which ends in front of the next one's (no rows where that is not
    above; no row of two requests), with max_query_len the most rows of one (or
    more; rows past it are not written, and it chooses the kernels: a limit
    above the need costs time); None: one row a request.  Row i of a request's n
    sees its tokens t <= seq_len - n + i; a row that sees none gives zeros.
    sm_scale defaults to 1 / sqrt(head_dim).  workspace: a Workspace, or a
    zero-filled uint8 tensor of fp8_kv_attention_workspace_size(); None: the
    default one of the stream that the call runs on.

    Scores and sums are 32-bit; a softmax weight has 11 bits in the second
    product.  fp8_kv_decode_attention (single tokens, head_dim 128) carries
    about 22, and is the faster call for many short contexts.  include/w8a8.h
    has the figures, and max_query_len's."""
    nb, bs, hkv, d = _fp8_caches(k_cache, v_cache)
    shape = q.shape
    if len(shape) != 3 or shape[2] != d:
        raise ValueError("q must be [tokens, num_q_heads, head_dim] with the cache's head_dim")
    tokens, hq, _ = shape
    qs, os_ = _heads("q", q, shape), _heads("out", out, shape)
    batch, max_blocks = _paged_rows(seq_lens, block_table, query_start)
    _one_scale(k_scale, v_scale)
    device = _cuda(q, k_cache, v_cache, seq_lens, block_table, k_scale, v_scale, out, query_start)
    handle = _stream(stream, device)
    if tokens == 0:
        return
    buf = _scratch(workspace, _fp8_attention_need(device, batch, max_query_len, hq, hkv, d), "fp8_attention", device, stream,
                   handle, q)
    if sm_scale is None:
        sm_scale = 1.0 / float(d) ** 0.5
    check(_lib.load().w8a8_fp8_kv_paged_attention(
        q.data_ptr(), _fkind(q), tokens, hq, hkv, d, *qs, k_cache.data_ptr(), v_cache.data_ptr(), nb, bs, block_table.data_ptr(),
        max_blocks, seq_lens.data_ptr(), _ptr(query_start), batch, max_query_len, k_scale.data_ptr(), v_scale.data_ptr(), sm_scale,
        out.data_ptr(), _fkind(out), *os_, buf.data_ptr(), buf.numel() * buf.element_size(), handle))


def _block_means(means: torch.Tensor, mean_scales: torch.Tensor) -> tuple:
    """(num_blocks, num_kv_heads, head_dim) of the blocks' means."""
    if means.dtype is not torch.int8 or means.ndim != 3 or not means.is_contiguous():
        raise ValueError("means must be a contiguous int8 [num_blocks, num_kv_heads, head_dim] tensor")
    if mean_scales.dtype is not torch.float32 or mean_scales.shape != means.shape[:2] or not mean_scales.is_contiguous():
        raise ValueError("mean_scales must be a contiguous float32 [num_blocks, num_kv_heads] tensor")
    return tuple(means.shape)


def fp8_kv_block_means(k_cache: torch.Tensor, seq_lens: torch.Tensor, block_table: torch.Tensor, means: torch.Tensor,
                       mean_scales: torch.Tensor, query_start: torch.Tensor | None = None, max_query_len: int = 1,
                       stream=None) -> None:
    """8-bit means of the keys of the blocks that a step wrote to, for
    fp8_kv_select_blocks.

    Written: the rows of means (int8 [num_blocks, num_kv_heads, head_dim]) and
    mean_scales (float32 [num_blocks, num_kv_heads]) of the blocks that hold
    the last n of each request's seq_len tokens, over the tokens that it
    holds; other rows stay.  No block may be among them twice, of two requests
    or two columns.  query_start: int32 [batch + 1], whose differences are the
    n, None: one each.  max_query_len: the largest n, or more (with less the
    means are the same, and take longer)."""
    nb, bs, h, d = _fp8_cache(k_cache, "k_cache")
    if _block_means(means, mean_scales) != (nb, h, d):
        raise ValueError("means must be [num_blocks, num_kv_heads, head_dim] of the cache")
    batch, max_blocks = _paged_rows(seq_lens, block_table, query_start)
    device = _cuda(k_cache, seq_lens, block_table, means, mean_scales, query_start)
    if batch == 0:
        return
    # no row of q is looked at: any number of them that the starts may name
    tokens = batch if query_start is None else (1 << 31) - 1
    check(_lib.load().w8a8_fp8_kv_block_means(
        k_cache.data_ptr(), nb, bs, h, d, block_table.data_ptr(), max_blocks, seq_lens.data_ptr(), _ptr(query_start), tokens, batch,
        max_query_len, means.data_ptr(), mean_scales.data_ptr(), _stream(stream, device)))


def fp8_kv_select_blocks_workspace_size(tokens: int, num_kv_heads: int, max_blocks: int) -> int:
    return int(_lib.load().w8a8_fp8_kv_select_blocks_workspace_size(tokens, num_kv_heads, max_blocks))


def fp8_kv_select_blocks(q: torch.Tensor, means: torch.Tensor, mean_scales: torch.Tensor, seq_lens: torch.Tensor,
                         block_table: torch.Tensor, block_size: int, selected: torch.Tensor,
                         query_start: torch.Tensor | None = None, max_query_len: int = 1, first_blocks: int = 1,
                         last_blocks: int = 2, workspace=None, stream=None) -> None:
    """The blocks that matter most to each new token and KV head, for
    fp8_kv_sparse_attention.

    Of the blocks up to the token's own, the first first_blocks and the last
    last_blocks are taken, then those of the highest scores, the lower block of
    equal ones: the largest product of the 8-bit mean of the block's keys
    (means and mean_scales of fp8_kv_block_means) with the query heads that
    share the KV head, each quantised to 8 bits.  selected: int32 [tokens,
    num_kv_heads, budget], columns of the block table in rising order, then
    -1.  q, seq_lens, block_table, query_start and max_query_len: as for
    fp8_kv_attention; rows of no request are not written.  workspace: a
    Workspace (the one of the attention calls is fine), or a uint8 tensor of
    fp8_kv_select_blocks_workspace_size()."""
    nb, hkv, d = _block_means(means, mean_scales)
    shape = q.shape
    if len(shape) != 3 or shape[2] != d:
        raise ValueError("q must be [tokens, num_q_heads, head_dim] with the means' head_dim")
    tokens, hq, _ = shape
    qs = _heads("q", q, shape)
    if selected.dtype is not torch.int32 or selected.ndim != 3 or not selected.is_contiguous() or \
            selected.shape[:2] != (tokens, hkv):
        raise ValueError("selected must be a contiguous int32 [tokens, num_kv_heads, budget] tensor")
    batch, max_blocks = _paged_rows(seq_lens, block_table, query_start)
    device = _cuda(q, means, mean_scales, seq_lens, block_table, selected, query_start)
    handle = _stream(stream, device)
    if tokens == 0:
        return
    lib = _lib.load()
    buf = _scratch(workspace, lib.w8a8_fp8_kv_select_blocks_workspace_size(tokens, hkv, max_blocks), "fp8_select", device, stream,
                   handle, q)
    check(lib.w8a8_fp8_kv_select_blocks(
        q.data_ptr(), _fkind(q), tokens, hq, hkv, d, *qs, means.data_ptr(), mean_scales.data_ptr(), nb, block_size,
        block_table.data_ptr(), max_blocks, seq_lens.data_ptr(), _ptr(query_start), batch, max_query_len, first_blocks, last_blocks,
        selected.shape[2], selected.data_ptr(), buf.data_ptr(), buf.numel() * buf.element_size(), handle))


def fp8_kv_sparse_attention_workspace_size(tokens: int, num_q_heads: int, num_kv_heads: int, head_dim: int, budget: int,
                                           block_size: int) -> int:
    return int(_lib.load().w8a8_fp8_kv_sparse_attention_workspace_size(tokens, num_q_heads, num_kv_heads, head_dim, budget,
                                                                       block_size))


@functools.lru_cache(maxsize=4096)
def _fp8_sparse_need(device_index: int, *sizes: int) -> int:
    """The same, looked up once for a device and sizes (it depends on nothing else)."""
    return fp8_kv_sparse_attention_workspace_size(*sizes)


def fp8_kv_sparse_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, seq_lens: torch.Tensor,
                            block_table: torch.Tensor, selected: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                            out: torch.Tensor, query_start: torch.Tensor | None = None, max_query_len: int = 1,
                            sm_scale: float | None = None, workspace=None, stream=None) -> None:
    """Attention of each new token over the blocks selected for it.

    selected: int32 [tokens, num_kv_heads, budget], columns of the block table
    (fp8_kv_select_blocks gives them); ones outside it are skipped, the tokens
    of a column named twice count twice.  A row sees the tokens of its columns
    up to its own position; one that sees none gives zeros.  The other
    arguments: as for fp8_kv_attention (workspace: of
    fp8_kv_sparse_attention_workspace_size())."""
    nb, bs, hkv, d = _fp8_caches(k_cache, v_cache)
    shape = q.shape
    if len(shape) != 3 or shape[2] != d:
        raise ValueError("q must be [tokens, num_q_heads, head_dim] with the cache's head_dim")
    tokens, hq, _ = shape
    qs, os_ = _heads("q", q, shape), _heads("out", out, shape)
    if selected.dtype is not torch.int32 or selected.ndim != 3 or not selected.is_contiguous() or \
            selected.shape[:2] != (tokens, hkv):
        raise ValueError("selected must be a contiguous int32 [tokens, num_kv_heads, budget] tensor")
    batch, max_blocks = _paged_rows(seq_lens, block_table, query_start)
    _one_scale(k_scale, v_scale)
    device = _cuda(q, k_cache, v_cache, seq_lens, block_table, selected, k_scale, v_scale, out, query_start)
    handle = _stream(stream, device)
    if tokens == 0:
        return
    budget = selected.shape[2]
    buf = _scratch(workspace, _fp8_sparse_need(device, tokens, hq, hkv, d, budget, bs), "fp8_sparse", device, stream, handle, q)
    if sm_scale is None:
        sm_scale = 1.0 / float(d) ** 0.5
    check(_lib.load().w8a8_fp8_kv_sparse_attention(
        q.data_ptr(), _fkind(q), tokens, hq, hkv, d, *qs, k_cache.data_ptr(), v_cache.data_ptr(), nb, bs, block_table.data_ptr(),
        max_blocks, seq_lens.data_ptr(), _ptr(query_start), batch, max_query_len, selected.data_ptr(), budget, k_scale.data_ptr(),
        v_scale.data_ptr(), sm_scale, out.data_ptr(), _fkind(out), *os_, buf.data_ptr(), buf.numel() * buf.element_size(), handle))
