"""Python binding of libmla_decode (argument marshalling only).

Every function here checks tensor dtypes/shapes, passes raw device pointers and sizes to
the C ABI declared in ``include/mla_decode.h`` and raises on a non-OK status.  All
computation happens in the library's CUDA kernels.  If the library has not been built,
the first call raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libmla_decode.so")

MLA_OK = 0
STATUS_NAMES = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED",
                3: "MLA_ERR_WORKSPACE", 4: "MLA_ERR_CUDA", 5: "MLA_ERR_INDEX",
                6: "MLA_ERR_TIMEOUT", 7: "MLA_ERR_RANGE"}
KV_BF16, KV_FP8 = 0, 1
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}

_lock = threading.Lock()
_lib = None


class MlaError(RuntimeError):
    def __init__(self, fn, status, text):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)} ({text})")
        self.status = status


def lib():
    """The loaded libmla_decode (ctypes.CDLL); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with `python -m mla_latent_kv_17_gb300.build`")
            L = ctypes.CDLL(LIB_PATH)
            P, I, I64, F, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                ctypes.c_size_t)
            L.mla_decode_workspace_size.argtypes = [I, I, I]
            L.mla_decode_workspace_size.restype = SZ
            L.mla_decode_plan.argtypes = [P, I, I, I, I, I, P, SZ, P]
            L.mla_decode_plan.restype = I
            L.mla_decode_plan_host.argtypes = [P, I, I, I, I, I, P, SZ]
            L.mla_decode_plan_host.restype = I
            L.mla_decode.argtypes = [P, SZ, P, P, P, I, I64, P, I, P, I, I, F, P, P, P]
            L.mla_decode.restype = I
            L.mla_decode_sparse.argtypes = [P, SZ, P, P, P, I64, P, I, P, P, I, I, I, F, P, P, P]
            L.mla_decode_sparse.restype = I
            L.mla_decode_static.argtypes = [P, P, P, I, I64, P, I, P, I, I, F, P, P, P, P]
            L.mla_decode_static.restype = I
            L.mla_cache_append.argtypes = [P, I, I64, P, I, P, P, P, I, P, P]
            L.mla_cache_append.restype = I
            L.mla_prefill_decompress.argtypes = [P, I, P, P, I, P, P, P, P]
            L.mla_prefill_decompress.restype = I
            L.mla_prefill_attention.argtypes = [P, P, P, P, P, I, I, F, P, P, P, P]
            L.mla_prefill_attention.restype = I
            L.mla_topk_select.argtypes = [P, I64, I, P, I, I, P, P, P]
            L.mla_topk_select.restype = I
            L.mla_absorb_query.argtypes = [P, P, I, I, P, P, P]
            L.mla_absorb_query.restype = I
            L.mla_project_output.argtypes = [P, P, I, I, P, P, P]
            L.mla_project_output.restype = I
            L.mla_rope.argtypes = [P, I64, I64, I64, I, I, I, I, P, P, F, P, I64, I64, P, I64, I64, P]
            L.mla_rope.restype = I
            L.mla_rope_axes.argtypes = [P, I64, I64, I64, I, I, I, I, P, I64, I64, I, P, P, F, P, I64, I64, P, I64, I64, P]
            L.mla_rope_axes.restype = I
            L.mla_cache_write_axes.argtypes = [P, I, I64, P, I, I, P, P, P, I64, I64, P, F, P, P, I64, I64, I, P, I, F, P,
                                               P]
            L.mla_cache_write_axes.restype = I
            L.mla_cache_write.argtypes = [P, I, I64, P, I, I, P, P, P, I64, I64, P, F, P, P, I, F, P, P]
            L.mla_cache_write.restype = I
            L.mla_cache_read.argtypes = [P, I, I64, P, I, I, P, P, I64, P, I64, P, P]
            L.mla_cache_read.restype = I
            L.mla_decode_tree_workspace_size.argtypes = [I, I, I, I]
            L.mla_decode_tree_workspace_size.restype = SZ
            L.mla_decode_tree_plan.argtypes = [P, P, I, I, I, I, I, P, SZ, P]
            L.mla_decode_tree_plan.restype = I
            L.mla_decode_tree_plan_host.argtypes = [P, P, I, I, I, I, I, P, SZ]
            L.mla_decode_tree_plan_host.restype = I
            L.mla_decode_tree.argtypes = [P, SZ, P, P, P, I, I64, P, I, P, P, P, I, I, I, F, P, I, P, P]
            L.mla_decode_tree.restype = I
            L.mla_verify_draft.argtypes = [P, P, P, P, P, P, I, I, I, P, P, P, P, P]
            L.mla_verify_draft.restype = I
            L.mla_cross_workspace_size.argtypes = [I, I, I64, I]
            L.mla_cross_workspace_size.restype = SZ
            L.mla_cross_plan.argtypes = [P, P, I, I, I64, I64, I, I, P, SZ, P]
            L.mla_cross_plan.restype = I
            L.mla_cross_attention.argtypes = [P, SZ, P, P, P, P, P, I, I, I64, I64, F, P, P, P, I, P, P]
            L.mla_cross_attention.restype = I
            L.mla_token_logprobs.argtypes = [P, I, I64, I64, I, P, F, I, P, P, P, P, P, P, P]
            L.mla_token_logprobs.restype = I
            L.mla_decode_status.argtypes = [P, SZ, P]
            L.mla_decode_status.restype = I
            L.mla_decode_inject_stall.argtypes = [I]
            L.mla_decode_inject_stall.restype = I
            L.mla_decode_set_wait_limit.argtypes = [I64]
            L.mla_decode_set_wait_limit.restype = I
            L.mla_status_string.argtypes = [I]
            L.mla_status_string.restype = ctypes.c_char_p
            _lib = L
    return _lib


def _check(fn, st):
    if st != MLA_OK:
        raise MlaError(fn, st, lib().mla_status_string(st).decode())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _stream_of(ws, stream):
    return ctypes.c_void_p(ws._on_stream(stream, torch.cuda.current_device()))


def workspace_size(B: int, H: int, num_sms: int = 0) -> int:
    n = lib().mla_decode_workspace_size(int(B), int(H), int(num_sms))
    if n == 0:
        raise MlaError("mla_decode_workspace_size", 1, "invalid arguments")
    return int(n)


class _Memory:
    """A workspace's device memory, made (and its header zeroed) on the then current stream.  What calls
    on any other stream do with it comes after that, and after the work of that stream before it, which
    the memory may have served; and it is not handed out again before they are done.  (In a captured
    graph streams are ordered by the capture alone.)"""

    def _made(self):
        """To be called once self.buf is made."""
        dev = self.buf.get_device()
        with _on(dev):
            self._event = None if torch.cuda.is_current_stream_capturing() else torch.cuda.current_stream().record_event()
        self._known = {_raw(None, dev)}  # streams whose calls come after the making

    def _on_stream(self, stream, dev) -> int:
        """The handle of the stream that a call of this workspace goes to, as _raw()."""
        raw = _raw(stream, dev)
        if raw not in self._known:
            if stream is None:
                stream = torch.cuda.current_stream(dev)
            with torch.cuda.stream(stream):
                capturing = torch.cuda.is_current_stream_capturing()
            if self._event is not None and not capturing:  # (no event of one can be waited for in the other)
                stream.wait_event(self._event)
                self.buf.record_stream(stream)
                self._known.add(raw)
        return raw


class Workspace(_Memory):
    """Device workspace holding a plan, the split-KV partials and the status word."""

    def __init__(self, B: int, H: int, num_sms: int = 0, device=None):
        self.B, self.H = int(B), int(H)
        self.nbytes = workspace_size(B, H, num_sms)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8,
                               device=device or torch.device("cuda", torch.cuda.current_device()))
        self._made()
        self.topk = None

    def ptr(self):
        return _ptr(self.buf)


def _i32(t, name):
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    return t


def _kv_code(kv_dtype) -> int:
    if kv_dtype in ("bf16", KV_BF16):
        return KV_BF16
    if kv_dtype in ("fp8", KV_FP8):
        return KV_FP8
    raise ValueError(f"kv_dtype must be 'bf16' or 'fp8', not {kv_dtype!r}")


def plan(ws: Workspace, seq_lens=None, topk: int = 0, num_sms: int = 0, stream=None,
         kv_dtype="bf16") -> Workspace:
    """Build the split-KV plan for seq_lens (device int32 [B]) or for topk index slots;
    kv_dtype ('bf16' or 'fp8') is the cache layout the decode will read."""
    if seq_lens is not None:
        _i32(seq_lens, "seq_lens")
    st = lib().mla_decode_plan(_ptr(seq_lens), ws.B, ws.H, int(topk), _kv_code(kv_dtype), int(num_sms),
                               ws.ptr(), ws.nbytes, _stream_of(ws, stream))
    _check("mla_decode_plan", st)
    ws.topk = int(topk)
    return ws


def _outputs(B, H, device, out, lse):
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.float32, device=device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=device)
    if out.dtype != torch.float32 or out.shape != (B, H, 512) or not out.is_contiguous():
        raise ValueError("out must be contiguous fp32 [B,H,512]")
    if lse.dtype != torch.float32 or lse.shape != (B, H) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [B,H]")
    return out, lse


def _queries(q_nope, q_rope):
    B, H, d = q_nope.shape
    if d != 512 or q_nope.dtype != torch.bfloat16 or not q_nope.is_contiguous():
        raise ValueError("q_nope must be contiguous bf16 [B,H,512]")
    if q_rope.shape != (B, H, 64) or q_rope.dtype != torch.bfloat16 or not q_rope.is_contiguous():
        raise ValueError("q_rope must be contiguous bf16 [B,H,64]")
    return B, H


def decode(ws: Workspace, q_nope, q_rope, cache, block_table, seq_lens, softmax_scale: float,
           out=None, lse=None, stream=None):
    """Dense decode; the cache is bf16 [P,64,576] or uint8 FP8 records [P,64,656]."""
    B, H = _queries(q_nope, q_rope)
    _i32(block_table, "block_table")
    _i32(seq_lens, "seq_lens")
    if cache.dtype == torch.bfloat16 and cache.shape[1:] == (64, 576):
        kv = KV_BF16
    elif cache.dtype == torch.uint8 and cache.shape[1:] == (64, 656):
        kv = KV_FP8
    else:
        raise ValueError("cache must be bf16 [P,64,576] or uint8 [P,64,656]")
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    out, lse = _outputs(B, H, q_nope.device, out, lse)
    st = lib().mla_decode(ws.ptr(), ws.nbytes, _ptr(q_nope), _ptr(q_rope), _ptr(cache), kv,
                          cache.shape[0], _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
                          B, H, float(softmax_scale), _ptr(out), _ptr(lse), _stream_of(ws, stream))
    _check("mla_decode", st)
    return out, lse


def cache_append(cache, block_table, positions, c_kv, k_rope, device_status=None, stream=None):
    """Writes request b's new token (c_kv [B,512], k_rope [B,64], bf16) at position positions[b]
    (int32 [B], < 0 skips) of the paged cache: bf16 [P,64,576] or uint8 FP8 records [P,64,656]
    (quantised on the way in).  device_status: optional int32 [1] tensor for MLA_ERR_INDEX."""
    _i32(block_table, "block_table")
    _i32(positions, "positions")
    if cache.dtype == torch.bfloat16 and cache.shape[1:] == (64, 576):
        kv = KV_BF16
    elif cache.dtype == torch.uint8 and cache.shape[1:] == (64, 656):
        kv = KV_FP8
    else:
        raise ValueError("cache must be bf16 [P,64,576] or uint8 [P,64,656]")
    B = positions.shape[0]
    for t, n, d in ((c_kv, "c_kv", 512), (k_rope, "k_rope", 64)):
        if t.dtype != torch.bfloat16 or t.shape != (B, d) or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{n} must be contiguous CUDA bf16 [{B},{d}]")
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    if device_status is not None:
        _i32(device_status, "device_status")
    st = lib().mla_cache_append(_ptr(cache), kv, cache.shape[0], _ptr(block_table), block_table.shape[1],
                                _ptr(positions), _ptr(c_kv), _ptr(k_rope), B, _ptr(device_status),
                                _stream(stream))
    _check("mla_cache_append", st)
    return cache


def topk_select(scores, seq_lens, k: int, indices=None, device_status=None, stream=None):
    """DSA indices int32 [B,k]: per request the k best-scored positions of [0, seq_len)
    (scores fp32 [B,Lmax], ties to the lower position), ascending, padded with -1."""
    if scores.dtype != torch.float32 or scores.dim() != 2 or not scores.is_cuda or scores.stride(1) != 1:
        raise ValueError("scores must be a CUDA fp32 [B,Lmax] tensor with unit column stride")
    _i32(seq_lens, "seq_lens")
    B, Lmax = scores.shape
    if indices is None:
        indices = torch.empty((B, k), dtype=torch.int32, device=scores.device)
    elif indices.dtype != torch.int32 or indices.shape != (B, k) or not indices.is_contiguous():
        raise ValueError(f"indices must be contiguous int32 [{B},{k}]")
    if device_status is not None:
        _i32(device_status, "device_status")
    st = lib().mla_topk_select(_ptr(scores), scores.stride(0), Lmax, _ptr(seq_lens), B, int(k), _ptr(indices),
                               _ptr(device_status), _stream(stream))
    _check("mla_topk_select", st)
    return indices


def _bf16(t, shape, name):
    if t.dtype != torch.bfloat16 or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be contiguous CUDA bf16 {list(shape)}")


def prefill_decompress(entries, w_uk, w_uv, k_nope=None, v=None, device_status=None, stream=None):
    """Per-head keys and values of a sequence: entries bf16 [L,576] (latent | RoPE key) ->
    k_nope, v bf16 [H,L,128] with k_nope[h,t] = w_uk[h] @ c_t and v[h,t] = w_uv[h] @ c_t."""
    if entries.dim() != 2:
        raise ValueError("entries must be [L,576]")
    L = entries.shape[0]
    H = w_uk.shape[0]
    _bf16(entries, (L, 576), "entries")
    _weights(w_uk, H, "w_uk")
    _weights(w_uv, H, "w_uv")
    if k_nope is None:
        k_nope = torch.empty((H, L, 128), dtype=torch.bfloat16, device=entries.device)
    if v is None:
        v = torch.empty((H, L, 128), dtype=torch.bfloat16, device=entries.device)
    _bf16(k_nope, (H, L, 128), "k_nope")
    _bf16(v, (H, L, 128), "v")
    if device_status is not None:
        _i32(device_status, "device_status")
    st = lib().mla_prefill_decompress(_ptr(entries), L, _ptr(w_uk), _ptr(w_uv), H, _ptr(k_nope), _ptr(v),
                                      _ptr(device_status), _stream(stream))
    _check("mla_prefill_decompress", st)
    return k_nope, v


def prefill_attention(q_nope, q_rope, entries, k_nope, v, softmax_scale: float, out=None, lse=None,
                      device_status=None, stream=None):
    """Causal prefill attention (non-absorbed): q_nope bf16 [L,H,128], q_rope bf16 [L,H,64],
    entries bf16 [L,576], k_nope / v bf16 [H,L,128] -> out fp32 [L,H,128], lse fp32 [L,H]."""
    if q_nope.dim() != 3:
        raise ValueError("q_nope must be [L,H,128]")
    L, H = q_nope.shape[0], q_nope.shape[1]
    _bf16(q_nope, (L, H, 128), "q_nope")
    _bf16(q_rope, (L, H, 64), "q_rope")
    _bf16(entries, (L, 576), "entries")
    _bf16(k_nope, (H, L, 128), "k_nope")
    _bf16(v, (H, L, 128), "v")
    if out is None:
        out = torch.empty((L, H, 128), dtype=torch.float32, device=q_nope.device)
    if lse is None:
        lse = torch.empty((L, H), dtype=torch.float32, device=q_nope.device)
    if device_status is not None:
        _i32(device_status, "device_status")
    st = lib().mla_prefill_attention(_ptr(q_nope), _ptr(q_rope), _ptr(entries), _ptr(k_nope), _ptr(v), L, H,
                                     float(softmax_scale), _ptr(out), _ptr(lse), _ptr(device_status),
                                     _stream(stream))
    _check("mla_prefill_attention", st)
    return out, lse


def _weights(w, H, name):
    if w.dtype != torch.bfloat16 or w.shape != (H, 128, 512) or not w.is_contiguous() or not w.is_cuda:
        raise ValueError(f"{name} must be contiguous CUDA bf16 [{H},128,512]")


def absorb_query(q_c, w_uk, q_nope=None, device_status=None, stream=None):
    """Absorbed decode query q_nope[b,h] = q_c[b,h] @ w_uk[h] (bf16 [B,H,128] x bf16 [H,128,512]
    -> bf16 [B,H,512], fp32 accumulation)."""
    if q_c.dtype != torch.bfloat16 or q_c.dim() != 3 or q_c.shape[2] != 128 or not q_c.is_contiguous() \
            or not q_c.is_cuda:
        raise ValueError("q_c must be contiguous CUDA bf16 [B,H,128]")
    B, H = q_c.shape[0], q_c.shape[1]
    _weights(w_uk, H, "w_uk")
    if q_nope is None:
        q_nope = torch.empty((B, H, 512), dtype=torch.bfloat16, device=q_c.device)
    elif q_nope.dtype != torch.bfloat16 or q_nope.shape != (B, H, 512) or not q_nope.is_contiguous():
        raise ValueError(f"q_nope must be contiguous bf16 [{B},{H},512]")
    if device_status is not None:
        _i32(device_status, "device_status")
    st = lib().mla_absorb_query(_ptr(q_c), _ptr(w_uk), B, H, _ptr(q_nope), _ptr(device_status), _stream(stream))
    _check("mla_absorb_query", st)
    return q_nope


def project_output(out, w_uv, y=None, device_status=None, stream=None):
    """Per-head value projection y[b,h] = w_uv[h] @ out[b,h] (fp32 [B,H,512], bf16 [H,128,512]
    -> fp32 [B,H,128]; the latent output enters the bf16 MMA rounded to bf16)."""
    if out.dtype != torch.float32 or out.dim() != 3 or out.shape[2] != 512 or not out.is_contiguous() \
            or not out.is_cuda:
        raise ValueError("out must be contiguous CUDA fp32 [B,H,512]")
    B, H = out.shape[0], out.shape[1]
    _weights(w_uv, H, "w_uv")
    if y is None:
        y = torch.empty((B, H, 128), dtype=torch.float32, device=out.device)
    elif y.dtype != torch.float32 or y.shape != (B, H, 128) or not y.is_contiguous():
        raise ValueError(f"y must be contiguous fp32 [{B},{H},128]")
    if device_status is not None:
        _i32(device_status, "device_status")
    st = lib().mla_project_output(_ptr(out), _ptr(w_uv), B, H, _ptr(y), _ptr(device_status), _stream(stream))
    _check("mla_project_output", st)
    return y


def decode_sparse(ws: Workspace, q_nope, q_rope, cache, block_table, seq_lens, indices,
                  softmax_scale: float, out=None, lse=None, stream=None):
    """Token-sparse decode over indices [B,topk] (int32, -1 = padding); bf16 cache."""
    B, H = _queries(q_nope, q_rope)
    _i32(block_table, "block_table")
    _i32(seq_lens, "seq_lens")
    _i32(indices, "indices")
    if cache.dtype != torch.bfloat16 or cache.shape[1:] != (64, 576) or not cache.is_contiguous():
        raise ValueError("cache must be contiguous bf16 [P,64,576]")
    out, lse = _outputs(B, H, q_nope.device, out, lse)
    st = lib().mla_decode_sparse(ws.ptr(), ws.nbytes, _ptr(q_nope), _ptr(q_rope), _ptr(cache),
                                 cache.shape[0], _ptr(block_table), block_table.shape[1],
                                 _ptr(seq_lens), _ptr(indices), indices.shape[1], B, H,
                                 float(softmax_scale), _ptr(out), _ptr(lse), _stream_of(ws, stream))
    _check("mla_decode_sparse", st)
    return out, lse


def decode_static(q_nope, q_rope, cache, block_table, seq_lens, softmax_scale: float,
                  out=None, lse=None, device_status=None, stream=None):
    """Dense plan + decode + merge with the library's fixed device scratch: no workspace
    argument and no allocation inside the call.  device_status: optional int32 CUDA
    tensor [1] that receives the call's device-side status word."""
    B, H = _queries(q_nope, q_rope)
    _i32(block_table, "block_table")
    _i32(seq_lens, "seq_lens")
    if cache.dtype == torch.bfloat16 and cache.shape[1:] == (64, 576):
        kv = KV_BF16
    elif cache.dtype == torch.uint8 and cache.shape[1:] == (64, 656):
        kv = KV_FP8
    else:
        raise ValueError("cache must be bf16 [P,64,576] or uint8 [P,64,656]")
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    out, lse = _outputs(B, H, q_nope.device, out, lse)
    if device_status is not None:
        _i32(device_status, "device_status")
    st = lib().mla_decode_static(_ptr(q_nope), _ptr(q_rope), _ptr(cache), kv, cache.shape[0],
                                 _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B, H,
                                 float(softmax_scale), _ptr(out), _ptr(lse), _ptr(device_status),
                                 _stream(stream))
    _check("mla_decode_static", st)
    return out, lse


def set_wait_limit(cycles: int = 0) -> None:
    """Limit of every pipeline wait of the decode kernel, and of cross_attention's long ones (more there
    for many keys), in SM clock cycles, for later calls (0 restores the default of about two seconds)."""
    _check("mla_decode_set_wait_limit", lib().mla_decode_set_wait_limit(int(cycles)))


def inject_stall(enable: bool) -> None:
    """Test hook: while enabled, decode and cross_attention calls make their MMA issuer wait on a barrier that
    nothing completes, so that the wait runs out (MLA_ERR_TIMEOUT) without any fault."""
    _check("mla_decode_inject_stall", lib().mla_decode_inject_stall(1 if enable else 0))


def status(ws: Workspace, stream=None) -> int:
    """Synchronise and return (and clear) the device-side status code of the workspace."""
    return int(lib().mla_decode_status(ws.ptr(), ws.nbytes, _stream_of(ws, stream)))


# ---- several tokens per request: rotary positions, cache write and read, verification ----
# These take tensors of any one CUDA device (the launch goes to that device's current stream,
# or to `stream`) and allocate the outputs they are not given.

# (A small call is bound by this file: tensors are checked by their device's number, pointers
# and the stream pass as plain integers.)

def _device_of(names, first, *others):
    """The number of the CUDA device that all given tensors (or None) live on; `first` decides."""
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            dev = -1
            break
    if dev < 0:
        for name, t in zip(names.split(), (first, *others)):
            if t is not None and not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
        raise ValueError("arguments are on different devices")
    return dev


class _Same:
    """Stands for torch.cuda.device(d) where d is the current device already."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_SAME = _Same()


def _on(dev: int):
    return _SAME if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _raw(stream, dev: int) -> int:
    """The handle of `stream`, or of the device's current stream (asked for without building the
    Stream object, a microsecond of a small call)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _at(t) -> int:
    return 0 if t is None else t.data_ptr()


def _new(like, shape, dtype, stream):
    """An output on `like`'s device.  What a given stream writes is allocated on that stream (memory
    of the current one may still be in use by work queued there) and recorded on the current one,
    where it will be read."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    reader = torch.cuda.current_stream(like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(reader)
    return t


def _ints(t, shape, name):
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 {list(shape)}")


def _status_word(t):
    if t is not None and (t.dtype != torch.int32 or t.numel() < 1 or not t.is_contiguous()):
        raise ValueError("device_status must be a contiguous int32 tensor")


def _layout(layout) -> int:
    try:
        return ROPE_LAYOUTS[layout]
    except (KeyError, TypeError):
        raise ValueError(f"layout must be 'interleaved' or 'half', not {layout!r}") from None


def _freqs(freqs, d_rot):
    if freqs.dtype != torch.float64 or freqs.shape != (d_rot // 2,) or not freqs.is_contiguous():
        raise ValueError(f"freqs must be contiguous float64 [{d_rot // 2}]")


def rope_frequencies(d_rot: int = 64, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained_length: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """(freqs float64 [d_rot/2] in radians per position, mscale) for rope() and cache_write().

    f_j = base^(-2j/d_rot), stretched for contexts beyond the trained length by `factor`:
    'none'; 'linear' (f / factor: positions interpolated); 'ntk' (base * factor^(d/(d-2)): the
    highest frequency kept, the lowest divided by factor); 'yarn' (frequencies that turn more
    than beta_fast times over the trained length kept, those below beta_slow turns divided by
    factor, a linear ramp over j between; mscale = 0.1 ln factor + 1 on the rotated values, of
    queries and keys alike).
    """
    import math
    if d_rot < 2 or d_rot % 2 or not base > 1.0 or not (math.isfinite(factor) and factor >= 1.0):
        raise ValueError("d_rot must be even and >= 2, base > 1, factor finite and >= 1")
    j = torch.arange(d_rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * j / d_rot)
    mscale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "ntk":
        if d_rot < 4:
            raise ValueError("'ntk' needs d_rot >= 4")
        f = (base * factor ** (d_rot / (d_rot - 2.0))) ** (-2.0 * j / d_rot)
    elif scaling == "yarn":
        if trained_length < 1 or not beta_fast > beta_slow > 0:
            raise ValueError("'yarn' needs trained_length >= 1 and beta_fast > beta_slow > 0")

        def place(turns):  # the j whose frequency makes that many turns over the trained length
            return d_rot * math.log(trained_length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        lo, hi = max(math.floor(place(beta_fast)), 0), min(math.ceil(place(beta_slow)), d_rot - 1)
        divided = ((j - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        f = f / factor * divided + f * (1.0 - divided)
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling != "none":
        raise ValueError(f"scaling must be 'none', 'linear', 'ntk' or 'yarn', not {scaling!r}")
    return f.to(device if device is not None else "cuda"), mscale


def rope_axes(sections, order: str = "blocks") -> bytes:
    """The axis of each pair of a rotated part, for rope() and cache_write() of tokens with a position per
    axis: sections[x] pairs turn by axis x (time, height, width, ...; 1 to 4 axes, len(freqs) pairs in
    all).  order 'blocks': one axis's pairs after the other's; 'interleaved': a pair of each axis in turn
    as long as the axis has pairs left."""
    counts = [int(n) for n in sections]
    if not 1 <= len(counts) <= 4 or any(n != m or n < 0 for n, m in zip(counts, sections)) or sum(counts) < 1:
        raise ValueError("sections must be 1 to 4 whole numbers of pairs, not all of them 0")
    if order == "blocks":
        return bytes(x for x, n in enumerate(counts) for _ in range(n))
    if order == "interleaved":
        return bytes(x for i in range(max(counts)) for x, n in enumerate(counts) if i < n)
    raise ValueError(f"order must be 'blocks' or 'interleaved', not {order!r}")


def _axis_places(positions, axes, N, pairs, name):
    """The number of axes after checks of positions [N,A] and of the pairs' axes."""
    if type(axes) is not bytes or len(axes) != pairs:
        raise ValueError(f"axes must be the bytes that rope_axes gives, of {pairs} pairs")
    if positions.dtype != torch.int32 or positions.dim() != 2 or positions.shape[0] != N or positions.shape[1] < 1:
        raise ValueError(f"{name} must be int32 [{N},axes]")
    return positions.shape[1]


def rope(x, positions, freqs, layout="interleaved", mscale: float = 1.0, out_pass=None, out_rot=None,
         copy_pass: bool = True, stream=None, axes=None):
    """Rotary positions of the last 2 len(freqs) values of every head: x bf16 [N,H,D] (rows of any
    stride, values adjacent), positions int32 [N], freqs float64 -> (x[..., :D-d] copied, the rotated
    part), bf16 [N,H,D-d] and [N,H,d]; None for the first part where it is empty or copy_pass=False
    leaves it out.  out_rot may be x[..., D-d:] itself (rotation in place).  With axes (from rope_axes)
    a token has a position per axis, positions int32 [N,A] (any strides), and pair j turns by that of
    axes[j]."""
    if x.dtype != torch.bfloat16 or x.dim() != 3:
        raise ValueError("x must be bf16 [N,H,D]")
    N, H, D = x.shape
    d_rot = 2 * freqs.numel()
    d_pass = D - d_rot
    if d_rot < 2 or d_pass < 0:
        raise ValueError(f"x has {D} values per head, freqs turns {d_rot}")
    dev = _device_of("x positions freqs out_pass out_rot", x, positions, freqs, out_pass, out_rot)
    if axes is None:
        _ints(positions, (N,), "positions")
    else:
        num_axes = _axis_places(positions, axes, N, d_rot // 2, "positions")
    _freqs(freqs, d_rot)
    code = _layout(layout)
    with _on(dev):
        ps = rs = (H * d_rot, d_rot, 1)
        if not copy_pass or d_pass == 0:
            out_pass = None
        elif out_pass is None:
            out_pass = _new(x, (N, H, d_pass), torch.bfloat16, stream)
            ps = (H * d_pass, d_pass, 1)
        elif out_pass.dtype != torch.bfloat16 or out_pass.shape != (N, H, d_pass):
            raise ValueError(f"out_pass must be bf16 [{N},{H},{d_pass}]")
        else:
            ps = out_pass.stride()
        if out_rot is None:
            out_rot = _new(x, (N, H, d_rot), torch.bfloat16, stream)
        elif out_rot.dtype != torch.bfloat16 or out_rot.shape != (N, H, d_rot):
            raise ValueError(f"out_rot must be bf16 [{N},{H},{d_rot}]")
        else:
            rs = out_rot.stride()
        xs = x.stride()
        if N == 0 or H == 0:
            return out_pass, out_rot
        if (xs[2] != 1 and D > 1) or rs[2] != 1 or (ps[2] != 1 and d_pass > 1):
            raise ValueError("x, out_pass and out_rot must have unit stride within a row")
        if axes is None:
            st = lib().mla_rope(x.data_ptr(), xs[0], xs[1], N, H, d_pass, d_rot, code, positions.data_ptr(),
                                freqs.data_ptr(), mscale, _at(out_pass), ps[0], ps[1], out_rot.data_ptr(), rs[0],
                                rs[1], _raw(stream, dev))
        else:
            at = positions.stride()
            st = lib().mla_rope_axes(x.data_ptr(), xs[0], xs[1], N, H, d_pass, d_rot, code, positions.data_ptr(), at[0],
                                     at[1], num_axes, axes, freqs.data_ptr(), mscale, _at(out_pass), ps[0], ps[1],
                                     out_rot.data_ptr(), rs[0], rs[1], _raw(stream, dev))
    if st:
        _check("mla_rope" if axes is None else "mla_rope_axes", st)
    return out_pass, out_rot


def _cache_kind(cache) -> int:
    shape = cache.shape
    width = shape[2] if len(shape) == 3 and shape[1] == 64 else 0
    if width == 576 and cache.dtype == torch.bfloat16:
        kv = KV_BF16
    elif width == 656 and cache.dtype == torch.uint8:
        kv = KV_FP8
    else:
        raise ValueError("cache must be bf16 [P,64,576] or uint8 [P,64,656]")
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    return kv


def _tokens(block_table, requests, positions):
    """N after checks of the block table and the tokens' places."""
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous int32 [B,max_pages]")
    if positions.dim() != 1:
        raise ValueError("positions must be int32 [N]")
    N = positions.shape[0]
    _ints(positions, (N,), "positions")
    if requests is not None:
        _ints(requests, (N,), "requests")
    return N


def _entry_rows(t, N, name):
    if t.dtype != torch.bfloat16 or t.shape != (N, 576) or (N and t.stride(1) != 1):
        raise ValueError(f"{name} must be bf16 [{N},576] with unit stride within a row")
    return t.stride(0) if N > 1 else 576


def cache_write(cache, block_table, requests, positions, kv, freqs=None, rope_positions=None,
                layout="interleaved", mscale: float = 1.0, norm_weight=None, norm_eps: float = 1e-6,
                device_status=None, stream=None, axes=None):
    """Writes many tokens' entries: token n (kv bf16 [N,576]: latent | key) goes to position
    positions[n] (< 0 skips) of request requests[n] (None: request n) of the paged cache, bf16
    [P,64,576] or uint8 FP8 records [P,64,656] (quantised on the way in).  With norm_weight
    (bf16 [512]) the latent is RMS-normalised first; with freqs (float64 [32]) the key is rotated
    at rope_positions (None: positions).  With axes (from rope_axes, 32 pairs) as well, rope_positions
    is int32 [N,A], a position per axis (any strides).  device_status: optional int32 [1] for
    MLA_ERR_INDEX."""
    dev = _device_of("cache block_table requests positions kv freqs rope_positions norm_weight device_status", cache,
                     block_table, requests, positions, kv, freqs, rope_positions, norm_weight, device_status)
    kind = _cache_kind(cache)
    N = _tokens(block_table, requests, positions)
    stride = _entry_rows(kv, N, "kv")
    if freqs is not None:
        _freqs(freqs, 64)
    if axes is not None:
        if freqs is None or rope_positions is None:
            raise ValueError("axes without freqs or without rope_positions")
        num_axes = _axis_places(rope_positions, axes, N, 32, "rope_positions")
    elif rope_positions is not None:
        if freqs is None:
            raise ValueError("rope_positions without freqs")
        _ints(rope_positions, (N,), "rope_positions")
    if norm_weight is not None and (norm_weight.dtype != torch.bfloat16 or norm_weight.shape != (512,)
                                    or not norm_weight.is_contiguous()):
        raise ValueError("norm_weight must be contiguous bf16 [512]")
    _status_word(device_status)
    code = _layout(layout)
    with _on(dev):
        if axes is None:
            st = lib().mla_cache_write(
                cache.data_ptr(), kind, cache.shape[0], block_table.data_ptr(), block_table.shape[0],
                block_table.shape[1], _at(requests), positions.data_ptr(), kv.data_ptr(), stride, N, _at(norm_weight),
                norm_eps, _at(freqs), _at(rope_positions), code, mscale, _at(device_status), _raw(stream, dev))
        else:
            at = rope_positions.stride()
            st = lib().mla_cache_write_axes(
                cache.data_ptr(), kind, cache.shape[0], block_table.data_ptr(), block_table.shape[0],
                block_table.shape[1], _at(requests), positions.data_ptr(), kv.data_ptr(), stride, N, _at(norm_weight),
                norm_eps, freqs.data_ptr(), rope_positions.data_ptr(), at[0], at[1], num_axes, axes, code, mscale,
                _at(device_status), _raw(stream, dev))
    if st:
        _check("mla_cache_write" if axes is None else "mla_cache_write_axes", st)
    return cache


def cache_read(cache, block_table, requests, positions, entries=None, device_status=None, stream=None):
    """Reads many tokens' entries back: bf16 [N,576], row n = position positions[n] of request
    requests[n] (None: request n); FP8 records are dequantised.  Rows of skipped tokens (negative
    or unmapped positions) stay as they were in `entries` (undefined where it is allocated here)."""
    dev = _device_of("cache block_table requests positions entries device_status", cache, block_table, requests, positions,
                     entries, device_status)
    kind = _cache_kind(cache)
    N = _tokens(block_table, requests, positions)
    _status_word(device_status)
    with _on(dev):
        if entries is None:
            entries, stride = _new(cache, (N, 576), torch.bfloat16, stream), 576
        else:
            stride = _entry_rows(entries, N, "entries")
        st = lib().mla_cache_read(
            cache.data_ptr(), kind, cache.shape[0], block_table.data_ptr(), block_table.shape[0],
            block_table.shape[1], _at(requests), positions.data_ptr(), N, entries.data_ptr(), stride,
            _at(device_status), _raw(stream, dev))
    if st:
        _check("mla_cache_read", st)
    return entries


class TreeWorkspace(_Memory):
    """Device workspace of a tree attention over B requests of T drafted tokens and H heads: its
    plan, split-KV partials and status word (status() reads it)."""

    def __init__(self, B: int, T: int, H: int, num_sms: int = 0, device=None):
        self.B, self.T, self.H = int(B), int(T), int(H)
        dev = torch.device(device if device is not None else "cuda")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        with _on(dev.index):
            self.nbytes = int(lib().mla_decode_tree_workspace_size(self.B, self.T, self.H, int(num_sms)))
            if self.nbytes == 0:
                raise MlaError("mla_decode_tree_workspace_size", 1, "invalid arguments")
            self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=dev)
            self.buf[:256].zero_()  # no plan yet, no error
            self._made()

    def ptr(self):
        return _ptr(self.buf)


def plan_tree(ws: TreeWorkspace, seq_lens, tree_lens=None, num_sms: int = 0, stream=None, kv_dtype="bf16"):
    """Builds the plan of decode_tree for seq_lens and tree_lens (device int32 [B]; tree_lens
    None: T); kv_dtype ('bf16' or 'fp8') is the cache layout the attention will read."""
    dev = _device_of("seq_lens tree_lens workspace", seq_lens, tree_lens, ws.buf)
    _ints(seq_lens, (ws.B,), "seq_lens")
    if tree_lens is not None:
        _ints(tree_lens, (ws.B,), "tree_lens")
    with _on(dev):
        st = lib().mla_decode_tree_plan(seq_lens.data_ptr(), _at(tree_lens), ws.B, ws.T, ws.H, _kv_code(kv_dtype),
                                        num_sms, ws.buf.data_ptr(), ws.nbytes, ws._on_stream(stream, dev))
    if st:
        _check("mla_decode_tree_plan", st)
    return ws


def decode_tree(ws: TreeWorkspace, q_nope, q_rope, cache, block_table, seq_lens, tree_lens, tree_mask,
                softmax_scale: float, out=None, lse=None, out_dtype=torch.float32, with_lse: bool = True,
                stream=None):
    """Tree attention with the plan in ws: q_nope bf16 [B,T,H,512], q_rope bf16 [B,T,H,64]; cache bf16
    [P,64,576] or uint8 FP8 records [P,64,656], holding seq_lens[b] entries of request b, the last
    tree_lens[b] (None: T) of them its drafted tokens'; tree_mask int64 [B,T]: bit j of [b,i] set:
    token i attends drafted token j.  -> (out fp32 or bf16 [B,T,H,512], lse fp32 [B,T,H] or None);
    NaN for a token that attends a drafted one whose entry is not finite."""
    B, T, H = ws.B, ws.T, ws.H
    dev = _device_of("q_nope q_rope cache block_table seq_lens tree_lens tree_mask out lse workspace", q_nope, q_rope,
                     cache, block_table, seq_lens, tree_lens, tree_mask, out, lse, ws.buf)
    for t, d, name in ((q_nope, 512, "q_nope"), (q_rope, 64, "q_rope")):
        if t.dtype != torch.bfloat16 or t.shape != (B, T, H, d) or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous bf16 [{B},{T},{H},{d}]")
    kind = _cache_kind(cache)
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B \
            or not block_table.is_contiguous():
        raise ValueError(f"block_table must be contiguous int32 [{B},max_pages]")
    _ints(seq_lens, (B,), "seq_lens")
    if tree_lens is not None:
        _ints(tree_lens, (B,), "tree_lens")
    if tree_mask.dtype != torch.int64 or tree_mask.shape != (B, T) or not tree_mask.is_contiguous():
        raise ValueError(f"tree_mask must be contiguous int64 [{B},{T}]")
    with _on(dev):
        if out is not None:
            out_dtype = out.dtype
        if out_dtype not in (torch.float32, torch.bfloat16) or out is not None and (
                out.shape != (B, T, H, 512) or not out.is_contiguous()):
            raise ValueError(f"out must be contiguous fp32 or bf16 [{B},{T},{H},512]")
        if out is None:
            out = _new(q_nope, (B, T, H, 512), out_dtype, stream)
        if lse is None:
            if with_lse:
                lse = _new(q_nope, (B, T, H), torch.float32, stream)
        elif (lse.dtype != torch.float32 or lse.shape != (B, T, H) or not lse.is_contiguous()):
            raise ValueError(f"lse must be contiguous fp32 [{B},{T},{H}]")
        st = lib().mla_decode_tree(
            ws.buf.data_ptr(), ws.nbytes, q_nope.data_ptr(), q_rope.data_ptr(), cache.data_ptr(), kind,
            cache.shape[0], block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), _at(tree_lens),
            tree_mask.data_ptr(), B, T, H, softmax_scale, out.data_ptr(), 1 if out_dtype == torch.bfloat16 else 0,
            _at(lse), ws._on_stream(stream, dev))
    if st:
        _check("mla_decode_tree", st)
    return out, lse


def verify_draft(target_probs, draft_probs, draft_tokens, uniforms, parents=None, tree_lens=None,
                 device_status=None, stream=None):
    """Which drafted tokens stand, and the next token: target_probs fp32 [B,T+1,V] (row 0 after
    the last committed token, row i+1 after drafted token i), draft_probs fp32 [B,T,V] (or None:
    the draft is certain of its tokens), draft_tokens int32 [B,T], uniforms fp32 [B,T+1] in
    [0,1), parents int32 [B,T] (-1: the last committed token; None: a chain), tree_lens int32 [B]
    -> (num_accepted int32 [B], depths int32 [B,T]: place among the accepted tokens or -1,
    next_token int32 [B])."""
    dev = _device_of("target_probs draft_probs draft_tokens uniforms parents tree_lens device_status", target_probs,
                     draft_probs, draft_tokens, uniforms, parents, tree_lens, device_status)
    if draft_tokens.dim() != 2 or target_probs.dim() != 3:
        raise ValueError("draft_tokens must be int32 [B,T], target_probs fp32 [B,T+1,V]")
    B, T = draft_tokens.shape
    V = target_probs.shape[2]
    _ints(draft_tokens, (B, T), "draft_tokens")
    for t, shape, name in ((target_probs, (B, T + 1, V), "target_probs"), (draft_probs, (B, T, V), "draft_probs"),
                           (uniforms, (B, T + 1), "uniforms")):
        if t is not None and (t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous fp32 {list(shape)}")
    if parents is not None:
        _ints(parents, (B, T), "parents")
    if tree_lens is not None:
        _ints(tree_lens, (B,), "tree_lens")
    _status_word(device_status)
    with _on(dev):
        num = _new(draft_tokens, (B,), torch.int32, stream)
        depths = _new(draft_tokens, (B, T), torch.int32, stream)
        nxt = _new(draft_tokens, (B,), torch.int32, stream)
        st = lib().mla_verify_draft(
            target_probs.data_ptr(), _at(draft_probs), draft_tokens.data_ptr(), _at(parents), _at(tree_lens),
            uniforms.data_ptr(), B, T, V, num.data_ptr(), depths.data_ptr(), nxt.data_ptr(), _at(device_status),
            _raw(stream, dev))
    if st:
        _check("mla_verify_draft", st)
    return num, depths, nxt


class CrossWorkspace(_Memory):
    """Device workspace of a cross attention of B query runs of H heads, total_q query rows in all: its
    plan, partial results (up to 147 MiB on 152 SMs) and status word (status() reads it)."""

    def __init__(self, B: int, H: int, total_q: int, num_sms: int = 0, device=None):
        self.B, self.H, self.total_q, self.num_sms = int(B), int(H), int(total_q), int(num_sms)
        self.total_k = None
        dev = torch.device(device if device is not None else "cuda")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        with _on(dev.index):
            self.nbytes = int(lib().mla_cross_workspace_size(self.B, self.H, self.total_q, self.num_sms))
            if self.nbytes == 0:
                raise MlaError("mla_cross_workspace_size", 1, "invalid arguments")
            self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=dev)
            self.buf[:256].zero_()  # no plan yet, no error
            self._made()

    def ptr(self):
        return _ptr(self.buf)


def plan_cross(ws: CrossWorkspace, cu_q, cu_k, total_k: int, causal: bool = False, stream=None):
    """Builds the plan of cross_attention: run b's queries are rows cu_q[b] .. cu_q[b+1] of ws.total_q, its
    keys rows cu_k[b] .. cu_k[b+1] of total_k (device int32 [B+1]); causal: a run's queries are its
    last keys (the last one sees all of them, the one before all but the last)."""
    dev = _device_of("cu_q cu_k workspace", cu_q, cu_k, ws.buf)
    _ints(cu_q, (ws.B + 1,), "cu_q")
    _ints(cu_k, (ws.B + 1,), "cu_k")
    with _on(dev):
        st = lib().mla_cross_plan(cu_q.data_ptr(), cu_k.data_ptr(), ws.B, ws.H, ws.total_q, total_k, 1 if causal else 0,
                                  ws.num_sms, ws.buf.data_ptr(), ws.nbytes, ws._on_stream(stream, dev))
    if st:
        _check("mla_cross_plan", st)
    ws.total_k = total_k
    return ws


def cross_attention(ws: CrossWorkspace, q_nope, q_rope, entries, k_nope, v, softmax_scale: float, before=None, out=None,
                    lse=None, out_dtype=torch.float32, with_lse: bool = True, stream=None):
    """Attention of the planned query runs to their key runs: q_nope bf16 [Nq,H,128], q_rope bf16
    [Nq,H,64] and entries bf16 [Nk,576] (the keys' RoPE part; None for both: no positions), k_nope and v
    bf16 [H,Nk,128] (as prefill_decompress gives them).  before = (out fp32, lse fp32): an earlier
    result over other keys, which this one is joined with (they may be `out` and `lse` themselves).
    -> (out fp32 or bf16 [Nq,H,128], lse fp32 [Nq,H] or None); rows outside every run are left as
    they were (undefined where out is allocated here)."""
    before_out, before_lse = before if before is not None else (None, None)
    H, Nq = ws.H, ws.total_q
    dev = _device_of("q_nope q_rope entries k_nope v before before_lse out lse workspace", q_nope, q_rope, entries, k_nope,
                     v, before_out, before_lse, out, lse, ws.buf)
    Nk = ws.total_k
    if Nk is None:
        raise ValueError("the workspace holds no plan (plan_cross)")
    bf16, fp32 = torch.bfloat16, torch.float32
    for t, shape, dtype, name in (
            (q_nope, (Nq, H, 128), bf16, "q_nope"), (q_rope, (Nq, H, 64), bf16, "q_rope"),
            (entries, (Nk, 576), bf16, "entries"), (k_nope, (H, Nk, 128), bf16, "k_nope"), (v, (H, Nk, 128), bf16, "v"),
            (before_out, (Nq, H, 128), fp32, "before's out"), (before_lse, (Nq, H), fp32, "before's lse")):
        if t is not None and (t.dtype != dtype or t.shape != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous {'bf16' if dtype == bf16 else 'fp32'} {list(shape)}")
    if (q_rope is None) != (entries is None):
        raise ValueError("q_rope and entries: both or neither")
    if (before_out is None) != (before_lse is None):
        raise ValueError("before must hold out and lse")
    with _on(dev):
        if out is not None:
            out_dtype = out.dtype
        if out_dtype not in (fp32, bf16) or out is not None and (out.shape != (Nq, H, 128) or not out.is_contiguous()):
            raise ValueError(f"out must be contiguous fp32 or bf16 [{Nq},{H},128]")
        if out is None:
            out = _new(q_nope, (Nq, H, 128), out_dtype, stream)
        if lse is None:
            if with_lse:
                lse = _new(q_nope, (Nq, H), fp32, stream)
        elif lse.dtype != fp32 or lse.shape != (Nq, H) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous fp32 [{Nq},{H}]")
        st = lib().mla_cross_attention(
            ws.buf.data_ptr(), ws.nbytes, q_nope.data_ptr(), _at(q_rope), _at(entries), k_nope.data_ptr(), v.data_ptr(),
            ws.B, H, Nq, Nk, softmax_scale, _at(before_out), _at(before_lse), out.data_ptr(),
            1 if out_dtype == bf16 else 0, _at(lse), ws._on_stream(stream, dev))
    if st:
        _check("mla_cross_attention", st)
    return out, lse


_LOGITS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def token_logprobs(logits, tokens, top: int = 0, scale: float = 1.0, device_status=None, stream=None):
    """Scores of given tokens: logits bf16, fp16 or fp32 [N,V] (rows of any stride; -inf masks a token),
    tokens int32 [N] (negative: none), scale = 1 / temperature -> (logprob fp32 [N], entropy fp32 [N],
    rank int32 [N]: 0 for the best, top_tokens int32 [N,top] best first, top_logprobs fp32 [N,top]; None
    for the last two where top is 0).  device_status: optional int32 [1] for MLA_ERR_INDEX."""
    dev = _device_of("logits tokens device_status", logits, tokens, device_status)
    kind = _LOGITS.get(logits.dtype)
    if kind is None or logits.dim() != 2:
        raise ValueError("logits must be bf16, fp16 or fp32 [N,V]")
    N, V = logits.shape
    row, col = logits.stride()
    if col != 1 and V > 1:
        raise ValueError("logits must have unit stride within a row")
    _ints(tokens, (N,), "tokens")
    _status_word(device_status)
    with _on(dev):
        logprob = _new(logits, (N,), torch.float32, stream)
        entropy = _new(logits, (N,), torch.float32, stream)
        rank = _new(logits, (N,), torch.int32, stream)
        ids = alt = None
        if top > 0:
            ids = _new(logits, (N, top), torch.int32, stream)
            alt = _new(logits, (N, top), torch.float32, stream)
        st = lib().mla_token_logprobs(
            logits.data_ptr(), kind, row, N, V, tokens.data_ptr(), scale, top, logprob.data_ptr(), entropy.data_ptr(),
            rank.data_ptr(), _at(ids), _at(alt), _at(device_status), _raw(stream, dev))
    if st:
        _check("mla_token_logprobs", st)
    return logprob, entropy, rank, ids, alt


def plan_tree_host(seq_lens, tree_lens, B: int, T: int, H: int, num_sms: int = 148, kv_dtype="bf16"):
    """Host twin of the tree planner: the plan bytes (numpy uint8) for host lengths."""
    import numpy as np
    n = lib().mla_decode_tree_workspace_size(int(B), int(T), int(H), int(num_sms))
    buf = np.zeros(n, dtype=np.uint8)
    ints = [None if x is None else np.ascontiguousarray(np.asarray(x, dtype=np.int32)) for x in (seq_lens, tree_lens)]
    ptrs = [None if x is None else x.ctypes.data_as(ctypes.c_void_p) for x in ints]
    _check("mla_decode_tree_plan_host", lib().mla_decode_tree_plan_host(
        *ptrs, int(B), int(T), int(H), _kv_code(kv_dtype), int(num_sms), buf.ctypes.data_as(ctypes.c_void_p), n))
    return buf


def plan_host(seq_lens, B: int, H: int, topk: int = 0, num_sms: int = 148, kv_dtype="bf16"):
    """Host twin of the planner: returns the plan bytes (numpy uint8) for host seq_lens."""
    import numpy as np
    n = lib().mla_decode_workspace_size(int(B), int(H), int(num_sms))
    buf = np.zeros(n, dtype=np.uint8)
    sl = None
    if seq_lens is not None:
        sl = np.ascontiguousarray(np.asarray(seq_lens, dtype=np.int32))
    st = lib().mla_decode_plan_host(
        sl.ctypes.data_as(ctypes.c_void_p) if sl is not None else None, int(B), int(H),
        int(topk), _kv_code(kv_dtype), int(num_sms), buf.ctypes.data_as(ctypes.c_void_p), n)
    _check("mla_decode_plan_host", st)
    return buf
