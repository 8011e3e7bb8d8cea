"""Serving operators next to the quantized projections: a paged 8-bit cache with the attention that
reads it, and low-rank adapters of many requests beside a shared projection.  As in the package's
other calls, only arguments are marshalled here; every step runs in the library's HIP kernels.

    cache = KVCache.allocate(num_pages, 16, kv_heads=8, head_dim=128, device="cuda")
    q = cache.append(k, v, page_table, start, cu, max_new=1, q=q, cos=cos, sin=sin)
    o = cache.attention(q, page_table, start + 1, cu, max_q=1)
    y = h.gemm(x); bank.add(y, x, ids, out=y)

Batches are packed: the tokens of sequence b are rows cu[b] .. cu[b + 1] of every packed tensor.
Tables, lengths and ids are int32 tensors on the GPU and are not copied to the host; entries outside
their range are treated as absent (include/gptq_mi355x.h says how at each call).
"""
from __future__ import annotations

import ctypes

import torch

from . import BF16, F16, F32, GPTQError, _OnStream, load_library

__all__ = ["KVCache", "LoraBank"]

_CODES = {torch.float16: F16, torch.bfloat16: BF16}
_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", _P), ("v_codes", _P), ("k_scale", _P), ("v_scale", _P), ("num_pages", _I64),
                ("kv_heads", _I32), ("page_size", _I32), ("head_dim", _I32), ("reserved", _I32)]


class _Batch(ctypes.Structure):
    _fields_ = [("page_table", _P), ("at", _P), ("cu", _P), ("rows", _I64), ("batch", _I32), ("table_width", _I32),
                ("max_rows", _I32), ("reserved", _I32)]


class _Rope(ctypes.Structure):
    _fields_ = [("cos", _P), ("sin", _P), ("rows", _I32), ("dim", _I32), ("interleaved", _I32), ("reserved", _I32)]


class _Attention(ctypes.Structure):
    _fields_ = [("q_heads", _I32), ("dtype", _I32), ("scale", ctypes.c_float), ("causal", _I32), ("window", _I32),
                ("max_kv", _I32), ("q_stride", _I64), ("out_stride", _I64)]


class _Bank(ctypes.Structure):
    _fields_ = [("a", _P), ("b", _P), ("scale", _P), ("adapters", _I32), ("rank", _I32), ("in_features", _I32),
                ("out_features", _I32), ("dtype", _I32), ("reserved", _I32)]


class _Here:
    """The current stream of the tensors' device, when that device is current: nothing to enter."""
    __slots__ = ("ptr",)

    def __init__(self, device):
        self.ptr = torch.cuda.current_stream(device).cuda_stream

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return None

    def keep(self, *tensors):
        pass


def _on(stream, device):
    if stream is None and device.index == torch.cuda.current_device():
        return _Here(device)
    return _OnStream(stream, device)


def _dtype(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float16 or bfloat16")
    return code


def _index(t, name, shape, device):
    if t.dtype is not torch.int32 or tuple(t.shape) != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)} on {device}")


def _packed(t, name, heads, dim, dtype, device):
    """A packed [rows, heads, dim] tensor with dense heads and rows 16 bytes aligned (copied if not)."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name} must be [rows, {heads}, {dim}]")
    if t.dtype is not dtype or t.device != device:
        raise TypeError(f"{name} must be {dtype} on {device}")
    return t if _strided(t) else t.clone(memory_format=torch.contiguous_format)


def _strided(t):
    s, rows, width = t.stride(), t.shape[0], t.shape[1] * t.shape[2]
    dense = s[2] == 1 and (t.shape[1] == 1 or s[1] == t.shape[2])
    return dense and (rows < 2 or (s[0] >= width and s[0] % 8 == 0)) and t.data_ptr() % 16 == 0


def _dense(t):
    """A contiguous 16-byte aligned tensor (copied if it is not)."""
    return t if t.is_contiguous() and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


def _row_stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


class KVCache:
    """One layer's keys and values in pages of 8-bit codes: codes int8 [pages, kv_heads, page_size,
    head_dim] and scales float32 [pages, kv_heads], value = code * scale.  The cache keeps the four
    tensors it is given; page sizes 16 to 256 (powers of two), head_dim 64 or 128."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale):
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [pages, kv_heads, page_size, head_dim]")
        for name, t, shape, dt in (("k_codes", k_codes, k_codes.shape, torch.int8),
                                   ("v_codes", v_codes, k_codes.shape, torch.int8),
                                   ("k_scale", k_scale, k_codes.shape[:2], torch.float32),
                                   ("v_scale", v_scale, k_codes.shape[:2], torch.float32)):
            if t.dtype != dt or t.shape != shape or not t.is_contiguous() or t.device != k_codes.device:
                raise ValueError(f"{name} must be a contiguous {dt} tensor of shape {list(shape)} on {k_codes.device}")
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k_codes.shape
        self.device = k_codes.device
        self._lib = load_library()
        self._c = _Cache(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                         self.num_pages, self.kv_heads, self.page_size, self.head_dim, 0)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def allocate(cls, num_pages, page_size, kv_heads, head_dim, device="cuda"):
        """A cache of zeros."""
        shape = (num_pages, kv_heads, page_size, head_dim)
        return cls(torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros(shape[:2], device=device), torch.zeros(shape[:2], device=device))

    def _batch(self, page_table, at, cu, rows, max_rows):
        n = cu.shape[0] - 1 if cu.dim() == 1 else -1
        if n < 0 or page_table.dim() != 2:
            raise ValueError("cu must be [batch + 1] and page_table [batch, pages]")
        _index(cu, "cu", (n + 1,), self.device)
        _index(at, "lengths", (n,), self.device)
        _index(page_table, "page_table", (n, page_table.shape[1]), self.device)
        return _Batch(page_table.data_ptr(), at.data_ptr(), cu.data_ptr(), rows, n, page_table.shape[1],
                      min(max_rows, rows), 0)

    def append(self, k, v, page_table, start, cu, *, max_new, q=None, cos=None, sin=None, interleaved=False,
               q_out=None, stream=None):
        """Append k and v [rows, kv_heads, head_dim] (fp16/bf16): row i of sequence b becomes its token
        start[b] + i; max_new is at least the rows of every sequence.  With cos and sin (float32
        [positions, rot / 2]) k is rotated at its position, and q [rows, q_heads, head_dim] too; the
        rotated q is returned (in q_out when given, which may be q).  Rotated pairs are halves of the
        first rot values, or neighbours when interleaved (gptq_kv_append)."""
        dt, device = k.dtype, self.device
        code = _dtype(k, "k")
        with _on(stream, device) as on:
            on.keep(k, v, q, q_out, page_table, start, cu, cos, sin, self.k_codes, self.v_codes, self.k_scale,
                    self.v_scale)
            k = _packed(k, "k", self.kv_heads, self.head_dim, dt, device)
            v = _packed(v, "v", self.kv_heads, self.head_dim, dt, device)
            rows = k.shape[0]
            if v.shape[0] != rows:
                raise ValueError("k and v must have the same rows")
            batch = self._batch(page_table, start, cu, rows, max_new)
            rope = None
            if (cos is None) != (sin is None):
                raise ValueError("cos and sin come together")
            if cos is not None:
                if (cos.dtype is not torch.float32 or sin.dtype is not torch.float32 or cos.dim() != 2
                        or cos.shape != sin.shape or not cos.is_contiguous() or not sin.is_contiguous()
                        or cos.device != device or sin.device != device):
                    raise ValueError(f"cos and sin must be contiguous float32 [positions, rot / 2] tensors on {device}")
                rope = _Rope(cos.data_ptr(), sin.data_ptr(), cos.shape[0], 2 * cos.shape[1], int(bool(interleaved)), 0)
            q_args = (None, 0, 0, None, 0)
            if q is not None:
                if rope is None:
                    raise ValueError("q is taken to be rotated: pass cos and sin")
                if q.dim() != 3 or q.shape[0] != rows:
                    raise ValueError("q must have k's rows")
                heads = q.shape[1]
                if q_out is None:
                    q_out = torch.empty((rows, heads, self.head_dim), dtype=dt, device=device)
                elif q_out.shape != q.shape or q_out.dtype is not dt or q_out.device != device or not _strided(q_out):
                    raise ValueError("q_out must have q's shape and type, dense heads and aligned rows")
                q = _packed(q, "q", heads, self.head_dim, dt, device)
                q_args = (q.data_ptr(), _row_stride(q), heads, q_out.data_ptr(), _row_stride(q_out))
            st = self._lib.gptq_kv_append(self._ref, ctypes.byref(batch), k.data_ptr(), _row_stride(k), v.data_ptr(),
                                          _row_stride(v), *q_args, code, ctypes.byref(rope) if rope else None, on.ptr)
        if st:
            raise GPTQError(st, "gptq_kv_append", self._lib)
        return q_out if q is not None else None

    def read(self, page_table, start, cu, *, rows, max_rows, dtype=torch.float16, stream=None):
        """Cached tokens as values: (k, v) [rows, kv_heads, head_dim] of dtype (fp16/bf16/fp32), row i
        of sequence b being its token start[b] + i; rows is cu's last entry (gptq_kv_read)."""
        code = F32 if dtype is torch.float32 else _CODES.get(dtype)
        if code is None:
            raise TypeError("dtype must be float16, bfloat16 or float32")
        batch = self._batch(page_table, start, cu, rows, max_rows)
        with _on(stream, self.device) as on:
            on.keep(page_table, start, cu, self.k_codes, self.v_codes, self.k_scale, self.v_scale)
            out = torch.empty((2, rows, self.kv_heads, self.head_dim), dtype=dtype, device=self.device)
            k, v = out[0], out[1]
            st = self._lib.gptq_kv_read(self._ref, ctypes.byref(batch), k.data_ptr(), v.data_ptr(), code, on.ptr)
        if st:
            raise GPTQError(st, "gptq_kv_read", self._lib)
        return k, v

    def attention(self, q, page_table, kv_len, cu, *, max_q, max_kv=None, scale=None, causal=True, window=0, out=None,
                  workspace=None, stream=None):
        """softmax(scale * q k^T) v of q [rows, q_heads, head_dim] (fp16/bf16) over each sequence's
        kv_len[b] cached tokens, the queries' own included: the last of a sequence's rows stands at its
        last token.  max_q is at least the rows of every sequence, max_kv at least every length (default:
        what the table holds).  scale defaults to head_dim ** -0.5; window > 0 hides tokens that are
        window or more before the query.  A query that sees nothing gives zeros (gptq_kv_attention)."""
        device = self.device
        code = _dtype(q, "q")
        heads = q.shape[1] if q.dim() == 3 else 0
        rows = q.shape[0]
        with _on(stream, device) as on:
            on.keep(q, out, workspace, page_table, kv_len, cu, self.k_codes, self.v_codes, self.k_scale, self.v_scale)
            q = _packed(q, "q", heads, self.head_dim, q.dtype, device)
            if out is None:
                out = torch.empty((rows, heads, self.head_dim), dtype=q.dtype, device=device)
            elif out.shape != q.shape or out.dtype is not q.dtype or out.device != device or not _strided(out):
                raise ValueError("out must have q's shape and type, dense heads and aligned rows")
            batch = self._batch(page_table, kv_len, cu, rows, max_q)
            call = _Attention(heads, code, self.head_dim ** -0.5 if scale is None else scale, int(bool(causal)), window,
                              page_table.shape[1] * self.page_size if max_kv is None else max_kv, _row_stride(q),
                              _row_stride(out))
            b, c = ctypes.byref(batch), ctypes.byref(call)
            n = ctypes.c_size_t(0)
            st = self._lib.gptq_kv_attention_workspace_size(self._ref, b, c, ctypes.byref(n))
            if st:
                raise GPTQError(st, "gptq_kv_attention_workspace_size", self._lib)
            if workspace is None and n.value:
                workspace = torch.empty(n.value, dtype=torch.uint8, device=device)
            ws, size = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) \
                if workspace is not None else (None, 0)
            st = self._lib.gptq_kv_attention(self._ref, b, c, q.data_ptr(), out.data_ptr(), ws, size, on.ptr)
        if st:
            raise GPTQError(st, "gptq_kv_attention", self._lib)
        return out


class LoraBank:
    """The low-rank adapters of one projection: a [adapters, rank, K], b [adapters, N, rank]
    (fp16/bf16) and scale float32 [adapters].  Adapters of a smaller rank are padded with zeros."""

    def __init__(self, a, b, scale):
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise ValueError("a must be [adapters, rank, K] and b [adapters, N, rank]")
        if a.dtype != b.dtype or not a.is_contiguous() or not b.is_contiguous() or a.device != b.device:
            raise ValueError("a and b must be contiguous tensors of one type and device")
        if scale.dtype != torch.float32 or tuple(scale.shape) != (a.shape[0],) or not scale.is_contiguous() \
                or scale.device != a.device:
            raise ValueError("scale must be a contiguous float32 [adapters] tensor on the same device")
        self.a, self.b, self.scale = a, b, scale
        self.adapters, self.rank, self.K = a.shape
        self.N, self.dtype, self.device = b.shape[1], a.dtype, a.device
        self._lib = load_library()
        self._c = _Bank(a.data_ptr(), b.data_ptr(), scale.data_ptr(), self.adapters, self.rank, self.K, self.N,
                        _dtype(a, "a"), 0)
        self._ref = ctypes.addressof(self._c)

    def workspace_size(self, M) -> int:
        n = ctypes.c_size_t(0)
        st = self._lib.gptq_lora_workspace_size(self._ref, M, ctypes.byref(n))
        if st:
            raise GPTQError(st, "gptq_lora_workspace_size", self._lib)
        return n.value

    def add(self, y, x, ids, out=None, workspace=None, stream=None):
        """y + scale[ids] * B (A x) for each row: y [M, N] is the shared projection's output, x [M, K]
        its input, ids int32 [M] (an id outside [0, adapters): no adapter).  out may be y."""
        device = self.device
        if x.dim() != 2 or x.shape[1] != self.K or y.dim() != 2 or y.shape[1] != self.N or x.shape[0] != y.shape[0]:
            raise ValueError(f"x must be [M, {self.K}] and y [M, {self.N}]")
        if x.dtype is not self.dtype or y.dtype is not self.dtype or x.device != device or y.device != device:
            raise TypeError(f"x and y must be {self.dtype} on {device}")
        M = x.shape[0]
        _index(ids, "ids", (M,), device)
        if out is not None and (out.shape != y.shape or out.dtype is not y.dtype or not out.is_contiguous()):
            raise ValueError("out must be a contiguous [M, N] tensor of y's dtype")
        with _on(stream, device) as on:
            on.keep(x, y, ids, out, workspace, self.a, self.b, self.scale)
            x, y = _dense(x), _dense(y)
            if out is None:
                out = torch.empty((M, self.N), dtype=y.dtype, device=device)
            if workspace is None:
                workspace = torch.empty(self.workspace_size(M), dtype=torch.uint8, device=device)
            st = self._lib.gptq_lora_add(self._ref, x.data_ptr(), y.data_ptr(), ids.data_ptr(), M, out.data_ptr(),
                                         workspace.data_ptr(), workspace.numel() * workspace.element_size(), on.ptr)
        if st:
            raise GPTQError(st, "gptq_lora_add", self._lib)
        return out
