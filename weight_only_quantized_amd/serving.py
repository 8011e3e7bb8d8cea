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
import struct

import torch

from . import BF16, F16, F32, GPTQError, _OnStream, load_library

__all__ = ["KVCache", "LoraBank"]

_CODES = {torch.float16: F16, torch.bfloat16: BF16}
_INT32, _FLOAT32 = torch.int32, torch.float32

# The C structures of include/gptq_mi355x.h, packed by call (natural alignment, trailing padding
# written out).  A few hundred nanoseconds each where a ctypes.Structure takes over a microsecond: a
# decode step's calls are as long as their launches.
_CACHE = struct.Struct("PPPPqiiii")        # gptq_kv_cache
_BATCH = struct.Struct("PPPqiiii")         # gptq_kv_batch
_ROPE = struct.Struct("PPiiii")            # gptq_rope
_ATTENTION = struct.Struct("iifiiiqq")     # gptq_attention
_BANK = struct.Struct("PPPiiiiii")         # gptq_lora_bank


def _here(stream, index):
    """The hipStream_t to queue on when nothing has to wait or be recorded: no stream given, and the
    tensors' device is the current one.  Else None."""
    if index < 0:
        raise ValueError("the call runs on a GPU: its tensors must be there")
    return torch._C._cuda_getCurrentRawStream(index) if stream is None and torch._C._cuda_getDevice() == index else None


class _Queue(_OnStream):
    """`with _Queue(stream, index, *tensors) as ptr`: ptr is the stream, and everything inside is
    allocated and queued on it after the current stream's work."""

    def __init__(self, stream, index, *tensors):
        super().__init__(stream, torch.device("cuda", index))
        self.tensors = tensors

    def __enter__(self):
        super().__enter__()
        self.keep(*self.tensors)
        return self.stream.cuda_stream


def _index(t, name, shape, device):
    if t.dtype is not _INT32 or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)} on cuda:{device}")
    return t.data_ptr()


def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float16 or bfloat16")
    return code


def _packed(t, name, heads, dim, dtype, device):
    """(tensor, row stride) of a packed [rows, heads, dim] tensor with dense heads and rows 16 bytes
    aligned; copied if it is not so."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [rows, {heads}, {dim}]")
    if t.dtype is not dtype or t.get_device() != device:
        raise TypeError(f"{name} must be {dtype} on cuda:{device}")
    if t.is_contiguous() and not t.data_ptr() & 15:
        return t, heads * dim
    stride = _row_stride(t, shape)
    if stride:
        return t, stride
    return t.clone(memory_format=torch.contiguous_format), heads * dim


def _row_stride(t, shape):
    """Elements between the rows of [rows, heads, dim], 0 when they are not laid out as the library
    takes them."""
    if t.data_ptr() & 15:
        return 0
    width = shape[1] * shape[2]
    if t.is_contiguous():
        return width
    row, head, one = t.stride()
    if shape[0] < 2:
        row = width
    return row if one == 1 and (shape[1] == 1 or head == shape[2]) and row >= width and row % 8 == 0 else 0


def _like(t):
    """A new contiguous tensor of t's shape and type (empty_like is the quicker call, but follows t's strides)."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _dense(t):
    """A contiguous 16-byte aligned tensor (copied if it is not)."""
    return t if t.is_contiguous() and not t.data_ptr() & 15 else t.clone(memory_format=torch.contiguous_format)


def _scratch(t, device):
    """(pointer, bytes) of a caller's workspace."""
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
    return t.data_ptr(), t.numel() * t.element_size()


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
        self._index = k_codes.get_device()
        self._lib = load_library()
        self._c = _CACHE.pack(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                              self.num_pages, self.kv_heads, self.page_size, self.head_dim, 0)
        self._sizes = {}          # workspace bytes by the sizes that they follow from

    @classmethod
    def allocate(cls, num_pages, page_size, kv_heads, head_dim, device="cuda"):
        """A cache of zeros."""
        shape = (num_pages, kv_heads, page_size, head_dim)
        return cls(torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros(shape[:2], device=device), torch.zeros(shape[:2], device=device))

    def _batch(self, page_table, at, cu, rows, max_rows):
        device, shape = self._index, page_table.shape
        if len(shape) != 2:
            raise ValueError("page_table must be [batch, pages]")
        n, width = shape
        return _BATCH.pack(_index(page_table, "page_table", shape, device), _index(at, "lengths", (n,), device),
                           _index(cu, "cu", (n + 1,), device), rows, n, width, max_rows if max_rows < rows else rows, 0)

    def _raise(self, st, where):
        raise GPTQError(st, where, self._lib)

    def append(self, k, v, page_table, start, cu, *, max_new, q=None, cos=None, sin=None, interleaved=False,
               q_out=None, stream=None):
        """Append k and v [rows, kv_heads, head_dim] (fp16/bf16): row i of sequence b becomes its token
        start[b] + i; max_new is at least the rows of every sequence.  With cos and sin (float32
        [positions, rot / 2]) k is rotated at its position, and q [rows, q_heads, head_dim] too; the
        rotated q is returned (in q_out when given, which may be q).  Rotated pairs are halves of the
        first rot values, or neighbours when interleaved (gptq_kv_append)."""
        ptr = _here(stream, self._index)
        if ptr is not None:
            return self._append(ptr, k, v, page_table, start, cu, max_new, q, cos, sin, interleaved, q_out)
        with _Queue(stream, self._index, k, v, q, q_out, page_table, start, cu, cos, sin, self.k_codes, self.v_codes,
                    self.k_scale, self.v_scale) as ptr:
            return self._append(ptr, k, v, page_table, start, cu, max_new, q, cos, sin, interleaved, q_out)

    def _append(self, ptr, k, v, page_table, start, cu, max_new, q, cos, sin, interleaved, q_out):
        dt, device, dim = k.dtype, self._index, self.head_dim
        code = _code(k, "k")
        k, k_stride = _packed(k, "k", self.kv_heads, dim, dt, device)
        v, v_stride = _packed(v, "v", self.kv_heads, dim, dt, device)
        rows = k.shape[0]
        if v.shape[0] != rows:
            raise ValueError("k and v must have the same rows")
        rope = None
        if cos is not None and sin is not None:
            shape = cos.shape
            if (cos.dtype is not _FLOAT32 or sin.dtype is not _FLOAT32 or len(shape) != 2 or sin.shape != shape
                    or not cos.is_contiguous() or not sin.is_contiguous() or cos.get_device() != device
                    or sin.get_device() != device):
                raise ValueError("cos and sin must be contiguous float32 [positions, rot / 2] tensors on "
                                 f"cuda:{device}")
            rope = _ROPE.pack(cos.data_ptr(), sin.data_ptr(), shape[0], 2 * shape[1], 1 if interleaved else 0, 0)
        elif cos is not None or sin is not None:
            raise ValueError("cos and sin come together")
        q_ptr, q_stride, heads, o_ptr, o_stride = None, 0, 0, None, 0
        if q is not None:
            if rope is None:
                raise ValueError("q is taken to be rotated: pass cos and sin")
            if q.dim() != 3 or q.shape[0] != rows:
                raise ValueError("q must have k's rows")
            heads = q.shape[1]
            if q_out is None:
                q_out, o_stride = _like(q), heads * dim
            elif q_out.shape != q.shape or q_out.dtype is not dt or q_out.get_device() != device:
                raise ValueError("q_out must have q's shape, type and device")
            else:
                o_stride = _row_stride(q_out, q_out.shape)
                if not o_stride:
                    raise ValueError("q_out must have dense heads and aligned rows")
            q, q_stride = _packed(q, "q", heads, dim, dt, device)
            q_ptr, o_ptr = q.data_ptr(), q_out.data_ptr()
        st = self._lib.gptq_kv_append(self._c, self._batch(page_table, start, cu, rows, max_new), k.data_ptr(),
                                      k_stride, v.data_ptr(), v_stride, q_ptr, q_stride, heads, o_ptr, o_stride,
                                      code, rope, ptr)
        if st:
            self._raise(st, "gptq_kv_append")
        return q_out if q is not None else None

    def read(self, page_table, start, cu, *, rows, max_rows, dtype=torch.float16, stream=None):
        """Cached tokens as values: (k, v) [rows, kv_heads, head_dim] of dtype (fp16/bf16/fp32), row i
        of sequence b being its token start[b] + i; rows is cu's last entry (gptq_kv_read)."""
        code = F32 if dtype is _FLOAT32 else _CODES.get(dtype)
        if code is None:
            raise TypeError("dtype must be float16, bfloat16 or float32")
        ptr = _here(stream, self._index)
        if ptr is not None:
            return self._read(ptr, page_table, start, cu, rows, max_rows, dtype, code)
        with _Queue(stream, self._index, page_table, start, cu, self.k_codes, self.v_codes, self.k_scale,
                    self.v_scale) as ptr:
            return self._read(ptr, page_table, start, cu, rows, max_rows, dtype, code)

    def _read(self, ptr, page_table, start, cu, rows, max_rows, dtype, code):
        k = torch.empty((rows, self.kv_heads, self.head_dim), dtype=dtype, device=self.device)
        v = torch.empty_like(k)
        st = self._lib.gptq_kv_read(self._c, self._batch(page_table, start, cu, rows, max_rows), k.data_ptr(),
                                    v.data_ptr(), code, ptr)
        if st:
            self._raise(st, "gptq_kv_read")
        return k, v

    def attention(self, q, page_table, kv_len, cu, *, max_q, max_kv=None, scale=None, causal=True, window=0, out=None,
                  workspace=None, stream=None):
        """softmax(scale * q k^T) v of q [rows, q_heads, head_dim] (fp16/bf16) over each sequence's
        kv_len[b] cached tokens, the queries' own included: the last of a sequence's rows stands at its
        last token.  max_q is at least the rows of every sequence, max_kv at least every length (default:
        what the table holds).  scale defaults to head_dim ** -0.5; window > 0 hides tokens that are
        window or more before the query.  A query that sees nothing gives zeros (gptq_kv_attention)."""
        ptr = _here(stream, self._index)
        if ptr is not None:
            return self._attention(ptr, q, page_table, kv_len, cu, max_q, max_kv, scale, causal, window, out, workspace)
        with _Queue(stream, self._index, q, out, workspace, page_table, kv_len, cu, self.k_codes, self.v_codes, self.k_scale,
                    self.v_scale) as ptr:
            return self._attention(ptr, q, page_table, kv_len, cu, max_q, max_kv, scale, causal, window, out, workspace)

    def _attention(self, ptr, q, page_table, kv_len, cu, max_q, max_kv, scale, causal, window, out, workspace):
        device, dim = self._index, self.head_dim
        code = _code(q, "q")
        if q.dim() != 3:
            raise ValueError(f"q must be [rows, heads, {dim}]")
        rows, heads = q.shape[0], q.shape[1]
        q, q_stride = _packed(q, "q", heads, dim, q.dtype, device)
        if out is None:
            out, out_stride = _like(q), heads * dim
        elif out.shape != q.shape or out.dtype is not q.dtype or out.get_device() != device:
            raise ValueError("out must have q's shape, type and device")
        else:
            out_stride = _row_stride(out, out.shape)
            if not out_stride:
                raise ValueError("out must have dense heads and aligned rows")
        batch = self._batch(page_table, kv_len, cu, rows, max_q)
        room = page_table.shape[1] * self.page_size
        if max_kv is None or max_kv > room:
            max_kv = room
        if window > 0x7fffffff:                 # past every position: hides nothing
            window = 0
        call = _ATTENTION.pack(heads, code, dim ** -0.5 if scale is None else scale, 1 if causal else 0, window, max_kv,
                               q_stride, out_stride)
        key = (rows, page_table.shape, max_q, heads, max_kv, causal, window)
        need = self._sizes.get(key)
        if need is None:
            need = self._workspace_size(batch, call, key)
        if workspace is not None:
            ws, need = _scratch(workspace, device)
        elif need:
            workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
            ws = workspace.data_ptr()
        else:
            ws = None
        st = self._lib.gptq_kv_attention(self._c, batch, call, q.data_ptr(), out.data_ptr(), ws, need, ptr)
        if st:
            self._raise(st, "gptq_kv_attention")
        return out

    def _workspace_size(self, batch, call, key):
        n = ctypes.c_size_t(0)
        st = self._lib.gptq_kv_attention_workspace_size(self._c, batch, call, ctypes.byref(n))
        if st:
            self._raise(st, "gptq_kv_attention_workspace_size")
        if len(self._sizes) > 4096:
            self._sizes.clear()
        self._sizes[key] = n.value
        return n.value


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
        self._index = a.get_device()
        self._lib = load_library()
        self._c = _BANK.pack(a.data_ptr(), b.data_ptr(), scale.data_ptr(), self.adapters, self.rank, self.K, self.N,
                             _code(a, "a"), 0)
        self._sizes = {}          # workspace bytes by rows

    def workspace_size(self, M) -> int:
        n = ctypes.c_size_t(0)
        st = self._lib.gptq_lora_workspace_size(self._c, M, ctypes.byref(n))
        if st:
            raise GPTQError(st, "gptq_lora_workspace_size", self._lib)
        if len(self._sizes) > 4096:
            self._sizes.clear()
        self._sizes[M] = n.value
        return n.value

    def add(self, y, x, ids, out=None, workspace=None, stream=None):
        """y + scale[ids] * B (A x) for each row: y [M, N] is the shared projection's output, x [M, K]
        its input, ids int32 [M] (an id outside [0, adapters): no adapter).  out may be y."""
        device, dt, M = self._index, self.dtype, x.shape[0]
        if x.shape != (M, self.K) or y.shape != (M, self.N):
            raise ValueError(f"x must be [M, {self.K}] and y [M, {self.N}]")
        if x.dtype is not dt or y.dtype is not dt or x.get_device() != device or y.get_device() != device:
            raise TypeError(f"x and y must be {dt} on {self.device}")
        id_ptr = _index(ids, "ids", (M,), device)
        if out is not None and (out.shape != y.shape or out.dtype is not dt or out.get_device() != device
                                or not out.is_contiguous()):
            raise ValueError("out must be a contiguous [M, N] tensor of y's dtype")
        ptr = _here(stream, device)
        if ptr is not None:
            return self._add(ptr, y, x, id_ptr, M, out, workspace)
        with _Queue(stream, device, x, y, ids, out, workspace, self.a, self.b, self.scale) as ptr:
            return self._add(ptr, y, x, id_ptr, M, out, workspace)

    def _add(self, ptr, y, x, id_ptr, M, out, workspace):
        x, y = _dense(x), _dense(y)
        if out is None:
            out = torch.empty_like(y)          # y is dense here
        if workspace is not None:
            ws, size = _scratch(workspace, self._index)
        else:
            size, ws = self._sizes.get(M), None
            if size is None:
                size = self.workspace_size(M)
            if size:
                workspace = torch.empty(size, dtype=torch.uint8, device=self.device)
                ws = workspace.data_ptr()
        st = self._lib.gptq_lora_add(self._c, x.data_ptr(), y.data_ptr(), id_ptr, M, out.data_ptr(), ws, size, ptr)
        if st:
            raise GPTQError(st, "gptq_lora_add", self._lib)
        return out
