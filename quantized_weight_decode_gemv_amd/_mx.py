"""Binding of libqwg's MXFP4 and 8-bit cache calls (include/qwg.h). Argument
marshalling only, as in _binding: every step of the computation runs in the library's
HIP kernels, calls enqueue on torch's current stream of the tensors' device, and no
call waits, allocates inside the library or keeps anything. Codes, pages, the activations of
gemm_mxfp4 and gemv_mxfp4 and dequant_mxfp4's result start on 16 bytes, as whole tensors do; a view
that does not is refused with a QwgError."""
from __future__ import annotations

import ctypes
import functools

import torch

from ._binding import _check, lib

MX_BLOCK = 32
MX_MAX_BATCH = 16
_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
KV8_HEAD_DIMS = (64, 96, 128, 192, 256)
KV8_PAGE_TOKENS = (16, 32, 64, 128)
# Positions in a table up to which qwg_kv8_attend_workspace is 0 for every call, by head_dim (qwg.h):
# such calls, whose time is the host's, do not ask.
_ALONE = {64: 1024, 96: 1024, 128: 1024, 192: 512, 256: 512}


class Kv8Desc(ctypes.Structure):
    """qwg_kv8: the pages and scales of an 8-bit key/value cache."""
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_tokens", ctypes.c_int)]


_Tensor = torch.Tensor
_U8, _I32 = torch.uint8, torch.int32


def _on_device(t, name: str, device=None) -> None:
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a tensor on a HIP device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _plain(t, name: str, dtype, device=None) -> None:
    # one expression for the usual case: a small call's time is the host's
    if (isinstance(t, _Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and (device is None or t.device == device)):
        return
    _on_device(t, name, device)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def _type(dtype, name: str) -> int:
    code = _TYPES.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {dtype}")
    return code


# torch's own accessors of the current device and of a stream's handle; torch.cuda's build a
# Stream object (1.9 us on the host, where a small call takes 8 to 12 in all).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_fns: dict = {}


def _run(fn: str, device, *args) -> None:
    """The call on the current stream of `device`, which becomes the current device for it."""
    f = _fns.get(fn)
    if f is None:
        f = _fns[fn] = getattr(lib(), fn)
    index = device.index
    if _current_device() == index:
        rc = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            rc = f(*args, _raw_stream(index))
    if rc:
        _check(rc, fn)


def _matrix(codes, scales, name: str, device=None):
    """Rows and columns of an MXFP4 matrix: codes uint8 [rows, n_in/2], scales uint8 [rows, n_in/32]."""
    _plain(codes, name, _U8, device)
    shape = codes.shape
    if len(shape) != 2 or shape[0] < 1 or shape[1] < 16 or shape[1] % 16:
        raise ValueError(f"{name} must be [rows, n_in/2] with n_in a positive multiple of 32")
    rows, half = shape
    _plain(scales, "scales", _U8, codes.device)
    if scales.shape != (rows, half // 16):
        raise ValueError(f"the scales of {name} must be [{rows}, {half // 16}], got {list(scales.shape)}")
    return rows, half * 2


def _out(out, shape, like, name: str = "out", dtype=None) -> torch.Tensor:
    """`out`, checked, or a new contiguous tensor on the device of `like` (of its type, or dtype)."""
    dtype = like.dtype if dtype is None else dtype
    if out is None:
        return like.new_empty(shape) if dtype == like.dtype else like.new_empty(shape, dtype=dtype)
    _plain(out, name, dtype, like.device)
    if out.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(out.shape)}")
    return out


def encode_mxfp4(x: torch.Tensor, codes: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None):
    """fp32, fp16 or bf16 x [rows, n_in] (n_in % 32 == 0; rows may lie apart, as in a slice of
    columns) -> MXFP4 (codes uint8 [rows, n_in/2], scales uint8 [rows, n_in/32])."""
    _on_device(x, "x")
    kind = _type(x.dtype, "x")
    shape = x.shape
    if len(shape) != 2 or shape[0] < 1 or shape[1] < MX_BLOCK or shape[1] % MX_BLOCK:
        raise ValueError("x must be [rows, n_in] with n_in a positive multiple of 32")
    rows, n_in = shape
    stride, each = x.stride()
    if rows == 1:
        stride = n_in
    if each != 1 or stride < n_in:
        raise ValueError("the values of a row of x must be contiguous, and rows must not overlap")
    codes = _out(codes, (rows, n_in // 2), x, "codes", _U8)
    scales = _out(scales, (rows, n_in // MX_BLOCK), x, "scales", _U8)
    _run("qwg_encode_mxfp4", x.device, codes.data_ptr(), scales.data_ptr(), x.data_ptr(), kind,
         rows, n_in, stride)
    return codes, scales


def dequant_mxfp4(codes: torch.Tensor, scales: torch.Tensor, dtype=torch.float32,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """MXFP4 codes [rows, n_in/2] and scales [rows, n_in/32] -> values [rows, n_in]."""
    rows, n_in = _matrix(codes, scales, "codes")
    kind = _type(dtype, "dtype")
    out = _out(out, (rows, n_in), codes, dtype=dtype)
    _run("qwg_dequant_mxfp4", codes.device, codes.data_ptr(), scales.data_ptr(), out.data_ptr(),
         kind, rows * n_in)
    return out


def gemm_mxfp4(w: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """Y = X W^T for MXFP4 weights (w uint8 [n_out, n_in/2], scales uint8 [n_out, n_in/32]) and
    X [batch, n_in] (1 <= batch <= 16; fp32, fp16 or bf16; starting on 16 bytes) -> [batch, n_out] of
    X's type."""
    n_out, n_in = _matrix(w, scales, "w")
    _on_device(x, "x", w.device)
    kind = _type(x.dtype, "x")
    shape = x.shape
    if len(shape) != 2 or not 1 <= shape[0] <= MX_MAX_BATCH or shape[1] != n_in:
        raise ValueError(f"x must be [batch, {n_in}] with 1 <= batch <= {MX_MAX_BATCH}")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    batch = shape[0]
    out = _out(out, (batch, n_out), x)
    _run("qwg_gemm_mxfp4", x.device, out.data_ptr(), x.data_ptr(), kind, w.data_ptr(),
         scales.data_ptr(), n_in, n_out, batch)
    return out


def gemv_mxfp4(w: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """y = W x for MXFP4 weights (as gemm_mxfp4) and x [n_in], starting on 16 bytes -> [n_out] of x's
    type."""
    n_out, n_in = _matrix(w, scales, "w")
    _plain(x, "x", x.dtype if isinstance(x, torch.Tensor) else None, w.device)
    kind = _type(x.dtype, "x")
    if x.shape != (n_in,):
        raise ValueError(f"x must be [{n_in}]")
    out = _out(out, (n_out,), x)
    _run("qwg_gemv_mxfp4", x.device, out.data_ptr(), x.data_ptr(), kind, w.data_ptr(),
         scales.data_ptr(), n_in, n_out)
    return out


def matmul_mxfp4(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                 dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """C = A W^T for two MXFP4 matrices (codes and scales of each, as encode_mxfp4 gives them),
    A [n_rows, n_in] and W [n_out, n_in] (at most 2^24 rows each and 2^38 outputs) -> [n_rows, n_out]
    of `dtype`."""
    n_rows, n_in = _matrix(a, a_scales, "a")
    n_out, w_in = _matrix(w, w_scales, "w", a.device)
    if w_in != n_in:
        raise ValueError(f"a has {n_in} columns and w {w_in}")
    kind = _type(dtype, "dtype")
    out = _out(out, (n_rows, n_out), a, dtype=dtype)
    _run("qwg_matmul_mxfp4", a.device, out.data_ptr(), kind, a.data_ptr(), a_scales.data_ptr(),
         w.data_ptr(), w_scales.data_ptr(), n_rows, n_in, n_out)
    return out


def kv8_pages(n_pages: int, n_kv_heads: int, head_dim: int, page_tokens: int = 64, device="cuda"):
    """The tensors of an 8-bit cache: (k_pages, k_scales, v_pages, v_scales), uint8 zeros."""
    if n_pages < 1 or n_kv_heads < 1:
        raise ValueError("a cache needs at least one page and one head")
    if head_dim not in KV8_HEAD_DIMS or page_tokens not in KV8_PAGE_TOKENS:
        raise ValueError(f"head_dim must be one of {KV8_HEAD_DIMS} and page_tokens of {KV8_PAGE_TOKENS}")

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device=device)

    return (zeros(n_pages, n_kv_heads, page_tokens, head_dim), zeros(n_pages, n_kv_heads),
            zeros(n_pages, n_kv_heads, head_dim, page_tokens), zeros(n_pages, n_kv_heads))


def _cache(k_pages, k_scales, v_pages, v_scales, device) -> Kv8Desc:
    _plain(k_pages, "k_pages", _U8, device)
    _plain(v_pages, "v_pages", _U8, device)
    _plain(k_scales, "k_scales", _U8, device)
    _plain(v_scales, "v_scales", _U8, device)
    shape = k_pages.shape
    if len(shape) != 4:
        raise ValueError("k_pages must be [n_pages, n_kv_heads, page_tokens, head_dim]")
    n_pages, heads, page, dim = shape
    if dim not in KV8_HEAD_DIMS or page not in KV8_PAGE_TOKENS:
        raise ValueError(f"head_dim must be one of {KV8_HEAD_DIMS} and page_tokens of {KV8_PAGE_TOKENS}")
    if v_pages.shape != (n_pages, heads, dim, page):
        raise ValueError(f"v_pages must be [{n_pages}, {heads}, {dim}, {page}]")
    if k_scales.shape != shape[:2] or v_scales.shape != shape[:2]:
        raise ValueError(f"k_scales and v_scales must be [{n_pages}, {heads}]")
    return Kv8Desc(k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                   n_pages, heads, dim, page)


def _sequences(table, lens, device):
    _plain(table, "table", _I32, device)
    _plain(lens, "lens", _I32, device)
    shape = table.shape
    if len(shape) != 2 or shape[0] < 1 or shape[1] < 1:
        raise ValueError("table must be [n_seqs, pages]")
    if lens.shape != shape[:1]:
        raise ValueError(f"lens must be [{shape[0]}]")
    return shape


def _tokens(x, name: str, heads: int, dim: int):
    """Tokens and token stride of [tokens, heads, dim] or [n_seqs, tokens, heads, dim]."""
    shape, strides = x.shape, x.stride()
    if len(shape) not in (3, 4) or shape[-2] != heads or shape[-1] != dim:
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}] or [n_seqs, tokens, {heads}, {dim}]")
    if strides[-1] != 1 or (heads > 1 and strides[-2] != dim):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    n, stride = shape[0], strides[-3]
    if len(shape) == 4:
        each = shape[1]
        if each == 1:
            stride = strides[0]
        elif n > 1 and strides[0] != each * stride:
            raise ValueError(f"the tokens of {name} must lie at one distance")
        n *= each
    if n > 1 and stride < heads * dim:
        raise ValueError(f"the tokens of {name} must not overlap")
    return n, stride


def kv8_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, k_scales: torch.Tensor,
               v_pages: torch.Tensor, v_scales: torch.Tensor, table: torch.Tensor,
               lens: torch.Tensor, starts: torch.Tensor | None = None,
               max_new: int | None = None) -> None:
    """Encode new keys and values into the pages of an 8-bit cache (kv8_pages).

    k, v: fp32, fp16 or bf16 [n_tokens, n_kv_heads, head_dim] or [n_seqs, tokens, n_kv_heads,
    head_dim] (slices of a fused q|k|v result may be given). table int32 [n_seqs, pages]: each
    sequence's pages in order; lens int32 [n_seqs]: the positions that each holds before the call.
    starts int32 [n_seqs + 1]: sequence s appends tokens starts[s] .. starts[s+1]-1; without it
    every sequence appends as many. max_new: the most that one appends, if known. The caller
    advances lens. A page that is written must belong to one sequence."""
    kind, cache, n_seqs, width, n, k_stride, v_stride, most = _new_tokens(
        k, v, k_pages, k_scales, v_pages, v_scales, table, lens, starts, max_new)
    _run("qwg_kv8_append", k.device, ctypes.byref(cache), k.data_ptr(), v.data_ptr(), kind,
         k_stride, v_stride, n, None if starts is None else starts.data_ptr(), table.data_ptr(),
         width, lens.data_ptr(), n_seqs, most)


def _new_tokens(k, v, k_pages, k_scales, v_pages, v_scales, table, lens, starts, max_new):
    """What kv8_append and kv8_append_rotary check alike."""
    _on_device(k, "k")
    _on_device(v, "v", k.device)
    kind = _type(k.dtype, "k")
    if v.dtype != k.dtype:
        raise ValueError("k and v must be of one type")
    cache = _cache(k_pages, k_scales, v_pages, v_scales, k.device)
    n_seqs, width = _sequences(table, lens, k.device)
    n, k_stride = _tokens(k, "k", cache.n_kv_heads, cache.head_dim)
    v_n, v_stride = _tokens(v, "v", cache.n_kv_heads, cache.head_dim)
    if n != v_n or n < 1:
        raise ValueError("k and v must hold the same tokens, one at least")
    if starts is None:
        if n % n_seqs or (k.dim() == 4 and k.shape[0] != n_seqs):
            raise ValueError(f"{n} tokens are not as many for each of {n_seqs} sequences")
        most = n // n_seqs
    else:
        _plain(starts, "starts", _I32, k.device)
        if starts.shape != (n_seqs + 1,):
            raise ValueError(f"starts must be [{n_seqs + 1}]")
        most = n if max_new is None else max_new
        if most < 1:
            raise ValueError("max_new must be at least 1")
    return kind, cache, n_seqs, width, n, k_stride, v_stride, most


def _out_tokens(out, like, name: str, heads: int, dim: int, n: int):
    """`out`, checked, or a new contiguous tensor of the shape of `like`; and its token stride."""
    if out is None:
        return like.new_empty(like.shape), heads * dim
    _on_device(out, name, like.device)
    if out.dtype != like.dtype or out.shape != like.shape:
        raise ValueError(f"{name} must be {like.dtype} {list(like.shape)}")
    return out, _tokens(out, name, heads, dim)[1]


def kv8_append_rotary(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, freqs: torch.Tensor,
                      k_pages: torch.Tensor, k_scales: torch.Tensor, v_pages: torch.Tensor,
                      v_scales: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                      starts: torch.Tensor | None = None, max_new: int | None = None,
                      interleaved: bool = False, out: torch.Tensor | None = None,
                      k_out: torch.Tensor | None = None,
                      prefix_len: torch.Tensor | None = None) -> torch.Tensor:
    """Rotate new queries and keys by their positions, and encode the keys and values into the
    pages of an 8-bit cache, as kv8_append does. Returns the rotated queries.

    q: [n_tokens, n_heads, head_dim] or [n_seqs, tokens, n_heads, head_dim], like k and v (slices of
    a fused q|k|v result may be given). Token i of sequence s is at position lens[s] + i
    (behind prefix_len others). freqs:
    fp32 [rotary_dim / 2] (rotary_dim a multiple of 16, head_dim at most), radians per position;
    the angle is computed in 64 bits. Channels (j, j + rotary_dim / 2), or with `interleaved`
    (2j, 2j + 1), turn by position * freqs[j]; those past rotary_dim stay. out: where the queries go
    (q itself may be given), else a new tensor. k_out: a tensor of k's shape that gets the rotated
    keys too (for prompt_attend); it must not overlap q, k or v. prefix_len int32 [1]: positions of a
    prefix that the sequences share (kv8_attend_shared), before the first of their own. Rows of tokens that belong to no
    sequence are left as they were."""
    kind, cache, n_seqs, width, n, k_stride, v_stride, most = _new_tokens(
        k, v, k_pages, k_scales, v_pages, v_scales, table, lens, starts, max_new)
    dim = cache.head_dim
    _on_device(q, "q", k.device)
    heads = q.shape[-2] if q.dim() in (3, 4) else 0
    if q.dtype != k.dtype:
        raise ValueError("q must be of the type of k and v")
    if heads < 1 or heads % cache.n_kv_heads or q.shape[:-2] != k.shape[:-2]:
        raise ValueError(f"q must hold the tokens of k, n_heads a multiple of {cache.n_kv_heads}")
    q_stride = _tokens(q, "q", heads, dim)[1]
    _plain(freqs, "freqs", torch.float32, k.device)
    rotary = 2 * freqs.numel()
    if freqs.dim() != 1 or rotary < 16 or rotary % 16 or rotary > dim:
        raise ValueError(f"freqs must be [rotary_dim / 2] with rotary_dim a multiple of 16, at most {dim}")
    if prefix_len is not None:
        _plain(prefix_len, "prefix_len", _I32, k.device)
        if prefix_len.numel() != 1:
            raise ValueError("prefix_len must be [1]")
    out, out_stride = _out_tokens(out, q, "out", heads, dim, n)
    k_out_stride = 0
    if k_out is not None:
        k_out, k_out_stride = _out_tokens(k_out, k, "k_out", cache.n_kv_heads, dim, n)
    _run("qwg_kv8_append_rotary", k.device, ctypes.byref(cache), out.data_ptr(), out_stride,
         None if k_out is None else k_out.data_ptr(), k_out_stride, q.data_ptr(), q_stride,
         k.data_ptr(), k_stride, v.data_ptr(), v_stride, kind, heads, freqs.data_ptr(), rotary,
         int(interleaved), None if prefix_len is None else prefix_len.data_ptr(), n,
         None if starts is None else starts.data_ptr(), table.data_ptr(), width, lens.data_ptr(), n_seqs, most)
    return out


def prompt_attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  starts: torch.Tensor | None = None, max_len: int | None = None,
                  scale: float | None = None, window: int = 0,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention over whole prompts.

    q: fp32, fp16 or bf16 [n_tokens, n_heads, head_dim], k and v [n_tokens, n_kv_heads, head_dim]
    (slices of a fused q|k|v result may be given), or all of them [n_seqs, tokens, ...]. starts int32
    [n_seqs + 1]: sequence s holds tokens starts[s] .. starts[s+1]-1; without it three-dimensional
    tensors hold one sequence, four-dimensional ones n_seqs. A token sees its sequence up to itself,
    the last `window` positions (0: all). scale defaults to head_dim ** -0.5. max_len: the longest
    sequence, if known: a hint that no result depends on, and that the present launch needs none of. out: where the result goes (a contiguous q
    itself may be given, else nothing that shares its memory or k's or v's), else a new tensor. Returns
    a contiguous tensor of q's shape and type; rows of tokens that belong to no sequence are left as they were (in a new tensor: undefined)."""
    _on_device(q, "q")
    device, dtype = q.device, q.dtype
    _on_device(k, "k", device)
    _on_device(v, "v", device)
    kind = _type(dtype, "q")
    if k.dtype != dtype or v.dtype != dtype:
        raise ValueError("q, k and v must be of one type")
    shape, of_k = q.shape, k.shape
    if len(shape) not in (3, 4) or v.shape != of_k or shape[:-2] != of_k[:-2] or len(of_k) != len(shape):
        raise ValueError("q must be [n_tokens, n_heads, head_dim] and k and v [n_tokens, n_kv_heads, head_dim], "
                         "or [n_seqs, tokens, ...] alike")
    heads, dim = shape[-2:]
    kv = of_k[-2]
    if dim not in KV8_HEAD_DIMS or kv < 1 or heads < 1 or heads % kv:
        raise ValueError(f"head_dim must be one of {KV8_HEAD_DIMS} and n_heads a multiple of n_kv_heads")
    n, q_stride = _tokens(q, "q", heads, dim)
    k_stride, v_stride = _tokens(k, "k", kv, dim)[1], _tokens(v, "v", kv, dim)[1]
    if n < 1:
        raise ValueError("a call needs at least one token")
    if starts is None:
        n_seqs = 1 if len(shape) == 3 else shape[0]
    else:
        _plain(starts, "starts", _I32, device)
        if starts.dim() != 1 or starts.shape[0] < 2:
            raise ValueError("starts must be [n_seqs + 1]")
        n_seqs = starts.shape[0] - 1
    if window < 0 or (max_len is not None and max_len < 0):
        raise ValueError("window and max_len must not be negative")
    out = _out(out, shape, q)
    _run("qwg_prompt_attend", device, out.data_ptr(), q.data_ptr(), q_stride, k.data_ptr(),
         k_stride, v.data_ptr(), v_stride, kind, n, None if starts is None else starts.data_ptr(),
         n_seqs, max_len or 0, heads, kv, dim, dim ** -0.5 if scale is None else scale, window)
    return out


def kv8_attend(q: torch.Tensor, k_pages: torch.Tensor, k_scales: torch.Tensor,
               v_pages: torch.Tensor, v_scales: torch.Tensor, table: torch.Tensor,
               lens: torch.Tensor, scale: float | None = None, window: int = 0,
               max_len: int | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the last tokens of each sequence over an 8-bit cache (kv8_pages).

    q: fp32, fp16 or bf16 [n_seqs, n_heads, head_dim] or [n_seqs, q_len, n_heads, head_dim] (a
    slice of a fused q|k|v result may be given). lens int32 [n_seqs]: the positions held, the
    queries' own among them; query t of a sequence sees positions up to lens - q_len + t, the last
    `window` of them (0: all). scale defaults to head_dim ** -0.5. max_len: the largest length, if
    known; a table cut to it is faster than one that is much wider. Returns a contiguous tensor of q's
    shape and type; rows that see nothing are zero."""
    _on_device(q, "q")
    kind = _type(q.dtype, "q")
    cache = _cache(k_pages, k_scales, v_pages, v_scales, q.device)
    n_seqs, width = _sequences(table, lens, q.device)
    heads, dim = q.shape[-2:] if q.dim() in (3, 4) else (0, 0)
    if dim != cache.head_dim or heads < 1 or heads % cache.n_kv_heads or q.shape[0] != n_seqs:
        raise ValueError(f"q must be [{n_seqs}, (q_len,) n_heads, {cache.head_dim}] with n_heads a "
                         f"multiple of {cache.n_kv_heads}")
    n, stride = _tokens(q, "q", heads, dim)
    q_len = n // n_seqs
    if q_len < 1 or q_len * heads > 65535:
        raise ValueError("q_len * n_heads must be in 1..65535")
    if window < 0 or (max_len is not None and max_len < 0):
        raise ValueError("window and max_len must not be negative")
    out = _out(out, q.shape, q)
    most = max_len or 0
    ref = ctypes.byref(cache)
    size = 0
    if width * cache.page_tokens > _ALONE[dim]:
        size = lib().qwg_kv8_attend_workspace(ref, width, n_seqs, q_len, heads, window, most)
        if size < 0:
            _check(-size, "qwg_kv8_attend_workspace")
    # of this call's stream (or of the graph that captures it): no two calls share one
    space = table.new_empty(size // 4) if size else None
    _run("qwg_kv8_attend", q.device, ref, out.data_ptr(), q.data_ptr(), kind, stride,
         table.data_ptr(), width, lens.data_ptr(), n_seqs, q_len, heads,
         dim ** -0.5 if scale is None else scale, window, most,
         space.data_ptr() if size else None, size)
    return out


@functools.lru_cache(maxsize=256)
def _shared_workspace(kind, n_pages, n_kv_heads, head_dim, page_tokens, *sizes) -> int:
    """Its bytes, by the call's sizes alone (asking the library takes 1.5 us of a call's 14)."""
    desc = Kv8Desc(1 << 12, 1 << 12, 1 << 12, 1 << 12, n_pages, n_kv_heads, head_dim, page_tokens)
    size = lib().qwg_kv8_attend_shared_workspace(ctypes.byref(desc), kind, *sizes)
    if size < 0:
        _check(-size, "qwg_kv8_attend_shared_workspace")
    return size


def kv8_attend_shared(q: torch.Tensor, k_pages: torch.Tensor, k_scales: torch.Tensor,
                      v_pages: torch.Tensor, v_scales: torch.Tensor, prefix: torch.Tensor,
                      prefix_len: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                      scale: float | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the last tokens of sequences that share a prefix, over an 8-bit cache
    (kv8_pages): kv8_attend over the prefix's positions and each sequence's own behind them, but the
    prefix is read once for all sequences.

    q: as kv8_attend's. prefix int32 [pages]: the shared pages in order; prefix_len int32 [1]: the
    positions that they hold (any number: the last page need not be full). table int32 [n_seqs, pages]
    and lens int32 [n_seqs]: each sequence's own pages and positions, the first right behind the
    prefix, the queries' own among them (kv8_append and kv8_append_rotary fill them; the latter's
    takes prefix_len too). scale defaults to head_dim ** -0.5. out: as prompt_attend's. A prefix and a
    table cut to what they hold are faster than ones that are much wider, and take a smaller workspace.
    Returns a contiguous tensor of q's shape and type."""
    _on_device(q, "q")
    kind = _type(q.dtype, "q")
    cache = _cache(k_pages, k_scales, v_pages, v_scales, q.device)
    n_seqs, width = _sequences(table, lens, q.device)
    _plain(prefix, "prefix", _I32, q.device)
    _plain(prefix_len, "prefix_len", _I32, q.device)
    pages = prefix.numel()
    if prefix.dim() != 1 or pages < 1 or prefix_len.numel() != 1:
        raise ValueError("prefix must be [pages] and prefix_len [1]")
    heads, dim = q.shape[-2:] if q.dim() in (3, 4) else (0, 0)
    if dim != cache.head_dim or heads < 1 or heads % cache.n_kv_heads or q.shape[0] != n_seqs:
        raise ValueError(f"q must be [{n_seqs}, (q_len,) n_heads, {cache.head_dim}] with n_heads a "
                         f"multiple of {cache.n_kv_heads}")
    n, stride = _tokens(q, "q", heads, dim)
    q_len = n // n_seqs
    if q_len < 1 or q_len * heads > 65535:
        raise ValueError("q_len * n_heads must be in 1..65535")
    out = _out(out, q.shape, q)
    ref = ctypes.byref(cache)
    size = _shared_workspace(kind, cache.n_pages, cache.n_kv_heads, dim, cache.page_tokens, pages,
                             width, n_seqs, q_len, heads)
    # of this call's stream (or of the graph that captures it): no two calls share one
    space = table.new_empty(size // 4)
    _run("qwg_kv8_attend_shared", q.device, ref, out.data_ptr(), q.data_ptr(), kind, stride,
         prefix.data_ptr(), pages, prefix_len.data_ptr(), table.data_ptr(), width,
         lens.data_ptr(), n_seqs, q_len, heads, dim ** -0.5 if scale is None else scale,
         space.data_ptr(), size)
    return out
