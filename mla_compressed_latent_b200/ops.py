"""Python binding of libmla: the C-ABI calls under the same names, taking torch CUDA tensors.

Argument marshalling only: shapes and dtypes are checked, device pointers and sizes are passed,
and a workspace is taken from torch's caching allocator when the caller gives none. Every step of
the computation runs in the library's CUDA kernels; a failing call raises MlaError.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

import torch

from . import _lib as L


class MlaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        lib = L.load()
        super().__init__(f"{fn}: {lib.mla_status_string(status).decode()} (status {status})")
        self.status = status


@dataclass(frozen=True)
class Dims:
    H: int
    D: int
    d_r: int
    d_c: int
    d_v: int
    g: int = 0
    page_size: int = 64
    sm_scale: float = 0.0
    rms_eps: float = 1e-6
    rope_base: float = 10000.0

    def c(self) -> L.MlaDims:
        # sm_scale 0 lets the library use its default, 1/sqrt(D + d_r)
        return L.MlaDims(self.H, self.D, self.d_r, self.d_c, self.d_v, self.g, self.page_size, self.sm_scale,
                         self.rms_eps, self.rope_base)

    @staticmethod
    def of(w) -> "Dims":
        """From any object with the attributes of a workload (H, D, d_r, d_c, d_v, g, ...)."""
        return Dims(w.H, w.D, w.d_r, w.d_c, w.d_v, getattr(w, "g", 0), getattr(w, "page_size", 64),
                    getattr(w, "sm_scale", 0.0), getattr(w, "rms_eps", 1e-6), getattr(w, "rope_base", 10000.0))


_DTYPES = {torch.float32: L.MLA_F32, torch.bfloat16: L.MLA_BF16}


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DTYPES[t.dtype]


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libmla takes device tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, rc):
    if rc != L.MLA_OK:
        raise MlaError(fn, rc)


def _i32(t):
    if t.dtype != torch.int32:
        raise TypeError("index tensors are int32")
    return t


@dataclass
class LatentCache:
    """Latent pool [num_pages*64, d_c] + RoPE-key pool [num_pages*64, d_r] (views may interleave)."""
    latent: torch.Tensor
    rope: torch.Tensor
    num_pages: int

    @staticmethod
    def interleaved(num_pages: int, d_c: int, d_r: int, dtype, device="cuda") -> "LatentCache":
        rows = torch.empty(num_pages * 64, d_c + d_r, dtype=dtype, device=device)
        return LatentCache(rows[:, :d_c], rows[:, d_c:], num_pages)

    def c(self) -> L.MlaLatentCache:
        return L.MlaLatentCache(self.latent.data_ptr(), self.latent.stride(0), self.rope.data_ptr(),
                                self.rope.stride(0), self.num_pages)


@dataclass
class GqaCache:
    k: torch.Tensor     # [num_pages*64, g, D]
    v: torch.Tensor     # [num_pages*64, g, d_v]
    rope: torch.Tensor  # [num_pages*64, d_r]
    num_pages: int

    def c(self) -> L.MlaGqaCache:
        return L.MlaGqaCache(self.k.data_ptr(), self.k.stride(0), self.v.data_ptr(), self.v.stride(0),
                             self.rope.data_ptr(), self.rope.stride(0), self.num_pages)


@dataclass
class LatentCacheFp8:
    """8-bit latent pool: E4M3 codes [num_pages*64, d_c] uint8 + fp32 scales [num_pages*64] + the
    16-bit RoPE-key pool [num_pages*64, d_r]."""
    codes: torch.Tensor
    scales: torch.Tensor
    rope: torch.Tensor
    num_pages: int

    @staticmethod
    def empty_like(cache: "LatentCache") -> "LatentCacheFp8":
        """Code and scale storage for every row of a 16-bit pool, sharing its RoPE keys."""
        rows, d_c = cache.latent.shape
        dev = cache.latent.device
        return LatentCacheFp8(torch.empty(rows, d_c, dtype=torch.uint8, device=dev),
                              torch.empty(rows, dtype=torch.float32, device=dev), cache.rope, cache.num_pages)

    def c(self) -> L.MlaLatentCacheFp8:
        return L.MlaLatentCacheFp8(self.codes.data_ptr(), self.codes.stride(0), self.scales.data_ptr(),
                                   self.rope.data_ptr(), self.rope.stride(0), self.num_pages)


def _workspace(nbytes, device, workspace):
    if nbytes == 0:
        return workspace, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------------------------------------
def mla_append_cache(dims: Dims, x, w_dkv_kr, gamma, seqlens, block_table, cache: LatentCache,
                     workspace=None, stream=None):
    lib = L.load()
    B, s_q, C = x.shape
    d = dims.c()
    need = lib.mla_append_workspace_size(ctypes.byref(d), B, s_q, C)
    workspace, wsb = _workspace(need, x.device, workspace)
    cc = cache.c()
    rc = lib.mla_append_cache(ctypes.byref(d), _dt(x), B, s_q, _ptr(x), C, _ptr(w_dkv_kr), _ptr(gamma),
                              _ptr(_i32(seqlens)), _ptr(_i32(block_table)), block_table.shape[1], ctypes.byref(cc),
                              _ptr(workspace) if workspace is not None else None, wsb, _stream(stream))
    _check("mla_append_cache", rc)


def mla_project_query(dims: Dims, x, w_dq, gamma_q, w_uq, w_qr, q_nope=None, q_rope_raw=None, workspace=None,
                      stream=None):
    """x [B, s_q, C] -> (q_nope [B, s_q, H, D], q_rope_raw [B, s_q, H, d_r]) through
    c_q = RMSNorm(x·W_DQ)·gamma_q (w_dq [C, d_q], w_uq [d_q, H*D], w_qr [d_q, H*d_r])."""
    lib = L.load()
    B, s_q, C = x.shape
    d_q = w_dq.shape[1]
    if q_nope is None:
        q_nope = torch.empty(B, s_q, dims.H, dims.D, dtype=x.dtype, device=x.device)
    if q_rope_raw is None:
        q_rope_raw = torch.empty(B, s_q, dims.H, dims.d_r, dtype=x.dtype, device=x.device)
    d = dims.c()
    need = lib.mla_query_workspace_size(ctypes.byref(d), B, s_q, C, d_q)
    workspace, wsb = _workspace(need, x.device, workspace)
    rc = lib.mla_project_query(ctypes.byref(d), _dt(x), B, s_q, _ptr(x), C, d_q, _ptr(w_dq), _ptr(gamma_q),
                               _ptr(w_uq), _ptr(w_qr), _ptr(q_nope), _ptr(q_rope_raw),
                               _ptr(workspace) if workspace is not None else None, wsb, _stream(stream))
    _check("mla_project_query", rc)
    return q_nope, q_rope_raw


def mla_absorb_q(dims: Dims, q_nope, q_rope_raw, w_uk, seqlens, q_abs=None, stream=None):
    lib = L.load()
    B, s_q, H, D = q_nope.shape
    if q_abs is None:
        q_abs = torch.empty(B, s_q, H, dims.d_c + dims.d_r, dtype=q_nope.dtype, device=q_nope.device)
    d = dims.c()
    rc = lib.mla_absorb_q(ctypes.byref(d), _dt(q_nope), B, s_q, _ptr(q_nope), _ptr(q_rope_raw), _ptr(w_uk),
                          _ptr(_i32(seqlens)), _ptr(q_abs), _stream(stream))
    _check("mla_absorb_q", rc)
    return q_abs


def mla_append_cache_absorb_q(dims: Dims, x, w_dkv_kr, gamma, q_nope, q_rope_raw, w_uk, seqlens, block_table,
                              cache: LatentCache, q_abs=None, workspace=None, stream=None):
    """mla_append_cache and mla_absorb_q of one step in one call (their projections share a launch);
    returns q_abs."""
    lib = L.load()
    B, s_q, C = x.shape
    if q_abs is None:
        q_abs = torch.empty(B, s_q, dims.H, dims.d_c + dims.d_r, dtype=q_nope.dtype, device=q_nope.device)
    d = dims.c()
    need = lib.mla_append_workspace_size(ctypes.byref(d), B, s_q, C)
    workspace, wsb = _workspace(need, x.device, workspace)
    cc = cache.c()
    rc = lib.mla_append_cache_absorb_q(ctypes.byref(d), _dt(x), B, s_q, _ptr(x), C, _ptr(w_dkv_kr), _ptr(gamma),
                                       _ptr(q_nope), _ptr(q_rope_raw), _ptr(w_uk), _ptr(_i32(seqlens)),
                                       _ptr(_i32(block_table)), block_table.shape[1], ctypes.byref(cc), _ptr(q_abs),
                                       _ptr(workspace) if workspace is not None else None, wsb, _stream(stream))
    _check("mla_append_cache_absorb_q", rc)
    return q_abs


def mla_decode_workspace_size(dims: Dims, dtype, B, s_q, max_pages) -> int:
    d = dims.c()
    return L.load().mla_decode_workspace_size(ctypes.byref(d), _DTYPES[dtype], B, s_q, max_pages)


def mla_decode_absorbed(dims: Dims, q_abs, cache: LatentCache, block_table, seqlens, o_lat=None, lse=None,
                        workspace=None, stream=None, seqlens_host=None):
    """a3 + a4. seqlens_host: optional host copy of seqlens (int32, B values; a numpy array or a CPU
    tensor) that lets the library launch the decode without the split machinery when nothing is
    cut (mla_decode_absorbed_hinted)."""
    lib = L.load()
    B, s_q, H, _ = q_abs.shape
    if o_lat is None:
        o_lat = torch.empty(B, s_q, H, dims.d_c, dtype=q_abs.dtype, device=q_abs.device)
    if lse is None:
        lse = torch.empty(B, s_q, H, dtype=torch.float32, device=q_abs.device)
    d = dims.c()
    max_pages = block_table.shape[1]
    need = lib.mla_decode_workspace_size(ctypes.byref(d), _dt(q_abs), B, s_q, max_pages)
    workspace, wsb = _workspace(need, q_abs.device, workspace)
    cc = cache.c()
    if seqlens_host is None:
        rc = lib.mla_decode_absorbed(ctypes.byref(d), _dt(q_abs), B, s_q, _ptr(q_abs), ctypes.byref(cc),
                                     _ptr(_i32(block_table)), max_pages, _ptr(_i32(seqlens)), _ptr(o_lat), _ptr(lse),
                                     _ptr(workspace) if workspace is not None else None, wsb, _stream(stream))
        _check("mla_decode_absorbed", rc)
    else:
        host = torch.as_tensor(seqlens_host, dtype=torch.int32).contiguous()
        if host.is_cuda or host.numel() != B:
            raise ValueError("seqlens_host: B int32 values in host memory")
        rc = lib.mla_decode_absorbed_hinted(ctypes.byref(d), _dt(q_abs), B, s_q, _ptr(q_abs), ctypes.byref(cc),
                                            _ptr(_i32(block_table)), max_pages, _ptr(_i32(seqlens)),
                                            ctypes.c_void_p(host.data_ptr()), _ptr(o_lat), _ptr(lse),
                                            _ptr(workspace) if workspace is not None else None, wsb, _stream(stream))
        _check("mla_decode_absorbed_hinted", rc)
    return o_lat, lse


def mla_quantize_latent_fp8(dims: Dims, latent, codes, scales, stream=None):
    """Rows of `latent` [rows, d_c] (dtype, rows may be a view of a pool) into E4M3 `codes` [rows, d_c]
    (uint8) and fp32 `scales` [rows]."""
    lib = L.load()
    rows = latent.shape[0]
    d = dims.c()
    rc = lib.mla_quantize_latent_fp8(ctypes.byref(d), _dt(latent), _ptr(latent), latent.stride(0), rows, _ptr(codes),
                                     codes.stride(0), _ptr(scales), _stream(stream))
    _check("mla_quantize_latent_fp8", rc)
    return codes, scales


def mla_decode_absorbed_fp8(dims: Dims, q_abs, cache: LatentCacheFp8, block_table, seqlens, o_lat=None, lse=None,
                            workspace=None, stream=None):
    lib = L.load()
    B, s_q, H, _ = q_abs.shape
    if o_lat is None:
        o_lat = torch.empty(B, s_q, H, dims.d_c, dtype=q_abs.dtype, device=q_abs.device)
    if lse is None:
        lse = torch.empty(B, s_q, H, dtype=torch.float32, device=q_abs.device)
    d = dims.c()
    max_pages = block_table.shape[1]
    need = lib.mla_decode_fp8_workspace_size(ctypes.byref(d), B, s_q, max_pages)
    workspace, wsb = _workspace(need, q_abs.device, workspace)
    cc = cache.c()
    rc = lib.mla_decode_absorbed_fp8(ctypes.byref(d), _dt(q_abs), B, s_q, _ptr(q_abs), ctypes.byref(cc),
                                     _ptr(_i32(block_table)), max_pages, _ptr(_i32(seqlens)), _ptr(o_lat), _ptr(lse),
                                     _ptr(workspace) if workspace is not None else None, wsb, _stream(stream))
    _check("mla_decode_absorbed_fp8", rc)
    return o_lat, lse


# ---- 8-bit cache written directly and read back; attention over selected pages -----------------
# These calls check what they are given: a tensor of another shape or dtype, one that is not contiguous
# where the library wants rows laid end to end, or one that is not on the current device raises before
# anything is enqueued.
# The checks of one tensor are a single condition (a decode step's calls are short, and so is the time to issue
# them); what was wrong is found out when it fails.
def _current(t: torch.Tensor) -> int:
    """The current device, which has to hold t (the library enqueues on it)."""
    if not t.is_cuda:
        raise ValueError(f"libmla takes device tensors, got {t.device}")
    dev = torch.cuda.current_device()
    if t.get_device() != dev:
        raise ValueError(f"libmla takes tensors of the current device (cuda:{dev}), got {t.device}")
    return dev


def _refuse(dev: int, name: str, t: torch.Tensor, dtype, what: str):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: libmla takes tensors of the current device (cuda:{dev}), got {t.device}")
    raise ValueError(f"{name}: expected {what}, got {tuple(t.shape)} with strides {t.stride()}")


def _need(dev: int, name: str, t: torch.Tensor, shape, dtype) -> int:
    """data_ptr of a contiguous tensor of this shape and dtype on device `dev`."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        _refuse(dev, name, t, dtype, f"a contiguous tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _need_rows(dev: int, name: str, t: torch.Tensor, rows: int, width: int, dtype):
    """(data_ptr, elements between rows) of a matrix of at least `rows` rows of `width` values laid end to end."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not dtype or t.get_device() != dev or len(shape) != 2 or shape[0] < rows or shape[1] != width or \
            (stride[1] != 1 and width > 1):
        _refuse(dev, name, t, dtype, f"at least {rows} rows of {width} values")
    return t.data_ptr(), stride[0]


def _cache_arg(dev: int, dims: Dims, cache, dtype):
    """The checked descriptor of a latent cache (LatentCache or LatentCacheFp8)."""
    n = cache.num_pages
    rope, rope_stride = _need_rows(dev, "cache.rope", cache.rope, n * 64, dims.d_r, dtype)
    if isinstance(cache, LatentCacheFp8):
        codes, code_stride = _need_rows(dev, "cache.codes", cache.codes, n * 64, dims.d_c, torch.uint8)
        scales = cache.scales
        if scales.dtype is not torch.float32 or scales.get_device() != dev or scales.dim() != 1 or \
                scales.numel() < n * 64 or not scales.is_contiguous():
            _refuse(dev, "cache.scales", scales, torch.float32, f"at least {n * 64} contiguous values")
        return L.MlaLatentCacheFp8(codes, code_stride, scales.data_ptr(), rope, rope_stride, n)
    latent, latent_stride = _need_rows(dev, "cache.latent", cache.latent, n * 64, dims.d_c, dtype)
    return L.MlaLatentCache(latent, latent_stride, rope, rope_stride, n)


def _table(dev: int, B: int, block_table, seqlens):
    """(block table, its row length, lengths) as pointers and sizes."""
    if block_table.dim() != 2:
        raise ValueError("block_table: expected [B, max_pages]")
    max_pages = block_table.shape[1]
    return (_need(dev, "block_table", block_table, (B, max_pages), torch.int32), max_pages,
            None if seqlens is None else _need(dev, "seqlens", seqlens, (B,), torch.int32))


def _new(dev: int, stream, make, *shape, dtype):
    """A tensor made by `make` (torch.empty, torch.zeros) for use on `stream`: taken from that stream's pool,
    so that no memory another stream still works on is handed out, nor this one's while it does."""
    if stream is None:
        return make(*shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return make(*shape, dtype=dtype, device=dev)


def _space(dev: int, nbytes: int, workspace, stream):
    """(workspace or None, its pointer, its size): taken from torch's allocator when none is given."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = _new(dev, stream, torch.empty, nbytes, dtype=torch.uint8)
    elif not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError(f"workspace: expected a contiguous tensor on cuda:{dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _stream_on(dev: int, stream) -> int:
    if stream is None:
        return _raw_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream: expected a stream of the current device (cuda:{dev})")
    return stream.cuda_stream


# the current stream's handle, without making a Stream object where this torch has the short way
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


@functools.lru_cache(maxsize=1024)
def _bytes_of(fn: str, dev: int, H: int, D: int, d_r: int, d_c: int, *args) -> int:
    return getattr(L.load(), fn)(ctypes.byref(Dims(H, D, d_r, d_c, d_c).c()), *args)


def _bytes(fn: str, dev: int, dims: Dims, *args) -> int:
    """A workspace size of the library: it depends on the head layout, the sizes and the device alone."""
    return _bytes_of(fn, dev, dims.H, dims.D, dims.d_r, dims.d_c, *args)


def _width(dims: Dims) -> int:
    return dims.d_c + dims.d_r


def mla_append_cache_fp8(dims: Dims, x, w_dkv_kr, gamma, seqlens, block_table, cache: LatentCacheFp8, workspace=None,
                         stream=None):
    """a1 into an 8-bit cache: the new tokens' latents leave the projection as E4M3 codes and one scale
    per row (quantised from fp32), their RoPE keys as in mla_append_cache. x [B, s_q, C], w_dkv_kr
    [C, d_c + d_r], gamma [d_c] or None."""
    lib = L.load()
    dt = _dt(x)
    B, s_q, C = x.shape
    dev = _current(x)
    px = _need(dev, "x", x, (B, s_q, C), x.dtype)
    pw = _need(dev, "w_dkv_kr", w_dkv_kr, (C, _width(dims)), x.dtype)
    pg = None if gamma is None else _need(dev, "gamma", gamma, (dims.d_c,), x.dtype)
    table, max_pages, lens = _table(dev, B, block_table, seqlens)
    cc = _cache_arg(dev, dims, cache, x.dtype)
    d = dims.c()
    workspace, ws, wsb = _space(dev, _bytes("mla_append_fp8_workspace_size", dev, dims, dt, B, s_q, C), workspace, stream)
    rc = lib.mla_append_cache_fp8(ctypes.byref(d), dt, B, s_q, px, C, pw, pg, lens, table, max_pages, ctypes.byref(cc),
                                  ws, wsb, _stream_on(dev, stream))
    _check("mla_append_cache_fp8", rc)


def mla_read_latent_fp8(dims: Dims, cache: LatentCacheFp8, block_table, row_offsets, out, first=None, stream=None):
    """Rows of an 8-bit cache back in storage type: out[row_offsets[b] + i] = [c ; k_r] of position
    first[b] + i (first None: from position 0) of sequence b. out [n_rows, d_c + d_r]; rows from
    row_offsets[B] on are left as they were. An out of no rows is a call without work."""
    lib = L.load()
    dt = _dt(out)
    dev = _current(out)
    B = block_table.shape[0]
    table, max_pages, _ = _table(dev, B, block_table, None)
    off = _need(dev, "row_offsets", row_offsets, (B + 1,), torch.int32)
    pf = None if first is None else _need(dev, "first", first, (B,), torch.int32)
    po, out_stride = _need_rows(dev, "out", out, 0, _width(dims), out.dtype)
    cc = _cache_arg(dev, dims, cache, out.dtype)
    if out.shape[0] == 0:   # a ragged batch without rows: nothing to enqueue (the library takes n_rows > 0)
        return out
    d = dims.c()
    rc = lib.mla_read_latent_fp8(ctypes.byref(d), dt, B, ctypes.byref(cc), table, max_pages, pf, off, out.shape[0],
                                 po, out_stride, _stream_on(dev, stream))
    _check("mla_read_latent_fp8", rc)
    return out


def mla_update_page_keys(dims: Dims, cache, block_table, seqlens, s_q: int, keys, stream=None):
    """keys [num_pages, d_c + d_r]: the mean row of every page that holds one of a sequence's s_q newest
    positions, from a LatentCache or a LatentCacheFp8. s_q >= the longest sequence rebuilds every key. A key
    holds all of a page's rows below seqlens: with several new tokens, scores of the earlier ones depend on the later
    ones unless keys and scores are made token by token (s_q = 1, seqlens lowered to the token's own)."""
    lib = L.load()
    dt = _dt(keys)
    dev = _current(keys)
    B = block_table.shape[0]
    table, max_pages, lens = _table(dev, B, block_table, seqlens)
    pk, key_stride = _need_rows(dev, "keys", keys, cache.num_pages, _width(dims), keys.dtype)
    cc = _cache_arg(dev, dims, cache, keys.dtype)
    name = "mla_update_page_keys_fp8" if isinstance(cache, LatentCacheFp8) else "mla_update_page_keys"
    d = dims.c()
    rc = getattr(lib, name)(ctypes.byref(d), dt, B, s_q, ctypes.byref(cc), table, max_pages, lens, pk, key_stride,
                            _stream_on(dev, stream))
    _check(name, rc)
    return keys


def mla_score_pages(dims: Dims, q_abs, keys, block_table, seqlens, scores=None, workspace=None, stream=None):
    """scores [B, s_q, max_pages] (fp32): for every page a token sees, the sum over the heads of the softmax
    over its pages of sm_scale * q_abs · key. Entries of pages it does not see are left as they were
    (zeros in a tensor made here)."""
    lib = L.load()
    dt = _dt(q_abs)
    dev = _current(q_abs)
    B, s_q = q_abs.shape[0], q_abs.shape[1]
    pq = _need(dev, "q_abs", q_abs, (B, s_q, dims.H, _width(dims)), q_abs.dtype)
    table, max_pages, lens = _table(dev, B, block_table, seqlens)
    pk, key_stride = _need_rows(dev, "keys", keys, 1, _width(dims), q_abs.dtype)
    if scores is None:
        scores = _new(dev, stream, torch.zeros, B, s_q, max_pages, dtype=torch.float32)
    ps = _need(dev, "scores", scores, (B, s_q, max_pages), torch.float32)
    d = dims.c()
    need = _bytes("mla_score_pages_workspace_size", dev, dims, dt, B, s_q, max_pages)
    workspace, ws, wsb = _space(dev, need, workspace, stream)
    rc = lib.mla_score_pages(ctypes.byref(d), dt, B, s_q, pq, pk, key_stride, keys.shape[0], table,
                             max_pages, lens, ps, ws, wsb, _stream_on(dev, stream))
    _check("mla_score_pages", rc)
    return scores


def mla_select_pages(dims: Dims, scores, seqlens, k: int, n_first: int = 0, n_recent: int = 1, pages=None, counts=None,
                     stream=None):
    """The k pages of largest score of each token, ascending: (pages [B, s_q, k] int32 with -1 after the
    last, counts [B, s_q] int32). The first n_first and last n_recent visible pages are always kept."""
    lib = L.load()
    dev = _current(scores)
    if scores.dim() != 3:
        raise ValueError("scores: expected [B, s_q, max_pages]")
    B, s_q, max_pages = scores.shape
    ps = _need(dev, "scores", scores, (B, s_q, max_pages), torch.float32)
    lens = _need(dev, "seqlens", seqlens, (B,), torch.int32)
    if pages is None:
        pages = _new(dev, stream, torch.empty, B, s_q, k, dtype=torch.int32)
    if counts is None:
        counts = _new(dev, stream, torch.empty, B, s_q, dtype=torch.int32)
    pp = _need(dev, "pages", pages, (B, s_q, k), torch.int32)
    pc = _need(dev, "counts", counts, (B, s_q), torch.int32)
    d = dims.c()
    rc = lib.mla_select_pages(ctypes.byref(d), B, s_q, ps, max_pages, lens, k, n_first, n_recent, pp, pc,
                              _stream_on(dev, stream))
    _check("mla_select_pages", rc)
    return pages, counts


def mla_decode_absorbed_sparse(dims: Dims, q_abs, cache, block_table, seqlens, pages, counts, o_lat=None, lse=None,
                               workspace=None, stream=None):
    """Absorbed decode over the visible positions of the listed pages (pages [B, s_q, k], counts [B, s_q] as
    mla_select_pages gives them) of a LatentCache or a LatentCacheFp8. A token with no page gets zeros
    and lse = -inf."""
    lib = L.load()
    dt = _dt(q_abs)
    dev = _current(q_abs)
    B, s_q = q_abs.shape[0], q_abs.shape[1]
    pq = _need(dev, "q_abs", q_abs, (B, s_q, dims.H, _width(dims)), q_abs.dtype)
    table, max_pages, lens = _table(dev, B, block_table, seqlens)
    k = pages.shape[-1]
    pp = _need(dev, "pages", pages, (B, s_q, k), torch.int32)
    pc = _need(dev, "counts", counts, (B, s_q), torch.int32)
    cc = _cache_arg(dev, dims, cache, q_abs.dtype)
    if o_lat is None:
        o_lat = _new(dev, stream, torch.empty, B, s_q, dims.H, dims.d_c, dtype=q_abs.dtype)
    if lse is None:
        lse = _new(dev, stream, torch.empty, B, s_q, dims.H, dtype=torch.float32)
    po = _need(dev, "o_lat", o_lat, (B, s_q, dims.H, dims.d_c), q_abs.dtype)
    pl = _need(dev, "lse", lse, (B, s_q, dims.H), torch.float32)
    fp8 = isinstance(cache, LatentCacheFp8)
    name = "mla_decode_absorbed_sparse_fp8" if fp8 else "mla_decode_absorbed_sparse"
    size = "mla_decode_sparse_fp8_workspace_size" if fp8 else "mla_decode_sparse_workspace_size"
    d = dims.c()
    workspace, ws, wsb = _space(dev, _bytes(size, dev, dims, dt, B, s_q, k), workspace, stream)
    rc = getattr(lib, name)(ctypes.byref(d), dt, B, s_q, pq, ctypes.byref(cc), table, max_pages, lens, pp, pc, k, po, pl,
                            ws, wsb, _stream_on(dev, stream))
    _check(name, rc)
    return o_lat, lse


def mla_out_proj(dims: Dims, o_lat, w_uv, out=None, w_o=None, out_model=None, stream=None):
    lib = L.load()
    B, s_q, H, _ = o_lat.shape
    if out is None:
        out = torch.empty(B, s_q, H, dims.d_v, dtype=o_lat.dtype, device=o_lat.device)
    C = 0
    if w_o is not None:
        C = w_o.shape[1]
        if out_model is None:
            out_model = torch.empty(B, s_q, C, dtype=o_lat.dtype, device=o_lat.device)
    d = dims.c()
    rc = lib.mla_out_proj(ctypes.byref(d), _dt(o_lat), B, s_q, _ptr(o_lat), _ptr(w_uv), _ptr(out), _ptr(w_o), C,
                          _ptr(out_model), _stream(stream))
    _check("mla_out_proj", rc)
    return (out, out_model) if w_o is not None else out


def mla_decode_gqla_grouped(dims: Dims, q_nope, q_rope_raw, cache: GqaCache, block_table, seqlens, out=None,
                            lse=None, workspace=None, stream=None):
    lib = L.load()
    B, s_q, H, _ = q_nope.shape
    if out is None:
        out = torch.empty(B, s_q, H, dims.d_v, dtype=q_nope.dtype, device=q_nope.device)
    if lse is None:
        lse = torch.empty(B, s_q, H, dtype=torch.float32, device=q_nope.device)
    d = dims.c()
    max_pages = block_table.shape[1]
    need = lib.mla_gqla_workspace_size(ctypes.byref(d), _dt(q_nope), B, s_q, max_pages)
    workspace, wsb = _workspace(need, q_nope.device, workspace)
    cc = cache.c()
    rc = lib.mla_decode_gqla_grouped(ctypes.byref(d), _dt(q_nope), B, s_q, _ptr(q_nope), _ptr(q_rope_raw),
                                     ctypes.byref(cc), _ptr(_i32(block_table)), max_pages, _ptr(_i32(seqlens)),
                                     _ptr(out), _ptr(lse), _ptr(workspace) if workspace is not None else None, wsb,
                                     _stream(stream))
    _check("mla_decode_gqla_grouped", rc)
    return out, lse


def mla_append_gqa_cache(dims: Dims, x, w_dkv_kr, gamma, w_uk_g, w_uv_g, seqlens, block_table, cache: GqaCache,
                         workspace=None, stream=None):
    """Append this step's tokens to the expanded GQA cache: k_r and, per group, K = W_UK[g]·c and
    V = c·W_UV[g] of c = RMSNorm(x·W_DKV) (x [B, s_q, C], w_uk_g [g, D, d_c], w_uv_g [g, d_c, d_v])."""
    lib = L.load()
    B, s_q, C = x.shape
    d = dims.c()
    need = lib.mla_gqa_append_workspace_size(ctypes.byref(d), B, s_q, C)
    workspace, wsb = _workspace(need, x.device, workspace)
    cc = cache.c()
    rc = lib.mla_append_gqa_cache(ctypes.byref(d), _dt(x), B, s_q, _ptr(x), C, _ptr(w_dkv_kr), _ptr(gamma),
                                  _ptr(w_uk_g), _ptr(w_uv_g), _ptr(_i32(seqlens)), _ptr(_i32(block_table)),
                                  block_table.shape[1], ctypes.byref(cc),
                                  _ptr(workspace) if workspace is not None else None, wsb, _stream(stream))
    _check("mla_append_gqa_cache", rc)


def mla_preabsorb_out_weights(dims: Dims, w_uv, w_o, w_uvo=None, stream=None):
    """W_UVO [H, d_c, C] with W_UVO[h] = W_UV[h] · W_O[h*d_v:(h+1)*d_v] (w_uv [H, d_c, d_v], w_o [H*d_v, C])."""
    lib = L.load()
    C = w_o.shape[1]
    if w_uvo is None:
        w_uvo = torch.empty(dims.H, dims.d_c, C, dtype=w_uv.dtype, device=w_uv.device)
    d = dims.c()
    rc = lib.mla_preabsorb_out_weights(ctypes.byref(d), _dt(w_uv), _ptr(w_uv), _ptr(w_o), C, _ptr(w_uvo),
                                       _stream(stream))
    _check("mla_preabsorb_out_weights", rc)
    return w_uvo


def mla_out_proj_preabsorbed(dims: Dims, o_lat, w_uvo, out_model=None, stream=None):
    """out_model [B, s_q, C] = concat_h(o_lat[..., h, :]) · W_UVO (o_lat [B, s_q, H, d_c], w_uvo [H, d_c, C])."""
    lib = L.load()
    B, s_q, H, _ = o_lat.shape
    C = w_uvo.shape[-1]
    if out_model is None:
        out_model = torch.empty(B, s_q, C, dtype=o_lat.dtype, device=o_lat.device)
    d = dims.c()
    rc = lib.mla_out_proj_preabsorbed(ctypes.byref(d), _dt(o_lat), B, s_q, _ptr(o_lat), _ptr(w_uvo), C,
                                      _ptr(out_model), _stream(stream))
    _check("mla_out_proj_preabsorbed", rc)
    return out_model


def mla_check_status(stream=None) -> int:
    return L.load().mla_check_status(_stream(stream))


def mla_status_string(status: int) -> str:
    return L.load().mla_status_string(status).decode()


def mla_build_info() -> str:
    return L.load().mla_build_info().decode()


def mla_launch_count() -> int:
    return int(L.load().mla_launch_count())
