"""Python binding over the kattn C ABI (argument marshalling only).

Every function takes torch CUDA tensors, checks dtypes/shapes/contiguity,
and passes raw device pointers plus torch's current CUDA stream to the
library.  All computation happens in the library's CUDA kernels.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib

P_MODES = {"f32": 0, "bf16": 1, "e4m3": 2, "e4m3x448": 3, "e4m3x256": 4, "e4m3direct": 5}

# Device error bits (KATTN_DEVERR_* in kattn.h), as get_device_status returns them.
DEVERR_BAD_SEQUENCE = 0x1
DEVERR_TIMEOUT = 0x2
DEVERR_BAD_PAGE = 0x4
DEVERR_NO_PAGES = 0x8


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _need(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def get_tiling() -> tuple:
    lib = _lib.load()
    c, bk = ctypes.c_int(), ctypes.c_int()
    lib.kattn_get_tiling(ctypes.byref(c), ctypes.byref(bk))
    return c.value, bk.value


def expf_constants() -> list:
    """The library's exact-mode exp constants: [K, C2, C0, C1, T[0..63]]."""
    lib = _lib.load()
    buf = (ctypes.c_double * 68)()
    _lib.check("kattn_expf_constants", lib.kattn_expf_constants(buf))
    return list(buf)


def decode_workspace_size(B: int, M: int, Hq: int, max_ctx: int) -> int:
    return int(_lib.load().kattn_decode_workspace_size(B, M, Hq, max_ctx))


def decode_launch_count(B: int, M: int, Hq: int, Hkv: int, max_ctx: int) -> int:
    """Kernels one fast-mode decode launches for these sizes on the current
    device (kattn_decode_launch_count)."""
    return int(_lib.load().kattn_decode_launch_count(B, M, Hq, Hkv, max_ctx))


def alloc_workspace(B: int, M: int, Hq: int, max_ctx: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace for kattn_decode (allocated by torch, not the library)."""
    n = decode_workspace_size(B, M, Hq, max_ctx)
    if n == 0:
        raise ValueError("invalid sizes for a decode workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def quantize_kv(x: torch.Tensor, out_q: torch.Tensor, out_scale: torch.Tensor,
                dst_row0: int = 0) -> None:
    """x [n_rows][Hkv][d] float32 -> out_q [Hkv][cap][d] int8, out_scale [Hkv][cap]."""
    _need(x, torch.float32, "x", 3)
    _need(out_q, torch.int8, "out_q", 3)
    _need(out_scale, torch.float32, "out_scale", 2)
    n_rows, n_kv, d = x.shape
    cap = out_q.shape[1]
    if out_q.shape[0] != n_kv or out_q.shape[2] != d or tuple(out_scale.shape) != (n_kv, cap):
        raise ValueError("cache shapes do not match x")
    lib = _lib.load()
    _lib.check("kattn_quantize_kv", lib.kattn_quantize_kv(
        _ptr(x), n_rows, n_kv, d, n_kv * d, _ptr(out_q), _ptr(out_scale), dst_row0, cap,
        _stream(x.device)))


def quantize_kv_rows(x: torch.Tensor, dst_rows: torch.Tensor, out_q: torch.Tensor,
                     out_scale: torch.Tensor) -> None:
    """Append form: row r of x [n_rows][Hkv][d] goes to cache row dst_rows[r]."""
    _need(x, torch.float32, "x", 3)
    _need(dst_rows, torch.int64, "dst_rows", 1)
    _need(out_q, torch.int8, "out_q", 3)
    _need(out_scale, torch.float32, "out_scale", 2)
    n_rows, n_kv, d = x.shape
    cap = out_q.shape[1]
    if dst_rows.numel() != n_rows:
        raise ValueError("dst_rows must have one entry per row of x")
    if out_q.shape[0] != n_kv or out_q.shape[2] != d or tuple(out_scale.shape) != (n_kv, cap):
        raise ValueError("cache shapes do not match x")
    lib = _lib.load()
    _lib.check("kattn_quantize_kv_rows", lib.kattn_quantize_kv_rows(
        _ptr(x), n_rows, n_kv, d, n_kv * d, _ptr(dst_rows), _ptr(out_q), _ptr(out_scale), cap,
        _stream(x.device)))


def decode(q, k, k_scale, v, v_scale, row_start, ctx_len, max_ctx: int, *,
           out=None, p_mode=0, exact_mode=False, sm_scale: float = 0.0, workspace=None):
    """Decode attention; returns out [B][M][Hq][d] float32.

    q [B][M][Hq][d] f32; k, v [Hkv][cap][d] int8; k_scale, v_scale [Hkv][cap]
    f32; row_start [B] int64; ctx_len [B] int32 (all on the same CUDA device).
    p_mode: an int or a name of P_MODES -- "f32", "bf16", "e4m3", "e4m3x448",
    "e4m3x256", or "e4m3direct" (e4m3 P fed straight to the P.V MMA as one
    f16 operand p~ * v_scale; fast mode only).
    workspace: a zeroed uint8 tensor of decode_workspace_size(...) bytes
    (fast mode); allocated here with torch if None.  Exact mode needs none; a
    zeroed one of at least 256 bytes, if given, receives the device error bits.
    """
    _need(q, torch.float32, "q", 4)
    _need(k, torch.int8, "k", 3)
    _need(v, torch.int8, "v", 3)
    _need(k_scale, torch.float32, "k_scale", 2)
    _need(v_scale, torch.float32, "v_scale", 2)
    _need(row_start, torch.int64, "row_start", 1)
    _need(ctx_len, torch.int32, "ctx_len", 1)
    B, M, Hq, d = q.shape
    Hkv, cap, _ = k.shape
    if tuple(v.shape) != tuple(k.shape) or tuple(k_scale.shape) != (Hkv, cap) \
            or tuple(v_scale.shape) != (Hkv, cap):
        raise ValueError("k/v/scales shapes disagree")
    if row_start.numel() != B or ctx_len.numel() != B:
        raise ValueError("row_start / ctx_len must have B entries")
    mode = P_MODES.get(p_mode, p_mode) if isinstance(p_mode, str) else int(p_mode)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, torch.float32, "out", 4)
    ws_bytes = 0
    if not exact_mode and workspace is None:
        workspace = alloc_workspace(B, M, Hq, max_ctx, q.device)
    if workspace is not None:                 # exact mode: optional, for the error word
        _need(workspace, torch.uint8, "workspace", 1)
        ws_bytes = workspace.numel()
    lib = _lib.load()
    _lib.check("kattn_decode", lib.kattn_decode(
        _ptr(q), _ptr(k), _ptr(k_scale), _ptr(v), _ptr(v_scale), _ptr(row_start), _ptr(ctx_len),
        B, M, Hq, Hkv, d, cap, int(max_ctx), float(sm_scale), mode, 1 if exact_mode else 0,
        _ptr(out), _ptr(workspace), ws_bytes, _stream(q.device)))
    return out


def decode_paged(q, k, k_scale, v, v_scale, block_table, page_rows: int, ctx_len, max_ctx: int,
                 *, out=None, p_mode=0, exact_mode=False, sm_scale: float = 0.0, workspace=None):
    """Decode attention over a paged cache; returns out [B][M][Hq][d] float32.

    Key t of sequence b is row block_table[b][t // page_rows] * page_rows +
    t % page_rows of every kv-head plane of k, v [Hkv][cap][d] (int8) and
    k_scale, v_scale [Hkv][cap] (f32).  block_table: int32 [B][max_pages];
    page_rows: 32 * 2^k, dividing cap.  Otherwise as decode().
    """
    _need(q, torch.float32, "q", 4)
    _need(k, torch.int8, "k", 3)
    _need(v, torch.int8, "v", 3)
    _need(k_scale, torch.float32, "k_scale", 2)
    _need(v_scale, torch.float32, "v_scale", 2)
    _need(block_table, torch.int32, "block_table", 2)
    _need(ctx_len, torch.int32, "ctx_len", 1)
    B, M, Hq, d = q.shape
    Hkv, cap, _ = k.shape
    if tuple(v.shape) != tuple(k.shape) or tuple(k_scale.shape) != (Hkv, cap) \
            or tuple(v_scale.shape) != (Hkv, cap):
        raise ValueError("k/v/scales shapes disagree")
    if block_table.shape[0] != B or ctx_len.numel() != B:
        raise ValueError("block_table / ctx_len must have B rows")
    mode = P_MODES.get(p_mode, p_mode) if isinstance(p_mode, str) else int(p_mode)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, torch.float32, "out", 4)
    ws_bytes = 0
    if not exact_mode and workspace is None:
        workspace = alloc_workspace(B, M, Hq, max_ctx, q.device)
    if workspace is not None:                 # exact mode: optional, for the error word
        _need(workspace, torch.uint8, "workspace", 1)
        ws_bytes = workspace.numel()
    lib = _lib.load()
    _lib.check("kattn_decode_paged", lib.kattn_decode_paged(
        _ptr(q), _ptr(k), _ptr(k_scale), _ptr(v), _ptr(v_scale), _ptr(block_table),
        int(block_table.shape[1]), int(page_rows), _ptr(ctx_len), B, M, Hq, Hkv, d, cap,
        int(max_ctx), float(sm_scale), mode, 1 if exact_mode else 0, _ptr(out),
        _ptr(workspace), ws_bytes, _stream(q.device)))
    return out


def decode_append(q, k_new, v_new, dst_rows, k, k_scale, v, v_scale, row_start, ctx_len,
                  max_ctx: int, *, out=None, p_mode=0, sm_scale: float = 0.0, workspace=None):
    """Append rows k_new / v_new [n][Hkv][d] f32 at cache rows dst_rows [n]
    (int64), then decode (fast mode): one call of kattn_decode_append."""
    _need(q, torch.float32, "q", 4)
    _need(k_new, torch.float32, "k_new", 3)
    _need(v_new, torch.float32, "v_new", 3)
    _need(dst_rows, torch.int64, "dst_rows", 1)
    _need(k, torch.int8, "k", 3)
    _need(v, torch.int8, "v", 3)
    _need(k_scale, torch.float32, "k_scale", 2)
    _need(v_scale, torch.float32, "v_scale", 2)
    _need(row_start, torch.int64, "row_start", 1)
    _need(ctx_len, torch.int32, "ctx_len", 1)
    B, M, Hq, d = q.shape
    Hkv, cap, _ = k.shape
    n_new = k_new.shape[0]
    if tuple(v_new.shape) != tuple(k_new.shape) or dst_rows.numel() != n_new \
            or k_new.shape[1] != Hkv or k_new.shape[2] != d:
        raise ValueError("k_new / v_new / dst_rows shapes disagree with the cache")
    if tuple(v.shape) != tuple(k.shape) or tuple(k_scale.shape) != (Hkv, cap) \
            or tuple(v_scale.shape) != (Hkv, cap):
        raise ValueError("k/v/scales shapes disagree")
    mode = P_MODES.get(p_mode, p_mode) if isinstance(p_mode, str) else int(p_mode)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, torch.float32, "out", 4)
    if workspace is None:
        workspace = alloc_workspace(B, M, Hq, max_ctx, q.device)
    _need(workspace, torch.uint8, "workspace", 1)
    lib = _lib.load()
    _lib.check("kattn_decode_append", lib.kattn_decode_append(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(dst_rows), n_new, Hkv * d, _ptr(k), _ptr(k_scale),
        _ptr(v), _ptr(v_scale), _ptr(row_start), _ptr(ctx_len), B, M, Hq, Hkv, d, cap,
        int(max_ctx), float(sm_scale), mode, _ptr(out), _ptr(workspace), workspace.numel(),
        _stream(q.device)))
    return out


def decode_paged_append(q, k_new, v_new, dst_rows, k, k_scale, v, v_scale, block_table,
                        page_rows: int, ctx_len, max_ctx: int, *, out=None, p_mode=0,
                        sm_scale: float = 0.0, workspace=None):
    """Append rows k_new / v_new [n][Hkv][d] f32 at PHYSICAL pool rows
    dst_rows [n] (int64), then decode the paged cache (fast mode): one call of
    kattn_decode_paged_append.  Paging arguments as decode_paged()."""
    _need(q, torch.float32, "q", 4)
    _need(k_new, torch.float32, "k_new", 3)
    _need(v_new, torch.float32, "v_new", 3)
    _need(dst_rows, torch.int64, "dst_rows", 1)
    _need(k, torch.int8, "k", 3)
    _need(v, torch.int8, "v", 3)
    _need(k_scale, torch.float32, "k_scale", 2)
    _need(v_scale, torch.float32, "v_scale", 2)
    _need(block_table, torch.int32, "block_table", 2)
    _need(ctx_len, torch.int32, "ctx_len", 1)
    B, M, Hq, d = q.shape
    Hkv, cap, _ = k.shape
    n_new = k_new.shape[0]
    if tuple(v_new.shape) != tuple(k_new.shape) or dst_rows.numel() != n_new \
            or k_new.shape[1] != Hkv or k_new.shape[2] != d:
        raise ValueError("k_new / v_new / dst_rows shapes disagree with the cache")
    if tuple(v.shape) != tuple(k.shape) or tuple(k_scale.shape) != (Hkv, cap) \
            or tuple(v_scale.shape) != (Hkv, cap):
        raise ValueError("k/v/scales shapes disagree")
    if block_table.shape[0] != B or ctx_len.numel() != B:
        raise ValueError("block_table / ctx_len must have B rows")
    mode = P_MODES.get(p_mode, p_mode) if isinstance(p_mode, str) else int(p_mode)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, torch.float32, "out", 4)
    if workspace is None:
        workspace = alloc_workspace(B, M, Hq, max_ctx, q.device)
    _need(workspace, torch.uint8, "workspace", 1)
    lib = _lib.load()
    _lib.check("kattn_decode_paged_append", lib.kattn_decode_paged_append(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(dst_rows), n_new, Hkv * d, _ptr(k), _ptr(k_scale),
        _ptr(v), _ptr(v_scale), _ptr(block_table), int(block_table.shape[1]), int(page_rows),
        _ptr(ctx_len), B, M, Hq, Hkv, d, cap, int(max_ctx), float(sm_scale), mode, _ptr(out),
        _ptr(workspace), workspace.numel(), _stream(q.device)))
    return out


WINDOW_KEYS = 512   # KATTN_WINDOW_KEYS: keys per window, the unit of a shard


def shard_partials_size(B: int, M: int, Hq: int, Hkv: int, win_per_shard: int) -> int:
    """Bytes of one shard's partials array (kattn_shard_partials_size)."""
    return int(_lib.load().kattn_shard_partials_size(B, M, Hq, Hkv, win_per_shard))


def partial_stride(R: int) -> int:
    """Floats per (sequence, window, kv head) partial: o[R][128], m[R], l[R],
    padded to a multiple of 4."""
    return R * 128 + (2 * R + 3) // 4 * 4


def decode_shard(q, k, k_scale, v, v_scale, row_start, ctx_len, max_ctx: int, shard: int,
                 win_per_shard: int, *, partials=None, p_mode=0, sm_scale: float = 0.0,
                 workspace=None):
    """Window partials of context-parallel shard `shard` (kattn_decode_shard).

    The cache k, v [Hkv][cap][d] (int8) and k_scale, v_scale [Hkv][cap] hold
    key t of sequence b, for the shard's keys t in [512 * shard * Ws,
    min(512 * (shard + 1) * Ws, ctx_len[b] + M - 1)), at row row_start[b] + t -
    512 * shard * Ws; ctx_len holds the global context lengths.  Returns
    partials float32 [B][Ws][Hkv][partial_stride(g * M)].
    """
    _need(q, torch.float32, "q", 4)
    _need(k, torch.int8, "k", 3)
    _need(v, torch.int8, "v", 3)
    _need(k_scale, torch.float32, "k_scale", 2)
    _need(v_scale, torch.float32, "v_scale", 2)
    _need(row_start, torch.int64, "row_start", 1)
    _need(ctx_len, torch.int32, "ctx_len", 1)
    B, M, Hq, d = q.shape
    Hkv, cap, _ = k.shape
    if tuple(v.shape) != tuple(k.shape) or tuple(k_scale.shape) != (Hkv, cap) \
            or tuple(v_scale.shape) != (Hkv, cap):
        raise ValueError("k/v/scales shapes disagree")
    if row_start.numel() != B or ctx_len.numel() != B:
        raise ValueError("row_start / ctx_len must have B entries")
    if Hq % Hkv != 0:
        raise ValueError("Hq must be a multiple of Hkv")
    stride = partial_stride(Hq // Hkv * M)
    shape = (B, win_per_shard, Hkv, stride)
    if partials is None:
        partials = torch.empty(shape, dtype=torch.float32, device=q.device)
    else:
        _need(partials, torch.float32, "partials", 4)
        if tuple(partials.shape) != shape:
            raise ValueError(f"partials must have shape {shape}")
    if workspace is None:
        workspace = alloc_workspace(B, M, Hq, max_ctx, q.device)
    _need(workspace, torch.uint8, "workspace", 1)
    mode = P_MODES.get(p_mode, p_mode) if isinstance(p_mode, str) else int(p_mode)
    lib = _lib.load()
    _lib.check("kattn_decode_shard", lib.kattn_decode_shard(
        _ptr(q), _ptr(k), _ptr(k_scale), _ptr(v), _ptr(v_scale), _ptr(row_start), _ptr(ctx_len),
        B, M, Hq, Hkv, d, cap, int(max_ctx), int(shard), int(win_per_shard), float(sm_scale),
        mode, _ptr(partials), _ptr(workspace), workspace.numel(), _stream(q.device)))
    return partials


def merge_shards(partials, ctx_len, M: int, Hq: int, max_ctx: int, *, out=None, workspace=None):
    """Combine gathered shard partials [n_shards][B][Ws][Hkv][stride] into
    out [B][M][Hq][128] float32 (kattn_merge_shards)."""
    _need(partials, torch.float32, "partials", 5)
    _need(ctx_len, torch.int32, "ctx_len", 1)
    n_shards, B, Ws, Hkv, stride = partials.shape
    if ctx_len.numel() != B:
        raise ValueError("ctx_len must have B entries")
    if Hq % Hkv != 0 or stride != partial_stride(Hq // Hkv * M):
        raise ValueError("partials do not match M, Hq")
    if out is None:
        out = torch.empty((B, M, Hq, 128), dtype=torch.float32, device=partials.device)
    else:
        _need(out, torch.float32, "out", 4)
        if tuple(out.shape) != (B, M, Hq, 128):
            raise ValueError("out must have shape [B][M][Hq][128]")
    if workspace is None:
        workspace = torch.zeros(256, dtype=torch.uint8, device=partials.device)
    _need(workspace, torch.uint8, "workspace", 1)
    lib = _lib.load()
    _lib.check("kattn_merge_shards", lib.kattn_merge_shards(
        _ptr(partials), _ptr(ctx_len), B, int(M), int(Hq), Hkv, 128, int(max_ctx), n_shards, Ws,
        _ptr(out), _ptr(workspace), workspace.numel(), _stream(partials.device)))
    return out


def hash_rows(x: torch.Tensor) -> torch.Tensor:
    """FNV-1a 64 of every row of x (a CUDA tensor whose last dimension is
    contiguous; rows = all leading indices).  Returns int64 [rows] holding
    the uint64 hash bits (kattn_hash_rows)."""
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    x2 = x.reshape(-1, x.shape[-1]) if x.dim() > 1 else x.reshape(1, -1)
    if x2.stride(-1) != 1:
        raise ValueError("the last dimension of x must be contiguous")
    out = torch.empty(x2.shape[0], dtype=torch.int64, device=x.device)
    row_bytes = x2.shape[1] * x2.element_size()
    stride = x2.stride(0) * x2.element_size()
    lib = _lib.load()
    _lib.check("kattn_hash_rows", lib.kattn_hash_rows(
        _ptr(x2), x2.shape[0], row_bytes, stride, _ptr(out), _stream(x.device)))
    return out


def qk_scores_debug(q, k, k_scale, row_start, ctx_len, max_ctx: int, *, scores=None,
                    want_q=False):
    """Integer QK scores [B][M][Hq][max_ctx + M - 1] (int32); entries t >= L_j
    keep their prior contents (filled with INT32_MIN when allocated here).
    With want_q, also returns (q_i8, q_scale)."""
    _need(q, torch.float32, "q", 4)
    _need(k, torch.int8, "k", 3)
    _need(k_scale, torch.float32, "k_scale", 2)
    _need(row_start, torch.int64, "row_start", 1)
    _need(ctx_len, torch.int32, "ctx_len", 1)
    B, M, Hq, d = q.shape
    Hkv, cap, _ = k.shape
    width = int(max_ctx) + M - 1
    if scores is None:
        scores = torch.full((B, M, Hq, width), -2 ** 31, dtype=torch.int32, device=q.device)
    else:
        _need(scores, torch.int32, "scores", 4)
    q_i8 = q_scale = None
    if want_q:
        q_i8 = torch.zeros((B, M, Hq, d), dtype=torch.int8, device=q.device)
        q_scale = torch.zeros((B, M, Hq), dtype=torch.float32, device=q.device)
    lib = _lib.load()
    _lib.check("kattn_qk_scores_debug", lib.kattn_qk_scores_debug(
        _ptr(q), _ptr(k), _ptr(k_scale), _ptr(row_start), _ptr(ctx_len), B, M, Hq, Hkv, d, cap,
        int(max_ctx), _ptr(scores), _ptr(q_i8), _ptr(q_scale), _stream(q.device)))
    return (scores, q_i8, q_scale) if want_q else scores


# ------------------------------------------------ differential attention --

# (the raw handle of torch's current stream: a Stream object costs 2 us more, as
# much as the launch of a kernel)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_entry = {}          # entry points of the library by name


def _check(t, dtype, index, name, ndim):
    """t is a contiguous tensor of the type and dimensions on CUDA device `index`."""
    try:
        if t.dtype is dtype and t.get_device() == index >= 0 and t.dim() == ndim and t.is_contiguous():
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.get_device() != index:
        where = f"cuda:{index}" if index >= 0 else "a CUDA device, as the others"
        raise ValueError(f"{name} must be a CUDA tensor on {where}, got {t.device}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    raise ValueError(f"{name} must be contiguous")


def _device_of(t, name):
    """The CUDA device index of a tensor (-1 on the host)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t.get_device()


def _launch(name, index, *args):
    """One library call on torch's current stream of device `index`, which need
    not be the current device."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(_lib.load(), name)
    if index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _lib.check(name, status)


def diff_workspace_size(B: int, M: int, Hq: int, max_ctx: int) -> int:
    return int(_lib.load().kattn_diff_workspace_size(B, M, Hq, max_ctx))


def alloc_diff_workspace(B: int, M: int, Hq: int, max_ctx: int, device="cuda") -> torch.Tensor:
    """A workspace for decode_diff with its header zeroed (allocated by torch, not
    the library)."""
    n = diff_workspace_size(B, M, Hq, max_ctx)
    if n == 0:
        raise ValueError("invalid sizes for a differential decode workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def _diff_args(q, k, k_scale, v, v_scale, ctx_len, max_ctx, lam, out, workspace):
    """Checks and defaults that decode_diff and decode_diff_paged share."""
    index = _device_of(q, "q")
    per_row = int(_device_of(lam, "lam") == index and lam.dim() == 3)
    _check(q, torch.float32, index, "q", 4)
    _check(k, torch.int8, index, "k", 3)
    _check(v, torch.int8, index, "v", 3)
    _check(k_scale, torch.float32, index, "k_scale", 2)
    _check(v_scale, torch.float32, index, "v_scale", 2)
    _check(ctx_len, torch.int32, index, "ctx_len", 1)
    _check(lam, torch.float32, index, "lam", 3 if per_row else 1)
    B, M, Hq, d = q.shape
    Hkv, cap, dk = k.shape
    if v.shape != k.shape or k_scale.shape != (Hkv, cap) or v_scale.shape != (Hkv, cap) or dk != d:
        raise ValueError("k/v/scales shapes disagree")
    if Hkv < 2 or Hkv % 2 or Hq % Hkv:
        raise ValueError("kv planes come in pairs, and Hq must be a multiple of Hkv")
    if ctx_len.shape[0] != B:
        raise ValueError("ctx_len must have B entries")
    if not 0 < max_ctx < 2 ** 30:
        raise ValueError("max_ctx out of range")
    H = Hq // 2
    if lam.shape != ((B, M, H) if per_row else (H,)):
        raise ValueError("lam must have shape [Hq/2] or [B][M][Hq/2]")
    if out is None:
        out = torch.empty((B, M, H, 2 * d), dtype=torch.float32, device=q.device)
    else:
        _check(out, torch.float32, index, "out", 4)
        if out.shape != (B, M, H, 2 * d):
            raise ValueError("out must have shape [B][M][Hq/2][256]")
    if workspace is None:
        workspace = (alloc_diff_workspace(B, M, Hq, max_ctx, q.device) if B else
                     torch.zeros(256, dtype=torch.uint8, device=q.device))
    else:
        _check(workspace, torch.uint8, index, "workspace", 1)
    return index, B, M, Hq, Hkv, d, cap, per_row, out, workspace


def decode_diff(q, k, k_scale, v, v_scale, row_start, ctx_len, max_ctx: int, lam, *, out=None,
                sm_scale: float = 0.0, workspace=None):
    """Differential decode attention; returns out [B][M][Hq/2][256] float32.

    Head i of the Hq/2 differential heads is softmax_1 V - lam softmax_2 V: its
    two maps come from query heads 2i, 2i+1 and key planes 2p, 2p+1, its V is
    the 256 channels of value planes 2p, 2p+1, with p = i // (Hq / Hkv).
    lam: float32 [Hq/2], or [B][M][Hq/2] for one value per row.  q and the cache
    as in decode(); Hkv even.  workspace: a uint8 tensor of
    diff_workspace_size(...) bytes, its first 256 zeroed before its first use,
    allocated here with torch if None.
    (kattn_decode_diff)
    """
    index, B, M, Hq, Hkv, d, cap, per_row, out, workspace = _diff_args(
        q, k, k_scale, v, v_scale, ctx_len, max_ctx, lam, out, workspace)
    _check(row_start, torch.int64, index, "row_start", 1)
    if row_start.shape[0] != B:
        raise ValueError("row_start must have B entries")
    _launch("kattn_decode_diff", index, q.data_ptr(), k.data_ptr(), k_scale.data_ptr(),
            v.data_ptr(), v_scale.data_ptr(), row_start.data_ptr(), ctx_len.data_ptr(),
            lam.data_ptr(), per_row, B, M, Hq, Hkv, d, cap, max_ctx, sm_scale, out.data_ptr(),
            workspace.data_ptr(), workspace.numel())
    return out


def decode_diff_paged(q, k, k_scale, v, v_scale, block_table, page_rows: int, ctx_len,
                      max_ctx: int, lam, *, out=None, sm_scale: float = 0.0, workspace=None):
    """decode_diff() over a paged cache; paging arguments as decode_paged().
    (kattn_decode_diff_paged)"""
    index, B, M, Hq, Hkv, d, cap, per_row, out, workspace = _diff_args(
        q, k, k_scale, v, v_scale, ctx_len, max_ctx, lam, out, workspace)
    _check(block_table, torch.int32, index, "block_table", 2)
    if block_table.shape[0] != B:
        raise ValueError("block_table must have B rows")
    _launch("kattn_decode_diff_paged", index, q.data_ptr(), k.data_ptr(), k_scale.data_ptr(),
            v.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), block_table.shape[1],
            page_rows, ctx_len.data_ptr(), lam.data_ptr(), per_row, B, M, Hq, Hkv, d, cap, max_ctx,
            sm_scale, out.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out


# ------------------------------------------------- norm with 8-bit output --

_NORM_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_CODE_TYPES = {torch.int8: 0, torch.float8_e4m3fn: 1}


def _row_stride(t, dtype, index, shape, name):
    """The row stride of t, rows of its last dimension: any for a 2-D tensor, else
    t is contiguous.  A single row keeps the stride of the buffer that it is a slice
    of: with the pointers it decides the width of the loads, and so the order of the
    row's sum."""
    d = shape[-1]
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on the device of x, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    if t.is_contiguous():
        return max(t.stride(0), d) if len(shape) == 2 and shape[0] == 1 else d
    if t.dim() != 2 or (d > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be contiguous, or 2-D with a contiguous last dimension")
    return t.stride(0) if shape[0] > 1 else d


def rms_norm_quant(x, weight, *, residual=None, residual_out=None, eps: float = 1e-6,
                   group: int = 0, out=None, out_scale=None, out_dtype=torch.int8):
    """Residual addition, RMS norm and 8-bit quantization of the rows of x.

    x [..., d] float32, bfloat16 or float16; weight [d] and residual (like x) of
    the same type.  h = x + residual (rounded to the type) is stored in
    residual_out (the residual itself if None).  Returns (codes, scales): codes
    like x in out_dtype (torch.int8 or torch.float8_e4m3fn), scales float32, one
    per row [...] or per 128 channels [..., d/128] (group = 128), so that codes *
    scales is h / rms(h) * weight.  Slices x[i:i+1] (and of the residual) give the
    bytes that row i has in the whole.  (kattn_rms_norm_quant)
    """
    index = _device_of(x, "x")
    dtype, shape = x.dtype, x.shape
    x_type = _NORM_TYPES.get(dtype)
    if x_type is None:
        raise TypeError(f"x must be float32, bfloat16 or float16, got {dtype}")
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError("x must have a last dimension of at least 1")
    if index < 0:
        raise ValueError("x must be a CUDA tensor")
    d = shape[-1]
    rows = x.numel() // d
    groups = 1
    if group:
        if group != 128 or d % 128:
            raise ValueError("group must be 0, or 128 for rows of a multiple of 128 channels")
        groups = d // 128
    x_stride = _row_stride(x, dtype, index, shape, "x")
    _check(weight, dtype, index, "weight", 1)
    if weight.shape[0] != d:
        raise ValueError("weight must have one entry per channel")
    res_stride = res_out_stride = d
    res_ptr = res_out_ptr = 0
    if residual is not None:
        res_stride = _row_stride(residual, dtype, index, shape, "residual")
        if residual_out is None:
            residual_out, res_out_stride = residual, res_stride
        else:
            res_out_stride = _row_stride(residual_out, dtype, index, shape, "residual_out")
        res_ptr, res_out_ptr = residual.data_ptr(), residual_out.data_ptr()
        if res_ptr == res_out_ptr and rows == 1:       # in place, whatever the views' strides say
            res_out_stride = res_stride
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=x.device)
    code_type = _CODE_TYPES.get(out.dtype)
    if code_type is None:
        raise TypeError(f"codes must be int8 or float8_e4m3fn, got {out.dtype}")
    _check(out, out.dtype, index, "out", len(shape))
    if out.shape != shape:
        raise ValueError("out must have the shape of x")
    if out_scale is None:
        out_scale = torch.empty(shape[:-1] + ((groups,) if group else ()), dtype=torch.float32,
                                device=x.device)
    else:
        _check(out_scale, torch.float32, index, "out_scale", out_scale.dim())
        if out_scale.numel() != rows * groups:
            raise ValueError("out_scale must have one entry per scale")
    _launch("kattn_rms_norm_quant", index, x.data_ptr(), res_ptr, weight.data_ptr(), x_type, rows, d,
            x_stride, res_stride, res_out_stride, eps, group, code_type, res_out_ptr, out.data_ptr(),
            out_scale.data_ptr())
    return out, out_scale


# -------------------------------------------------------- page operations --

def page_workspace_size(n_slots: int, n_pages: int) -> int:
    return int(_lib.load().kattn_page_workspace_size(n_slots, n_pages))


def alloc_page_workspace(n_slots: int, n_pages: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace for the page operations of one table of n_slots rows over
    one pool of n_pages pages."""
    n = page_workspace_size(n_slots, n_pages)
    if n == 0:
        raise ValueError("invalid sizes for a page workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _page_args(block_table, ref_count, seqs, name, workspace):
    """Checks that the page operations share; seqs: the list of slots, or None.
    Returns (device index, n_slots, max_pages, n_pages, n, workspace)."""
    index = _device_of(block_table, "block_table")
    _check(block_table, torch.int32, index, "block_table", 2)
    _check(ref_count, torch.int32, index, "ref_count", 1)
    n_slots, max_pages = block_table.shape
    n_pages = ref_count.shape[0]
    n = 0
    if name:
        _check(seqs, torch.int32, index, name, 1)
        n = seqs.shape[0]
    if workspace is None:
        workspace = alloc_page_workspace(n_slots, n_pages, block_table.device)
    else:
        _check(workspace, torch.uint8, index, "workspace", 1)
    return index, n_slots, max_pages, n_pages, n, workspace


def _check_list(t, index, name, n):
    _check(t, torch.int32, index, name, 1)
    if t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries")


def reserve_pages(block_table, ref_count, seqs, lens, page_rows: int, *, workspace=None) -> None:
    """Pages from the pool for lens[i] rows of slot seqs[i] (kattn_reserve_pages).

    block_table int32 [n_slots][max_pages] (unused entries below 0), ref_count
    int32 [n_pages], seqs and lens int32 [n]; both tables are updated in place.
    """
    index, S, mp, P, n, ws = _page_args(block_table, ref_count, seqs, "seqs", workspace)
    _check_list(lens, index, "lens", n)
    _launch("kattn_reserve_pages", index, block_table.data_ptr(), S, mp,
            ref_count.data_ptr(), P, page_rows, seqs.data_ptr(), lens.data_ptr(), n, ws.data_ptr(),
            ws.numel())


def free_sequences(block_table, ref_count, seqs, *, workspace=None) -> None:
    """Release the pages of the slots seqs (int32 [n]); in place
    (kattn_free_sequences)."""
    index, S, mp, P, n, ws = _page_args(block_table, ref_count, seqs, "seqs", workspace)
    _launch("kattn_free_sequences", index, block_table.data_ptr(), S, mp,
            ref_count.data_ptr(), P, seqs.data_ptr(), n, ws.data_ptr(), ws.numel())


def fork_sequences(block_table, ref_count, parents, children, lens, page_rows: int, *, src=None,
                   dst=None, workspace=None):
    """Slot children[i] becomes a branch of the first lens[i] rows of slot
    parents[i]: full pages shared, the last partial one to be copied.  Returns
    (src, dst), int32 [n], for copy_pages() (kattn_fork_sequences)."""
    index, S, mp, P, n, ws = _page_args(block_table, ref_count, children, "children", workspace)
    _check_list(parents, index, "parents", n)
    _check_list(lens, index, "lens", n)
    if src is None:
        src = torch.empty_like(lens)
    else:
        _check_list(src, index, "src", n)
    if dst is None:
        dst = torch.empty_like(lens)
    else:
        _check_list(dst, index, "dst", n)
    _launch("kattn_fork_sequences", index, block_table.data_ptr(), S, mp, ref_count.data_ptr(), P,
            page_rows, parents.data_ptr(), children.data_ptr(), lens.data_ptr(), n, src.data_ptr(),
            dst.data_ptr(), ws.data_ptr(), ws.numel())
    return src, dst


def compact_pages(block_table, ref_count, *, table_out=None, ref_out=None, src=None, dst=None,
                  counts=None, workspace=None):
    """The moves that bring the live pages to the front of the pool.

    Returns (table_out, ref_out, src, dst, counts): the table and counts after
    the moves (new tensors unless given; the inputs themselves for an update in
    place), the moves for copy_pages() (int32 [max(1, n_pages // 2)], -1 past
    the last), and counts = int32 [n_live, n_moves] (kattn_compact_pages)."""
    index, S, mp, P, _, ws = _page_args(block_table, ref_count, None, None, workspace)
    most = max(1, P // 2)

    if table_out is None:
        table_out = torch.empty_like(block_table)
    else:
        _check(table_out, torch.int32, index, "table_out", 2)
        if table_out.shape != block_table.shape:
            raise ValueError("table_out must have the shape of block_table")
    if ref_out is None:
        ref_out = torch.empty_like(ref_count)
    else:
        _check_list(ref_out, index, "ref_out", P)
    if src is None:
        src = torch.empty(most, dtype=torch.int32, device=ref_count.device)
    else:
        _check_list(src, index, "src", most)
    if dst is None:
        dst = torch.empty_like(src)
    else:
        _check_list(dst, index, "dst", most)
    if counts is None:
        counts = torch.empty(2, dtype=torch.int32, device=ref_count.device)
    else:
        _check_list(counts, index, "counts", 2)
    _launch("kattn_compact_pages", index, block_table.data_ptr(), S, mp, ref_count.data_ptr(), P,
            table_out.data_ptr(), ref_out.data_ptr(), src.data_ptr(), dst.data_ptr(),
            counts.data_ptr(), ws.data_ptr(), ws.numel())
    return table_out, ref_out, src, dst, counts


def copy_pages(k, k_scale, v, v_scale, src, dst, page_rows: int, *, count=None,
               workspace=None) -> None:
    """Copy page src[i] to page dst[i] in every plane of one cache, k and v
    [Hkv][cap][128] int8 with their scales [Hkv][cap]; entries below 0 are
    skipped.  count: an int32 tensor of one entry; only the first min(n, count)
    moves are made.  workspace: any workspace of the library (its error word
    takes the checks of the entries); allocated here if None.
    (kattn_copy_pages)"""
    index = _device_of(k, "k")
    _check(k, torch.int8, index, "k", 3)
    _check(v, torch.int8, index, "v", 3)
    _check(k_scale, torch.float32, index, "k_scale", 2)
    _check(v_scale, torch.float32, index, "v_scale", 2)
    _check(src, torch.int32, index, "src", 1)
    n = src.shape[0]
    _check_list(dst, index, "dst", n)
    Hkv, cap, d = k.shape
    if v.shape != k.shape or k_scale.shape != (Hkv, cap) or v_scale.shape != (Hkv, cap):
        raise ValueError("k/v/scales shapes disagree")
    count_ptr = 0
    if count is not None:
        _check_list(count, index, "count", 1)
        count_ptr = count.data_ptr()
    if workspace is None:
        workspace = torch.zeros(256, dtype=torch.uint8, device=k.device)
    else:
        _check(workspace, torch.uint8, index, "workspace", 1)
    _launch("kattn_copy_pages", index, k.data_ptr(), k_scale.data_ptr(), v.data_ptr(),
            v_scale.data_ptr(), Hkv, d, cap, page_rows, src.data_ptr(), dst.data_ptr(), n, count_ptr,
            workspace.data_ptr(), workspace.numel())


def get_device_status(workspace: torch.Tensor) -> int:
    """Read and clear the device error bits of a workspace."""
    _need(workspace, torch.uint8, "workspace", 1)
    lib = _lib.load()
    err = ctypes.c_int(0)
    _lib.check("kattn_get_device_status", lib.kattn_get_device_status(
        _ptr(workspace), workspace.numel(), ctypes.byref(err), _stream(workspace.device)))
    return err.value
