"""Binding of the operators around the KDA core (include/kda_hybrid.h): page
tables, residual + RMS norm, the paged latent cache and latent attention.

Arguments are checked on the host, nothing is synchronised.  What a call on a
given stream allocates is that stream's memory.
Small calls are dominated by the host, so the checks test all of a tensor's
properties at once and name the property only when one of them fails.
"""
from __future__ import annotations

import torch

import kimi_delta_attention_07_gb300 as _core

KDA_QUANT_NONE, KDA_QUANT_ROW, KDA_QUANT_BLOCK = range(3)
KDA_BF16 = _core.KDA_BF16
LATENT_DIM, ROPE_DIM, LATENT_ROW, NOPE_DIM, VALUE_DIM = 512, 64, 576, 128, 128
KDA_LATENT_PREFILL_SPLIT_KEYS = 1024
_QUANT = {"none": KDA_QUANT_NONE, None: KDA_QUANT_NONE, "row": KDA_QUANT_ROW, "block": KDA_QUANT_BLOCK}
_bf16, _f32, _i32, _u8, _e4m3 = (torch.bfloat16, torch.float32, torch.int32, torch.uint8,
                                 torch.float8_e4m3fn)
_current_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_empty = _core._empty
_lib = None


def _library():
    global _lib
    _lib = _core.load()
    return _lib


def _device(t, name):
    """The device of t, which is the current one: kernels are launched there, and their grids and
    workspaces are sized for it."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{_current_device()}")
    return dev


def _need(t, name, dtype, shape, dev):
    """The address of t: a contiguous CUDA tensor of this dtype and shape on device `dev`."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _core._check(t, name, dtype, shape)
    raise ValueError(f"{name} must be on the same device as the other tensors")


def _rows(t, name, dtype, shape, dev):
    """The same for a tensor whose first stride is free (a slice of a wider
    projection); returns (address, elements between rows)."""
    strides = t.stride()
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        # below the first axis the strides are those of a contiguous tensor
        inner = shape[-1] if len(shape) == 2 else shape[-1] * shape[-2]
        if strides[-1] == 1 and (len(shape) == 2 or strides[1] == shape[2] or shape[1] == 1):
            stride = strides[0] if shape[0] > 1 else inner
            if stride >= inner and stride % 8 == 0:
                return t.data_ptr(), stride
            raise ValueError(f"{name}: its row stride must be a multiple of 8 of at least {inner}, got {stride}")
        raise ValueError(f"{name} must be contiguous but for its row stride")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")
    raise ValueError(f"{name} must be on the same device as the other tensors")


def kda_page_tables(ctx_lens, new_lens, free_pages, block_table, *, page_size, n_pages, max_tokens=None,
                    free_start=None, cu_seqlens=None, seq_lens=None, slots=None, positions=None,
                    status=None, stream=None):
    """Block table, slot map, positions and offsets of one step, from request
    lengths on the device (kda_page_tables in kda_hybrid.h).

    ctx_lens, new_lens int32 [N] (tokens in the cache; tokens this step adds);
    free_pages int32 [F]; block_table int32 [N, max_pages], extended in place.
    max_tokens sizes slots and positions (the length of the packed, possibly
    padded batch) unless they are given.  free_start int32 [1] (status[:1] of
    the step before) or None.  Returns (cu_seqlens [N+1], seq_lens [N], slots
    [max_tokens], positions [max_tokens], status [2] = (position in free_pages
    after the step, requests refused)), all int32.
    """
    dev = _device(ctx_lens, "ctx_lens")
    n = ctx_lens.numel()
    if slots is not None:
        max_tokens = slots.numel()
    elif max_tokens is None:
        raise ValueError("pass max_tokens, or slots and positions")
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [N, max_pages]")
    max_pages, n_free = block_table.shape[1], free_pages.numel()
    shape = (n,)
    pc = _need(ctx_lens, "ctx_lens", _i32, shape, dev)
    pn = _need(new_lens, "new_lens", _i32, shape, dev)
    pf = _need(free_pages, "free_pages", _i32, (n_free,), dev)
    pb = _need(block_table, "block_table", _i32, (n, max_pages), dev)
    ps = None if free_start is None else _need(free_start, "free_start", _i32, (1,), dev)

    def fresh(size):
        return _empty(size, _i32, ctx_lens.device, stream)

    cu_seqlens = fresh(n + 1) if cu_seqlens is None else cu_seqlens
    seq_lens = fresh(n) if seq_lens is None else seq_lens
    slots = fresh(max_tokens) if slots is None else slots
    positions = fresh(max_tokens) if positions is None else positions
    status = fresh(2) if status is None else status
    st = (_lib or _library()).kda_page_tables(
        pc, pn, pf, n_free, ps, pb, _need(cu_seqlens, "cu_seqlens", _i32, (n + 1,), dev),
        _need(seq_lens, "seq_lens", _i32, shape, dev), _need(slots, "slots", _i32, (max_tokens,), dev),
        _need(positions, "positions", _i32, (max_tokens,), dev), _need(status, "status", _i32, (2,), dev), n,
        max_tokens, max_pages, page_size, n_pages,
        _current_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise _core.KdaError(st, "kda_page_tables")
    return cu_seqlens, seq_lens, slots, positions, status


def kda_rms_norm(x, weight=None, *, residual=None, eps=1e-6, quant="none", residual_out=None, y=None,
                 scales=None, stream=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight over the last axis.

    x, residual [..., D] bf16 or fp32; weight [D] fp32 or None.  quant "none":
    y in x's dtype; "row" / "block": y in float8_e4m3fn with fp32 scales
    [...] (shape [..., 1]) / [..., D / 128], y * scale standing for the value.
    With a residual, h (rounded to x's dtype) is returned too, in residual_out
    (allocated unless given; may be residual or x).  Returns (y, residual_out
    or None, scales or None).
    """
    dev = _device(x, "x")
    shape, dtype = x.shape, x.dtype
    D = shape[-1]
    q = _QUANT[quant]
    px = _need(x, "x", dtype, shape, dev)
    if residual is None:
        pr = None
    else:
        pr = _need(residual, "residual", dtype, shape, dev)
        if residual_out is None:
            residual_out = _empty(shape, dtype, x.device, stream)
    po = None if residual_out is None else _need(residual_out, "residual_out", dtype, shape, dev)
    pw = None if weight is None else _need(weight, "weight", _f32, (D,), dev)
    ydt = _e4m3 if q else dtype
    if y is None:
        y = _empty(shape, ydt, x.device, stream)
    py = _need(y, "y", ydt, shape, dev)
    if q:
        groups = (*shape[:-1], 1 if q == KDA_QUANT_ROW else D // 128)
        if scales is None:
            scales = _empty(groups, _f32, x.device, stream)
        ps = _need(scales, "scales", _f32, groups, dev)
    else:
        scales = ps = None
    st = (_lib or _library()).kda_rms_norm(
        px, pr, pw, py, ps, po, eps, x.numel() // D if D else 0, D, q,
        KDA_BF16 if dtype is _bf16 else _core._dtype_code(x),
        _current_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise _core.KdaError(st, "kda_rms_norm")
    return y, residual_out, scales


def kda_latent_cache_write(kv, weight, cache, slots, *, eps=1e-6, stream=None):
    """cache row slots[t] = [rms_norm(kv[t, :512]) * weight ; kv[t, 512:]].

    kv [T, 576] bf16 (its row stride is free: a slice of a fused projection);
    weight fp32 [512], or None to store the latent as it is; cache [n_pages,
    page_size, 576] bf16, written in place; slots int32 [T] (others than cache
    rows, such as -1, are skipped).  Returns cache.
    """
    dev = _device(kv, "kv")
    T = kv.shape[0]
    pk, stride = _rows(kv, "kv", _bf16, (T, LATENT_ROW), dev)
    if cache.dim() != 3:
        raise ValueError(f"cache must be [n_pages, page_size, {LATENT_ROW}]")
    n_pages, page_size, _ = cache.shape
    pc = _need(cache, "cache", _bf16, (n_pages, page_size, LATENT_ROW), dev)
    pw = None if weight is None else _need(weight, "weight", _f32, (LATENT_DIM,), dev)
    ps = _need(slots, "slots", _i32, (T,), dev)
    st = (_lib or _library()).kda_latent_cache_write(
        pk, stride, pw, eps, pc, ps, T, n_pages, page_size,
        _current_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise _core.KdaError(st, "kda_latent_cache_write")
    return cache


def kda_latent_decode_workspace_bytes(n_seqs: int, S: int, H: int) -> int:
    return int((_lib or _library()).kda_latent_decode_workspace_bytes(n_seqs, S, H))


def kda_latent_decode(q, cache, block_table, seq_lens, *, scale=None, o=None, lse=None, workspace=None,
                      stream=None):
    """Absorbed latent attention of S new tokens a request over the paged cache.

    q [N, S, H, 576] (or [N, H, 576]: S = 1) bf16; cache [n_pages, page_size,
    576] bf16; block_table int32 [N, max_pages]; seq_lens int32 [N], the S new
    tokens among them: token s sees positions below seq_lens[n] - S + 1 + s.
    scale defaults to 192 ** -0.5 (the expanded query's width).  lse, if given,
    is fp32 [N, S, H] (or [N, H]).  Returns o, q's shape with 512 for 576.
    """
    dev = _device(q, "q")
    shape = q.shape
    if len(shape) == 4:
        n, S, H, _ = shape
    elif len(shape) == 3:
        (n, H, _), S = shape, 1
    else:
        raise ValueError("q must be [N, S, H, 576] or [N, H, 576]")
    pq = _need(q, "q", _bf16, (*shape[:-1], LATENT_ROW), dev)
    if cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("cache must be [n_pages, page_size, 576], block_table [N, max_pages]")
    n_pages, page_size, _ = cache.shape
    pc = _need(cache, "cache", _bf16, (n_pages, page_size, LATENT_ROW), dev)
    pb = _need(block_table, "block_table", _i32, (n, block_table.shape[1]), dev)
    pl = _need(seq_lens, "seq_lens", _i32, (n,), dev)
    out = (*shape[:-1], LATENT_DIM)
    if o is None:
        o = _empty(out, _bf16, q.device, stream)
    po = _need(o, "o", _bf16, out, dev)
    ple = None if lse is None else _need(lse, "lse", _f32, shape[:-1], dev)
    lib = _lib or _library()
    if workspace is None:
        workspace = _empty(max(256, lib.kda_latent_decode_workspace_bytes(n, S, H)), _u8, q.device, stream, scratch=True)
    ws = workspace.numel()
    st = lib.kda_latent_decode(
        pq, pc, pb, pl, po, ple, n, S, H, n_pages, page_size, block_table.shape[1],
        192 ** -0.5 if scale is None else scale, _need(workspace, "workspace", _u8, (ws,), dev), ws,
        _current_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise _core.KdaError(st, "kda_latent_decode")
    return o


def kda_latent_prefill_workspace_bytes(n_seqs: int, total_q: int, total_k: int, H: int) -> int:
    return int((_lib or _library()).kda_latent_prefill_workspace_bytes(n_seqs, total_q, total_k, H))


def kda_latent_prefill(q, kv, k_rope, *, cu_seqlens_q, cu_seqlens_k=None, causal=True, scale=None, o=None,
                       lse=None, workspace=None, stream=None):
    """Expanded latent attention over packed sequences.

    q [Tq, H, 192] bf16; kv [Tk, H, 256] bf16 (a head's key part, then its
    value); k_rope [Tk, 64] bf16, shared by the heads; the token strides of the
    three are free.  cu_seqlens_q / cu_seqlens_k int32 [N+1] (k None: the same
    as q).  causal: query i of lq sees keys j <= i + lk - lq.  scale defaults to
    192 ** -0.5.  lse, if given, is fp32 [Tq, H].  workspace is allocated where one
    is needed, unless given (kda_latent_prefill_workspace_bytes).  Returns o [Tq, H, 128].
    """
    dev = _device(q, "q")
    if q.dim() != 3 or kv.dim() != 3:
        raise ValueError("q must be [Tq, H, 192], kv [Tk, H, 256]")
    Tq, H, _ = q.shape
    Tk = kv.shape[0]
    pq, sq = _rows(q, "q", _bf16, (Tq, H, NOPE_DIM + ROPE_DIM), dev)
    pk, sk = _rows(kv, "kv", _bf16, (Tk, H, NOPE_DIM + VALUE_DIM), dev)
    pr, sr = _rows(k_rope, "k_rope", _bf16, (Tk, ROPE_DIM), dev)
    n = cu_seqlens_q.numel() - 1
    if n < 1:
        raise ValueError("cu_seqlens_q must be int32 [N+1] with N >= 1")
    pcq = _need(cu_seqlens_q, "cu_seqlens_q", _i32, (n + 1,), dev)
    pck = None if cu_seqlens_k is None else _need(cu_seqlens_k, "cu_seqlens_k", _i32, (n + 1,), dev)
    if o is None:
        o = _empty((Tq, H, VALUE_DIM), _bf16, q.device, stream)
    po = _need(o, "o", _bf16, (Tq, H, VALUE_DIM), dev)
    ple = None if lse is None else _need(lse, "lse", _f32, (Tq, H), dev)
    lib = _lib or _library()
    pw, ws = None, 0
    if workspace is not None:
        ws = workspace.numel()
        pw = _need(workspace, "workspace", _u8, (ws,), dev)
    elif Tk >= KDA_LATENT_PREFILL_SPLIT_KEYS:
        ws = lib.kda_latent_prefill_workspace_bytes(n, Tq, Tk, H)
        if ws:
            workspace = _empty(ws, _u8, q.device, stream, scratch=True)
            pw = workspace.data_ptr()
    st = lib.kda_latent_prefill(
        pq, sq, pk, sk, pr, sr, po, ple, pcq, pck, n, Tq, Tk, H, 1 if causal else 0,
        192 ** -0.5 if scale is None else scale, pw, ws,
        _current_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise _core.KdaError(st, "kda_latent_prefill")
    return o
