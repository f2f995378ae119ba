"""Binding of the linear-attention layer with one decay a head and of the head
norm and rotation in front of it (include/kda_linear.h).

Arguments are checked on the host, nothing is synchronised.  What a call on a
given stream allocates is that stream's memory.
"""
from __future__ import annotations

import ctypes

import torch

import kimi_delta_attention_07_gb300 as _core
from ._hybrid import _current_stream, _device, _need, _rows

_f32, _i32, _u8 = torch.float32, torch.int32, torch.uint8
_empty = _core._empty
_lib = None


def _library():
    global _lib
    _lib = _core.load()
    return _lib


def _stream_of(stream, dev):
    return _current_stream(dev) if stream is None else stream.cuda_stream


def _decay(g, tokens, H, dev):
    """The address of g and its elements between tokens: [H] (0), or tokens' shape with H behind it, whose
    tokens are all at one stride (a slice of a projection, or one row expanded)."""
    if g.dim() == 1:
        return _need(g, "g", _f32, (H,), dev), 0
    if g.is_contiguous():
        return _need(g, "g", _f32, (*tokens, H), dev), H
    if g.dtype is not _f32 or g.shape != (*tokens, H) or g.get_device() != dev:
        _need(g.contiguous(), "g", _f32, (*tokens, H), dev)  # names what is wrong
    steps = [s for s, n in zip(g.stride(), tokens) if n > 1]
    stride = steps[-1] if steps else H
    if (H > 1 and g.stride(-1) != 1) or (0 < stride < H) or (len(steps) == 2 and steps[0] != tokens[1] * stride):
        raise ValueError(f"g: its heads must be next to each other and all tokens at one stride of at least {H} (or 0)")
    return g.data_ptr(), stride


def _states(t, name, H, dev):
    """The address of a pool or batch of states, and how many it holds."""
    if t.dim() != 4:
        raise ValueError(f"{name} must be [states, {H}, 128, 128]")
    return _need(t, name, _f32, (t.shape[0], H, 128, 128), dev), t.shape[0]


def kda_head_norm_rope(q, k=None, *, positions=None, inv_freq=None, sections=None, rot_offset=0, interleaved=False,
                       norm=True, q_weight=None, k_weight=None, eps=1e-6, q_out=None, k_out=None, stream=None):
    """RMS norm of each head of q (and k) and rotation by the token's position, in
    one pass (kda_head_norm_rope in kda_linear.h).

    q [T, Hq, D], k [T, Hk, D] or None, bf16 or fp32; their token strides are free
    (slices of a fused projection).  norm: x / sqrt(mean(x^2) + eps) * weight over the
    D channels of a head (weights fp32 [D], None: ones; refused without the norm).  inv_freq fp32
    [rot_dim / 2] (None: no rotation) turns the rot_dim channels from rot_offset
    on, in pairs (i, i + rot_dim / 2), or (2 i, 2 i + 1) if interleaved; positions int32
    [T], or [A, T] with `sections`, the pairs of each axis.  A token whose first
    position is negative is padding: its rows are not written.  q_out and k_out are
    allocated unless given; they may be q and k.  Returns (q_out, k_out or None).
    """
    dev = _device(q, "q")
    dtype = q.dtype
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k must be [T, heads, D]")
    T, Hq, D = q.shape
    code = _core._dtype_code(q)
    pq, sq = _rows(q, "q", dtype, (T, Hq, D), dev)
    if q_out is None:
        q_out = _empty((T, Hq, D), dtype, q.device, stream)
    poq, soq = _rows(q_out, "q_out", dtype, (T, Hq, D), dev)
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    pk = pok = None
    Hk = sk = sok = 0
    if k is not None:
        Hk = k.shape[1]
        pk, sk = _rows(k, "k", dtype, (T, Hk, D), dev)
        if k_out is None:
            k_out = _empty((T, Hk, D), dtype, q.device, stream)
        pok, sok = _rows(k_out, "k_out", dtype, (T, Hk, D), dev)
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("weights without the norm: they would not be applied")
    pwq = None if q_weight is None else _need(q_weight, "q_weight", _f32, (D,), dev)
    pwk = None if k_weight is None else _need(k_weight, "k_weight", _f32, (D,), dev)
    axes = 1
    pp = pf = ps = None
    if positions is not None:
        axes = 1 if positions.dim() == 1 else positions.shape[0]
        pp = _need(positions, "positions", _i32, (T,) if positions.dim() == 1 else (axes, T), dev)
    rot = 0
    if inv_freq is not None:
        if positions is None:
            raise ValueError("a rotation needs positions")
        rot = 2 * inv_freq.numel()
        pf = _need(inv_freq, "inv_freq", _f32, (rot // 2,), dev)
    if sections is not None:
        if len(sections) != axes or sum(sections) != rot // 2:
            raise ValueError(f"sections must name the pairs of each of {axes} axes, {rot // 2} in all, got {list(sections)}")
        if axes > 1:
            ps = (ctypes.c_int * axes)(*sections)
    st = (_lib or _library()).kda_head_norm_rope(
        pq, sq, pk, sk, pwq, pwk, eps, 1 if norm else 0, pp, ps, axes, pf, rot_offset, rot, 1 if interleaved else 0,
        poq, soq, pok, sok, T, Hq, Hk, D, code, _stream_of(stream, dev))
    if st:
        raise _core.KdaError(st, "kda_head_norm_rope")
    return q_out, k_out


def kda_linear_chunk_workspace_bytes(total_tokens: int, n_seqs: int, H: int, dtype: int = _core.KDA_BF16) -> int:
    return int((_lib or _library()).kda_linear_chunk_workspace_bytes(total_tokens, n_seqs, H, dtype))


def kda_linear_chunk_fwd(q, k, v, g, *, cu_seqlens=None, n_seqs=None, initial_state=None, final_state=None,
                         state_indices=None, n_slots=None, scale=None, output_final_state=True, o=None,
                         workspace=None, stream=None):
    """Linear attention with one decay a head over packed sequences:
    S <- exp(g) S + k v^T, o = scale S^T q (kda_linear_chunk_fwd in kda_linear.h).

    q, k [T, Hk, 128], v [T, H, 128] (Hk divides H; head h reads q and k of head
    h // (H // Hk)), bf16 or fp32; g fp32 [T, H], or [H] for fixed decays; token
    strides free.  cu_seqlens int32 [N+1] or None (n_seqs equal lengths, default 1).  States are [N, H, 128, 128] ([V, K]) fp32, or with state_indices (int32
    [N]) pools of them; final_state may be initial_state.  scale defaults to 128 ** -0.5.
    workspace is allocated where one is needed, unless given
    (kda_linear_chunk_workspace_bytes).  Returns (o, final_state).
    """
    dev = _device(q, "q")
    dtype = q.dtype
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and k must be [T, Hk, 128], v [T, H, 128]")
    T, Hk, K = q.shape
    H, V = v.shape[1:]
    code = _core._dtype_code(q)
    pq, sq = _rows(q, "q", dtype, (T, Hk, K), dev)
    pk, sk = _rows(k, "k", dtype, (T, Hk, K), dev)
    pv, sv = _rows(v, "v", dtype, (T, H, V), dev)
    pg, sg = _decay(g, (T,), H, dev)
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        if N < 1:
            raise ValueError("cu_seqlens must be int32 [N+1] with N >= 1")
        pc = _need(cu_seqlens, "cu_seqlens", _i32, (N + 1,), dev)
    else:
        N, pc = (1 if n_seqs is None else int(n_seqs)), None
    pi = None if state_indices is None else _need(state_indices, "state_indices", _i32, (N,), dev)
    if state_indices is None:
        if final_state is None and output_final_state:
            final_state = _empty((N, H, V, K), _f32, q.device, stream)
        slots = N
    else:
        held = [t.shape[0] for t in (initial_state, final_state) if t is not None]
        if not held or (final_state is None and output_final_state):
            raise ValueError("with state_indices, final_state must be the destination pool")
        slots = min(held) if n_slots is None else int(n_slots)
    p0 = pf = None
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        if t is None:
            continue
        p, held = _states(t, name, H, dev)
        if held < slots or (state_indices is None and held != N):
            raise ValueError(f"{name} holds {held} states, {slots} are needed")
        p0, pf = (p, pf) if name == "initial_state" else (p0, p)
    if o is None:
        o = _empty((T, H, V), dtype, q.device, stream)
    po = _need(o, "o", dtype, (T, H, V), dev)
    lib = _lib or _library()
    pw, ws = None, 0
    if workspace is not None:
        ws = workspace.numel()
        pw = _need(workspace, "workspace", _u8, (ws,), dev)
    else:
        ws = lib.kda_linear_chunk_workspace_bytes(T, N, H, code)
        if ws:
            workspace = _empty(ws, _u8, q.device, stream, scratch=True)
            pw = workspace.data_ptr()
    st = lib.kda_linear_chunk_fwd(
        pq, sq, pk, sk, pv, sv, pg, sg, p0, pf, pi, slots, po, pc, N, T, H, Hk, K, V,
        K ** -0.5 if scale is None else scale, code, pw, ws, _stream_of(stream, dev))
    if st:
        raise _core.KdaError(st, "kda_linear_chunk_fwd")
    return o, final_state


def _tokens(t, name, dtype, shape, dev):
    """The address and token stride of [N, heads, 128], or of [N, S, heads, 128] whose sequences follow one
    another at the same stride."""
    if len(shape) == 3:
        return _rows(t, name, dtype, shape, dev)
    if tuple(t.shape) == shape and shape[0] > 1 and shape[1] > 1 and t.stride(0) != shape[1] * t.stride(1):
        raise ValueError(f"{name}: the tokens of all sequences must be at one stride")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {shape}")
    return _rows(t.flatten(0, 1) if shape[0] and shape[1] else t.reshape(0, *shape[2:]), name, dtype,
                 (shape[0] * shape[1], *shape[2:]), dev)


def _step(name, q, k, v, g, state_pool, state_indices, num_accepted, scale, o, stream, lead):
    dev = _device(q, "q")
    dtype = q.dtype
    if q.dim() != len(lead) + 2 or v.dim() != len(lead) + 2:
        raise ValueError(f"q, k and v must be [{'N, S' if len(lead) == 2 else 'N'}, heads, 128]")
    Hk, K = q.shape[-2:]
    H, V = v.shape[-2:]
    code = _core._dtype_code(q)
    pq, sq = _tokens(q, "q", dtype, (*lead, Hk, K), dev)
    pk, sk = _tokens(k, "k", dtype, (*lead, Hk, K), dev)
    pv, sv = _tokens(v, "v", dtype, (*lead, H, V), dev)
    pg, sg = _decay(g, lead, H, dev)
    pp, slots = _states(state_pool, "state_pool", H, dev)
    pi = None if state_indices is None else _need(state_indices, "state_indices", _i32, lead, dev)
    if o is None:
        o = _empty((*lead, H, V), dtype, q.device, stream)
    po = _need(o, "o", dtype, (*lead, H, V), dev)
    lib = _lib or _library()
    scale = K ** -0.5 if scale is None else scale
    if len(lead) == 1:
        st = lib.kda_linear_step(pq, sq, pk, sk, pv, sv, pg, sg, pp, pi, slots, po, lead[0], H, Hk, K, V, scale, code,
                                 _stream_of(stream, dev))
    else:
        pa = None if num_accepted is None else _need(num_accepted, "num_accepted", _i32, lead[:1], dev)
        st = lib.kda_linear_multi_step(pq, sq, pk, sk, pv, sv, pg, sg, pp, pi, pa, slots, po, *lead, H, Hk, K, V, scale,
                                       code, _stream_of(stream, dev))
    if st:
        raise _core.KdaError(st, name)
    return o


def kda_linear_step(q, k, v, g, state_pool, *, state_indices=None, scale=None, o=None, stream=None):
    """One decode token per sequence, updating ``state_pool`` [slots, H, 128, 128] in place.

    q, k [N, Hk, 128]; v [N, H, 128]; g fp32 [N, H] (token strides free) or [H];
    state_indices int32 [N] or None (slot n).  Returns o [N, H, 128].
    """
    return _step("kda_linear_step", q, k, v, g, state_pool, state_indices, None, scale, o, stream, (q.shape[0],))


def kda_linear_multi_step(q, k, v, g, state_pool, state_indices, *, num_accepted=None, scale=None, o=None, stream=None):
    """Speculative decode: S tokens per sequence.  q, k [N, S, Hk, 128]; v [N, S, H,
    128]; g fp32 [N, S, H] or [H]; state_indices int32 [N, S] (the state after token t goes to slot
    state_indices[n, t]); num_accepted int32 [N] or None (start from slot state_indices[n, a - 1], else
    [n, 0]).  Updates state_pool in place; returns o [N, S, H, 128].
    """
    if state_indices is None:
        raise ValueError("state_indices is required")
    if q.dim() != 4:
        raise ValueError("q, k and v must be [N, S, heads, 128]")
    return _step("kda_linear_multi_step", q, k, v, g, state_pool, state_indices, num_accepted, scale, o, stream,
                 tuple(q.shape[:2]))
