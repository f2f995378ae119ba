"""The linear-attention layer with one decay a head, and the head norm and rotation,
against plain implementations in 64 bits.

Bounds, element by element, from the roundings that an output passes (a
rounding is off by at most half a step, eps / 2 of its type: bf16 2^-8, fp32 2^-24):
  rope    norm factor, weight, angle (2^-20 of a radian) and the rotation's products:
          2^-18 (|a| + |b|) of a pair, then the output's own rounding
  state   a decay e^x enters with the relative error of its exponent, at most 7 roundings
          of |x| <= 24 (smaller weights than e^-24 do not count), below 2^-16, and of the
          exponential, 2^-22 a chunk; k v^T is split to 2^-24: (2^-16 + chunks 2^-21)
          of the state of |k| |v|, called A.  fp32 inputs, token by token: T 2^-22 A
  o       bf16: p_ij = (q_i . k_j) e^.. is rounded to bf16, weighing sum_j |p_ij v_j| over
          the chunk of 128, and so is the state in front of the chunk, weighing |q| . |S|;
          2^-12 of both for fp32 scores, decays and sums; then o's rounding
          fp32: T 2^-22 |q| . A
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
C = 128


@pytest.fixture(scope="module")
def kda():
    import kimi_delta_attention_07_gb300 as m
    m.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(shape, seed, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * std).to(dtype)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def within(got, ref, bound, what):
    got, ref = got.double(), ref.double()
    off = (got - ref).abs()
    bad = ~((off <= bound) | (got.isnan() & ref.isnan()) | (got == ref))
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, worst {float((off / bound.clamp(min=1e-300)).nan_to_num(INF).max()):.3g} of its bound"


# ---- head norm and rotation --------------------------------------------------------


def rope_ref(x, weight, positions, inv_freq, sections, off, interleaved, norm, eps=1e-6):
    """(y, |a| + |b| of each element's pair) in 64 bits."""
    y = x.double()
    if norm:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        if weight is not None:
            y = y * weight.double()
    size = y.abs().clone()
    if inv_freq is None:
        return y, size
    half = inv_freq.numel()
    axis = torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], device="cuda", dtype=torch.long)
    t = (positions.double()[axis].t() * inv_freq.double())[:, None]
    i = torch.arange(half, device="cuda")
    a, b = (off + 2 * i, off + 2 * i + 1) if interleaved else (off + i, off + half + i)
    out = y.clone()
    out[..., a] = y[..., a] * t.cos() - y[..., b] * t.sin()
    out[..., b] = y[..., b] * t.cos() + y[..., a] * t.sin()
    size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
    return out, size


def check_rope(kda, T, Hq, Hk, D, rot, off=0, interleaved=False, norm=True, weights=True, axes=1, far=5000,
               dtype=torch.bfloat16, pad=0, in_place=False, seed=0):
    fused = normal((T, (Hq + Hk) * D + 24), seed, dtype, 3.0)
    q = fused[:, 8: 8 + Hq * D].unflatten(1, (Hq, D))
    k = fused[:, 8 + Hq * D: 8 + (Hq + Hk) * D].unflatten(1, (Hk, D)) if Hk else None
    pos = torch.randint(0, far, (axes, T), generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    if pad:
        pos[0, torch.randperm(T, generator=torch.Generator().manual_seed(seed))[:pad].cuda()] = -1
    half = rot // 2
    freq = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float().cuda() if rot else None
    sections = [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    w = [normal((D,), seed + 1 + i, torch.float32) if weights and norm else None for i in range(2)]
    refs = [None if x is None else (x.clone(), *rope_ref(x, wt, pos, freq, sections, off, interleaved, norm))
            for x, wt in ((q, w[0]), (k, w[1]))]
    outs = [None if x is None else x if in_place else torch.full((T, x.shape[1] + 1, D), 7.0, dtype=dtype, device="cuda")[:, 1:]
            for x in (q, k)]
    before = fused.clone()
    kda.kda_head_norm_rope(q, k, positions=pos[0] if axes == 1 else pos, inv_freq=freq,
                           sections=None if axes == 1 else sections, rot_offset=off, interleaved=interleaved, norm=norm,
                           q_weight=w[0], k_weight=w[1], q_out=outs[0], k_out=outs[1])
    real = (pos[0] >= 0)[:, None, None]
    for ref, out, name in zip(refs, outs, "qk"):
        if ref is None:
            continue
        x, y, size = ref
        half_step = torch.finfo(dtype).eps / 2
        bound = half_step * y.abs() * (1 + 2.0 ** -10) + 2.0 ** -18 * size + 1e-38
        old = x.double() if in_place else torch.full_like(y, 7.0)
        within(out, torch.where(real, y, old), torch.where(real, bound, 0.0), name)
    if in_place:
        assert torch.equal(fused[:, :8], before[:, :8]) and torch.equal(fused[:, -16:], before[:, -16:])


@pytest.mark.parametrize("T,Hq,Hk,D,rot,off", [
    (1, 1, 0, 64, 64, 0), (1, 32, 8, 128, 64, 0), (3, 5, 1, 128, 128, 0), (130, 7, 3, 128, 32, 96), (33, 2, 2, 16, 16, 0),
    (700, 1, 0, 64, 64, 0), (65, 4, 0, 192, 64, 128), (40, 3, 2, 256, 256, 0), (9, 64, 64, 96, 48, 16),
    (257, 1, 1, 48, 32, 8), (21, 6, 1, 208, 96, 104), (5, 33, 0, 128, 0, 0), (2000, 9, 4, 80, 64, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope(kda, T, Hq, Hk, D, rot, off, interleaved, dtype):
    check_rope(kda, T, Hq, Hk, D, rot, off, interleaved, dtype=dtype, seed=T + D)


@pytest.mark.parametrize("norm,weights", [(False, False), (True, False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_without_norm_or_weights(kda, norm, weights, dtype):
    check_rope(kda, 77, 6, 2, 192, 64, 128, True, norm, weights, dtype=dtype)
    check_rope(kda, 77, 6, 2, 128, 0, 0, False, norm, weights, dtype=dtype)


@pytest.mark.parametrize("axes,rot", [(2, 64), (3, 96), (4, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_axes(kda, axes, rot, interleaved):
    check_rope(kda, 150, 4, 2, 128, rot, 0, interleaved, axes=axes, dtype=torch.float32)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_leaves_padding_alone(kda, in_place, dtype):
    check_rope(kda, 90, 5, 2, 128, 64, 32, pad=31, in_place=in_place, dtype=dtype)
    check_rope(kda, 6, 2, 0, 64, 64, 0, pad=6, in_place=in_place, dtype=dtype)


@pytest.mark.parametrize("far", [1 << 17, (1 << 24) - 1])
def test_rope_far_positions(kda, far):
    check_rope(kda, 500, 2, 1, 128, 128, far=far, dtype=torch.float32)


def test_rope_negative_positions_of_other_axes(kda):
    q = normal((3, 2, 64), 0, torch.float32)
    pos = i32([[0, 5, 9], [-7, -70000, -1]])
    freq = torch.rand(32, generator=gen(1), device="cuda")
    got, _ = kda.kda_head_norm_rope(q, positions=pos, inv_freq=freq, sections=[8, 24], norm=False)
    ref, size = rope_ref(q, None, pos, freq, [8, 24], 0, False, False)
    within(got, ref, 2.0 ** -18 * size, "q")


def test_rope_empty_and_refused(kda):
    q = normal((0, 2, 64), 0)
    assert kda.kda_head_norm_rope(q, positions=i32([]), inv_freq=torch.ones(32, device="cuda"))[0].shape == (0, 2, 64)
    q = normal((4, 2, 64), 0)
    with pytest.raises(ValueError, match="positions"):
        kda.kda_head_norm_rope(q, inv_freq=torch.ones(32, device="cuda"))
    with pytest.raises(ValueError, match="sections"):
        kda.kda_head_norm_rope(q, positions=i32([[0] * 4] * 2), inv_freq=torch.ones(32, device="cuda"), sections=[30, 1])
    with pytest.raises(ValueError, match="positions"):
        kda.kda_head_norm_rope(q, positions=i32([0] * 5), inv_freq=torch.ones(32, device="cuda"))
    with pytest.raises(TypeError, match="bf16 or fp32"):
        kda.kda_head_norm_rope(q.half())
    with pytest.raises(ValueError, match="stride"):
        kda.kda_head_norm_rope(normal((4, 132), 0)[:, :128].unflatten(1, (2, 64)))
    with pytest.raises(kda.KdaError):
        kda.kda_head_norm_rope(normal((4, 2, 72), 0))


def test_rope_zero_row_and_not_finite(kda):
    q = normal((4, 1, 128), 0, torch.float32)
    q[1] = 0.0
    q[2, 0, 5] = INF
    q[3, 0, 100] = NAN
    got, _ = kda.kda_head_norm_rope(q, positions=i32([3] * 4), inv_freq=torch.ones(32, device="cuda"))
    assert (got[1] == 0).all() and got[0].isfinite().all()
    assert got[2, 0, 5].isnan() and got[3].isnan().all()


# ---- the layer -----------------------------------------------------------------------


def layer_ref(q, k, v, g, s0, scale):
    """One sequence in 64 bits: q, k [T, Hk, K], v [T, H, V], g [T, H], s0 [H, V, K].  Returns (o, bound of o's bf16
    products, |q| . A, states behind each token [T, H, V, K] for short ones, S, A)."""
    T, H = v.shape[:2]
    rep = H // q.shape[1]
    q, k = (x.double().repeat_interleave(rep, 1) for x in (q, k))
    v, g = v.double(), g.double()
    S, A = s0.double().clone(), s0.double().abs()
    o, inner, outer = (torch.zeros((T, H, 128), dtype=torch.float64, device="cuda") for _ in range(3))
    for t in range(T):
        if t % C == 0:
            inside, start, decay = [], S.clone(), torch.ones(H, dtype=torch.float64, device="cuda")
        d = g[t].exp()
        S = S * d[:, None, None] + v[t][:, :, None] * k[t][:, None, :]
        A = A * d[:, None, None] + v[t].abs()[:, :, None] * k[t].abs()[:, None, :]
        decay = decay * d
        o[t] = (S @ q[t][:, :, None])[..., 0] * scale
        outer[t] = (A @ q[t].abs()[:, :, None])[..., 0] * abs(scale)
        # the roundings of the chunk's scores and of the state in front of it
        if t % C == 0:
            weight = torch.zeros((C, H), dtype=torch.float64, device="cuda")
        weight = weight * d[None]
        weight[t % C] = 1.0
        rows = slice(t - t % C, t + 1)
        p = (k[rows] * q[t]).sum(-1).abs() * weight[: t % C + 1]
        inner[t] = ((p[..., None] * v[rows].abs()).sum(0)
                    + decay[:, None] * (start.abs() @ q[t].abs()[:, :, None])[..., 0]) * abs(scale)
    return o, inner, outer, S, A


def o_bound(o, inner, outer, T, dtype):
    if dtype is torch.float32:
        return 2.0 ** -24 * o.abs() + T * 2.0 ** -22 * outer + 1e-37
    return 2.0 ** -8 * o.abs() * (1 + 2.0 ** -8) + 2.0 ** -8 * inner * (1 + 2.0 ** -7) + 2.0 ** -12 * outer + 1e-37


def s_bound(A, T, dtype):
    return (T * 2.0 ** -22 if dtype is torch.float32 else 2.0 ** -16 + (-(-T // C)) * 2.0 ** -21) * A + 1e-37


def decays(T, H, seed, kind):
    rate = torch.exp2(-8.0 * torch.arange(H, device="cuda") / max(1, H - 1))
    if kind == "head":
        return -rate
    if kind == "none":
        return torch.zeros((T, H), device="cuda")
    if kind == "strong":
        return -40.0 * torch.rand((T, H), generator=gen(seed), device="cuda")
    g = -rate * torch.nn.functional.softplus(torch.randn((T, H), generator=gen(seed), device="cuda"))
    if kind == "reset":
        g[torch.rand((T, H), generator=gen(seed + 1), device="cuda") < 0.02] = -INF
    return g


def layer_inputs(T, H, Hk, dtype, seed, kind="token"):
    fused = normal((T, 2 * Hk * 128 + H * 128 + 8), seed, dtype)
    q, k, v = fused[:, : Hk * 128], fused[:, Hk * 128: 2 * Hk * 128], fused[:, 2 * Hk * 128: (2 * Hk + H) * 128]
    return (q.unflatten(1, (Hk, 128)), k.unflatten(1, (Hk, 128)), v.unflatten(1, (H, 128)), decays(T, H, seed + 1, kind))


def check_chunk(kda, lens, H, Hk, dtype=torch.bfloat16, kind="token", carry=True, in_place=False, extra=0, seed=0, cu=True,
                scale=128 ** -0.5, **kw):
    T, N = sum(lens), len(lens)
    q, k, v, g = layer_inputs(T + extra, H, Hk, dtype, seed, kind)
    s0 = normal((N, H, 128, 128), seed + 2, torch.float32) if carry else None
    start = s0.clone() if carry else torch.zeros((N, H, 128, 128), device="cuda")
    offsets = [0]
    for n in lens:
        offsets.append(offsets[-1] + n)
    o = torch.full((T + extra, H, 128), 7.0, dtype=dtype, device="cuda")
    _, sf = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32(offsets) if cu else None, n_seqs=N, initial_state=s0,
                                     final_state=s0 if in_place else None, scale=scale, o=o, **kw)
    torch.cuda.synchronize()
    for n, (a, b) in enumerate(zip(offsets, offsets[1:])):
        gn = g.expand(T + extra, H)[a:b]
        ref, inner, outer, S, A = layer_ref(q[a:b], k[a:b], v[a:b], gn, start[n], scale)
        within(o[a:b], ref, o_bound(ref, inner, outer, b - a, dtype), f"o of sequence {n}")
        within(sf[n], S, s_bound(A, b - a, dtype), f"state of sequence {n}")
    assert (o[T:] == 7.0).all()
    return o, sf


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("lens", [[1], [127], [128], [129], [0], [5, 0, 300, 1, 64], [256, 128, 33], [2, 3] * 9])
@pytest.mark.parametrize("dtype", DTYPES)
def test_chunk_lengths(kda, lens, dtype):
    check_chunk(kda, lens, 3, 3, dtype)
    check_chunk(kda, lens, 2, 1, dtype, carry=False, seed=5)


@pytest.mark.parametrize("kind", ["head", "none", "strong", "reset"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_chunk_decays(kda, kind, dtype):
    check_chunk(kda, [200, 391], 4, 2, dtype, kind)


@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (8, 1), (5, 5)])
def test_chunk_heads(kda, H, Hk):
    check_chunk(kda, [70, 190], H, Hk)


@pytest.mark.parametrize("lens,H", [([1500], 1), ([2048, 5, 1100], 1), ([1000, 1], 2), ([130] * 7 + [1700], 2), ([3333], 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_chunk_long_sequences_are_cut(kda, lens, H, in_place):
    check_chunk(kda, lens, H, H, in_place=in_place)
    check_chunk(kda, lens, H, H, carry=False, kind="head", seed=9)


@pytest.mark.parametrize("dtype", DTYPES)
def test_chunk_equal_lengths_rows_behind_and_scale(kda, dtype):
    check_chunk(kda, [150] * 4, 2, 2, dtype, cu=False)
    check_chunk(kda, [150, 20], 2, 2, dtype, extra=77)
    check_chunk(kda, [150, 20], 2, 2, dtype, scale=-3.0)
    check_chunk(kda, [150, 20], 2, 2, dtype, scale=0.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("long", [0, 1500])
def test_chunk_pools_and_refused_sequences(kda, dtype, long):
    # sequence 1 has no slot in the pool, sequence 3 ends behind the last token, sequence 4's offsets run backwards
    H, end = 2, 370 + long
    T = end + 60
    q, k, v, g = layer_inputs(T, H, 1, dtype, 0)
    pool = normal((9, H, 128, 128), 3, torch.float32)
    start = pool.clone()
    cu = [0, 40, 170, end, T + 5, T]
    o = torch.full((T, H, 128), 7.0, dtype=dtype, device="cuda")
    kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32(cu), initial_state=pool, final_state=pool,
                             state_indices=i32([6, 9, 0, 2, 4]), o=o)
    torch.cuda.synchronize()
    for n, slot in ((0, 6), (2, 0)):
        a, b = cu[n], cu[n + 1]
        ref, inner, outer, S, A = layer_ref(q[a:b], k[a:b], v[a:b], g[a:b], start[slot], 128 ** -0.5)
        within(o[a:b], ref, o_bound(ref, inner, outer, b - a, dtype), f"o of sequence {n}")
        within(pool[slot], S, s_bound(A, b - a, dtype), f"state of sequence {n}")
    assert o[40:170].isnan().all() and (o[end:] == 7.0).all()
    for slot in (1, 2, 3, 4, 5, 7, 8):
        assert torch.equal(pool[slot], start[slot])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_chunk_not_finite_stays_in_its_sequence(kda, dtype, value):
    lens, H = [200, 150, 90], 2
    T = sum(lens)
    q, k, v, g = (x.clone() for x in layer_inputs(T, H, H, dtype, 0))
    clean, sc = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32([0, 200, 350, 440]))
    for at, x in ((200, k), (201, q), (202, v)):
        x[at] = value
    g[203] = NAN
    o, s = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32([0, 200, 350, 440]))
    for a, b, n in ((0, 200, 0), (350, 440, 2)):
        assert torch.equal(o[a:b], clean[a:b]) and torch.equal(s[n], sc[n])
    assert not o[204:350].isfinite().any() and not s[1].isfinite().any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("which", ["k", "v", "q"])
@pytest.mark.parametrize("value", [NAN, INF])
def test_chunk_not_finite_leaves_the_rows_before_it(kda, dtype, which, value):
    q, k, v, g = (x.clone() for x in layer_inputs(300, 1, 1, dtype, 0))
    clean, _ = kda.kda_linear_chunk_fwd(q, k, v, g)
    at = 170
    dict(q=q, k=k, v=v)[which][at, 0, 77] = value
    o, s = kda.kda_linear_chunk_fwd(q, k, v, g)
    assert torch.equal(o[:at], clean[:at])
    if which == "v":    # the channel, and no other
        other = torch.arange(128, device="cuda") != 77
        assert not o[at:, 0, 77].isfinite().any() and not s[0, 0, 77].isfinite().any()
        assert torch.equal(o[:, :, other], clean[:, :, other]) and s[0, 0, other].isfinite().all()
    elif which == "k":
        assert not o[at:].isfinite().any() and not s[0, 0, :, 77].isfinite().any()
    else:
        assert not o[at].isfinite().any() and torch.equal(o[at + 1:], clean[at + 1:]) and s.isfinite().all()


def test_rope_refuses_a_destination_without_its_source(kda):
    q = normal((4, 2, 128), 0)
    with pytest.raises(ValueError, match="k_out without k"):
        kda.kda_head_norm_rope(q, k_out=torch.empty_like(q))


def test_chunk_repeats_bit_for_bit_and_in_a_graph(kda):
    q, k, v, g = layer_inputs(2500, 2, 2, torch.bfloat16, 0)
    cu = i32([0, 1900, 2500])
    o, s = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=cu)
    out, sf = torch.empty_like(o), torch.empty_like(s)
    ws = torch.empty(max(256, kda.kda_linear_chunk_workspace_bytes(2500, 2, 2)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=cu, o=out, final_state=sf, workspace=ws)
    for _ in range(3):
        out.zero_(), sf.zero_(), ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(sf, s)


def test_chunk_on_another_stream_and_many_calls(kda):
    a, b = (layer_inputs(1400, 2, 1, torch.bfloat16, seed) for seed in (0, 50))
    ref = [kda.kda_linear_chunk_fwd(*x) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, x in enumerate((a, b)):
            got[i].append(kda.kda_linear_chunk_fwd(*x, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, s in got[i]:
            assert torch.equal(o, ref[i][0]) and torch.equal(s, ref[i][1])


def test_chunk_many_sequences(kda):
    lens = [(7 * i) % 40 for i in range(500)]
    T = sum(lens)
    q, k, v, g = layer_inputs(T, 2, 2, torch.bfloat16, 0)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    o, s = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=cu)
    for n in (0, 1, 17, 250, 499):
        x, y = int(cu[n]), int(cu[n + 1])
        ref, inner, outer, S, A = layer_ref(q[x:y], k[x:y], v[x:y], g[x:y], torch.zeros_like(s[n]), 128 ** -0.5)
        within(o[x:y], ref, o_bound(ref, inner, outer, y - x, torch.bfloat16), f"o of sequence {n}")
        within(s[n], S, s_bound(A, y - x, torch.bfloat16), f"state of sequence {n}")


def test_chunk_refuses(kda):
    q, k, v, g = layer_inputs(64, 4, 2, torch.bfloat16, 0)
    pool = torch.zeros((3, 4, 128, 128), device="cuda")
    with pytest.raises(ValueError, match="k shape"):
        kda.kda_linear_chunk_fwd(q, k[:, :1], v, g)
    with pytest.raises(TypeError, match="v must be"):
        kda.kda_linear_chunk_fwd(q, k, v.float(), g)
    with pytest.raises(ValueError, match="g shape"):
        kda.kda_linear_chunk_fwd(q, k, v, g[:, :2].contiguous())
    with pytest.raises(ValueError, match="states"):
        kda.kda_linear_chunk_fwd(q, k, v, g, initial_state=pool)
    with pytest.raises(ValueError, match="destination pool"):
        kda.kda_linear_chunk_fwd(q, k, v, g, initial_state=pool, state_indices=i32([0]))
    with pytest.raises(ValueError, match="holds"):
        kda.kda_linear_chunk_fwd(q, k, v, g, final_state=pool, state_indices=i32([0]), n_slots=4)
    with pytest.raises(kda.KdaError):
        kda.kda_linear_chunk_fwd(q, k, v, g, n_seqs=3)
    with pytest.raises(kda.KdaError):
        kda.kda_linear_chunk_fwd(normal((64, 3, 128), 0), normal((64, 3, 128), 0), v, g)


# ---- steps -----------------------------------------------------------------------------


def check_step(kda, N, H, Hk, dtype, kind="token", slots=None, seed=0):
    q, k, v, g = layer_inputs(N, H, Hk, dtype, seed, kind)
    pool = normal((N + 2, H, 128, 128), seed + 3, torch.float32)
    start = pool.clone()
    index = list(range(N)) if slots is None else slots
    o = kda.kda_linear_step(q, k, v, g, pool, state_indices=None if slots is None else i32(slots))
    torch.cuda.synchronize()
    for n in {0, N // 2, N - 1}:
        if not 0 <= index[n] < N + 2:
            assert o[n].isnan().all()
            continue
        gn = g.expand(N, H)[n: n + 1]
        ref, _, outer, S, A = layer_ref(q[n: n + 1], k[n: n + 1], v[n: n + 1], gn, start[index[n]], 128 ** -0.5)
        half = torch.finfo(dtype).eps / 2
        within(o[n], ref[0], half * ref[0].abs() * (1 + half) + 2.0 ** -19 * outer[0] + 1e-37, f"o of sequence {n}")
        within(pool[index[n]], S, 2.0 ** -21 * A, f"state of sequence {n}")
    held = {s for s in index if 0 <= s < N + 2}
    for s in set(range(min(N + 2, 40))) - held:
        assert torch.equal(pool[s], start[s])


@pytest.mark.parametrize("N,H,Hk", [(1, 1, 1), (3, 2, 1), (50, 6, 3), (90, 7, 7), (160, 8, 2)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["token", "head", "reset"])
def test_step(kda, N, H, Hk, dtype, kind):
    check_step(kda, N, H, Hk, dtype, kind)
    order = torch.randperm(N + 2, generator=torch.Generator().manual_seed(N))[:N].tolist()
    check_step(kda, N, H, Hk, dtype, kind, slots=order, seed=11)


def test_step_refused_slots_and_no_sequence(kda):
    for dtype in DTYPES:
        check_step(kda, 5, 2, 2, dtype, slots=[-1, 3, 7, 0, 6])
    q, k, v, g = layer_inputs(0, 2, 2, torch.bfloat16, 0)
    assert kda.kda_linear_step(q, k, v, g, torch.zeros((1, 2, 128, 128), device="cuda")).shape == (0, 2, 128)


@pytest.mark.parametrize("S", [1, 2, 3, 6])
@pytest.mark.parametrize("N,H,Hk", [(1, 1, 1), (4, 6, 2), (90, 8, 8), (320, 4, 4)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["token", "head"])
def test_multi_step(kda, S, N, H, Hk, dtype, kind):
    q, k, v, g = (x if x.dim() == 1 else x.unflatten(0, (N, S)) for x in layer_inputs(N * S, H, Hk, dtype, S, kind))
    pool = normal((N * S + 1, H, 128, 128), 3, torch.float32)
    start = pool.clone()
    index = torch.randperm(N * S + 1, generator=torch.Generator().manual_seed(S))[: N * S].view(N, S).to(torch.int32).cuda()
    accepted = torch.randint(1, S + 1, (N,), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    if N > 2:
        accepted[1] = 0
        index[2, S - 1] = N * S + 1
    count = None if S == 2 else accepted
    o = kda.kda_linear_multi_step(q, k, v, g, pool, index, num_accepted=count)
    torch.cuda.synchronize()
    bad = [] if N <= 2 else [2] if count is None else [1, 2]
    touched = torch.zeros(N * S + 1, dtype=torch.bool)
    for n in {0, 1 % N, 2 % N, N // 2, N - 1}:
        if n in bad:
            assert o[n].isnan().all()
            continue
        state = start[index[n, 0 if count is None else accepted[n] - 1]]
        gn = g.expand(N, S, H)[n]
        for t in range(S):
            ref, _, outer, state, A = layer_ref(q[n, : t + 1], k[n, : t + 1], v[n, : t + 1], gn[: t + 1],
                                                start[index[n, 0 if count is None else accepted[n] - 1]], 128 ** -0.5)
            half = torch.finfo(dtype).eps / 2
            within(o[n, t], ref[t], half * ref[t].abs() * (1 + half) + (t + 1) * 2.0 ** -19 * outer[t] + 1e-37, f"o {n} {t}")
            within(pool[index[n, t]], state, (t + 1) * 2.0 ** -21 * A, f"state {n} {t}")
    for n in range(N):
        if n not in bad:
            touched[index[n].long().cpu()] = True
    kept = (~touched).nonzero()[:, 0].cuda()
    assert torch.equal(pool[kept], start[kept])


def test_step_in_a_graph_and_on_another_stream(kda):
    q, k, v, g = layer_inputs(6, 4, 2, torch.bfloat16, 0)
    pool = normal((6, 4, 128, 128), 3, torch.float32)
    start = pool.clone()
    for _ in range(3):
        ref = kda.kda_linear_step(q, k, v, g, pool)
    end, o = pool.clone(), torch.empty_like(ref)
    pool.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_linear_step(q, k, v, g, pool, o=o)
    pool.copy_(start)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, ref) and torch.equal(pool, end)
    pool.copy_(start)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = kda.kda_linear_step(q, k, v, g, pool, stream=side)
    side.synchronize()
    assert torch.equal(got, ref) and torch.equal(pool, end)


def test_step_refuses(kda):
    q, k, v, g = layer_inputs(4, 4, 2, torch.bfloat16, 0)
    pool = torch.zeros((4, 4, 128, 128), device="cuda")
    with pytest.raises(ValueError, match="state_pool"):
        kda.kda_linear_step(q, k, v, g, pool[:, :2].contiguous())
    with pytest.raises(TypeError, match="state_pool"):
        kda.kda_linear_step(q, k, v, g, pool.double())
    with pytest.raises(kda.KdaError):
        kda.kda_linear_step(q, k, v, g, pool[:3])
    with pytest.raises(ValueError, match="one stride"):
        x = normal((2, 3, 4, 128), 0)[:, :2]
        kda.kda_linear_multi_step(x, x, x, g.view(2, 2, 4), pool, i32([[0, 1], [2, 3]]))


# ---- together ---------------------------------------------------------------------------


def test_prompt_then_steps_follow_one_longer_prompt(kda):
    """rope -> chunk -> gate norm over prompts, then steps from the pool: against one call over all tokens."""
    H, Hk, lens, more = 4, 2, [300, 1, 1200], 3
    freq = (10000.0 ** (-torch.arange(32) / 32)).cuda()
    w = normal((128,), 1, torch.float32)
    g = -torch.exp2(-torch.arange(1, H + 1, device="cuda").float())
    data = [normal((n + more, (2 * Hk + 2 * H) * 128), 10 + i) for i, n in enumerate(lens)]

    def layer(x, pos, core):
        q, k, v, gate = x.split([Hk * 128, Hk * 128, H * 128, H * 128], 1)
        q, k = kda.kda_head_norm_rope(q.unflatten(1, (Hk, 128)), k.unflatten(1, (Hk, 128)), positions=i32(pos),
                                      inv_freq=freq, q_weight=w, k_weight=w)
        o = core(q, k, v.unflatten(1, (H, 128)))
        return kda.kda_output_gate_norm(o, gate.unflatten(1, (H, 128)).contiguous(), w)

    def prompts(rows, pool):
        cu = [0]
        for r in rows:
            cu.append(cu[-1] + len(r))
        o = layer(torch.cat(rows), [p for r in rows for p in range(len(r))],
                  lambda q, k, v: kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32(cu), final_state=pool,
                                                           state_indices=i32([2, 0, 1]))[0])
        return [o[a:b] for a, b in zip(cu, cu[1:])]

    whole = prompts(data, torch.zeros((3, H, 128, 128), device="cuda"))
    pool = torch.zeros((3, H, 128, 128), device="cuda")
    prompts([x[:n] for x, n in zip(data, lens)], pool)
    for s in range(more):
        got = layer(torch.stack([x[n + s] for x, n in zip(data, lens)]), [n + s for n in lens],
                    lambda q, k, v: kda.kda_linear_step(q, k, v, g, pool, state_indices=i32([2, 0, 1])))
        for i, n in enumerate(lens):
            # two bf16 products and roundings against one: a few half steps of an output row
            off = (got[i].double() - whole[i][n + s].double()).norm() / whole[i][n + s].double().norm()
            assert off < 2.0 ** -6, (i, s, float(off))


# ---- calls that share something, sizes at the ends ----------------------------------------


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [NAN, INF])
def test_chunk_decay_not_finite_leaves_the_rows_before_it(kda, dtype, value):
    q, k, v, g = (x.clone() for x in layer_inputs(300, 2, 1, dtype, 0))
    at = 170
    g[at, 1] = value
    o, s = kda.kda_linear_chunk_fwd(q, k, v, g)
    ref, inner, outer, S, A = layer_ref(q[:at], k[:at], v[:at], g[:at], torch.zeros_like(s[0]), 128 ** -0.5)
    within(o[:at], ref, o_bound(ref, inner, outer, at, dtype), "o before it")
    assert not o[at:, 1].isfinite().any() and not s[0, 1].isfinite().any()
    assert o[:, 0].isfinite().all() and s[0, 0].isfinite().all()


@pytest.mark.parametrize("lens,H", [([700] * 14, 8), ([1000, 1], 2), ([900, 0, 650], 20)])
def test_chunk_sequences_that_could_be_cut_and_are_not(kda, lens, H):
    check_chunk(kda, lens, H, H, in_place=True)


def test_chunk_fp32_sequences_that_are_not_cut(kda):
    check_chunk(kda, [200, 30, 140, 0, 90] * 12, 16, 4, torch.float32)


def test_two_graphs_share_a_workspace(kda):
    cu = i32([0, 1900, 2500])
    ws = torch.empty(max(256, kda.kda_linear_chunk_workspace_bytes(2500, 2, 2)), dtype=torch.uint8, device="cuda")
    graphs = []
    for seed in (0, 40):
        x = layer_inputs(2500, 2, 2, torch.bfloat16, seed)
        ref = kda.kda_linear_chunk_fwd(*x, cu_seqlens=cu)
        out = tuple(torch.empty_like(t) for t in ref)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kda.kda_linear_chunk_fwd(*x, cu_seqlens=cu, o=out[0], final_state=out[1], workspace=ws)
        graphs.append((graph, x, ref, out))
    for _ in range(4):
        for graph, _, _, out in graphs:
            out[0].zero_(), out[1].zero_()
            graph.replay()
    torch.cuda.synchronize()
    for _, _, ref, out in graphs:
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])


def test_steps_and_rope_on_two_streams_at_once(kda):
    freq = (100.0 ** (-torch.arange(16) / 16)).cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]

    def run(seed, stream):
        q, k, v, g = layer_inputs(40, 4, 2, torch.bfloat16, seed)
        pool = normal((40, 4, 128, 128), seed + 3, torch.float32)
        pos = torch.arange(40, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        yield
        for _ in range(20):
            a, b = kda.kda_head_norm_rope(q, k, positions=pos, inv_freq=freq, stream=stream)
            o = kda.kda_linear_step(a, b, v, g, pool, stream=stream)
            yield
        torch.cuda.synchronize()
        yield o, pool

    alone = [list(run(seed, None))[-1] for seed in (0, 60)]
    together = list(zip(*(run(seed, streams[i]) for i, seed in enumerate((0, 60)))))[-1]
    for x, y in zip(alone, together):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_chunk_thousands_of_sequences_and_a_long_one(kda):
    lens = [3] * 2500 + [1500, 0] + [3, 7] * 1300
    N, T, H = len(lens), sum(lens), 2
    q, k, v, g = layer_inputs(T, H, 2, torch.bfloat16, 0)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    pool = normal((N + 1, H, 128, 128), 3, torch.float32)
    start = pool.clone()
    index = (torch.arange(N - 1, -1, -1) + 1).to(torch.int32)
    gone = [0, 2400, 4000]
    index[gone] = torch.tensor([-1, N + 1, -5], dtype=torch.int32)
    o = torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=cu, initial_state=pool, final_state=pool, state_indices=index.cuda(), o=o)
    for n in (1, 2399, 2499, 2500, 2501, 2502, 3999, N - 1):
        a, b, slot = int(cu[n]), int(cu[n + 1]), int(index[n])
        if a == b:
            assert torch.equal(pool[slot], start[slot])
            continue
        ref, inner, outer, S, A = layer_ref(q[a:b], k[a:b], v[a:b], g[a:b], start[slot], 128 ** -0.5)
        within(o[a:b], ref, o_bound(ref, inner, outer, b - a, torch.bfloat16), f"o of sequence {n}")
        within(pool[slot], S, s_bound(A, b - a, torch.bfloat16), f"state of sequence {n}")
    rows = torch.zeros(T, dtype=torch.bool, device="cuda")
    for n in gone:
        rows[int(cu[n]): int(cu[n + 1])] = True
    assert o[rows].isnan().all() and o[~rows].isfinite().all() and not (o[~rows] == 7.0).all(-1).any()
    for slot in [0] + [N - n for n in gone]:
        assert torch.equal(pool[slot], start[slot])


@pytest.mark.parametrize("dtype", DTYPES)
def test_chunk_more_heads_than_sms_and_no_token(kda, dtype):
    check_chunk(kda, [130, 0, 10], 170, 1, dtype)
    check_chunk(kda, [0, 0, 0], 2, 2, dtype)
    check_chunk(kda, [0, 0, 0], 2, 2, dtype, carry=False)
    check_chunk(kda, [20, 0, 30], 3, 3, dtype, in_place=True)


def test_multi_step_keeps_the_last_state_of_a_slot_that_it_repeats(kda):
    N, S, H = 3, 4, 2
    q, k, v, g = layer_inputs(N * S, H, H, torch.bfloat16, 0)
    pool = normal((N, H, 128, 128), 3, torch.float32)
    one = pool.clone()
    shape = lambda x: x.unflatten(0, (N, S))  # noqa: E731
    o = kda.kda_linear_multi_step(shape(q), shape(k), shape(v), shape(g), pool, i32([[n] * S for n in range(N)]))
    for t in range(S):
        got = kda.kda_linear_step(*(shape(x)[:, t].contiguous() for x in (q, k, v, g)), one)
        assert torch.equal(o[:, t], got)
    assert torch.equal(pool, one)


def test_offsets_behind_32_bits(kda):
    """Slots and tokens whose elements lie behind 2^31 of their buffers."""
    pool = torch.empty((140000, 1, 128, 128), device="cuda")
    slot, T, stride = 139990, 18, 1 << 27
    x = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda").view(T, 1, stride)
    q, k, v = (x[:, :, 128 * i: 128 * i + 128] for i in range(3))
    for i, t in enumerate((q, k, v)):
        t.copy_(normal((T, 1, 128), i))
    g = decays(T, 1, 5, "token")
    s0 = normal((1, 128, 128), 6, torch.float32)
    ref, inner, outer, S, A = layer_ref(q, k, v, g, s0, 128 ** -0.5)
    pool[slot] = s0
    o, _ = kda.kda_linear_chunk_fwd(q, k, v, g, initial_state=pool, final_state=pool, state_indices=i32([slot]))
    within(o, ref, o_bound(ref, inner, outer, T, torch.bfloat16), "o")
    within(pool[slot], S, s_bound(A, T, torch.bfloat16), "state")
    pool[slot] = s0
    for t in range(T):
        one = kda.kda_linear_step(q[t:], k[t:], v[t:], g[t:], pool, state_indices=i32([slot] + [-1] * (T - t - 1)))
        within(one[0], ref[t], 2.0 ** -8 * ref[t].abs() * (1 + 2.0 ** -8) + (t + 1) * 2.0 ** -19 * outer[t] + 1e-37, f"o of token {t}")
    within(pool[slot], S, T * 2.0 ** -21 * A, "state of the steps")
    freq, pos = (10000.0 ** (-torch.arange(64) / 64)).cuda(), torch.arange(T, dtype=torch.int32, device="cuda")
    a, _ = kda.kda_head_norm_rope(q, positions=pos, inv_freq=freq)
    b, _ = kda.kda_head_norm_rope(q.contiguous(), positions=pos, inv_freq=freq)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
def test_chunk_decays_above_zero(kda, dtype):
    # (their sum over 128 tokens stays below 20)
    q, k, v, _ = layer_inputs(300, 2, 2, dtype, 0)
    g = torch.rand((300, 2), generator=gen(9), device="cuda") * 0.25 - 0.1
    o, s = kda.kda_linear_chunk_fwd(q, k, v, g)
    ref, inner, outer, S, A = layer_ref(q, k, v, g, torch.zeros_like(s[0]), 128 ** -0.5)
    within(o, ref, o_bound(ref, inner, outer, 300, dtype), "o")
    within(s[0], S, s_bound(A, 300, dtype), "state")
