"""Precision of the linear-attention layer with one decay a head over long runs and in mixed
batches, against 64 bits, by the norm of the error where roundings add up as independent ones do
(a rounding of fp32 is off by at most 2^-24 of the value, 2^-24 / sqrt 3 in the root mean square)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def kda():
    import kimi_delta_attention_07_gb300 as m
    m.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    return m


def normal(shape, seed, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


# ---- a decay that is applied again and again ------------------------------------------


@pytest.mark.parametrize("S", [1, 4])
@pytest.mark.parametrize("dtype", DTYPES)
def test_steps_keep_a_slow_fixed_decay(kda, S, dtype):
    """1024 steps at decays of 2^-6 to 2^-9 a token.  A step rounds an element of the state twice; behind m = 2^9
    tokens of memory these add up to 2^-24 sqrt(2 / 3) sqrt(m / 2) = 13 x 2^-24 of the state's norm, below 2^-20.  The
    decay as the sum of two floats adds 2^-22 at most, as one float up to m 2^-25 = 2^-16."""
    H, N, steps = 4, 2, 1024
    g = -torch.exp2(-torch.arange(6.0, 10.0, device="cuda"))
    d = g.double().exp()[:, None, None]
    pool = torch.zeros((N * S, H, 128, 128), device="cuda")
    ref = torch.zeros((N, H, 128, 128), dtype=torch.float64, device="cuda")
    slots = torch.arange(N * S, dtype=torch.int32, device="cuda").view(N, S)
    for t in range(0, steps, S):
        q, k, v = (normal((N, S, H, 128), 3 * t + i, dtype) for i in range(3))
        if S == 1:
            kda.kda_linear_step(q[:, 0], k[:, 0], v[:, 0], g, pool)
        else:
            kda.kda_linear_multi_step(q, k, v, g, pool, slots, num_accepted=i32([S] * N))
        for s in range(S):
            ref = ref * d + v[:, s].double()[..., :, None] * k[:, s].double()[..., None, :]
    for h in range(H):
        assert rel(pool[S - 1::S, h], ref[:, h]) < 2.0 ** -19, h


def final_state(k, v, g):
    """[H, V, K] behind tokens k, v [T, H, 128] with decays g [T, H], from zero, in 64 bits."""
    g = g.double()
    behind = (g.flip(0).cumsum(0).flip(0) - g).exp()
    return torch.einsum("the,thd->hed", v.double() * behind[..., None], k.double())


@pytest.mark.parametrize("dtype,T,n", [(torch.bfloat16, 131072, 1), (torch.bfloat16, 20000, 1), (torch.bfloat16, 6000, 3),
                                       (torch.float32, 32768, 1), (torch.float32, 9000, 2)])
@pytest.mark.parametrize("fixed", [True, False])
def test_chunks_keep_slow_decays(kda, dtype, T, n, fixed):
    """Decays of 2^-8 to 2^-20 a token over whole prompts, chunk by chunk and segment by segment.  A token's weight
    carries two exponentials (2^-22 each), three products and its exponent's rounding (2^-24 each, relative to
    exponents that are at most some units while the weight counts); the sums, a rounding of 2^-24 / sqrt 3 for each of
    some hundreds of chunks, segments or tokens in a row, add sqrt(200) of those: 2^-20 of the norm in all.  A decay as one
    float adds 2^-25 for each time that it is applied within its memory: 200 segments 2^-17."""
    H = 4
    rate = torch.exp2(-torch.tensor([8.0, 12.0, 16.0, 20.0], device="cuda"))
    g = (-0.9 * rate if fixed else -rate * torch.rand((T, H), generator=torch.Generator("cuda").manual_seed(5), device="cuda"))
    q, k, v = (normal((T, H, 128), i, dtype) for i in range(3))
    cu = [0] + [T * (2 * i + 1) // (2 * n) for i in range(1, n)] + [T]
    _, s = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32(cu))
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        ref = final_state(k[a:b], v[a:b], g.expand(T, H)[a:b])
        for h in range(H):
            assert rel(s[i, h], ref[h]) < 2.0 ** -20, (i, h)


# ---- rows of a few tokens, alone and beside others -------------------------------------


def run(kda, data, order, H):
    """o of the sequences data[i] for i in order, packed, each with 0.5 in its initial state."""
    q, k, v, g = (torch.cat([data[i][j] for i in order]) for j in range(4))
    cu = [0]
    for i in order:
        cu.append(cu[-1] + data[i][0].shape[0])
    s0 = torch.full((len(order), H, 128, 128), 0.5, device="cuda")
    o, s = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32(cu), initial_state=s0)
    return {i: (o[a:b], s[n]) for n, (i, a, b) in enumerate(zip(order, cu, cu[1:]))}


@pytest.mark.parametrize("H,Hk", [(8, 2), (90, 1)])
def test_a_sequence_does_not_depend_on_the_others(kda, H, Hk):
    """Short sequences, which no call cuts, bit for bit: alone, a few together, and beside a long one."""
    lens = [4, 1, 130, 77, 512, 300, 1900]
    data = [(normal((n, Hk, 128), 5 * i), normal((n, Hk, 128), 5 * i + 1), normal((n, H, 128), 5 * i + 2),
             -torch.rand((n, H), generator=torch.Generator("cuda").manual_seed(i), device="cuda")) for i, n in enumerate(lens)]
    together = [run(kda, data, order, H) for order in ([0, 1, 2, 3], [6, 0, 1, 2, 3, 4, 5], [5, 4, 3, 2, 1, 0, 6])]
    for i in range(6):
        o, s = run(kda, data, [i], H)[i]
        for others in together:
            if i in others:
                assert torch.equal(others[i][0], o) and torch.equal(others[i][1], s), i


@pytest.mark.parametrize("lens", [[4], [4] * 200, [1, 2, 3, 31, 33, 128] * 6, [3, 2500, 5]])
@pytest.mark.parametrize("decay", [0.0, -0.05, -3.0])
def test_first_rows_are_off_by_little_more_than_their_own_rounding(kda, lens, decay):
    """o of a sequence's first 128 tokens from zero: rounded to bf16 (2^-8), behind scores as two bf16 terms (2^-16 of each
    p_ij v_j) and fp32 sums and decays (2^-17 of |q| |k| |v|, weighed alike: 8 steps of 2^-22 and three exponentials)."""
    H, T = 4, sum(lens)
    q, k, v = (normal((T, H, 128), i) for i in range(3))
    g = torch.full((H,), decay, device="cuda")
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    o, _ = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32(cu))
    for a, b in zip(cu, cu[1:]):
        b = min(b, a + 128)
        x, y, z = (t[a:b].double().transpose(0, 1) for t in (q, k, v))
        at = torch.arange(b - a, device="cuda", dtype=torch.float64)
        weight = ((at[:, None] - at) * g.double()[0]).exp().tril() * 128 ** -0.5
        p = x @ y.transpose(1, 2) * weight
        ref = p @ z
        bound = (2.0 ** -8 * (1 + 2.0 ** -7) * ref.abs() + 2.0 ** -16 * (p.abs() @ z.abs())
                 + 2.0 ** -17 * (x.abs() @ y.abs().transpose(1, 2) * weight @ z.abs()))
        off = (o[a:b].double().transpose(0, 1) - ref).abs()
        assert (off <= bound).all(), float((off / bound).max())


def test_ragged_sequences_of_many_heads_are_listed(kda):
    """More than half as many heads as SMs: nothing is cut, and the sequences' order still comes from a list, which
    takes a workspace.  Against each sequence alone, bit for bit."""
    H, lens = 96, [100, 3000, 1, 0, 777, 1500, 128, 640]
    assert kda.kda_linear_chunk_workspace_bytes(sum(lens), len(lens), H) > 0
    assert kda.kda_linear_chunk_workspace_bytes(sum(lens), 1, H) == 0
    data = [(normal((n, 2, 128), 5 * i), normal((n, 2, 128), 5 * i + 1), normal((n, H, 128), 5 * i + 2),
             -torch.rand((n, H), generator=torch.Generator("cuda").manual_seed(i), device="cuda")) for i, n in enumerate(lens)]
    together = run(kda, data, list(range(len(lens))), H)
    for i in range(len(lens)):
        o, s = run(kda, data, [i], H)[i]
        assert torch.equal(together[i][0], o) and torch.equal(together[i][1], s), i
    # of one length: as they come
    q, k, v, g = (torch.cat([d[j] for d in data])[:6000] for j in range(4))
    o, s = kda.kda_linear_chunk_fwd(q, k, v, g, n_seqs=4)
    o2, s2 = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32([0, 1500, 3000, 4500, 6000]))
    assert torch.equal(o, o2) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype,T,H,cut", [
    (torch.float32, 65, 16, False), (torch.float32, 128, 1, False), (torch.float32, 256, 64, False), (torch.float32, 512, 16, True),
    (torch.float32, 1024, 4, True), (torch.bfloat16, 641, 64, False), (torch.bfloat16, 1024, 64, False),
    (torch.bfloat16, 1024, 4, True), (torch.bfloat16, 4096, 32, True), (torch.bfloat16, 2500, 100, False)])
def test_one_sequence_is_cut_where_it_pays(kda, dtype, T, H, cut):
    """By the rule that several sequences are cut by; what is cut takes a workspace.  State and last outputs against 64 bits."""
    code = kda.KDA_BF16 if dtype is torch.bfloat16 else kda.KDA_F32
    assert (kda.kda_linear_chunk_workspace_bytes(T, 1, H, code) > 0) == cut
    q, k, v = (normal((T, H, 128), i, dtype) for i in range(3))
    g = -torch.rand((T, H), generator=torch.Generator("cuda").manual_seed(5), device="cuda") / 64
    o, s = kda.kda_linear_chunk_fwd(q, k, v, g)
    ref = final_state(k, v, g)
    assert rel(s[0], ref) < 2.0 ** -20
    # (bf16: o's rounding, and those of P and of the state in front of the chunk, 2^-8 / sqrt 3 at most each)
    last = torch.einsum("hed,hd->he", ref, q[-1].double()) * 128 ** -0.5
    assert rel(o[-1], last) < (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -20)


@pytest.mark.parametrize("lens,H,workspace", [([200, 154, 108, 62, 17, 90, 120], 8, False), ([500, 600], 8, False), ([4, 1100], 2, False),
                                              ([200] * 12, 8, True), ([3000, 20], 8, True), ([40] * 20, 16, True), ([300, 500], 40, False)])
def test_nothing_is_launched_for_a_cut_that_cannot_pay(kda, lens, H, workspace):
    """By their tokens and heads alone; what may be cut, or is listed for its order, takes a workspace."""
    assert (kda.kda_linear_chunk_workspace_bytes(sum(lens), len(lens), H) > 0) == workspace
    data = [(normal((n, 2, 128), 5 * i), normal((n, 2, 128), 5 * i + 1), normal((n, H, 128), 5 * i + 2),
             -torch.rand((n, H), generator=torch.Generator("cuda").manual_seed(i), device="cuda")) for i, n in enumerate(lens)]
    together = run(kda, data, list(range(len(lens))), H)
    for i, n in enumerate(lens):
        if n <= 512 or not workspace:
            o, s = run(kda, data, [i], H)[i]
            assert torch.equal(together[i][0], o) or n > 512
            assert rel(together[i][0], o.double()) < 2.0 ** -7 and rel(together[i][1], s.double()) < 2.0 ** -19


# ---- states behind every way of finding the segments ------------------------------------


@pytest.mark.parametrize("lens,H", [([100], 4), ([200, 154, 108, 62, 17], 4), ([700] * 14, 8), ([3000], 4), ([1900, 40, 1500], 2)])
@pytest.mark.parametrize("rate", [2.0 ** -3, 2.0 ** -5, 2.0 ** -8])
def test_states_of_bf16_prompts_are_as_exact_as_fp32_sums(kda, lens, H, rate):
    """A token's weight carries two exponentials (2^-22), three products and some roundings of its exponent (2^-24 each), the sums
    a few more: 2^-20 of the norm.  Decayed keys as two bf16 terms instead of three would be off by 2.1e-6 to 2.5e-6,
    more than twice as much, as one term by 1.6e-3."""
    T = sum(lens)
    q, k, v = (normal((T, H, 128), i) for i in range(3))
    g = torch.full((H,), -rate, device="cuda")
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    _, s = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32(cu))
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        assert rel(s[n], final_state(k[a:b], v[a:b], g.expand(T, H)[a:b])) < 2.0 ** -20, n


# ---- sequences that are cut: values that are not finite, slots that are refused ----------------


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("which", ["k", "v", "g"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens,at", [([3000], 300), ([3000], 2999), ([40, 2900, 60], 1500)])
def test_not_finite_in_a_sequence_that_is_cut(kda, dtype, which, value, lens, at):
    H, T = 2, sum(lens)
    q, k, v = (normal((T, H, 128), i, dtype) for i in range(3))
    g = -torch.rand((T, H), generator=torch.Generator("cuda").manual_seed(5), device="cuda") / 16
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    n = next(i for i in range(len(lens)) if cu[i] <= at < cu[i + 1])
    end = cu[n + 1]
    clean, sc = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32(cu))
    x = dict(k=k, v=v, g=g)[which]
    x[(at, 1) if which == "g" else (at, 1, 77)] = value
    o, s = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32(cu))
    # (fp32: eight tokens of which one has no finite decay go token by token instead of by their common reference, and round
    # otherwise: some products more or fewer, 2^-24 each, of |q| |k| |v|, which is ten times o)
    same = at - (at - cu[n]) % 8 if which == "g" and dtype is torch.float32 else at
    assert same == at or rel(o[same:at], clean[same:at].double()) < 2.0 ** -18
    assert torch.equal(o[:same], clean[:same]) and torch.equal(o[end:], clean[end:]) and torch.equal(o[:, 0], clean[:, 0])
    assert torch.equal(s[:, 0], sc[:, 0])
    for i in range(len(lens)):
        assert i == n or torch.equal(s[i], sc[i])
    if which == "v":
        other = torch.arange(128, device="cuda") != 77
        assert not o[at:end, 1, 77].isfinite().any() and not s[n, 1, 77].isfinite().any()
        assert torch.equal(o[:, 1, other], clean[:, 1, other]) and torch.equal(s[n, 1, other], sc[n, 1, other])
    else:
        assert not o[at:end, 1].isfinite().any()
        assert not (s[n, 1, :, 77] if which == "k" else s[n, 1]).isfinite().any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_long_sequence_without_a_slot(kda, dtype):
    """Long enough to be cut, refused, beside one that is cut and one that is not: alone they come to the same within the
    rounding of another cut (2^-18 of the state's norm, a rounding of bf16 of o's)."""
    H, lens = 1, [2100, 1700, 50]
    T, cu = sum(lens), [0, 2100, 3800, 3850]
    q, k, v = (normal((T, H, 128), i, dtype) for i in range(3))
    g = -torch.rand((T, H), generator=torch.Generator("cuda").manual_seed(5), device="cuda") / 16
    pool = normal((5, H, 128, 128), 9, torch.float32)
    start = pool.clone()
    for slot in (-1, 5):
        pool.copy_(start)
        o, _ = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32(cu), initial_state=pool, final_state=pool, state_indices=i32([slot, 3, 1]))
        assert o[:2100].isnan().all()
        for unused in (0, 2, 4):
            assert torch.equal(pool[unused], start[unused])
        for n, at in ((1, 3), (2, 1)):
            rows = slice(cu[n], cu[n + 1])
            one, s = kda.kda_linear_chunk_fwd(q[rows], k[rows], v[rows], g[rows], initial_state=start[at:at + 1])
            assert rel(pool[at], s[0].double()) < 2.0 ** -18
            assert rel(o[rows], one.double()) < (2.0 ** -7 if dtype is torch.bfloat16 else 2.0 ** -18)


def test_one_sequence_without_a_slot(kda):
    for dtype, T in ((torch.bfloat16, 3000), (torch.float32, 900), (torch.bfloat16, 30)):
        q, k, v = (normal((T, 2, 128), i, dtype) for i in range(3))
        pool = normal((3, 2, 128, 128), 9, torch.float32)
        start = pool.clone()
        o, _ = kda.kda_linear_chunk_fwd(q, k, v, torch.zeros(2, device="cuda"), initial_state=pool, final_state=pool, state_indices=i32([3]))
        assert o.isnan().all() and torch.equal(pool, start)


def test_one_sequence_that_ends_before_the_last_token(kda):
    """A padded batch of one sequence: cut or not by all tokens, computed as far as it goes, the rows behind it left."""
    for dtype, T, H in ((torch.bfloat16, 3000, 2), (torch.float32, 900, 2), (torch.float32, 200, 4)):
        q, k, v = (normal((T, H, 128), i, dtype) for i in range(3))
        g = torch.full((H,), -2.0 ** -6, device="cuda")
        for n in (0, 1, 64, 65, 130, T // 2, T - 1):
            o = torch.full((T, H, 128), 7.0, dtype=dtype, device="cuda")
            _, s = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32([0, n]), o=o)
            assert (o[n:] == 7.0).all()
            if n == 0:
                assert (s == 0).all()
                continue
            ref = final_state(k[:n], v[:n], g.expand(T, H)[:n])
            last = torch.einsum("hed,hd->he", ref, q[n - 1].double()) * 128 ** -0.5
            assert rel(s[0], ref) < 2.0 ** -20 and rel(o[n - 1], last) < (2.0 ** -7 if dtype is torch.bfloat16 else 2.0 ** -20)


# ---- a captured call whose offsets change, offsets that are out of order ----------------------


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", [(2000, 8), (2000, 90), (1100, 8), (600, 2)])
def test_a_captured_call_follows_its_offsets(kda, dtype, T, H):
    """What is launched follows from the tokens and heads; which sequences there are, from the offsets at replay."""
    q, k, v = (normal((T, n, 128), i, dtype) for i, n in enumerate((2, 2, H)))
    g = -torch.rand((T, H), generator=torch.Generator("cuda").manual_seed(5), device="cuda") / 8
    code = kda.KDA_BF16 if dtype is torch.bfloat16 else kda.KDA_F32
    offsets = [[0, 40, 300, 310, T], [0, 0, 0, T, T], [0, T - 1, T - 1, T, T], [0, 1, 2, 3, 4], [0, T // 4, T // 2, T - T // 4, T]]
    cu, o, s = i32(offsets[0]), torch.empty((T, H, 128), dtype=dtype, device="cuda"), torch.empty((4, H, 128, 128), device="cuda")
    ws = torch.empty(max(256, kda.kda_linear_chunk_workspace_bytes(T, 4, H, code)), dtype=torch.uint8, device="cuda")
    kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=cu, o=o, final_state=s, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=cu, o=o, final_state=s, workspace=ws)
    for new in offsets:
        cu.copy_(i32(new))
        o.fill_(7.0), s.fill_(7.0), ws.fill_(255)
        graph.replay()
        want, end = kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32(new))
        assert torch.equal(o[:new[-1]], want[:new[-1]]) and torch.equal(s, end) and (o[new[-1]:] == 7.0).all()
        for n, (a, b) in enumerate(zip(new, new[1:])):
            assert (s[n] == 0).all() if a == b else rel(s[n], final_state(k[a:b].repeat_interleave(H // 2, 1), v[a:b], g[a:b])) < 2.0 ** -20


@pytest.mark.parametrize("dtype", DTYPES)
def test_refused_sequences_of_many_heads(kda, dtype):
    """Listed though nothing is cut: a sequence without a slot, one that ends behind the last token, one that runs backwards."""
    H, T = 80, 1000
    q, k, v = (normal((T, n, 128), i, dtype) for i, n in enumerate((1, 1, H)))
    g = torch.full((H,), -2.0 ** -5, device="cuda")
    pool = normal((9, H, 128, 128), 3, torch.float32)
    start, cu, slots = pool.clone(), [0, 400, 530, 900, T + 5, T], [6, 9, 0, 2, 4]
    o = torch.full((T, H, 128), 7.0, dtype=dtype, device="cuda")
    kda.kda_linear_chunk_fwd(q, k, v, g, cu_seqlens=i32(cu), final_state=pool, state_indices=i32(slots), o=o)
    for n in (0, 2):
        a, b = cu[n], cu[n + 1]
        assert rel(pool[slots[n]], final_state(k[a:b].expand(-1, H, -1), v[a:b], g.expand(b - a, H))) < 2.0 ** -20
        assert o[a:b].isfinite().all() and not (o[a:b] == 7.0).all(-1).any()
    assert o[400:530].isnan().all() and (o[900:] == 7.0).all()
    for slot in (1, 2, 3, 4, 5, 7, 8):
        assert torch.equal(pool[slot], start[slot])
