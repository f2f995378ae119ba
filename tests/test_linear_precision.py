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
