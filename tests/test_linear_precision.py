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
