"""What the binding of the linear-attention layer takes beside contiguous tensors, and what it refuses."""
import pytest
import torch

pytestmark = pytest.mark.gpu


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


def tokens(*lead, H=4):
    """q, k, v and decays as a slice of a wider fp32 projection."""
    q, k, v = (normal((*lead, H, 128), i) for i in range(3))
    return q, k, v, (-normal((*lead, 3 * H + 1), 3, torch.float32).abs())[..., H + 1: 2 * H + 1]


def test_decays_are_taken_from_a_wider_projection(kda):
    q, k, v, g = tokens(700)
    assert not g.is_contiguous()
    for x, y in zip(kda.kda_linear_chunk_fwd(q, k, v, g), kda.kda_linear_chunk_fwd(q, k, v, g.contiguous())):
        assert torch.equal(x, y)
    pools = [torch.zeros((12, 4, 128, 128), device="cuda") for _ in range(2)]
    for pool, d in zip(pools, (g[:12], g[:12].contiguous())):
        kda.kda_linear_step(q[:12], k[:12], v[:12], d, pool)
    assert torch.equal(*pools)
    for n, s in ((4, 3), (1, 6), (6, 1)):
        q, k, v, g = tokens(n, s)
        index = i32(list(range(n * s))).view(n, s)
        pools = [torch.zeros((n * s, 4, 128, 128), device="cuda") for _ in range(2)]
        for pool, d in zip(pools, (g, g.contiguous())):
            kda.kda_linear_multi_step(q, k, v, d, pool, index)
        assert torch.equal(*pools)


def test_one_row_of_decays_is_expanded(kda):
    q, k, v, g = tokens(300)
    row = g[:1].contiguous()
    one = kda.kda_linear_chunk_fwd(q, k, v, row.expand(300, 4))
    for x, y, z in zip(one, kda.kda_linear_chunk_fwd(q, k, v, row[0]), kda.kda_linear_chunk_fwd(q, k, v, row.repeat(300, 1))):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_decays_that_are_refused(kda):
    q, k, v, g = tokens(60)
    wide = normal((60, 9), 1, torch.float32)
    for bad, error, match in ((wide[:, ::2][:, :4], ValueError, "next to each other"), (g[:59], ValueError, "g shape"),
                              (normal((4, 60), 1, torch.float32).t(), ValueError, "next to each other"),
                              (normal((60, 9), 1, torch.bfloat16)[:, :4], TypeError, "g must be"),
                              (torch.as_strided(wide, (60, 4), (3, 1)), ValueError, "at least 4"),
                              (wide[:, :4].cpu(), ValueError, "CUDA")):
        with pytest.raises(error, match=match):
            kda.kda_linear_chunk_fwd(q, k, v, bad)
    q, k, v, g = tokens(4, 3)
    pool, index = torch.zeros((12, 4, 128, 128), device="cuda"), i32(list(range(12))).view(4, 3)
    for bad in (normal((4, 5, 4), 1, torch.float32)[:, :3], normal((4, 1, 4), 1, torch.float32).expand(4, 3, 4)):
        with pytest.raises(ValueError, match="one stride"):
            kda.kda_linear_multi_step(q, k, v, bad, pool, index)


def test_weights_without_the_norm_are_refused(kda):
    q, k, w = normal((5, 2, 128), 0), normal((5, 1, 128), 1), torch.ones(128, device="cuda")
    for weights in (dict(q_weight=w), dict(k_weight=w), dict(q_weight=w, k_weight=w)):
        with pytest.raises(ValueError, match="without the norm"):
            kda.kda_head_norm_rope(q, k, norm=False, **weights)
        kda.kda_head_norm_rope(q, k, **weights)
    a, b = kda.kda_head_norm_rope(q, k, norm=False)
    assert torch.equal(a, q) and torch.equal(b, k)
