"""The rotation in front of the latent layer: positions from the page tables, queries and key rotated in place in
their projection, the key into the cache, then prompts and one token a request, against 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

H, HEAD, ROPE, LATENT = 4, 128, 64, 512


def normal(shape, seed, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def turned(x, positions, freq):
    """Adjacent pairs of x [T, heads, 64] by their position, in 64 bits."""
    t = (positions.double()[:, None] * freq.double())[:, None]
    z = torch.view_as_complex(x.double().unflatten(-1, (-1, 2)).contiguous()) * torch.polar(torch.ones_like(t), t)
    return torch.view_as_real(z).flatten(-2)


def attend(scores, values):
    return torch.einsum("hqk,khd->qhd", torch.softmax(scores, -1), values)


def test_rotated_queries_and_keys_through_the_latent_layer():
    import kimi_delta_attention_07_gb300 as kda
    kda.load()
    lens, N, far = [70, 1, 200], 3, 5  # and a request's `far` tokens more, one at a time
    freq = (10000.0 ** (-torch.arange(32) / 32)).cuda()
    width = H * (HEAD + ROPE)
    cache = torch.zeros((12, 64, LATENT + ROPE), dtype=torch.bfloat16, device="cuda")
    table, free = torch.full((N, 6), -1, dtype=torch.int32, device="cuda"), torch.arange(12, dtype=torch.int32, device="cuda")
    norm, start, ctx = torch.ones(LATENT, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), i32([0] * N)
    keys = [torch.empty((0, 1, ROPE), dtype=torch.float64, device="cuda")] * N  # of each request, rotated in 64 bits

    def step(new, pad, seed):
        """Projection (rotated), q in 64 bits, slots, offsets of a step of `new` tokens and `pad` rows of padding."""
        nonlocal start, ctx
        T = sum(new) + pad
        cu, ctx, slots, positions, status = kda.kda_page_tables(ctx, i32(new), free, table, page_size=64, n_pages=12,
                                                                max_tokens=T, free_start=start)
        start = status[:1].clone()
        fused = normal((T, width + LATENT + ROPE), seed)
        q, k = fused[:, :width].unflatten(1, (H, HEAD + ROPE)), fused[:, width + LATENT:].unflatten(1, (1, ROPE))
        real = torch.cat([torch.arange(p, p + n) for p, n in zip((ctx - i32(new)).tolist(), new)]).cuda()
        assert torch.equal(positions[:sum(new)].long(), real) and (positions[sum(new):] < 0).all()
        exact = q[:sum(new)].double()
        exact = torch.cat([exact[..., :HEAD], turned(exact[..., HEAD:], real, freq)], -1)
        for n, x in enumerate(turned(k[:sum(new)], real, freq).split(new)):
            keys[n] = torch.cat([keys[n], x])
        before = fused.clone()
        for x, offset in ((q, HEAD), (k, 0)):
            kda.kda_head_norm_rope(x, positions=positions, inv_freq=freq, rot_offset=offset, interleaved=True, norm=False, q_out=x)
        assert torch.equal(fused[sum(new):], before[sum(new):]) and torch.equal(fused[:, width: width + LATENT], before[:, width: width + LATENT])
        kda.kda_latent_cache_write(fused[:, width:], norm, cache, slots)
        return q, exact, cu, k

    # Rotated rows are rounded once (2^-8 / sqrt 3 in the root mean square), which moves a score by some 2^-9; p and o are
    # rounded likewise: some 2^-8 of o's norm in all.  Rows that were not rotated, or by another position, are off by 1 and more.
    q, exact, cu, k = step(lens, 3, 0)
    kv = normal((sum(lens) + 3, H, 2 * HEAD), 9)
    o = kda.kda_latent_prefill(q, kv, k[:, 0], cu_seqlens_q=cu)
    at = 0
    for n, length in enumerate(lens):
        rows = slice(at, at + length)
        key = torch.cat([kv[rows, :, :HEAD].double(), keys[n].expand(-1, H, -1)], -1)
        scores = torch.einsum("qhd,khd->hqk", exact[rows], key) * (HEAD + ROPE) ** -0.5
        scores = scores.masked_fill(torch.ones(length, length, device="cuda").triu(1).bool(), float("-inf"))
        ref = attend(scores, kv[rows, :, HEAD:].double())
        assert float((o[rows].double() - ref).norm() / ref.norm()) < 2.0 ** -6
        at += length
    for s in range(far):
        q, exact, _, _ = step([1] * N, 0, 10 + s)
        absorbed = normal((N, H, LATENT), 100 + s, 0.3)
        o = kda.kda_latent_decode(torch.cat([absorbed, q[..., HEAD:]], -1), cache, table, ctx, scale=(HEAD + ROPE) ** -0.5)
        for n, length in enumerate(ctx.tolist()):
            rows = cache[table[n, : -(-length // 64)].long()].flatten(0, 1)[:length, :LATENT].double()
            scores = torch.einsum("hd,kd->hk", absorbed[n].double(), rows) + torch.einsum("hd,kd->hk", exact[n, :, HEAD:], keys[n][:, 0])
            ref = torch.softmax(scores * (HEAD + ROPE) ** -0.5, -1) @ rows
            assert float((o[n].double() - ref).norm() / ref.norm()) < 2.0 ** -6, (s, n)
