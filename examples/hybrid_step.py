#!/usr/bin/env python3
"""A server's steps through a small hybrid decoder: a KDA layer and a latent
attention layer, prompts first, then one token a request.

The operators are the package's own; the projections between them are plain
matrix products on random weights.  One page table serves the latent cache,
one slot per request the KDA state pool:

  kda_page_tables          lengths -> new table rows, slots, positions, offsets
  kda_rms_norm             residual + norm in front of each layer
  kda_chunk_fwd_gated      KDA layer, prompts (final states into the pool)
  kda_recurrent_step_gated KDA layer, one token, in place on the pool
  kda_head_norm_rope       latent layer: queries' and key's positional channels
                           turn by the token's position
  kda_latent_cache_write   normed latent and key into the pages
  kda_latent_prefill       prompts, expanded keys and values
  kda_latent_decode        one token, on the cached vectors themselves

The final norm is taken in e4m3 with a scale per 128 channels, as an 8-bit
output head would read it.

  python examples/hybrid_step.py     # checks steps against one longer prompt
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kimi_delta_attention_07_gb300 as kda  # noqa: E402

LATENT, ROPE, HEAD = 512, 64, 128


class HybridDecoder:
    def __init__(self, hidden=512, heads=4, requests=8, n_pages=64, page_size=64, max_pages=16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=gen, device="cuda") * shape[-2] ** -0.5).to(torch.bfloat16)

        self.heads, self.page_size, self.n_pages = heads, page_size, n_pages
        self.norms = [torch.ones(hidden, device="cuda") for _ in range(3)]
        # KDA layer: q, k, v, gate, beta; output
        self.kda_in = weight(hidden, 4 * heads * HEAD + heads)
        self.a_log = torch.zeros(heads, device="cuda")
        self.dt_bias = torch.zeros((heads, HEAD), device="cuda")
        self.kda_out = weight(heads * HEAD, hidden)
        # latent layer: queries, latent and positional key in one projection; up-projection; output
        self.q_width = heads * (HEAD + ROPE)
        self.latent_in = weight(hidden, self.q_width + LATENT + ROPE)
        self.inv_freq = 10000.0 ** (-torch.arange(ROPE // 2, device="cuda") / (ROPE // 2))
        self.latent_norm = torch.ones(LATENT, device="cuda")
        self.up = weight(heads, LATENT, 2 * HEAD)     # a head's key part and value
        self.latent_out = weight(heads * HEAD, hidden)
        # what lives between steps
        self.states = torch.zeros((requests, heads, HEAD, HEAD), device="cuda")
        self.cache = torch.empty((n_pages, page_size, LATENT + ROPE), dtype=torch.bfloat16, device="cuda")
        self.table = torch.full((requests, max_pages), -1, dtype=torch.int32, device="cuda")
        self.free_pages = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        self.free_start = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.slots = torch.arange(requests, dtype=torch.int32, device="cuda")
        self.begun = False

    def step(self, x, new_lens, prompts):
        """x [T, hidden]: the packed new tokens' embeddings (one a request when
        `prompts` is false); new_lens int32 [N].  Prompts come first: they begin at
        position 0 and from zero states.  Raises, and changes nothing that a later
        step reads, if a request is refused (out of pages or of its table's row).
        Returns the normed output as e4m3 values and scales, and those values in
        fp32."""
        T, H = x.shape[0], self.heads
        if prompts and self.begun:
            raise ValueError("a prompt needs requests without cached tokens")
        if not prompts and T != self.lens.numel():
            raise ValueError("a decode step takes one token a request")
        cu, lens, slots, positions, status = kda.kda_page_tables(
            self.lens, new_lens, self.free_pages, self.table, page_size=self.page_size, n_pages=self.n_pages,
            max_tokens=T, free_start=self.free_start)
        # A refused request's tokens have slot -1 and its length stays.  (A server that counts its pages on the host
        # does not wait for the device here.)
        if int(status[1]):
            raise RuntimeError(f"{int(status[1])} requests refused: more pages are needed than are free or fit a row")
        self.free_start, self.begun = status[:1].clone(), True
        # KDA layer
        y, _, _ = kda.kda_rms_norm(x, self.norms[0])
        q, k, v, gate, beta = (y @ self.kda_in).split([H * HEAD] * 4 + [H], -1)
        q, k, v, gate = (t.reshape(T, H, HEAD).contiguous() for t in (q, k, v, gate))
        beta = beta.contiguous()
        if prompts:
            o, _ = kda.kda_chunk_fwd_gated(q, k, v, gate, beta, self.a_log, self.dt_bias, cu_seqlens=cu,
                                           final_state=self.states, state_indices=self.slots)
        else:
            o = kda.kda_recurrent_step_gated(q, k, v, gate, beta, self.a_log, self.dt_bias, self.states,
                                             state_indices=self.slots)
        # latent layer
        y, x, _ = kda.kda_rms_norm(o.view(T, -1) @ self.kda_out, self.norms[1], residual=x)
        fused = y @ self.latent_in
        q = fused[:, :self.q_width].unflatten(1, (H, HEAD + ROPE))
        k_rope = fused[:, self.q_width + LATENT:].unflatten(1, (1, ROPE))
        for t, offset in ((q, HEAD), (k_rope, 0)):  # in place, in the projection
            kda.kda_head_norm_rope(t, positions=positions, inv_freq=self.inv_freq, rot_offset=offset, interleaved=True,
                                   norm=False, q_out=t)
        kda.kda_latent_cache_write(fused[:, self.q_width:], self.latent_norm, self.cache, slots)
        if prompts:
            rows = self.cache.view(-1, LATENT + ROPE)[slots.long()]
            kv = torch.einsum("tc,hcd->thd", rows[:, :LATENT], self.up).contiguous()
            o = kda.kda_latent_prefill(q, kv, rows[:, LATENT:], cu_seqlens_q=cu)
        else:
            absorbed = torch.einsum("thd,hcd->thc", q[..., :HEAD], self.up[..., :HEAD])
            o = kda.kda_latent_decode(torch.cat([absorbed, q[..., HEAD:]], -1), self.cache, self.table, lens)
            o = torch.einsum("thc,hcd->thd", o, self.up[..., HEAD:])
        self.lens = lens
        y, _, scales = kda.kda_rms_norm(o.reshape(T, -1) @ self.latent_out, self.norms[2], residual=x, quant="block")
        return y, scales, (y.float().unflatten(-1, (-1, 128)) * scales[..., None]).flatten(-2)


def main(lengths=(70, 1, 129, 300), steps=3):
    """The outputs of `steps` decode steps behind prompts, against the last rows
    of one prompt call over the same tokens.  Returns the largest relative
    difference of a request's rows."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    n, hidden = len(lengths), 512
    tokens = [torch.randn((length + steps, hidden), generator=gen, device="cuda").to(torch.bfloat16) for length in lengths]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    whole = HybridDecoder(requests=n)
    _, _, ref = whole.step(torch.cat(tokens), i32([length + steps for length in lengths]), True)
    ends = torch.tensor(lengths).add(steps).cumsum(0).tolist()

    model = HybridDecoder(requests=n)
    model.step(torch.cat([t[:length] for t, length in zip(tokens, lengths)]), i32(lengths), True)
    worst = 0.0
    for s in range(steps):
        _, _, out = model.step(torch.stack([t[length + s] for t, length in zip(tokens, lengths)]), i32([1] * n), False)
        for b in range(n):
            want = ref[ends[b] - steps + s]
            worst = max(worst, float((out[b] - want).norm() / want.norm()))
    return worst


if __name__ == "__main__":
    print(f"decode steps against one longer prompt: largest relative difference {main():.2e}")
