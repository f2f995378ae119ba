"""Workloads of the operators around the KDA core in a hybrid serving step.

A hybrid decoder interleaves KDA layers with latent-attention layers, whose
keys and values come from one 576-wide vector a token (a normalised latent of
512 and a shared positional key of 64), kept in a paged cache.  One step of a
server runs, for these layers, the five operators measured here:

  tables   block table, slot map, positions and offsets from request lengths
  norm     residual addition + RMS norm, output in the input type or in e4m3
  write    latent norm + scatter of the step's tokens into the paged cache
  decode   absorbed attention over the paged latent cache (1 to 4 new tokens)
  prefill  expanded causal attention over packed sequences, with cached prefixes

``run`` computes each in elementary torch operations (fp32), or, with ``own``
set, through the package's entry points.  Lengths are spread evenly between
their bounds and shuffled by the seed, so that a case's work is the same for
every seed.
"""
from __future__ import annotations

import math

import torch

own = False

LATENT, ROPE = 512, 64
ROW = LATENT + ROPE          # one token of the latent cache
NOPE, VDIM = 128, 128        # expanded key part and value, per head
QK = NOPE + ROPE
EPS = 1e-6
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-30           # smallest |y| maximum that a scale stands for
SCALE = QK ** -0.5


# ---- cases ------------------------------------------------------------------


def listed():
    return [
        # a small server's decode step: eight requests, one new token each
        dict(name="tables_step_8", op="tables", n=8, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=4000, page=64),
        # a batch of prompts entering the cache, some behind a cached prefix: the slot map of 1.1M tokens
        dict(name="tables_prompts_256", op="tables", n=256, new_lo=512, new_hi=8192, ctx_lo=0, ctx_hi=1000, page=64),
        # decode of a single request: the norm in front of every layer, where only latency counts
        dict(name="norm_token", op="norm", t=1, d=4096, dtype="bf16", quant="none"),
        # a prompt's residual stream, normalised straight into e4m3 with a scale per 128 channels
        dict(name="norm_4096_block", op="norm", t=4096, d=4096, dtype="bf16", quant="block"),
        # fp32 residual stream of an odd batch, one e4m3 scale a row
        dict(name="norm_777_fp32_row", op="norm", t=777, d=2304, dtype="fp32", quant="row"),
        # the cache write of a decode step of 256 requests
        dict(name="write_256", op="write", t=256, page=64),
        # the cache write of a prefill step
        dict(name="write_16384", op="write", t=16384, page=64),
        # a few interactive requests verifying four speculative tokens each: latency
        dict(name="decode_verify_4x4", op="decode", n=4, s=4, h=32, lo=60, hi=700, page=64),
        # the decode batch: 256 ragged requests of 32 heads
        dict(name="decode_256", op="decode", n=256, s=1, h=32, lo=512, hi=4096, page=64),
        # one long document: the cache split over the whole GPU
        dict(name="decode_131k", op="decode", n=1, s=1, h=32, lo=131072, hi=131072, page=64),
        # one prompt of 4096 tokens and 32 heads
        dict(name="prefill_4k", op="prefill", n=1, h=32, q_lo=4096, q_hi=4096, p_lo=0, p_hi=0),
        # eight packed prompts behind cached prefixes of up to 2048 tokens
        dict(name="prefill_packed_8", op="prefill", n=8, h=32, q_lo=512, q_hi=2048, p_lo=0, p_hi=2048),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "norm", "write", "decode", "prefill"])
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        n = _log(rng, 1, 1024)
        new_hi = _log(rng, 1, max(1, min(8192, 1100000 // n)))
        ctx_hi = _log(rng, 1, 131072 if n <= 64 else 4096)
        return dict(op=op, n=n, new_lo=rng.randint(1, new_hi), new_hi=new_hi, ctx_lo=rng.randint(0, ctx_hi),
                    ctx_hi=ctx_hi, page=page)
    if op == "norm":
        quant, dtype = rng.choice(["none", "row", "block"]), rng.choice(["bf16", "fp32"])
        d = 128 * rng.randint(1, 64) if quant == "block" else 8 * rng.randint(8, 1024)
        most = 4096 * 4096 // (2 if dtype == "fp32" else 1)
        return dict(op=op, t=_log(rng, 1, max(1, min(65536, most // d))), d=d, dtype=dtype, quant=quant)
    if op == "write":
        return dict(op=op, t=_log(rng, 1, 16384), page=page)
    if op == "decode":
        n, s, h = _log(rng, 1, 256), rng.randint(1, 4), rng.choice([1, 2, 5, 8, 16, 32, 64])
        most = min(256 * 4096, 256 * 4096 * 32 // (s * h)) // n
        hi = _log(rng, s, max(s, min(131072, most)))
        return dict(op=op, n=n, s=s, h=h, lo=rng.randint(s, hi), hi=hi, page=page)
    n, h = _log(rng, 1, 8), rng.choice([1, 2, 5, 8, 16, 32])
    q_hi = _log(rng, 1, 2048)
    p_hi = rng.choice([0, _log(rng, 1, 2048)])
    return dict(op=op, n=n, h=h, q_lo=rng.randint(1, q_hi), q_hi=q_hi, p_lo=0, p_hi=p_hi)


def _spread(n, lo, hi):
    """n lengths spread evenly over [lo, hi]."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _pages(length, page):
    return -(-length // page)


def _prefill_lengths(case):
    q = _spread(case["n"], case["q_lo"], case["q_hi"])
    p = _spread(case["n"], case["p_lo"], case["p_hi"])
    k = case["n"] // 2
    return q, p[k:] + p[:k]


def _tables_lengths(case):
    new = _spread(case["n"], case["new_lo"], case["new_hi"])
    ctx = _spread(case["n"], case["ctx_lo"], case["ctx_hi"])
    k = case["n"] // 2
    return new, ctx[k:] + ctx[:k]


# ---- inputs -----------------------------------------------------------------


def _shuffled(gen, *lists):
    order = torch.randperm(len(lists[0]), generator=gen).tolist()
    return [[v[i] for i in order] for v in lists]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lengths):
    return _i32([0] + torch.tensor(lengths).cumsum(0).tolist())


def prepare(case, seed):
    host = torch.Generator().manual_seed(int(seed))
    dev = torch.Generator(device="cuda").manual_seed(int(seed))
    return dict(_PREPARE[case["op"]](case, host, dev), op=case["op"], case=dict(case))


def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _prepare_tables(case, host, dev):
    page, n = case["page"], case["n"]
    new, ctx = _shuffled(host, *_tables_lengths(case))
    max_pages = _pages(case["new_hi"] + case["ctx_hi"], page)
    held = [_pages(c, page) for c in ctx]
    need = [_pages(c + t, page) - h for c, t, h in zip(ctx, new, held)]
    n_pages = sum(held) + sum(need) + 32
    pages = torch.randperm(n_pages, generator=host).to(torch.int32)
    lens = torch.tensor(held)
    mask = torch.arange(max_pages)[None, :] < lens[:, None]
    table = torch.full((n, max_pages), -1, dtype=torch.int32)
    table[mask] = pages[: sum(held)]
    max_tokens = -(-sum(new) // 8) * 8          # the batch's token buffers, padded
    return dict(ctx=_i32(ctx), new=_i32(new), free=pages[sum(held):].cuda(), table=table.cuda(), page=page,
                n_pages=n_pages, max_tokens=max_tokens, cu=_i32([0] * (n + 1)), lens=_i32([0] * n),
                slots=_i32([0] * max_tokens), pos=_i32([0] * max_tokens), status=_i32([0, 0]))


def _prepare_norm(case, host, dev):
    t, d = case["t"], case["d"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    s = dict(x=_normal((t, d), dev, dtype), residual=_normal((t, d), dev, dtype) * 4,
             weight=torch.rand((d,), generator=dev, device="cuda") + 0.5, quant=case["quant"])
    s["residual_out"] = torch.empty_like(s["x"])
    groups = {"none": 0, "row": 1, "block": d // 128}[case["quant"]]
    s["y"] = torch.empty((t, d), dtype=torch.float8_e4m3fn if groups else dtype, device="cuda")
    s["scales"] = torch.empty((t, groups), dtype=torch.float32, device="cuda") if groups else None
    return s


def _prepare_write(case, host, dev):
    t, page = case["t"], case["page"]
    n_pages = _pages(2 * t, page)
    slots = torch.randperm(n_pages * page, generator=host)[:t].to(torch.int32)
    slots[torch.randperm(t, generator=host)[: t // 64]] = -1      # padding tokens of the batch
    fused = _normal((t, 2048 + ROW), dev)                         # the layer's fused down-projection
    return dict(kv=fused[:, 2048:], weight=torch.rand((LATENT,), generator=dev, device="cuda") + 0.5,
                cache=_normal((n_pages, page, ROW), dev), slots=slots.cuda())


def _prepare_decode(case, host, dev):
    n, s, h, page = case["n"], case["s"], case["h"], case["page"]
    (lens,) = _shuffled(host, _spread(n, case["lo"], case["hi"]))
    held = torch.tensor([_pages(v, page) for v in lens])
    max_pages = int(held.max())
    n_pages = int(held.sum()) + 1
    table = torch.full((n, max_pages), -1, dtype=torch.int32)
    table[torch.arange(max_pages)[None, :] < held[:, None]] = \
        torch.randperm(n_pages, generator=host)[: n_pages - 1].to(torch.int32)
    state = dict(q=_normal((n, s, h, ROW), dev), cache=_normal((n_pages, page, ROW), dev), table=table.cuda(),
                 lens=_i32(lens), longest=max(lens), o=torch.empty((n, s, h, LATENT), dtype=torch.bfloat16, device="cuda"))
    if own:
        import kimi_delta_attention_07_gb300 as kda
        state["workspace"] = torch.empty(kda.kda_latent_decode_workspace_bytes(n, s, h), dtype=torch.uint8, device="cuda")
    return state


def _prepare_prefill(case, host, dev):
    h = case["h"]
    q_lens, p_lens = _shuffled(host, *_prefill_lengths(case))
    k_lens = [a + b for a, b in zip(q_lens, p_lens)]
    tq, tk = sum(q_lens), sum(k_lens)
    return dict(q=_normal((tq, h, QK), dev), kv=_normal((tk, h, NOPE + VDIM), dev), k_rope=_normal((tk, ROPE), dev),
                cu_q=_cu(q_lens), cu_k=_cu(k_lens), longest_q=max(q_lens), longest_k=max(k_lens),
                o=torch.empty((tq, h, VDIM), dtype=torch.bfloat16, device="cuda"))


_PREPARE = dict(tables=_prepare_tables, norm=_prepare_norm, write=_prepare_write, decode=_prepare_decode,
                prefill=_prepare_prefill)


# ---- one pass ---------------------------------------------------------------


def run(state):
    return (_run_own if own else _PLAIN[state["op"]])(state)


def _run_own(s):
    import kimi_delta_attention_07_gb300 as kda
    op = s["op"]
    if op == "tables":
        kda.kda_page_tables(s["ctx"], s["new"], s["free"], s["table"], page_size=s["page"], n_pages=s["n_pages"],
                            max_tokens=s["max_tokens"], cu_seqlens=s["cu"], seq_lens=s["lens"], slots=s["slots"],
                            positions=s["pos"], status=s["status"])
        return s["table"], s["cu"], s["lens"], s["slots"], s["pos"], s["status"]
    if op == "norm":
        return kda.kda_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quant=s["quant"],
                                residual_out=s["residual_out"], y=s["y"], scales=s["scales"])
    if op == "write":
        return kda.kda_latent_cache_write(s["kv"], s["weight"], s["cache"], s["slots"], eps=EPS)
    if op == "decode":
        return kda.kda_latent_decode(s["q"], s["cache"], s["table"], s["lens"], scale=SCALE, o=s["o"],
                                     workspace=s["workspace"])
    return kda.kda_latent_prefill(s["q"], s["kv"], s["k_rope"], cu_seqlens_q=s["cu_q"], cu_seqlens_k=s["cu_k"],
                                  scale=SCALE, o=s["o"])


def _plain_tables(s):
    ctx, new, free, table, page = s["ctx"].long(), s["new"].long(), s["free"], s["table"], s["page"]
    n, max_pages = table.shape
    held = (ctx + page - 1) // page
    total = (ctx + new + page - 1) // page
    fits = (ctx >= 0) & (new >= 0) & (total <= max_pages)
    need = torch.where(fits, total - held, 0)
    end = need.cumsum(0)
    fits &= (need == 0) | (end <= free.numel())
    taken = torch.where(fits, end, 0).amax()
    cols = torch.arange(max_pages, device=table.device)[None, :]
    fresh = fits[:, None] & (cols >= held[:, None]) & (cols < total[:, None])
    at = ((end - need - held)[:, None] + cols).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[at], table))
    cu = torch.cat([end.new_zeros(1), new.clamp(min=0).cumsum(0)])
    t = torch.arange(s["max_tokens"], device=table.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    real = (r < n)
    r = r.clamp(max=n - 1)
    pos = ctx[r] + t - cu[r]
    real = real & fits[r]
    entry = table[r, (pos // page).clamp(0, max_pages - 1)].long()
    real = real & (entry >= 0) & (entry < s["n_pages"])
    slots = torch.where(real, entry * page + pos % page, -1)
    pos = torch.where(real, pos, -1)
    lens = torch.where(fits, ctx + new, ctx.clamp(min=0))
    status = torch.stack([taken, (~fits).sum()])
    return (table,) + tuple(v.to(torch.int32) for v in (cu, lens, slots, pos, status))


def _plain_norm(s):
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"]
    residual = h.to(s["x"].dtype)
    if s["quant"] == "none":
        return y.to(s["x"].dtype), residual, None
    t, d = y.shape
    g = y.view(t, 1 if s["quant"] == "row" else d // 128, -1)
    scales = g.abs().amax(-1).clamp(min=AMAX_FLOOR) / E4M3_MAX
    q = (g / scales[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(t, d), residual, scales


def _plain_write(s):
    rows = s["cache"].view(-1, ROW)
    kept = (s["slots"] >= 0) & (s["slots"] < rows.shape[0])
    x = s["kv"].float()
    c = x[:, :LATENT]
    c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["weight"]
    x = torch.cat([c, x[:, LATENT:]], -1).to(torch.bfloat16)
    rows[s["slots"][kept].long()] = x[kept]
    return s["cache"]


def _softmax_times(scores, seen, v):
    """softmax over the seen entries of the last axis, times v; rows that see nothing are zero."""
    scores = scores.masked_fill_(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, 1.0)


def _plain_decode(s):
    n, steps, h, _ = s["q"].shape
    page = s["cache"].shape[1]
    at = torch.arange(s["longest"], device="cuda")
    table = s["table"].long()
    rows = table[:, at // page] * page + at % page                       # [n, longest]
    held = at[None, :] < s["lens"][:, None]
    k = s["cache"].view(-1, ROW)[torch.where(held, rows, 0)].float()     # [n, longest, ROW]
    k = k.masked_fill_(~held[..., None], 0.0)
    scores = torch.matmul(s["q"].float().view(n, steps * h, ROW), k.transpose(1, 2)) * SCALE
    last = s["lens"][:, None] - steps + torch.arange(steps, device="cuda")  # newest position a row sees
    seen = at[None, None, :] <= last[:, :, None].expand(n, steps, 1)
    seen = seen[:, :, None, :].expand(n, steps, h, at.numel()).reshape(n, steps * h, -1)
    return _softmax_times(scores, seen, k[..., :LATENT]).view(n, steps, h, LATENT).to(torch.bfloat16)


def _padded(x, cu, longest):
    """[T, ...] packed by cu to [N, longest, ...] (rows past a sequence's end: any) and which rows are real."""
    at = cu[:-1, None].long() + torch.arange(longest, device=x.device)
    real = at < cu[1:, None]
    return x[at.clamp(max=x.shape[0] - 1)], real


def _plain_prefill(s):
    h = s["q"].shape[1]
    q, _ = _padded(s["q"].float(), s["cu_q"], s["longest_q"])
    kv, real = _padded(s["kv"].float(), s["cu_k"], s["longest_k"])
    rope, _ = _padded(s["k_rope"].float(), s["cu_k"], s["longest_k"])
    k = torch.cat([kv[..., :NOPE], rope[:, :, None, :].expand(-1, -1, h, -1)], -1)
    scores = torch.matmul(q.transpose(1, 2), k.permute(0, 2, 3, 1)).mul_(SCALE)      # [N, h, lq, lk]
    lens_q, lens_k = s["cu_q"].diff(), s["cu_k"].diff()
    i = torch.arange(s["longest_q"], device="cuda")
    j = torch.arange(s["longest_k"], device="cuda")
    seen = real[:, None, :] & (j[None, None, :] <= i[None, :, None] + (lens_k - lens_q)[:, None, None])
    o = _softmax_times(scores, seen[:, None], kv[..., NOPE:].transpose(1, 2)).transpose(1, 2)
    t = torch.arange(s["q"].shape[0], device="cuda")
    n = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    return o[n, t - s["cu_q"][n]].to(torch.bfloat16)


_PLAIN = dict(tables=_plain_tables, norm=_plain_norm, write=_plain_write, decode=_plain_decode, prefill=_plain_prefill)


# ---- what a pass cannot do without --------------------------------------------


def work(case):
    op = case["op"]
    if op == "tables":
        new, ctx = _tables_lengths(case)
        fresh = sum(_pages(a + b, case["page"]) - _pages(b, case["page"]) for a, b in zip(new, ctx))
        n, t = case["n"], sum(new)
        # lengths in; offsets and lengths out; a free page in and a table entry out; a slot and a position a token;
        # the table entry of each partly filled page
        return {"bytes": 8 * n + 8 * n + 8 * fresh + 8 * t + 4 * n, "flops": 0}
    if op == "norm":
        e = 2 if case["dtype"] == "bf16" else 4
        t, d = case["t"], case["d"]
        groups = {"none": 0, "row": 1, "block": d // 128}[case["quant"]]
        return {"bytes": t * d * (3 * e + (1 if groups else e)) + 4 * t * groups + 4 * d, "flops": 6 * t * d}
    if op == "write":
        return {"bytes": case["t"] * (2 * 2 * ROW + 4) + 4 * LATENT, "flops": 4 * LATENT * case["t"]}
    if op == "decode":
        tokens = sum(_spread(case["n"], case["lo"], case["hi"]))
        rows = case["s"] * case["h"]
        return {"bytes": tokens * ROW * 2 + case["n"] * rows * (ROW + LATENT) * 2 + 4 * tokens // case["page"],
                "flops": 2 * tokens * rows * (ROW + LATENT)}
    q, p = _prefill_lengths(case)
    h, tq, tk = case["h"], sum(q), sum(q) + sum(p)
    pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(q, p))
    return {"bytes": 2 * (tq * h * (QK + VDIM) + tk * (h * (NOPE + VDIM) + ROPE)),
            "flops": 2 * pairs * h * (QK + VDIM)}


# ---- the definitions, in 64 bits ----------------------------------------------


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "tables":
        return None
    if op == "norm":
        h = s["x"].double() + s["residual"].double()
        rms = (h.pow(2).sum(-1, keepdim=True) / h.shape[-1] + EPS).sqrt()
        y = h / rms * s["weight"].double()
        if s["quant"] == "none":
            return y, h, None
        t, d = y.shape
        width = d if s["quant"] == "row" else 128
        g = y.reshape(t, d // width, width)
        scales = g.abs().max(-1).values / E4M3_MAX
        return (g / scales.unsqueeze(-1)).reshape(t, d), h, scales
    if op == "write":
        cache = s["cache"].double()
        c = s["kv"][:, :LATENT].double()
        c = c / (c.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["weight"].double()
        keep = s["slots"] >= 0
        at = s["slots"][keep].long()
        page = cache.shape[1]
        cache[at // page, at % page, :LATENT] = c[keep]
        cache[at // page, at % page, LATENT:] = s["kv"][keep][:, LATENT:].double()
        return cache
    if op == "decode":
        n, steps, h, _ = s["q"].shape
        page = s["cache"].shape[1]
        o = torch.zeros((n, steps, h, LATENT), dtype=torch.float64, device="cuda")
        for b, length in enumerate(s["lens"].tolist()):
            pages = s["table"][b, : _pages(length, page)].long()
            k = s["cache"][pages].reshape(-1, ROW)[:length].double()
            for i in range(max(0, steps - length), steps):
                visible = length - steps + 1 + i
                w = torch.softmax(s["q"][b, i].double() @ k[:visible].T * SCALE, -1)
                o[b, i] = w @ k[:visible, :LATENT]
        return o
    h = s["q"].shape[1]
    o = torch.zeros((s["q"].shape[0], h, VDIM), dtype=torch.float64, device="cuda")
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(len(cu_q) - 1):
        q = s["q"][cu_q[b]:cu_q[b + 1]].double()
        kv = s["kv"][cu_k[b]:cu_k[b + 1]].double()
        rope = s["k_rope"][cu_k[b]:cu_k[b + 1]].double()
        nq, nk = q.shape[0], kv.shape[0]
        hidden = torch.ones((nq, nk), dtype=torch.bool, device="cuda").triu(nk - nq + 1)
        for head in range(h):
            x = q[:, head, :NOPE] @ kv[:, head, :NOPE].T + q[:, head, NOPE:] @ rope.T
            w = torch.softmax((x * SCALE).masked_fill(hidden, float("-inf")), -1)
            o[cu_q[b]:cu_q[b + 1], head] = w @ kv[:, head, NOPE:]
    return o
