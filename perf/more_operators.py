"""Workloads of a linear-attention layer with one decay a head, and of the head
norms and rotations in front of it.

The layer's state is S [V, K] in fp32 per (sequence, head), K = V = 128:

    S <- exp(g_t) S + v_t k_t^T        o_t = scale * S q_t

with g a number a head (a fixed slope) or a number a token and head, and q, k
shared by H / Hk heads.  A hybrid decoder runs it as

  rope    RMS norm of each head of q and k and the rotation by the token's
          position (one axis, or time, height and width), in one pass
  chunk   the prompts' tokens, packed, states into the pool's slots
  step    one new token a request, or S tokens of a speculative verify whose
          states each go to a slot of their own

``run`` computes each in elementary torch operations (fp32, angles and sums of
decays in fp64), or, with ``own`` set, through the package's entry points.
Lengths are spread evenly between their bounds and shuffled by the seed, so that
a case's work is the same for every seed.
"""
from __future__ import annotations

import math

import torch

own = False

DIM = 128                    # key and value width of the linear layer
EPS = 1e-6
SCALE = DIM ** -0.5
BASE = 10000.0               # of the rotation's frequencies
C = 128                      # chunk of the plain form


# ---- cases ------------------------------------------------------------------


def listed():
    return [
        # decode of a single request: norm and rotation of one token's heads, latency only
        dict(name="rope_token", op="rope", t=1, hq=32, hk=8, d=128, rot=64, offset=0, pairs="half", norm=True,
             axes=1, far=131072, pad=0, dtype="bf16"),
        # a prompt's queries and keys in front of the linear layer, some padding at the batch's end
        dict(name="rope_4096", op="rope", t=4096, hq=32, hk=32, d=128, rot=128, offset=0, pairs="half", norm=True,
             axes=1, far=131072, pad=37, dtype="bf16"),
        # tokens of a video: time, height and width; every channel rotated
        dict(name="rope_video_10000", op="rope", t=10000, hq=16, hk=4, d=128, rot=128, offset=0, pairs="half",
             norm=True, axes=3, far=4096, pad=0, dtype="bf16"),
        # the latent layer's queries: no norm, the 64 positional channels behind 128 others, adjacent pairs, fp32
        dict(name="rope_latent_777", op="rope", t=777, hq=32, hk=0, d=192, rot=64, offset=128, pairs="adjacent",
             norm=False, axes=1, far=131072, pad=0, dtype="fp32"),
        # a few interactive requests, one token each: latency
        dict(name="step_4x8", op="step", n=4, s=1, h=8, hk=8, decay="head", dtype="bf16"),
        # the decode batch
        dict(name="step_256x32", op="step", n=256, s=1, h=32, hk=32, decay="token", dtype="bf16"),
        # speculative verify of four tokens, shared keys
        dict(name="step_verify_64x4", op="step", n=64, s=4, h=32, hk=8, decay="head", dtype="bf16"),
        # a few short prompts
        dict(name="chunk_short_5", op="chunk", n=5, lo=17, hi=200, h=8, hk=8, decay="head", carry=False, dtype="bf16"),
        # one prompt of 4096 tokens and 32 heads
        dict(name="chunk_4k", op="chunk", n=1, lo=4096, hi=4096, h=32, hk=32, decay="token", carry=False, dtype="bf16"),
        # packed prompts behind carried states, ragged, shared keys
        dict(name="chunk_packed_8", op="chunk", n=8, lo=333, hi=4001, h=32, hk=8, decay="head", carry=True, dtype="bf16"),
        # one long document
        dict(name="chunk_131k", op="chunk", n=1, lo=131072, hi=131072, h=8, hk=8, decay="token", carry=False,
             dtype="bf16"),
        # two prompts in fp32
        dict(name="chunk_fp32_2", op="chunk", n=2, lo=500, hi=1001, h=16, hk=16, decay="token", carry=True, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "step", "chunk", "chunk"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "rope":
        d = rng.choice([64, 128, 192, 256])
        rot = rng.choice([r for r in (32, 64, 96, 128, 192, 256) if r <= d])
        hq, hk = rng.choice([1, 4, 7, 16, 32, 64]), rng.choice([0, 1, 2, 8, 32])
        most = 4096 * 64 * 128 // ((hq + hk) * d * (2 if dtype == "fp32" else 1))
        t = _log(rng, 1, max(1, min(32768, most)))
        return dict(op=op, t=t, hq=hq, hk=hk, d=d, rot=rot, offset=8 * rng.randint(0, (d - rot) // 8),
                    pairs=rng.choice(["half", "adjacent"]), norm=rng.random() < 0.7, axes=rng.choice([1, 1, 2, 3]),
                    far=_log(rng, 16, 1 << 20), pad=rng.choice([0, 0, t // 5]), dtype=dtype)
    hk = rng.choice([1, 2, 3, 8, 16])
    h = hk * rng.choice([1, 1, 2, 4])
    decay = rng.choice(["head", "token"])
    if op == "step":
        s = rng.choice([1, 1, 1, 2, 3, 4, 6])
        n = _log(rng, 1, max(1, min(512, 256 * 32 // (s * h))))
        return dict(op=op, n=n, s=s, h=h, hk=hk, decay=decay, dtype=dtype)
    n = _log(rng, 1, 64)
    most = ((1 << 20) if dtype == "bf16" else 32768) // (n * h)
    hi = _log(rng, 1, min(131072 if n == 1 else 16384, max(1, most)))
    return dict(op=op, n=n, lo=rng.randint(1, hi), hi=hi, h=h, hk=hk, decay=decay, carry=rng.random() < 0.5, dtype=dtype)


def _lengths(case):
    """n lengths spread evenly over [lo, hi]."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _sections(case):
    """Pairs of each axis: the first a half, the others share the rest."""
    half, axes = case["rot"] // 2, case["axes"]
    if axes == 1:
        return [half]
    rest = [half // (2 * (axes - 1))] * (axes - 1)
    return [half - sum(rest)] + rest


# ---- inputs -----------------------------------------------------------------


def _i32(v):
    return torch.as_tensor(v, dtype=torch.int32).to("cuda")


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _unit(shape, gen, dtype):
    """Heads of mean square 1: what a head norm leaves."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True))).to(dtype)


def _decays(case, tokens, gen):
    """Slopes from 1 down to 2^-8 over the heads, or those times a softplus of the token's own."""
    h = case["h"]
    rate = torch.exp2(-8.0 * torch.arange(h, device="cuda", dtype=torch.float32) / max(1, h - 1))
    if case["decay"] == "head":
        return -rate * (0.5 + torch.rand((h,), generator=gen, device="cuda"))
    x = torch.randn((*tokens, h), generator=gen, device="cuda", dtype=torch.float32)
    return -rate * torch.nn.functional.softplus(x)


def prepare(case, seed):
    host = torch.Generator().manual_seed(int(seed))
    dev = torch.Generator(device="cuda").manual_seed(int(seed))
    return dict(_PREPARE[case["op"]](case, host, dev), op=case["op"], case=dict(case))


def _prepare_rope(case, host, dev):
    t, hq, hk, d, dtype = case["t"], case["hq"], case["hk"], case["d"], _dtype(case)
    fused = _normal((t, (hq + hk) * d + 64), dev, dtype)          # the layer's fused projection
    half = case["rot"] // 2
    pos = torch.randint(0, case["far"], (case["axes"], t), generator=host)
    if case["pad"]:
        pos[:, t - case["pad"]:] = -1                              # the batch's padding
    weight = lambda: torch.rand((d,), generator=dev, device="cuda") + 0.5 if case["norm"] else None  # noqa: E731
    return dict(q=fused[:, : hq * d].unflatten(1, (hq, d)),
                k=fused[:, hq * d: (hq + hk) * d].unflatten(1, (hk, d)) if hk else None,
                q_weight=weight(), k_weight=weight() if hk else None, positions=_i32(pos), sections=_sections(case),
                inv_freq=(BASE ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda(),
                q_out=torch.zeros((t, hq, d), dtype=dtype, device="cuda"),
                k_out=torch.zeros((t, hk, d), dtype=dtype, device="cuda") if hk else None)


def _prepare_step(case, host, dev):
    n, s, h, hk, dtype = case["n"], case["s"], case["h"], case["hk"], _dtype(case)
    slots = n * s + 3
    index = torch.randperm(slots, generator=host)[: n * s].view(n, s)
    lead = (n,) if s == 1 else (n, s)
    fused = _normal((n * s, 2 * h * DIM), dev, dtype)             # value and output gate
    v = fused[:, : h * DIM].unflatten(1, (h, DIM))
    return dict(q=_unit((*lead, hk, DIM), dev, dtype), k=_unit((*lead, hk, DIM), dev, dtype),
                v=v if s == 1 else v.unflatten(0, lead), g=_decays(case, lead, dev),
                pool=torch.randn((slots, h, DIM, DIM), generator=dev, device="cuda", dtype=torch.float32),
                index=_i32(index[:, 0] if s == 1 else index),
                accepted=None if s == 1 else _i32(torch.randint(1, s + 1, (n,), generator=host)),
                o=torch.empty((*lead, h, DIM), dtype=dtype, device="cuda"))


def _prepare_chunk(case, host, dev):
    n, h, hk, dtype = case["n"], case["h"], case["hk"], _dtype(case)
    lens = torch.tensor(_lengths(case))[torch.randperm(n, generator=host)]
    t = int(lens.sum())
    fused = _normal((t, 2 * h * DIM), dev, dtype)                 # value and output gate
    pool = torch.randn((n + 3, h, DIM, DIM), generator=dev, device="cuda", dtype=torch.float32)
    return dict(q=_unit((t, hk, DIM), dev, dtype), k=_unit((t, hk, DIM), dev, dtype),
                v=fused[:, : h * DIM].unflatten(1, (h, DIM)), g=_decays(case, (t,), dev), pool=pool,
                index=_i32(torch.randperm(n + 3, generator=host)[:n]), carry=case["carry"],
                cu=_i32(torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])), longest=int(lens.max()),
                o=torch.empty((t, h, DIM), dtype=dtype, device="cuda"))


_PREPARE = dict(rope=_prepare_rope, step=_prepare_step, chunk=_prepare_chunk)


# ---- one pass ---------------------------------------------------------------


def run(state):
    return (_run_own if own else _PLAIN[state["op"]])(state)


def _run_own(s):
    import kimi_delta_attention_07_gb300 as kda
    if s["op"] == "rope":
        case = s["case"]
        return kda.kda_head_norm_rope(s["q"], s["k"], positions=s["positions"], inv_freq=s["inv_freq"],
                                      sections=s["sections"], rot_offset=case["offset"],
                                      interleaved=case["pairs"] == "adjacent", norm=case["norm"],
                                      q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, q_out=s["q_out"],
                                      k_out=s["k_out"])
    if s["op"] == "step":
        if s["accepted"] is None:
            o = kda.kda_linear_step(s["q"], s["k"], s["v"], s["g"], s["pool"], state_indices=s["index"], scale=SCALE,
                                    o=s["o"])
        else:
            o = kda.kda_linear_multi_step(s["q"], s["k"], s["v"], s["g"], s["pool"], s["index"],
                                          num_accepted=s["accepted"], scale=SCALE, o=s["o"])
        return o, s["pool"]
    return kda.kda_linear_chunk_fwd(s["q"], s["k"], s["v"], s["g"], cu_seqlens=s["cu"],
                                    initial_state=s["pool"] if s["carry"] else None, final_state=s["pool"],
                                    state_indices=s["index"], scale=SCALE, o=s["o"])


def _plain_rope(s):
    case = s["case"]
    rot, off, adjacent = case["rot"], case["offset"], case["pairs"] == "adjacent"
    axis = torch.repeat_interleave(torch.tensor(s["sections"])).to("cuda")
    angle = s["positions"].double()[axis].t() * s["inv_freq"].double()       # [T, rot / 2]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    real = (s["positions"][0] >= 0)[:, None, None]

    def one(x, weight, out):
        if x is None:
            return None
        y = x.float()
        if case["norm"]:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight
        r = y[..., off: off + rot]
        r = r.unflatten(-1, (rot // 2, 2)).movedim(-1, 0) if adjacent else r.unflatten(-1, (2, rot // 2)).movedim(-2, 0)
        a, b = r[0] * cos - r[1] * sin, r[1] * cos + r[0] * sin
        r = torch.stack([a, b], -1 if adjacent else -2).flatten(-2)
        y = torch.cat([y[..., :off], r, y[..., off + rot:]], -1).to(x.dtype)
        return out.copy_(torch.where(real, y, out))

    return one(s["q"], s["q_weight"], s["q_out"]), one(s["k"], s["k_weight"], s["k_out"])


def _heads(x, h):
    """[..., Hk, D] as fp32 [..., H, D], each head by the H / Hk that share it."""
    return x.float().repeat_interleave(h // x.shape[-2], -2)


def _plain_step(s):
    case, pool = s["case"], s["pool"]
    n, steps, h = case["n"], case["s"], case["h"]
    lead = (n, steps)
    q, k, v = (_heads(x.reshape(*lead, *x.shape[-2:]), h).transpose(1, 2) for x in (s["q"], s["k"], s["v"]))   # [n, h, s, 128]
    g = s["g"].double().expand(*lead, h) if case["decay"] == "head" else s["g"].double().view(*lead, h)
    total = g.transpose(1, 2).cumsum(-1)                                                    # [n, h, s]
    index = s["index"].long().view(*lead)
    first = index[:, 0] if s["accepted"] is None else index.gather(1, s["accepted"].long()[:, None] - 1)[:, 0]
    weight = torch.exp(total[..., :, None] - total[..., None, :]).float().tril()            # [n, h, t, j]
    new = torch.matmul((weight[..., None] * v[:, :, None]).transpose(-1, -2).flatten(2, 3), k)  # [n, h, s V, K]
    states = new.unflatten(2, (steps, DIM)) + torch.exp(total).float()[..., None, None] * pool[first][:, :, None]
    o = torch.matmul(states, q[..., None])[..., 0] * SCALE                                   # [n, h, s, V]
    pool[index.flatten()] = states.transpose(1, 2).flatten(0, 1)
    return o.transpose(1, 2).reshape(s["o"].shape).to(s["o"].dtype), pool


def _plain_chunk(s):
    case, cu, pool = s["case"], s["cu"].long(), s["pool"]
    n, h = case["n"], case["h"]
    m = -(-s["longest"] // C)
    at = cu[:-1, None] + torch.arange(m * C, device="cuda")
    real = (at < cu[1:, None])[..., None]                                                   # [n, m C, 1]
    at = at.clamp(max=s["q"].shape[0] - 1)
    chunks = lambda x: x.unflatten(1, (m, C)).movedim(3, 1)                                  # noqa: E731  [n, h, m, C, ...]
    q, k, v = (chunks(_heads(x, h)[at].masked_fill_(~real[..., None], 0.0)) for x in (s["q"], s["k"], s["v"]))
    g = s["g"].double().expand(s["q"].shape[0], h)[at].masked_fill(~real, 0.0)
    upto = chunks(g).cumsum(-1)                                                              # [n, h, m, C]
    whole = upto[..., -1]
    weight = torch.exp(upto[..., :, None] - upto[..., None, :]).float().tril_()
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)).mul_(weight), v)
    k = k * torch.exp(whole[..., None] - upto).float()[..., None]
    local = torch.matmul(v.transpose(-1, -2), k).flatten(-2)                                 # [n, h, m, V K]
    # the state behind chunk c: sum over c' <= c of exp(decays of c' + 1 .. c) local_c', and the initial one
    after = whole.cumsum(-1)
    first = pool[s["index"].long()].flatten(-2) if s["carry"] else local.new_zeros((n, h, DIM * DIM))
    behind = torch.matmul(torch.exp(after[..., :, None] - after[..., None, :]).float().tril_(), local)
    behind += torch.exp(after).float()[..., None] * first[:, :, None]
    before = torch.cat([first[:, :, None], behind[:, :, :-1]], 2).unflatten(-1, (DIM, DIM))
    o += torch.matmul(q * torch.exp(upto).float()[..., None], before.transpose(-1, -2))
    o = o.movedim(1, 3).flatten(1, 2)                                                        # [n, m C, h, V]
    pool[s["index"].long()] = behind[:, :, -1].unflatten(-1, (DIM, DIM))
    return (o[real[..., 0]] * SCALE).to(s["o"].dtype), pool


_PLAIN = dict(rope=_plain_rope, step=_plain_step, chunk=_plain_chunk)


# ---- what a pass cannot do without --------------------------------------------


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        t, heads, d = case["t"] - case["pad"], case["hq"] + case["hk"], case["d"]
        return {"bytes": t * heads * d * 2 * e + 4 * case["t"] * case["axes"] + 2 * case["rot"],
                "flops": t * heads * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    h, hk = case["h"], case["hk"]
    state = 4 * DIM * DIM * h
    t = case["n"] * case["s"] if case["op"] == "step" else sum(_lengths(case))
    tokens = e * t * DIM * 2 * (hk + h) + (4 * t * h if case["decay"] == "token" else 4 * h)
    states = case["n"] * state * (1 + case["s"] if case["op"] == "step" else 1 + case["carry"])
    return {"bytes": tokens + states, "flops": 4 * DIM * DIM * t * h}


# ---- the definitions, in 64 bits ----------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "step": _exact_step, "chunk": _exact_chunk}[case["op"]](case, s)


def _exact_rope(case, s):
    half, first = case["rot"] // 2, case["offset"]
    pos = s["positions"].double()
    turn = torch.empty((case["t"], half), dtype=torch.float64, device="cuda")
    at = 0
    for axis, pairs in enumerate(s["sections"]):
        turn[:, at: at + pairs] = pos[axis][:, None] * s["inv_freq"][at: at + pairs].double()
        at += pairs
    rotate = torch.polar(torch.ones_like(turn), turn)[:, None]
    i = torch.arange(half, device="cuda")
    left, right = (first + 2 * i, first + 2 * i + 1) if case["pairs"] == "adjacent" else (first + i, first + half + i)
    outs = []
    for x, weight in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        if x is None:
            outs.append(None)
            continue
        y = x.double()
        if case["norm"]:
            y = y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt() * weight.double()
        z = torch.complex(y[..., left], y[..., right]) * rotate
        y = y.clone()
        y[..., left], y[..., right] = z.real, z.imag
        y[case["t"] - case["pad"]:] = 0.0
        outs.append(y)
    return tuple(outs)


def _exact_step(case, s):
    n, steps, h = case["n"], case["s"], case["h"]
    head = torch.arange(h, device="cuda") * case["hk"] // h
    q, k, v = (x.double().reshape(n, steps, -1, DIM) for x in (s["q"], s["k"], s["v"]))
    g = s["g"].double().reshape(-1, h)
    index = s["index"].long().reshape(n, steps)
    begin = torch.ones(n, dtype=torch.long, device="cuda") if s["accepted"] is None else s["accepted"].long()
    state = s["pool"][index[torch.arange(n, device="cuda"), begin - 1]].double()
    o = torch.empty((n, steps, h, DIM), dtype=torch.float64, device="cuda")
    pool = s["pool"].double()
    for t in range(steps):
        decay = g if case["decay"] == "head" else g.view(n, steps, h)[:, t]
        state = state * decay.exp()[..., None, None] + v[:, t, :, :, None] * k[:, t, head][:, :, None, :]
        o[:, t] = (state * q[:, t, head][:, :, None, :]).sum(-1) * SCALE
        pool[index[:, t]] = state
    return o.view(s["o"].shape), pool


def _exact_chunk(case, s):
    n, h, lens = case["n"], case["h"], s["cu"].diff().long()
    head = torch.arange(h, device="cuda") * case["hk"] // h
    index, start = s["index"].long(), s["cu"][:-1].long()
    state = s["pool"][index].double() if s["carry"] else torch.zeros((n, h, DIM, DIM), dtype=torch.float64, device="cuda")
    state = state.flatten(0, 1)
    total = s["q"].shape[0]
    o = torch.zeros((total + n, h, DIM), dtype=torch.float64, device="cuda")   # (a place for each sequence that has ended)
    g = s["g"].double().expand(total, h)
    for t in range(s["longest"]):
        live = t < lens
        at = torch.where(live, start + t, 0)
        mask = live[:, None, None].double()
        decay = torch.where(live[:, None], g[at], 0.0).exp().reshape(-1, 1, 1)
        v = (s["v"][at].double() * mask).reshape(n * h, DIM, 1)
        k = s["k"][at][:, head].double().reshape(n * h, 1, DIM)
        state = torch.baddbmm(state * decay, v, k)
        row = torch.bmm(state, s["q"][at][:, head].double().reshape(n * h, DIM, 1)).view(n, h, DIM)
        o[torch.where(live, at, total + torch.arange(n, device="cuda"))] = row * SCALE
    pool = s["pool"].double()
    pool[index] = state.view(n, h, DIM, DIM)
    return o[:total], pool
