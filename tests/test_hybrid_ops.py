"""The operators around the core against plain implementations in 64 bits.

Bounds, element by element, from the roundings that an output passes (a
rounding is off by at most half a step, eps / 2 of its type):
  norms      the fp32 sum of squares and the products: at most 64 roundings of
             2^-24, then the output's own (bf16 2^-8, fp32 2^-24, e4m3 2^-4 or
             half its smallest step, 2^-10 of the scale)
  attention  o = sum_j p_j v_j: an fp32 score of K products is off by at most
             K 2^-24 sum_d |q_d k_d| scale =: e, which enters p (and its sum) as a factor within
             1 +- 2e; the bf16 rounding of p by 2^-8; both weigh sum_j p_j |v_j|; 2^-12 of that for the
             exponential and the fp32 sums; then the output's bf16 rounding, 2^-8 |o|
  lse        e + 2^-16 (1 + |lse|)
Whole numbers are equal.
"""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

E_BF16, E_F32 = 2.0 ** -8, 2.0 ** -24
NAN, INF = float("nan"), float("inf")


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
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, worst {float((off / bound.clamp(min=1e-300)).nan_to_num(INF).max()):.3g} of its bound"


# ---- page tables ----------------------------------------------------------------


def tables_ref(ctx, new, free, table, page, n_pages, max_tokens, start=0):
    table = [list(r) for r in table]
    max_pages = len(table[0]) if table else 0
    cu, lens, slots, pos, at, top, refused = [0], [], [], [], start, start, 0
    for n, (c, t) in enumerate(zip(ctx, new)):
        cu.append(cu[-1] + max(t, 0))
        held, total = -(-c // page), -(-(c + t) // page)
        ok = c >= 0 and t >= 0 and total <= max_pages
        if ok:
            need = total - held
            if need and at + need > len(free):
                ok = False
            elif need:
                table[n][held:total] = free[at:at + need]
                top = max(top, at + need)
            at += need
        refused += not ok
        lens.append(c + t if ok else max(c, 0))
        for p in range(c, c + max(t, 0)):
            entry = table[n][p // page] if ok else -1
            good = 0 <= entry < n_pages
            slots.append(entry * page + p % page if good else -1)
            pos.append(p if good else -1)
    pad = [-1] * max(0, max_tokens - len(slots))
    return table, cu, lens, (slots + pad)[:max_tokens], (pos + pad)[:max_tokens], [top, refused]


def check_tables(kda, ctx, new, free, table, page, n_pages, max_tokens, start=None, **kw):
    t = i32(table).view(len(ctx), -1)
    got = kda.kda_page_tables(i32(ctx), i32(new), i32(free), t, page_size=page, n_pages=n_pages,
                              max_tokens=max_tokens, free_start=None if start is None else i32([start]), **kw)
    torch.cuda.synchronize()
    ref = tables_ref(ctx, new, free, table, page, n_pages, max_tokens, start or 0)
    for name, a, b in zip(("table", "cu", "lens", "slots", "positions", "status"), (t, *got), ref):
        assert a.tolist() == b, name


@pytest.mark.parametrize("page", [16, 64, 256])
def test_page_tables_ragged(kda, page):
    ctx, new = [0, 5, page, page - 1, 3 * page + 7, 0], [1, 0, 1, 1, 2 * page, 5 * page]
    held = [-(-c // page) for c in ctx]
    ids = list(range(90, 10, -1))
    table, k = [], 0
    for h in held:
        table.append(ids[k:k + h] + [-7] * (8 - h))
        k += h
    check_tables(kda, ctx, new, ids[k:], table, page, 100, sum(new) + 5)


def test_page_tables_refusals_leave_the_others_alone(kda):
    ctx = [10, -1, 0, 70, 0, 64]
    new = [60, 4, -3, 5, 64 * 9, 1]              # negative context, negative count, too many pages for the row
    table = [[3, -9, -9, -9], [-9] * 4, [-9] * 4, [5, 6, -9, -9], [-9] * 4, [7, -9, -9, -9]]
    check_tables(kda, ctx, new, [20, 21, 22], table, 64, 32, sum(v for v in new if v > 0))


def test_page_tables_free_list_runs_out(kda):
    # the second request passes the end; the third needs no page and stands; the fourth is behind the second
    check_tables(kda, [0, 0, 3, 0], [40, 64, 2, 1], [4, 5, 6], [[-1] * 5, [-1] * 5, [9] + [-1] * 4, [-1] * 5],
                 16, 12, 107)


def test_page_tables_start_of_the_free_list_chains(kda):
    free, table = list(range(40, 60)), [[-1] * 4] * 3
    check_tables(kda, [0, 0, 0], [20, 3, 33], free, table, 16, 64, 56, start=7)
    t = i32(table)
    first = kda.kda_page_tables(i32([0, 0, 0]), i32([20, 3, 16]), i32(free), t, page_size=16, n_pages=64, max_tokens=39)
    kda.kda_page_tables(i32([20, 3, 16]), i32([14, 1, 1]), i32(free), t, page_size=16, n_pages=64, max_tokens=16,
                        free_start=first[4][:1].clone())
    assert t.tolist() == [[40, 41, 44, -1], [42, -1, -1, -1], [43, 45, -1, -1]]


def test_page_tables_bad_page_ids_and_short_outputs(kda):
    # a page of the context and a free page outside the pool; only the first 9 tokens fit the outputs
    check_tables(kda, [3, 0], [6, 20], [200, 1, -4], [[99, -1], [-1, -1]], 16, 50, 9)
    check_tables(kda, [3, 0], [14, 20], [200, 1, -4], [[9, -1], [-1, -1]], 16, 50, 40)


def test_page_tables_empty(kda):
    got = kda.kda_page_tables(i32([]), i32([]), i32([]), torch.empty((0, 4), dtype=torch.int32, device="cuda"),
                              page_size=16, n_pages=4, max_tokens=6)
    torch.cuda.synchronize()
    assert [g.tolist() for g in got] == [[0], [], [-1] * 6, [-1] * 6, [0, 0]]
    check_tables(kda, [4], [0], [], [[2]], 16, 4, 0)


@pytest.mark.parametrize("n", [1, 255, 1500])
def test_page_tables_many_requests(kda, n):
    r = torch.Generator().manual_seed(n)
    ctx = torch.randint(0, 300, (n,), generator=r).tolist()
    new = torch.randint(0, 90, (n,), generator=r).tolist()
    ids = torch.randperm(40 * n, generator=r).tolist()
    table, k = [], 0
    for c in ctx:
        h = -(-c // 32)
        table.append(ids[k:k + h] + [-1] * (13 - h))
        k += h
    check_tables(kda, ctx, new, ids[k:], table, 32, 40 * n, sum(new) + 3)


@pytest.mark.parametrize("n", [1024, 1025, 4097, 16384])
def test_page_tables_many_requests_of_few_tokens(kda, n):
    r = torch.Generator().manual_seed(n)
    ctx = torch.randint(-1, 40, (n,), generator=r).tolist()
    new = torch.randint(-1, 4, (n,), generator=r).tolist()
    ids = torch.randperm(5 * n, generator=r).tolist()
    table, k = [], 0
    for c in ctx:
        h = max(0, -(-c // 16))
        table.append(ids[k:k + h] + [-1] * (4 - h))
        k += h
    check_tables(kda, ctx, new, ids[k:k + n // 10], table, 16, 5 * n, sum(v for v in new if v > 0) + 3)


def test_page_tables_request_counts_around_48_kb_of_shared_memory():
    # in a process of its own: what a call with more requests raises stays raised for the calls after it
    code = """
import torch
import kimi_delta_attention_07_gb300 as kda
i32 = lambda v: v.to(torch.int32).cuda()
for n in (4082, 4083, 4084, 4085, 4090, 4095, 4096):
    t = i32(torch.full((n, 1), -1))
    got = kda.kda_page_tables(i32(torch.zeros(n)), i32(torch.ones(n)), i32(torch.arange(n)), t, page_size=16, n_pages=n, max_tokens=n)
    assert t[:, 0].tolist() == list(range(n)) and got[2].tolist() == list(range(0, 16 * n, 16)) and got[4].tolist() == [n, 0], n
print("all right")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.stdout.strip() == "all right", run.stderr[-2000:]


def test_page_tables_lengths_near_the_type_limit(kda):
    big = 2 ** 31 - 1
    t = i32([[1, 2]])
    got = kda.kda_page_tables(i32([big]), i32([big]), i32([3]), t, page_size=16, n_pages=4, max_tokens=4)
    torch.cuda.synchronize()
    assert t.tolist() == [[1, 2]] and got[2].tolist() == [-1] * 4 and got[4].tolist() == [0, 1]


def test_page_tables_sums_of_lengths_past_the_type(kda):
    # a table row wide enough for the sum: what refuses it is the length itself
    big = 2 ** 31 - 1
    t = torch.full((1, 2 ** 28), 3, dtype=torch.int32, device="cuda")
    for new, ok in ((2, False), (1, False), (0, True)):
        cu, lens, slots, pos, status = kda.kda_page_tables(i32([big]), i32([new]), i32([3]), t, page_size=16,
                                                           n_pages=4, max_tokens=2)
        torch.cuda.synchronize()
        assert lens.tolist() == [big] and slots.tolist() == pos.tolist() == [-1, -1] and status.tolist() == [0, int(not ok)]


# ---- rms norm ---------------------------------------------------------------------


def norm_ref(x, residual, weight, eps):
    h = x.double() + (0 if residual is None else residual.double())
    y = h / (h.square().mean(-1, keepdim=True) + eps).sqrt()
    return h, y * (1 if weight is None else weight.double())


def check_norm(x, residual, weight, quant, got, eps=1e-6):
    y, h_out, scales = got
    h, ref = norm_ref(x, residual, weight, eps)
    half = E_BF16 if x.dtype is torch.bfloat16 else E_F32
    if h_out is not None:
        within(h_out, h, h.abs() * (half + 2 * E_F32), "residual_out")
    calc = 64 * E_F32
    if quant == "none":
        return within(y, ref, ref.abs() * (half * (1 + calc) + calc), "y")
    g = ref.reshape(*ref.shape[:-1], scales.shape[-1], -1)
    s = g.abs().amax(-1).clamp(min=1e-30) / 448
    within(scales, s, s * (calc + 2 * E_F32), "scales")
    stood = y.double().reshape(g.shape) * scales.double()[..., None]
    within(stood, g, g.abs() * (2.0 ** -4 * (1 + 2 * calc) + 2 * calc) + s[..., None] * 2.0 ** -10 * (1 + 2 * calc), "y")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(1, 8), (3, 24), (5, 128), (2, 1000), (300, 2304), (1, 4096), (7, 4104), (2, 16384), (3, 32768)])
def test_rms_norm(kda, dtype, rows, D):
    x, r = normal((rows, D), 1, dtype), normal((rows, D), 2, dtype, 3.0)
    w = torch.rand(D, generator=gen(3), device="cuda") + 0.5
    for quant in ("none", "row") + (("block",) if D % 128 == 0 else ()):
        check_norm(x, r, w, quant, kda.kda_rms_norm(x, w, residual=r, quant=quant))
        got = kda.kda_rms_norm(x, quant=quant)
        assert got[1] is None
        check_norm(x, None, None, quant, got)


def test_rms_norm_in_place_and_leading_axes(kda):
    x, r = normal((2, 3, 512), 4), normal((2, 3, 512), 5)
    w = torch.ones(512, device="cuda")
    r0, x0 = r.clone(), x.clone()
    got = kda.kda_rms_norm(x, w, residual=r, residual_out=r, quant="block")
    assert got[1] is r
    check_norm(x0, r0, w, "block", got)
    r = r0.clone()
    got = kda.kda_rms_norm(x, w, residual=r, residual_out=x, y=r)      # both inputs overwritten
    check_norm(x0, r0, w, "none", got)


def test_rms_norm_zero_rows_and_zero_row_count(kda):
    x = torch.zeros((2, 256), dtype=torch.bfloat16, device="cuda")
    for quant in ("row", "block"):
        y, _, s = kda.kda_rms_norm(x, quant=quant)
        assert (y.float() == 0).all() and torch.isfinite(s).all() and (s > 0).all()
    y, _, _ = kda.kda_rms_norm(x, eps=0.0)
    assert y.isnan().all()                                               # 0 / 0, as the formula says
    assert kda.kda_rms_norm(x[:0])[0].shape == (0, 256)


@pytest.mark.parametrize("value", [NAN, INF])
def test_rms_norm_not_finite(kda, value):
    x = normal((3, 512), 6)
    x[1, 300] = value
    y, _, _ = kda.kda_rms_norm(x)
    _, ref = norm_ref(x, None, None, 1e-6)
    assert torch.equal(y.isnan(), ref.isnan()) and y[[0, 2]].isfinite().all()
    y, _, s = kda.kda_rms_norm(x, quant="block")
    # inf turns its own channel to NaN (inf * 0) and the others to 0; NaN turns the row to NaN
    groups = [True] * 4 if value != value else [False, False, True, False]
    assert s[1].isnan().tolist() == groups and s[[0, 2]].isfinite().all() and y.float()[[0, 2]].isfinite().all()


def test_rms_norm_large_values(kda):
    # bf16 values whose squares pass fp16 and whose sum stays in fp32
    x = normal((2, 1024), 7, std=1e15)
    check_norm(x, None, None, "none", kda.kda_rms_norm(x))
    check_norm(x, None, None, "row", kda.kda_rms_norm(x, quant="row"))


# ---- cache write ------------------------------------------------------------------


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("T", [1, 3, 130])
def test_cache_write(kda, T, page):
    fused = normal((T, 64 + 576 + 8), 1)
    kv = fused[:, 64:640]
    w = torch.rand(512, generator=gen(2), device="cuda") + 0.5
    cache = normal((T // page + 2, page, 576), 3)
    rows = cache.shape[0] * page
    slots = torch.randperm(rows, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32)
    if T > 2:
        slots[1], slots[2] = -1, rows          # padding, one past the pool
    before = cache.clone().view(-1, 576)
    assert kda.kda_latent_cache_write(kv, w, cache, slots.cuda()) is cache
    got = cache.view(-1, 576)
    keep = ((slots >= 0) & (slots < rows)).nonzero()[:, 0]
    at, src = slots[keep].long().cuda(), kv[keep.cuda()]
    _, ref = norm_ref(src[:, :512], None, w, 1e-6)
    within(got[at, :512], ref, ref.abs() * (E_BF16 * (1 + 2.0 ** -16) + 64 * E_F32), "latent")
    assert torch.equal(got[at, 512:], src[:, 512:])
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(got[rest], before[rest])
    kda.kda_latent_cache_write(kv, None, cache, slots.cuda())
    assert torch.equal(cache.view(-1, 576)[at], src)


def test_cache_write_past_32_bits(kda):
    page = 64
    n_pages = 2 ** 31 // (576 * page) + 40                              # over 2^31 elements
    cache = torch.empty((n_pages, page, 576), dtype=torch.bfloat16, device="cuda")
    kv = normal((4, 576), 5)
    slots = [n_pages * page - 1, 0, n_pages * page - 70, 2 ** 31 // 576 + 3]
    kda.kda_latent_cache_write(kv, None, cache, i32(slots))
    assert torch.equal(cache.view(-1, 576)[torch.tensor(slots, device="cuda")], kv)


# ---- absorbed attention -------------------------------------------------------------


def attention_ref(q, k, v, visible, scale):
    """One sequence: q [lq, H, D], k [lk, H or 1, D], v [lk, H or 1, Dv] in 64 bits; query i sees keys below
    visible[i].  Returns o, lse and the two bounds."""
    q, k, v = q.double(), k.double(), v.double()
    H, lk = q.shape[1], k.shape[0]
    k, v = k.expand(lk, H, -1), v.expand(lk, H, -1)
    x = torch.einsum("qhd,khd->hqk", q, k) * scale
    e = torch.einsum("qhd,khd->hqk", q.abs(), k.abs()) * (abs(scale) * q.shape[-1] * E_F32)
    hidden = torch.arange(lk, device=q.device)[None, :] >= torch.as_tensor(visible, device=q.device)[:, None]
    x = x.masked_fill(hidden, -INF)
    e = e.masked_fill(hidden, 0.0).amax(-1) if lk else x.new_zeros(H, q.shape[0])
    lse = torch.logsumexp(x, -1) if lk else x.new_full((H, q.shape[0]), -INF)
    p = torch.where(hidden, 0.0, torch.exp(x - lse[..., None].clamp(min=-1e300)))
    o = torch.einsum("hqk,khd->qhd", p, v)
    weigh = torch.einsum("hqk,khd->qhd", p, v.abs())
    bound = E_BF16 * o.abs() + weigh * (E_BF16 + 2.0 ** -12 + 4 * e.T[..., None])
    lse_bound = e + 2.0 ** -16 * (1 + lse.abs().nan_to_num(0, 0, 0))
    return o, lse.T, bound + 1e-30, lse_bound.T


def decode_case(lens, S, H, page, seed, spare=3, poison=True, high=False):
    g = torch.Generator().manual_seed(seed)
    held = [max(0, -(-v // page)) for v in lens]
    n_pages = sum(held) + spare
    ids = torch.randperm(n_pages, generator=g).tolist()
    width = max(held + [1]) + 1
    table, k = [], 0
    for h in held:
        table.append(ids[k:k + h] + [-1] * (width - h))
        k += h
    cache = normal((n_pages, page, 576), seed)
    if poison:   # what no request holds may be anything
        used = torch.zeros((n_pages, page), dtype=torch.bool)
        for row, v in zip(table, lens):
            for p in range(v):
                used[row[p // page], p % page] = True
        cache[~used.cuda()] = NAN
    return normal((len(lens), S, H, 576), seed + 1), cache, i32(table).view(len(lens), width), i32(lens)


def check_decode(kda, case, scale=192 ** -0.5, **kw):
    q, cache, table, lens = case
    n, S, H, _ = q.shape
    page = cache.shape[1]
    lse = torch.full((n, S, H), 7.0, device="cuda")
    o = torch.full((n, S, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    assert kda.kda_latent_decode(q, cache, table, lens, scale=scale, o=o, lse=lse, **kw) is o
    torch.cuda.synchronize()
    for b, length in enumerate(lens.tolist()):
        rows = cache[table[b, : -(-length // page)].long()].reshape(-1, 576)[:length][:, None]
        ref, ref_lse, bound, lse_bound = attention_ref(q[b], rows, rows[..., :512],
                                                       [length - S + 1 + s for s in range(S)], scale)
        within(o[b], ref, bound, f"o of request {b} ({length} tokens)")
        seen = ref_lse.isfinite()
        assert torch.equal(lse[b][~seen].double(), ref_lse[~seen])
        within(lse[b][seen], ref_lse[seen], lse_bound[seen], f"lse of request {b}")
    return o, lse


EDGES = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_lengths_and_pages(kda, page):
    check_decode(kda, decode_case(EDGES, 1, 32, page, 10))


@pytest.mark.parametrize("H", [1, 2, 5, 8, 16, 31, 33, 40, 64, 100])
def test_decode_heads(kda, H):
    check_decode(kda, decode_case([3, 200, 131], 1, H, 64, 20))


@pytest.mark.parametrize("S,H", [(2, 32), (3, 5), (4, 32), (7, 16), (4, 9)])
def test_decode_several_tokens(kda, S, H):
    # lengths below S leave the first tokens without a position: zeros and -inf
    check_decode(kda, decode_case([0, 1, S - 1, S, S + 1, 127, 128, 129, 128 + S, 300], S, H, 32, 30))


def test_decode_single_short_request(kda):
    for length in (0, 1, 5):
        check_decode(kda, decode_case([length], 1, 32, 64, 40))


def test_decode_long_request_is_split(kda):
    check_decode(kda, decode_case([20011], 1, 32, 64, 50))


@pytest.mark.parametrize("n", [40, 300])
def test_decode_many_ragged_requests(kda, n):
    g = torch.Generator().manual_seed(n)
    lens = (torch.rand(n, generator=g) ** 4 * 1500).int().tolist()
    check_decode(kda, decode_case(lens, 1, 8, 64, 60))


def test_decode_large_scores(kda):
    # scores of some hundreds, rising and falling along the cache: the running maximum moves often
    q, cache, table, lens = decode_case([700, 129], 2, 32, 64, 70)
    ramp = torch.linspace(0.2, 6.0, 700, device="cuda")
    rows = cache[table[0, :11].long()].reshape(-1, 576)
    rows[:700] *= ramp[:, None].to(torch.bfloat16)
    cache[table[0, :11].long()] = rows.view(11, 64, 576)
    check_decode(kda, (q * 4, cache, table, lens))
    check_decode(kda, (q, cache, table, lens), scale=-0.3)
    check_decode(kda, (q, cache, table, lens), scale=0.0)


def test_decode_requests_that_cannot_be_read(kda):
    """Bad lengths and page ids give NaN for their request alone."""
    case = decode_case([100, 100, 100, 100, 300, 50], 1, 4, 64, 80, poison=False)
    q, cache, table, lens = case
    o0 = kda.kda_latent_decode(q, cache, table, lens)
    bad_table, bad_lens = table.clone(), lens.clone()
    bad_lens[0], bad_lens[1] = -5, table.shape[1] * 64 + 1
    bad_table[2, 1], bad_table[4, 3] = cache.shape[0], -1
    bad_table[3, 2] = 2 ** 31 - 1                                        # past request 3's length: not used
    o = kda.kda_latent_decode(q, cache, bad_table, bad_lens)
    for b, nan in enumerate([True, True, True, False, True, False]):
        assert o[b].isnan().all() if nan else torch.equal(o[b], o0[b]), b


def test_decode_nan_and_inf_in_the_cache_stay_in_their_request(kda):
    q, cache, table, lens = decode_case([200, 200], 1, 8, 64, 90)
    clean = kda.kda_latent_decode(q, cache, table, lens)
    cache[table[0, 1].long(), 5, 100] = NAN
    o = kda.kda_latent_decode(q, cache, table, lens)
    assert o[0].isnan().all() and torch.equal(o[1], clean[1])


def test_decode_nan_in_a_new_token_stays_with_the_rows_that_see_it(kda):
    q, cache, table, lens = decode_case([200, 97], 3, 16, 64, 95)
    clean = kda.kda_latent_decode(q, cache, table, lens)
    cache[table[0, 3].long(), 199 - 192, 7] = NAN                        # the last of request 0's three tokens
    cache[table[1, 1].long(), 95 - 64, 300] = INF                        # the second of request 1's
    o = kda.kda_latent_decode(q, cache, table, lens)
    assert torch.equal(o[0, :2], clean[0, :2]) and o[0, 2].isnan().all()
    assert torch.equal(o[1, 0], clean[1, 0])


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("lens,S,H,wide", [([200, 97], 3, 16, False), ([200, 97], 3, 16, True), ([49, 65], 2, 8, False),
                                           ([20011, 3], 4, 8, False), ([20011, 96], 4, 32, True)])
def test_decode_not_finite_in_a_new_token_reaches_the_rows_that_see_it(kda, lens, S, H, wide, value):
    """The newest but one token of the first request has a latent value that is not finite.  Rows whose query is of the
    other sign score -inf there: p = 0, NaN in that channel (0 * inf), and the others as if the token were not there.
    Every other row that sees it is NaN.  (49 and 65: the new tokens lie in two tiles.)"""
    case = decode_case(lens, S, H, 64, 96)
    q, cache, table, lens = widened(case) if wide else case
    length, d = int(lens[0]), 300
    q[..., d] = torch.where(q[..., d] == 0, 1.0, q[..., d])
    clean = kda.kda_latent_decode(q, cache, table, lens)
    at = length - 2
    cache[table[0, at // 64].long(), at % 64, d] = value
    lse = torch.empty((len(lens), S, H), device="cuda")
    o = kda.kda_latent_decode(q, cache, table, lens, lse=lse)
    assert torch.equal(o[1:], clean[1:]) and torch.equal(o[0, :S - 2], clean[0, :S - 2])
    rows = cache[table[0, : -(-length // 64)].long()].reshape(-1, 576)[:length]
    hidden = q[0, S - 2:, :, d].float() * value == -INF
    assert (value != value) == (not hidden.any()) and not hidden.all()
    assert o[0, S - 2:][~hidden].isnan().all() and lse[0, S - 2:][~hidden].isnan().all()
    rows = torch.cat([rows[:at], rows[at + 1:]])[:, None]
    ref, ref_lse, bound, lse_bound = attention_ref(q[0, S - 2:], rows, rows[..., :512], [at, at + 1], 192 ** -0.5)
    got, rest = o[0, S - 2:], torch.arange(512, device="cuda") != d
    assert got[hidden][:, d].isnan().all()
    within(got[hidden][:, rest], ref[hidden][:, rest], bound[hidden][:, rest], "rows that score -inf")
    within(lse[0, S - 2:][hidden], ref_lse[hidden], lse_bound[hidden], "their lse")


def test_decode_many_rows_and_tokens(kda):
    # more rows than one CTA takes, over a table that holds many tokens
    check_decode(kda, decode_case([9000, 5, 0, 7777, 300], 2, 48, 64, 96))
    check_decode(kda, decode_case([20000], 1, 33, 16, 97))


def widened(case):
    """The same requests with a table that could hold many more tokens."""
    q, cache, table, lens = case
    more = 200000 // (table.shape[0] * cache.shape[1]) + 1
    return q, cache, torch.cat([table, table.new_full((table.shape[0], more), -1)], 1), lens


@pytest.mark.parametrize("S,H,page", [(1, 33, 16), (1, 64, 64), (2, 32, 256), (4, 32, 32), (3, 48, 128), (16, 8, 64)])
def test_decode_many_rows_over_a_wide_table(kda, S, H, page):
    check_decode(kda, widened(decode_case([0, S - 1, S, 48, 49, *EDGES, 700], S, H, page, 98)))


def test_decode_many_rows_over_a_wide_table_large_scores(kda):
    q, cache, table, lens = decode_case([1500, 129, 64], 2, 32, 64, 71)
    ramp = torch.linspace(0.2, 6.0, 1500, device="cuda")
    rows = cache[table[0, :24].long()].reshape(-1, 576)
    rows[:1500] *= ramp[:, None].to(torch.bfloat16)
    cache[table[0, :24].long()] = rows.view(24, 64, 576)
    check_decode(kda, widened((q * 4, cache, table, lens)))
    check_decode(kda, widened((q, cache, table, lens)), scale=-0.3)


def test_decode_many_rows_over_a_wide_table_not_finite(kda):
    q, cache, table, lens = widened(decode_case([200, 97, 90, 300], 3, 16, 64, 99))
    clean = kda.kda_latent_decode(q, cache, table, lens)
    cache[table[0, 3].long(), 199 - 192, 7] = NAN                        # the last of request 0's three tokens
    cache[table[1, 1].long(), 95 - 64, 530] = INF                        # the key of the second of request 1's
    table[2, 1] = cache.shape[0]
    o = kda.kda_latent_decode(q, cache, table, lens)
    assert torch.equal(o[0, :2], clean[0, :2]) and o[0, 2].isnan().all()
    assert torch.equal(o[1, 0], clean[1, 0])
    assert o[2].isnan().all() and torch.equal(o[3], clean[3])


@pytest.mark.parametrize("S,H,wide", [(1, 1, False), (1, 5, False), (1, 8, False), (2, 3, False), (1, 40, False), (1, 40, True), (3, 16, True)])
def test_decode_rows_do_not_depend_on_what_lies_beside_them(kda, S, H, wide):
    """Bit for bit: not on cache rows past the length, nor on another request's or another head's query.  Enough requests
    that a CTA takes several tiles of each, where a score far above the first tile's raises the reference."""
    case = decode_case([97 + 7 * b % 60 for b in range(500)], S, H, 64, 120, poison=False)
    q, cache, table, lens = widened(case) if wide else case
    plain = kda.kda_latent_decode(q, cache, table, lens)
    held = torch.zeros(cache.shape[:2], dtype=torch.bool)
    for row, length in zip(table.tolist(), lens.tolist()):
        for p in range(length):
            held[row[p // 64], p % 64] = True
    other = torch.where(held.cuda()[..., None], cache, cache * 3e4)
    assert torch.equal(kda.kda_latent_decode(q, other, table, lens), plain)
    other = q.clone()
    other[1::2] *= 50
    assert torch.equal(kda.kda_latent_decode(other, cache, table, lens)[::2], plain[::2])
    other = q.clone()
    other[:, :, 0] *= 50
    assert torch.equal(kda.kda_latent_decode(other, cache, table, lens)[:, :, 1:], plain[:, :, 1:])


@pytest.mark.parametrize("n", [5000, 65535])
def test_decode_thousands_of_requests(kda, n):
    # of one tile each, so that a request's bits are the same in a call with fewer of them
    g = torch.Generator().manual_seed(n)
    cache, q = normal((300, 16, 576), 121), normal((n, 4, 576), 122)
    table = torch.randint(0, 300, (n, 3), generator=g).to(torch.int32).cuda()
    lens = torch.randint(0, 49, (n,), generator=g).to(torch.int32).cuda()
    o = kda.kda_latent_decode(q, cache, table, lens)
    for a in range(0, n, n // 5 - 7):
        part = slice(a, a + 700)
        assert torch.equal(o[part], kda.kda_latent_decode(q[part], cache, table[part], lens[part])), a
    check_decode(kda, (q[-40:, None], cache, table[-40:], lens[-40:]))


def test_decode_past_32_bits(kda):
    page, n_pages = 64, 2 ** 31 // (576 * 64) + 200
    cache = torch.empty((n_pages, page, 576), dtype=torch.bfloat16, device="cuda")
    ids = [n_pages - 1, 3, n_pages - 120, 2 ** 31 // (576 * 64) + 1]
    cache[torch.tensor(ids, device="cuda")] = normal((4, page, 576), 1)
    check_decode(kda, (normal((1, 1, 32, 576), 2), cache, i32([ids]), i32([250])))


def test_decode_repeats_bit_for_bit_and_on_another_stream(kda):
    case = decode_case([5000, 3, 900], 1, 32, 64, 100)
    o = kda.kda_latent_decode(*case)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        assert torch.equal(kda.kda_latent_decode(*case), o)
    other = kda.kda_latent_decode(*case, stream=s)
    s.synchronize()
    assert torch.equal(other, o)


def test_decode_in_a_graph_follows_the_lengths(kda):
    q, cache, table, lens = decode_case([640, 500], 1, 32, 64, 110, poison=False)
    ws = torch.empty(kda.kda_latent_decode_workspace_bytes(2, 1, 32), dtype=torch.uint8, device="cuda")
    o = torch.empty((2, 1, 32, 512), dtype=torch.bfloat16, device="cuda")
    run = lambda: kda.kda_latent_decode(q, cache, table, lens, o=o, workspace=ws)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for v in ([640, 500], [1, 0], [130, 499]):
        lens.copy_(i32(v))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, kda.kda_latent_decode(q, cache, table, lens))


# ---- expanded attention ---------------------------------------------------------------


def prefill_case(lens_q, lens_k, H, seed, slack=0):
    tq, tk = sum(lens_q) + slack, sum(lens_k) + slack
    cu = lambda v: i32([0] + torch.tensor(v).cumsum(0).tolist())  # noqa: E731
    return (normal((tq, H, 192), seed), normal((tk, H, 256), seed + 1), normal((tk, 64), seed + 2), cu(lens_q), cu(lens_k))


def check_prefill(kda, case, causal=True, scale=192 ** -0.5, **kw):
    q, kv, rope, cq, ck = case
    H = q.shape[1]
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    o = torch.full((*q.shape[:2], 128), 7.0, dtype=torch.bfloat16, device="cuda")
    assert kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck, causal=causal, scale=scale, o=o,
                                  lse=lse, **kw) is o
    torch.cuda.synchronize()
    cq, ck = cq.tolist(), ck.tolist()
    for b in range(len(cq) - 1):
        qs, ks = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        lq, lk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        if not lq:
            continue
        k = torch.cat([kv[ks, :, :128], rope[ks, None].expand(-1, H, -1)], -1)
        seen = [max(0, i + 1 + lk - lq) if causal else lk for i in range(lq)]
        ref, ref_lse, bound, lse_bound = attention_ref(q[qs], k, kv[ks, :, 128:], seen, scale)
        within(o[qs], ref, bound, f"o of sequence {b} ({lq} queries, {lk} keys)")
        some = ref_lse.isfinite()
        assert torch.equal(lse[qs][~some].double(), ref_lse[~some])
        within(lse[qs][some], ref_lse[some], lse_bound[some], f"lse of sequence {b}")
    rest = o[cq[-1]:]
    assert (rest == 7).all() and (lse[cq[-1]:] == 7).all()               # tokens past the last sequence
    return o, lse


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("length", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513])
def test_prefill_one_sequence(kda, length, causal):
    check_prefill(kda, prefill_case([length], [length], 2, length), causal)


@pytest.mark.parametrize("H", [1, 3, 32])
def test_prefill_packed(kda, H):
    lens = [70, 1, 0, 300, 128, 5]
    check_prefill(kda, prefill_case(lens, lens, H, 5))


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_behind_a_prefix_and_with_empty_rows(kda, causal):
    # more keys than queries, fewer (the first queries see nothing), no key at all, one of either
    check_prefill(kda, prefill_case([100, 200, 40, 1, 260, 3], [230, 70, 0, 500, 1, 129], 4, 6), causal)


def test_prefill_tokens_past_the_last_sequence(kda):
    check_prefill(kda, prefill_case([30, 140], [30, 200], 2, 7, slack=19))


def test_prefill_longer(kda):
    check_prefill(kda, prefill_case([1500, 33], [2100, 1033], 2, 8))


def test_prefill_large_scores(kda):
    q, kv, rope, cq, ck = prefill_case([400], [700], 2, 9)
    kv *= torch.linspace(0.2, 5.0, 700, device="cuda")[:, None, None].to(torch.bfloat16)
    check_prefill(kda, (q * 6, kv, rope, cq, ck))
    check_prefill(kda, (q, kv, rope, cq, ck), scale=-0.4)
    check_prefill(kda, (q, kv, rope, cq, ck), scale=0.0, causal=False)


@pytest.mark.parametrize("scale", [0.0, -0.4, 0.1])
def test_prefill_nan_query_keeps_to_its_row(kda, scale):
    # 0 times a NaN score is NaN too
    q, kv, rope, cq, ck = prefill_case([300], [300], 2, 24)
    plain = kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck, scale=scale)
    q[140, 1, 3] = NAN
    lse = torch.empty(q.shape[:2], device="cuda")
    o = kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck, scale=scale, lse=lse)
    assert o[140, 1].isnan().all() and lse[140, 1].isnan()
    o[140, 1] = plain[140, 1]
    assert torch.equal(o, plain)


def test_prefill_strided_inputs(kda):
    H = 3
    q, kv, rope, cq, ck = prefill_case([90, 31], [150, 31], H, 10)
    wide_q = torch.full((q.shape[0], H * 192 + 40), NAN, dtype=torch.bfloat16, device="cuda")
    wide_q[:, 8:8 + H * 192] = q.view(q.shape[0], -1)
    wide_kv = torch.full((kv.shape[0], H * 256 + 8), NAN, dtype=torch.bfloat16, device="cuda")
    wide_kv[:, :H * 256] = kv.view(kv.shape[0], -1)
    wide_r = torch.full((kv.shape[0], 512 + 64), NAN, dtype=torch.bfloat16, device="cuda")
    wide_r[:, 512:] = rope
    a = check_prefill(kda, (q, kv, rope, cq, ck))
    b = check_prefill(kda, (wide_q[:, 8:8 + H * 192].unflatten(1, (H, 192)), wide_kv[:, :H * 256].unflatten(1, (H, 256)),
                            wide_r[:, 512:], cq, ck))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_prefill_not_finite_values_stay_where_they_are_seen(kda):
    q, kv, rope, cq, ck = prefill_case([200, 150], [200, 150], 2, 11)
    clean, _ = check_prefill(kda, (q, kv, rope, cq, ck))
    kv[77, 1, 200] = NAN                       # a value: seen by queries 77.. of head 1
    o = kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck)
    seen = torch.zeros_like(o, dtype=torch.bool)
    seen[77:200, 1, 72] = True
    assert torch.equal(o.isnan(), seen) and torch.equal(o[~seen], clean[~seen])
    kv[77, 1, 200] = 0.0
    clean = kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck)
    kv[300, 0, 3] = INF                        # a key of the second sequence, head 0
    o = kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck)
    assert torch.equal(o[:300], clean[:300]) and torch.equal(o[:, 1], clean[:, 1])


@pytest.mark.parametrize("lq,lk,at", [(300, 300, 200), (300, 300, 20), (200, 2000, 1900), (129, 199, 198)])
@pytest.mark.parametrize("value", [INF, -INF])
def test_prefill_infinite_value_of_a_token_that_scores_minus_infinity(kda, lq, lk, at, value):
    """p = 0 there, and 0 times the value is NaN in its channel; the other channels are as if the token were not there.
    (In a tile with hidden places, in one without, with split keys, and as the last key.)"""
    q, kv, rope, cq, ck = prefill_case([lq], [lk], 2, 36)
    q[..., 7] = torch.where(q[..., 7] == 0, 1.0, q[..., 7])
    kv[at, :, 7], kv[at, 1, 128 + 40] = INF, value
    lse = torch.empty(q.shape[:2], device="cuda")
    o = kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck, lse=lse)
    sees = (torch.arange(lq, device="cuda") + lk - lq >= at)[:, None].expand(lq, 2)
    below = sees & (q[..., 7] < 0)
    assert o[sees & ~below].isnan().all() and o[below & (torch.arange(2, device="cuda") == 1)][:, 40].isnan().all()
    rest = [j for j in range(lk) if j != at]
    k = torch.cat([kv[..., :128], rope[:, None].expand(-1, 2, -1)], -1)[rest]
    seen = [i + 1 + lk - lq - (i + lk - lq >= at) for i in range(lq)]
    ref, ref_lse, bound, lse_bound = attention_ref(q, k, kv[rest][..., 128:], seen, 192 ** -0.5)
    fine = (below | ~sees)[..., None].expand(lq, 2, 128).clone()
    fine[:, 1, 40] &= ~sees[:, 1]
    within(o[fine], ref[fine], bound[fine], "o")
    within(lse[below | ~sees], ref_lse[below | ~sees], lse_bound[below | ~sees], "lse")


def test_prefill_bad_offsets_write_nothing_of_their_sequence(kda):
    q, kv, rope, _, _ = prefill_case([300], [300], 2, 12)
    o = torch.full((300, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    cq, ck = i32([0, 100, 90, 160, 300]), i32([0, 100, 120, 200, 900])     # decreasing queries, keys out of range
    kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck, o=o)
    torch.cuda.synchronize()
    assert (o[160:] == 7).all() and not (o[:90] == 7).all()


def test_prefill_other_stream_and_repeats(kda):
    q, kv, rope, cq, ck = prefill_case([500, 20], [600, 20], 4, 13)
    o = kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck, stream=s)
    s.synchronize()
    assert torch.equal(o, other)


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_many_short_sequences(kda, causal):
    # more blocks of queries than the GPU runs at once, most of at most 128 queries (which take either half of a block)
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 129, (90,), generator=g).tolist()
    lens[7], lens[40], lens[41] = 257, 128, 129
    keys = [n + int(p) for n, p in zip(lens, torch.randint(0, 200, (90,), generator=g))]
    keys[3], keys[4] = 0, 1
    case = prefill_case(lens, keys, 8, 41, slack=3)
    o, _ = check_prefill(kda, case, causal)
    q, kv, rope, cq, ck = case
    starts = cq.tolist()
    b = next(i for i in range(50, 90) if lens[i] > 3 and keys[i] >= lens[i])
    kv[ck[b + 1] - 2, 5, 200] = INF                                      # seen by the last two queries (or all)
    cq = cq.clone()
    cq[20] = -1                                                          # sequences 19 and 20: not written
    again = torch.full_like(o, 7.0)
    kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck, causal=causal, o=again)
    want = o.clone()
    want[starts[19]:starts[21]] = 7.0
    want[starts[b + 1] - 2 if causal else starts[b]:starts[b + 1], 5, 72] = INF
    assert torch.equal(again, want)


def test_prefill_thousands_of_sequences(kda):
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(0, 4, (5000,), generator=g).tolist()
    lens[4321], lens[17] = 300, 257
    keys = [v + int(p) for v, p in zip(lens, torch.randint(0, 5, (5000,), generator=g))]
    q, kv, rope, cq, ck = prefill_case(lens, keys, 2, 42, slack=1)
    o = kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck)
    aq, ak = cq.tolist(), ck.tolist()
    for a in range(0, 5000, 500):
        rows, cols = slice(aq[a], aq[a + 500]), slice(ak[a], ak[a + 500])
        part = (q[rows], kv[cols], rope[cols], cq[a:a + 501] - aq[a], ck[a:a + 501] - ak[a])
        got = kda.kda_latent_prefill(*part[:3], cu_seqlens_q=part[3], cu_seqlens_k=part[4])
        assert torch.equal(o[rows], got), a
    check_prefill(kda, (part[0], part[1], part[2], part[3][-61:], part[4][-61:]))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens_q,lens_k,H", [([64], [1500], 3), ([1], [2049], 1), ([300], [5000], 2), ([100, 1, 260], [1400, 2000, 1100], 2),
                                             ([5, 0, 9], [4000, 3000, 3], 4), ([700], [1100], 1), ([400], [65], 1)])
def test_prefill_few_queries_split_their_keys(kda, lens_q, lens_k, H, causal):
    case = prefill_case(lens_q, lens_k, H, 31, slack=sum(lens_k) % 7 + 1)
    need = kda.kda_latent_prefill_workspace_bytes(len(lens_q), case[0].shape[0], case[1].shape[0], H)
    assert (need > 0) == (sum(lens_k) > 1000)
    o, lse = check_prefill(kda, case, causal)
    ws = torch.full((need + 8,), 255, dtype=torch.uint8, device="cuda")   # NaN wherever it is read before it is written
    again, lse2 = check_prefill(kda, case, causal, workspace=ws)
    assert torch.equal(o, again) and torch.equal(lse, lse2)


def test_prefill_split_keys_not_finite(kda):
    q, kv, rope, cq, ck = prefill_case([200, 30], [2000, 1700], 2, 33)
    run = lambda: kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck)  # noqa: E731
    assert kda.kda_latent_prefill_workspace_bytes(2, 230, 3700, 2) > 0
    clean = run()
    kv[1900, 1, 130] = INF                                               # seen by query 100 of sequence 0 and later ones
    kv[1999, 0, 128] = NAN                                               # by its last one
    kv[2000 + 1690, 0, 140] = NAN                                        # by query 20 of sequence 1 and later ones
    q[50, 1, 3] = NAN
    o = run()
    want = clean.clone()
    want[100:200, 1, 2] = INF
    want[199, 0, 0] = NAN
    want[220:, 0, 12] = NAN
    want[50, 1] = NAN
    assert torch.equal(o.nan_to_num(7.0, 8.0), want.nan_to_num(7.0, 8.0))
    q[199] = INF                                                         # scores of +-inf and NaN: one row of either head
    o2 = run()
    assert torch.equal(o2[:199].nan_to_num(7.0, 8.0), o[:199].nan_to_num(7.0, 8.0))


def test_prefill_split_keys_in_a_graph_and_on_another_stream(kda):
    q, kv, rope, cq, ck = prefill_case([90], [3000], 2, 35)
    eager = kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck, stream=s)
    s.synchronize()
    assert torch.equal(other, eager)
    o = torch.empty_like(eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck, o=o)
    for keys in (3000, 1, 700):
        ck[1] = keys
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck))


def test_prefill_past_32_bits(kda):
    # the second sequence's keys lie past 2^31 elements of kv, its queries behind an empty sequence
    H, first, lk = 32, 2 ** 31 // (32 * 256) + 500, 300
    kv = torch.empty((first + lk, H, 256), dtype=torch.bfloat16, device="cuda")
    rope = torch.empty((first + lk, 64), dtype=torch.bfloat16, device="cuda")
    kv[first:], rope[first:] = normal((lk, H, 256), 1), normal((lk, 64), 2)
    q = normal((5, H, 192), 3)
    a = kda.kda_latent_prefill(q, kv, rope, cu_seqlens_q=i32([0, 0, 5]), cu_seqlens_k=i32([0, first, first + lk]))
    b = kda.kda_latent_prefill(q, kv[first:].clone(), rope[first:].clone(), cu_seqlens_q=i32([0, 5]),
                               cu_seqlens_k=i32([0, lk]))
    assert torch.equal(a, b) and a.isfinite().all()


def test_a_step_in_a_graph(kda):
    """All operators in one captured graph, replayed on other lengths and data."""
    H, N, page, pages = 4, 3, 32, 40
    g = torch.Generator().manual_seed(1)
    new, ctx = i32([5, 1, 40]), i32([0, 0, 0])
    free, table = torch.randperm(pages, generator=g).to(torch.int32).cuda(), i32([[-1] * 8] * N)
    x, w = normal((64, 576), 2), torch.rand(512, generator=gen(3), device="cuda") + 0.5
    cache = torch.zeros((pages, page, 576), dtype=torch.bfloat16, device="cuda")
    q, kv, qa = normal((64, H, 192), 4), normal((64, H, 256), 5), normal((N, H, 576), 6)
    ws = torch.empty(kda.kda_latent_decode_workspace_bytes(N, 1, H), dtype=torch.uint8, device="cuda")
    out = {}

    def step():
        cu, lens, slots, pos, status = kda.kda_page_tables(ctx, new, free, table, page_size=page, n_pages=pages, max_tokens=64)
        y, _, _ = kda.kda_rms_norm(x, residual=x)
        kda.kda_latent_cache_write(y, w, cache, slots)
        o = kda.kda_latent_prefill(q, kv, y[:, 512:], cu_seqlens_q=cu)
        d = kda.kda_latent_decode(qa, cache, table, lens, workspace=ws)
        out.update(o=o, d=d, lens=lens, slots=slots)
        return out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    captured = dict(out)
    for lens, seed in (([5, 1, 40], 7), ([0, 33, 2], 8), ([20, 20, 20], 9)):
        new.copy_(i32(lens))
        x.copy_(normal((64, 576), seed))
        for t in (cache, captured["o"], captured["d"]):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in captured.items()}
        cache.zero_()
        want = step()
        n = sum(lens)
        assert torch.equal(got["o"][:n], want["o"][:n])   # (rows past the last sequence are not written)
        for k in ("d", "lens", "slots"):
            assert torch.equal(got[k], want[k]), k


def test_prefill_agrees_with_decode(kda):
    """The two forms on the same layer: k = [U c; r], v = W c against q' = [U^T q; q_r] and W applied after."""
    H, n = 4, 90
    c, r = normal((n, 512), 1), normal((n, 64), 2)
    U, W = normal((H, 128, 512), 3, torch.float32, 512 ** -0.5), normal((H, 128, 512), 4, torch.float32, 512 ** -0.5)
    q = normal((n, H, 192), 5)
    kv = torch.cat([torch.einsum("hkc,tc->thk", U, c.float()), torch.einsum("hvc,tc->thv", W, c.float())], -1)
    a = kda.kda_latent_prefill(q, kv.to(torch.bfloat16), r, cu_seqlens_q=i32([0, n]))
    qa = torch.cat([torch.einsum("thk,hkc->thc", q[..., :128].float(), U).to(torch.bfloat16), q[..., 128:]], -1)
    cache = torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda")
    kda.kda_latent_cache_write(torch.cat([c, r], -1), None, cache, torch.arange(n, dtype=torch.int32, device="cuda"))
    b = kda.kda_latent_decode(qa[None], cache, i32([[0, 1]]), i32([n]))[0]
    b = torch.einsum("hvc,thc->thv", W, b.float())
    # both round their operands to bf16: k, v and p here, q' and p there
    assert float((a.float() - b).norm() / b.norm()) < 4 * E_BF16
