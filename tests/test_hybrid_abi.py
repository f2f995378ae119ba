"""Refusals of the operators around the core (include/kda_hybrid.h) and of
their binding, on the host: nothing here launches a kernel."""
import ctypes

import pytest
import torch

import kimi_delta_attention_07_gb300 as kda

BASE = 1 << 20  # a fake, never dereferenced address
INVALID, UNSUPPORTED, WORKSPACE, OK = (kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED,
                                       kda.KDA_ERR_WORKSPACE, kda.KDA_OK)


@pytest.fixture(scope="module")
def lib():
    from kimi_delta_attention_07_gb300 import _build
    _build.build()
    return kda.load()


def _call(fn, order, defaults, kw):
    a = {**defaults, **kw}
    assert set(a) == set(order)
    return fn(*[a[k] for k in order])


def _tables(lib, **kw):
    order = ("ctx", "new", "free", "n_free", "start", "table", "cu", "lens", "slots", "pos", "status", "n",
             "tokens", "max_pages", "page", "n_pages", "stream")
    d = {k: BASE + 256 * i for i, k in enumerate(order)}
    d.update(n_free=8, start=None, n=2, tokens=8, max_pages=4, page=64, n_pages=16, stream=None)
    return _call(lib.kda_page_tables, order, d, kw)


@pytest.mark.parametrize("kw", [dict(page=0), dict(page=8), dict(page=48), dict(page=512), dict(n=-1),
                                dict(tokens=-1), dict(tokens=1 << 31), dict(n_free=-1), dict(max_pages=0),
                                dict(n_pages=0), dict(n_pages=1 << 25), dict(ctx=None), dict(new=None),
                                dict(free=None), dict(table=None), dict(cu=None), dict(lens=None),
                                dict(slots=None), dict(pos=None), dict(status=None), dict(ctx=BASE + 2)])
def test_page_tables_refuses(lib, kw):
    assert _tables(lib, **kw) == INVALID


@pytest.mark.parametrize("which", ["ctx", "new", "free", "start"])
@pytest.mark.parametrize("out", ["cu", "lens", "slots", "pos", "status", "table"])
def test_page_tables_refuses_an_output_that_is_an_input(lib, which, out):
    assert _tables(lib, **{which: BASE + 1024 * 1024, out: BASE + 1024 * 1024}) == INVALID


@pytest.mark.parametrize("kw", [
    dict(ctx=BASE, lens=BASE + 4), dict(lens=BASE, ctx=BASE + 4),                      # one entry apart, two requests
    dict(new=BASE, cu=BASE + 4), dict(cu=BASE, new=BASE + 8),                          # offsets hold one entry more
    dict(free=BASE, slots=BASE + 28), dict(pos=BASE, free=BASE + 28),                  # the last of eight
    dict(start=BASE + 4, status=BASE), dict(table=BASE, start=BASE + 28),
    dict(table=BASE, slots=BASE + 16), dict(pos=BASE, table=BASE + 28), dict(table=BASE, status=BASE - 4)])
def test_page_tables_refuses_an_output_that_shares_memory_with_an_input(lib, kw):
    assert _tables(lib, **{k: v + 1024 * 1024 for k, v in kw.items()}) == INVALID


def test_page_tables_refuses_too_many_requests(lib):
    assert _tables(lib, n=16385) == UNSUPPORTED


def _norm(lib, **kw):
    order = ("x", "res", "w", "y", "scales", "out", "eps", "rows", "D", "quant", "dtype", "stream")
    d = dict.fromkeys(order, BASE)
    d.update(eps=1e-6, rows=4, D=256, quant=0, dtype=kda.KDA_BF16, stream=None)
    return _call(lib.kda_rms_norm, order, d, kw)


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(quant=3), dict(quant=-1), dict(rows=-1), dict(D=0),
                                dict(D=12), dict(D=136, quant=2), dict(eps=float("nan")), dict(eps=-1.0),
                                dict(x=None), dict(y=None), dict(quant=1, scales=None), dict(x=BASE + 8),
                                dict(res=BASE + 8), dict(out=BASE + 8), dict(w=BASE + 8), dict(y=BASE + 8),
                                dict(y=BASE + 4, quant=1)])
def test_rms_norm_refuses(lib, kw):
    assert _norm(lib, **kw) == INVALID


def test_rms_norm_other_statuses(lib):
    assert _norm(lib, D=32776) == UNSUPPORTED
    assert _norm(lib, rows=0) == OK


def _write(lib, **kw):
    order = ("kv", "stride", "w", "eps", "cache", "slots", "T", "n_pages", "page", "stream")
    d = dict.fromkeys(order, BASE)
    d.update(stride=576, eps=1e-6, T=4, n_pages=4, page=64, stream=None)
    return _call(lib.kda_latent_cache_write, order, d, kw)


@pytest.mark.parametrize("kw", [dict(stride=568), dict(stride=580), dict(T=-1), dict(page=24), dict(n_pages=0),
                                dict(kv=None), dict(cache=None), dict(slots=None), dict(kv=BASE + 8),
                                dict(cache=BASE + 8), dict(w=BASE + 4), dict(eps=float("inf"))])
def test_cache_write_refuses(lib, kw):
    assert _write(lib, **kw) == INVALID


def test_cache_write_nothing_to_do(lib):
    assert _write(lib, T=0) == OK


def _decode(lib, **kw):
    order = ("q", "cache", "table", "lens", "o", "lse", "n", "S", "H", "n_pages", "page", "max_pages", "scale",
             "ws", "wsb", "stream")
    d = dict.fromkeys(order, BASE)
    d.update(lse=None, n=2, S=1, H=4, n_pages=8, page=64, max_pages=4, scale=0.1, wsb=1 << 30, stream=None)
    return _call(lib.kda_latent_decode, order, d, kw)


@pytest.mark.parametrize("kw", [dict(n=-1), dict(S=0), dict(H=0), dict(max_pages=0), dict(page=100),
                                dict(n_pages=0), dict(scale=float("nan")), dict(q=None), dict(cache=None),
                                dict(table=None), dict(lens=None), dict(o=None), dict(q=BASE + 8),
                                dict(cache=BASE + 8), dict(o=BASE + 8), dict(lse=BASE + 2)])
def test_decode_refuses(lib, kw):
    assert _decode(lib, **kw) == INVALID


def test_decode_other_statuses(lib):
    assert _decode(lib, S=64, H=128) == UNSUPPORTED
    assert _decode(lib, n=65536) == UNSUPPORTED
    assert _decode(lib, n=1 << 10, page=256, max_pages=1 << 18) == UNSUPPORTED
    assert _decode(lib, ws=None) == WORKSPACE
    assert _decode(lib, ws=BASE + 16) == WORKSPACE
    assert _decode(lib, wsb=0) == WORKSPACE
    assert _decode(lib, n=0) == OK
    f = kda.kda_latent_decode_workspace_bytes
    assert f(4, 1, 32) > 0 and f(-1, 1, 1) == 0 and f(1, 0, 1) == 0 and f(1, 64, 128) == 0
    assert _decode(lib, wsb=f(2, 1, 4) - 1) == WORKSPACE


def _prefill(lib, **kw):
    order = ("q", "sq", "kv", "sk", "rope", "sr", "o", "lse", "cq", "ck", "n", "Tq", "Tk", "H", "causal", "scale",
             "ws", "ws_bytes", "stream")
    d = dict.fromkeys(order, BASE)
    d.update(ws=None, ws_bytes=0, sq=768, sk=1024, sr=64, lse=None, n=2, Tq=16, Tk=32, H=4, causal=1, scale=0.1, stream=None)
    return _call(lib.kda_latent_prefill, order, d, kw)


@pytest.mark.parametrize("kw", [dict(n=0), dict(H=0), dict(Tq=-1), dict(Tk=-1), dict(scale=float("inf")),
                                dict(sq=760), dict(sq=772), dict(sk=1016), dict(sr=56), dict(sr=66),
                                dict(q=None), dict(kv=None), dict(rope=None), dict(o=None), dict(cq=None),
                                dict(ck=None), dict(q=BASE + 8), dict(kv=BASE + 8), dict(rope=BASE + 8),
                                dict(o=BASE + 8), dict(lse=BASE + 1)])
def test_prefill_refuses(lib, kw):
    assert _prefill(lib, **kw) == INVALID


def test_prefill_unsupported(lib):
    wide = dict(sq=192 * 65535, sk=256 * 65535)
    assert _prefill(lib, H=65536, sq=192 * 65536, sk=256 * 65536) == UNSUPPORTED
    assert _prefill(lib, n=65536) == UNSUPPORTED
    # more blocks of queries and heads than a grid has
    assert _prefill(lib, Tq=(1 << 31) - 1, n=1, H=65535, **wide) == UNSUPPORTED
    assert _prefill(lib, Tq=40000, n=40000, H=65535, **wide) == UNSUPPORTED


def test_prefill_workspace(lib):
    # few queries behind many keys: the keys are split; enough queries, or few keys: they are not
    need = kda.kda_latent_prefill_workspace_bytes(1, 64, 65536, 4)
    assert need > 4 * 64 * 132 * 4
    assert kda.kda_latent_prefill_workspace_bytes(1, 64, kda.KDA_LATENT_PREFILL_SPLIT_KEYS - 1, 4) == 0
    assert kda.kda_latent_prefill_workspace_bytes(1, 65536, 65536, 32) == 0
    for bad in ((0, 64, 65536, 4), (1, -1, 65536, 4), (1, 64, -1, 4), (1, 64, 65536, 0), (1, 64, 65536, 65536)):
        assert kda.kda_latent_prefill_workspace_bytes(*bad) == 0
    few = dict(n=1, Tq=64, Tk=65536)
    for ws, size in ((None, need), (BASE, need - 1), (BASE + 128, need)):
        assert _prefill(lib, ws=ws, ws_bytes=size, **few) == WORKSPACE


def test_prefill_needs_no_workspace_below_the_documented_number_of_keys(lib):
    below = kda.KDA_LATENT_PREFILL_SPLIT_KEYS - 1
    for n in (1, 2, 3, 8):
        for tq in (1, 64, 256, 257, 1024):
            for H in (*range(1, 34), 64, 100, 128, 149, 150, 153, 200, 300, 305):
                assert all(kda.kda_latent_prefill_workspace_bytes(n, tq, tk, H) == 0 for tk in (0, 1, 500, 896, 897, 960, below))


def test_prefill_nothing_to_do(lib):
    assert _prefill(lib, Tq=0) == OK
    assert _prefill(lib, Tq=0, ck=None, Tk=0) == OK


def test_binding_refuses_host_tensors(lib):
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kda_page_tables(i, i, i, t, page_size=64, n_pages=4, max_tokens=8)
    b = torch.zeros((2, 576), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kda.kda_rms_norm(b)
    with pytest.raises(ValueError):
        kda.kda_latent_cache_write(b, None, torch.zeros((1, 16, 576), dtype=torch.bfloat16), i)
    with pytest.raises(ValueError):
        kda.kda_latent_decode(b[:, None], torch.zeros((1, 16, 576), dtype=torch.bfloat16), t, i)
    with pytest.raises(ValueError):
        kda.kda_latent_prefill(b[:, None, :192], b[:, None, :256], b[:, :64], cu_seqlens_q=i)


class Fake:
    """Stands for a CUDA tensor (default: an aligned address on device 1)."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.bfloat16, dev=1):
        self.shape, self.dtype, self.dev, self.device = torch.Size(shape), dtype, dev, torch.device("cuda", dev)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return BASE


def ints(*shape):
    return Fake(*shape, dtype=torch.int32)


def calls_on_fakes():
    """One call of each entry point, with every output given."""
    return {
        "page_tables": lambda: kda.kda_page_tables(
            ints(2), ints(2), ints(8), ints(2, 4), page_size=64, n_pages=16, cu_seqlens=ints(3), seq_lens=ints(2),
            slots=ints(8), positions=ints(8), status=ints(2)),
        "rms_norm": lambda: kda.kda_rms_norm(Fake(4, 256), y=Fake(4, 256)),
        "cache_write": lambda: kda.kda_latent_cache_write(Fake(2, 576), None, Fake(1, 16, 576), ints(2)),
        "decode": lambda: kda.kda_latent_decode(Fake(2, 4, 576), Fake(8, 16, 576), ints(2, 4), ints(2), o=Fake(2, 4, 512),
                                                workspace=Fake(1 << 28, dtype=torch.uint8)),
        "prefill": lambda: kda.kda_latent_prefill(Fake(6, 2, 192), Fake(6, 2, 256), Fake(6, 64), cu_seqlens_q=ints(3),
                                                  o=Fake(6, 2, 128)),
        "recurrent_step": lambda: kda.kda_recurrent_step(
            Fake(2, 4, 128), Fake(2, 4, 128), Fake(2, 4, 128), Fake(2, 4, 128, dtype=torch.float32),
            Fake(2, 4, dtype=torch.float32), Fake(2, 4, 128, 128, dtype=torch.float32), o=Fake(2, 4, 128)),
        "output_gate_norm": lambda: kda.kda_output_gate_norm(Fake(3, 128), Fake(3, 128), Fake(128, dtype=torch.float32)),
    }


class FakeLibrary:
    def __init__(self):
        self.launched = []

    def __getattr__(self, name):
        return lambda *a: self.launched.append(name) or 0


@pytest.fixture
def fake_library(monkeypatch):
    """Device 0 is current, every call of the library succeeds and is noted."""
    from kimi_delta_attention_07_gb300 import _hybrid
    library = FakeLibrary()
    monkeypatch.setattr(_hybrid, "_lib", library)
    monkeypatch.setattr(kda, "load", lambda: library)
    for module in (kda, _hybrid):
        monkeypatch.setattr(module, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(_hybrid, "_current_stream", lambda dev: 0)
    monkeypatch.setattr(kda, "_stream", lambda stream: 0)
    return library


@pytest.mark.parametrize("name", sorted(calls_on_fakes()))
def test_binding_refuses_tensors_of_another_device_than_the_current_one(fake_library, name):
    with pytest.raises(ValueError, match="current device"):
        calls_on_fakes()[name]()
    assert not fake_library.launched
    kda._current_device = kda._hybrid._current_device = lambda: 1     # (put back by the fixture)
    calls_on_fakes()[name]()
    assert fake_library.launched


def test_every_entry_point_of_the_header_has_argument_types(lib):
    for name in ("kda_page_tables", "kda_rms_norm", "kda_latent_cache_write", "kda_latent_decode", "kda_latent_prefill"):
        fn = getattr(lib, name)
        assert fn.argtypes and fn.restype is ctypes.c_int
