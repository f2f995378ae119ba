"""Refusals of the linear-attention layer with one decay a head and of the head
norm and rotation (include/kda_linear.h), on the host: nothing here launches a
kernel."""
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


def _rope(lib, sections=None, **kw):
    import ctypes
    order = ("q", "sq", "k", "sk", "wq", "wk", "eps", "norm", "pos", "sections", "axes", "freq", "off", "rot", "inter",
             "oq", "soq", "ok", "sok", "T", "Hq", "Hk", "D", "dtype", "stream")
    d = {n: BASE + 4096 * i for i, n in enumerate(order)}
    d.update(sq=1024, sk=256, soq=1024, sok=256, eps=1e-6, norm=1, axes=1, off=0, rot=128, inter=0, T=5, Hq=8, Hk=2,
             D=128, dtype=kda.KDA_BF16, stream=None,
             sections=None if sections is None else (ctypes.c_int * len(sections))(*sections))
    return _call(lib.kda_head_norm_rope, order, d, kw)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(T=-1), dict(T=1 << 31), dict(Hq=0), dict(Hk=-1), dict(D=0), dict(D=120), dict(rot=-16),
    dict(rot=24), dict(rot=144), dict(off=-8), dict(off=8), dict(off=4, rot=64), dict(off=72, rot=64),
    dict(eps=float("nan")), dict(eps=-1.0), dict(axes=0), dict(axes=5, sections=[16] * 4), dict(axes=2), dict(pos=None),
    dict(freq=None), dict(sq=1016), dict(sq=1028), dict(soq=1016), dict(sk=248), dict(sok=248), dict(q=None),
    dict(oq=None), dict(k=None), dict(ok=None), dict(q=BASE + 8), dict(oq=BASE + 8), dict(k=BASE + 8), dict(ok=BASE + 8),
    dict(wq=BASE + 8), dict(wk=BASE + 4), dict(pos=BASE + 2), dict(freq=BASE + 2),
    dict(q=BASE, oq=BASE, soq=2048), dict(k=BASE, ok=BASE, sok=512),
    dict(axes=3, sections=[32, 16, 8]), dict(axes=3, sections=[80, -16, 0]), dict(axes=2, sections=[1 << 30, 1 << 30]),
    dict(axes=1, sections=[63])])
def test_rope_refuses(lib, kw):
    assert _rope(lib, **kw) == INVALID


def test_rope_limits(lib):
    assert _rope(lib, D=272, sq=8 * 272, soq=8 * 272, sk=2 * 272, sok=2 * 272, rot=0) == UNSUPPORTED
    assert _rope(lib, Hq=65536, sq=65536 * 128, soq=65536 * 128) == UNSUPPORTED
    assert _rope(lib, T=1 << 28) == UNSUPPORTED
    # nothing to do: no pointer is looked at
    assert _rope(lib, T=0, q=None, k=None, oq=None, ok=None) == OK
    assert _rope(lib, T=0, rot=0, pos=None, freq=None) == OK


LAYER = ("q", "sq", "k", "sk", "v", "sv", "g", "sg")


def _chunk(lib, **kw):
    order = LAYER + ("s0", "sf", "idx", "slots", "o", "cu", "N", "T", "H", "Hk", "K", "V", "scale", "dtype", "ws",
                     "ws_bytes", "stream")
    d = {n: BASE + 4096 * i for i, n in enumerate(order)}
    d.update(sq=256, sk=256, sv=1024, sg=8, slots=4, N=2, T=64, H=8, Hk=2, K=128, V=128, scale=1.0, dtype=kda.KDA_BF16,
             ws=None, ws_bytes=0, stream=None)
    return _call(lib.kda_linear_chunk_fwd, order, d, kw)


BAD_LAYER = [dict(H=0), dict(Hk=0), dict(Hk=3), dict(H=-8), dict(K=0), dict(V=-1), dict(dtype=2),
             dict(scale=float("inf")), dict(scale=float("nan")), dict(sq=248), dict(sq=260), dict(sk=128), dict(sv=1016),
             dict(sg=7), dict(sg=-1), dict(slots=-1), dict(q=None), dict(k=None), dict(v=None), dict(g=None),
             dict(o=None), dict(q=BASE + 8), dict(k=BASE + 2), dict(v=BASE + 8), dict(o=BASE + 8), dict(g=BASE + 2),
             dict(idx=BASE + 1)]


@pytest.mark.parametrize("kw", BAD_LAYER + [dict(N=0), dict(N=-1), dict(T=-1), dict(T=1 << 31), dict(s0=BASE + 8),
                                            dict(sf=BASE + 4), dict(cu=BASE + 2), dict(cu=None, N=3)])
def test_chunk_refuses(lib, kw):
    assert _chunk(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(K=64), dict(V=256), dict(N=65536), dict(H=65536, Hk=2, sv=65536 * 128, sg=0),
                                dict(T=(1 << 31) - 1, H=128, Hk=2, sv=16384, sg=128)])
def test_chunk_limits(lib, kw):
    assert _chunk(lib, **kw) == UNSUPPORTED


def test_chunk_workspace(lib):
    size = kda.kda_linear_chunk_workspace_bytes
    assert size(-1, 1, 8) == size(1 << 31, 1, 8) == size(64, 0, 8) == size(64, 65536, 8) == size(64, 1, 0) == 0
    assert size(1 << 20, 1, 8, 2) == 0


def _step(lib, **kw):
    order = LAYER + ("pool", "idx", "slots", "o", "N", "H", "Hk", "K", "V", "scale", "dtype", "stream")
    d = {n: BASE + 4096 * i for i, n in enumerate(order)}
    d.update(sq=256, sk=256, sv=1024, sg=8, slots=4, N=2, H=8, Hk=2, K=128, V=128, scale=1.0, dtype=kda.KDA_BF16,
             stream=None)
    return _call(lib.kda_linear_step, order, d, kw)


@pytest.mark.parametrize("kw", BAD_LAYER + [dict(N=-1), dict(pool=None), dict(pool=BASE + 8), dict(idx=None, slots=1)])
def test_step_refuses(lib, kw):
    assert _step(lib, **kw) == INVALID


def test_step_limits(lib):
    assert _step(lib, K=64) == UNSUPPORTED
    assert _step(lib, N=1 << 29) == UNSUPPORTED
    assert _step(lib, N=0, q=None, k=None, v=None, g=None, pool=None, o=None) == OK


def _multi(lib, **kw):
    order = LAYER + ("pool", "idx", "acc", "slots", "o", "N", "S", "H", "Hk", "K", "V", "scale", "dtype", "stream")
    d = {n: BASE + 4096 * i for i, n in enumerate(order)}
    d.update(sq=256, sk=256, sv=1024, sg=8, slots=4, N=2, S=3, H=8, Hk=2, K=128, V=128, scale=1.0, dtype=kda.KDA_BF16,
             stream=None)
    return _call(lib.kda_linear_multi_step, order, d, kw)


@pytest.mark.parametrize("kw", BAD_LAYER + [dict(N=-1), dict(S=0), dict(pool=None), dict(idx=None), dict(acc=BASE + 2),
                                            dict(N=1 << 20, S=1 << 20)])
def test_multi_step_refuses(lib, kw):
    assert _multi(lib, **kw) == INVALID


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_host_tensors(lib):
    f32 = torch.float32
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_head_norm_rope(_cpu(4, 2, 128))
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_linear_chunk_fwd(_cpu(4, 2, 128), _cpu(4, 2, 128), _cpu(4, 2, 128), _cpu(4, 2, dtype=f32))
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_linear_step(_cpu(4, 2, 128), _cpu(4, 2, 128), _cpu(4, 2, 128), _cpu(4, 2, dtype=f32),
                            _cpu(4, 2, 128, 128, dtype=f32))
    with pytest.raises(ValueError, match="state_indices"):
        kda.kda_linear_multi_step(_cpu(4, 1, 2, 128), _cpu(4, 1, 2, 128), _cpu(4, 1, 2, 128), _cpu(4, 1, 2, dtype=f32),
                                  _cpu(4, 2, 128, 128, dtype=f32), None)
