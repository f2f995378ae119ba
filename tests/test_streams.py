"""Memory that a call on a given stream allocates: that stream's own, so that neither what is still running on the
current stream nor what comes next there shares it with the call."""
import contextlib

import pytest
import torch

import kimi_delta_attention_07_gb300 as kda

# ---- on the host, with a torch allocator and streams that note what is asked of them ----


class Tensor:
    is_cuda = True

    def __init__(self, shape, dtype, on=None):
        self.shape = torch.Size((shape,) if isinstance(shape, int) else shape)
        self.dtype, self.on, self.device, self.recorded = dtype, on, torch.device("cuda", 0), []

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return tuple(self.shape[i + 1:].numel() for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, stream):
        self.recorded.append(stream)


def t(*shape, dtype=torch.bfloat16):
    return Tensor(shape, dtype)


def i32(*shape):
    return Tensor(shape, torch.int32)


def f32(*shape):
    return Tensor(shape, torch.float32)


CALLS = {
    "page_tables": lambda s: kda.kda_page_tables(i32(2), i32(2), i32(8), i32(2, 4), page_size=64, n_pages=16, max_tokens=8, stream=s),
    "rms_norm": lambda s: kda.kda_rms_norm(t(4, 256), residual=t(4, 256), quant="block", stream=s),
    "decode": lambda s: kda.kda_latent_decode(t(2, 4, 576), t(8, 16, 576), i32(2, 4), i32(2), stream=s),
    "prefill": lambda s: kda.kda_latent_prefill(t(6, 2, 192), t(2000, 2, 256), t(2000, 64), cu_seqlens_q=i32(3), cu_seqlens_k=i32(3),
                                                stream=s),
    "chunk_fwd": lambda s: kda.kda_chunk_fwd(t(9, 4, 128), t(9, 4, 128), t(9, 4, 128), f32(9, 4, 128), f32(9, 4), stream=s),
    "recurrent_step": lambda s: kda.kda_recurrent_step(t(2, 4, 128), t(2, 4, 128), t(2, 4, 128), f32(2, 4, 128), f32(2, 4),
                                                       f32(2, 4, 128, 128), stream=s),
    "recurrent_multi_step": lambda s: kda.kda_recurrent_multi_step(
        t(2, 3, 4, 128), t(2, 3, 4, 128), t(2, 3, 4, 128), f32(2, 3, 4, 128), f32(2, 3, 4), f32(6, 4, 128, 128), i32(2, 3), stream=s),
    "short_conv_fwd": lambda s: kda.kda_short_conv_fwd(t(9, 64), t(4, 64), stream=s),
    "short_conv_update": lambda s: kda.kda_short_conv_update(t(2, 64), t(4, 64), t(2, 3, 64), stream=s),
    "short_conv_multi_update": lambda s: kda.kda_short_conv_multi_update(t(2, 3, 64), t(4, 64), t(6, 3, 64), i32(2, 3), stream=s),
}


class Library:
    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("workspace_bytes") else 0


class Stream:
    cuda_stream = 77


@pytest.mark.parametrize("name", sorted(CALLS))
def test_allocations_are_the_given_streams_own(monkeypatch, name):
    from kimi_delta_attention_07_gb300 import _hybrid
    current, side, made, plain = ["current"], Stream(), [], torch.empty

    @contextlib.contextmanager
    def stream_context(s):
        before, current[0] = current[0], s
        yield
        current[0] = before

    def empty(shape, dtype=None, device=None):
        if getattr(device, "type", None) != "cuda":
            return plain(shape, dtype=dtype, device=device)
        made.append(Tensor(shape, dtype, current[0]))
        return made[-1]

    monkeypatch.setattr(_hybrid, "_lib", Library())
    monkeypatch.setattr(kda, "load", lambda: Library())
    for module in (kda, _hybrid):
        monkeypatch.setattr(module, "_current_device", lambda: 0)
    monkeypatch.setattr(_hybrid, "_current_stream", lambda dev: 0)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda x: empty(x.shape, x.dtype, x.device))
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[0])

    out = CALLS[name](side)
    returned = [x for x in (out if isinstance(out, tuple) else (out,)) if x in made]
    assert returned and made and all(x.on is side for x in made)
    assert all(x.recorded == ["current"] for x in returned)


# ---- on the GPU ----------------------------------------------------------------------


SLEEP = 40_000_000  # clocks, about 20 ms


def gpu_cases():
    def n(*shape, seed=0, dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    def i(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    x, r = n(300, 512, seed=1), n(300, 512, seed=2)
    q, cache = n(1, 32, 576, seed=3), n(80, 64, 576, seed=4)
    table, lens = torch.arange(80, dtype=torch.int32, device="cuda")[None], i(5000)
    pq, kv, rope, cq, ck = n(90, 2, 192, seed=5), n(3000, 2, 256, seed=6), n(3000, 64, seed=7), i(0, 90), i(0, 3000)
    k = [n(200, 4, 128, seed=s) for s in (8, 9, 10)]
    g, beta = -n(200, 4, 128, seed=11, dtype=torch.float32).abs() * 0.1, n(200, 4, seed=12, dtype=torch.float32).sigmoid()
    return {
        "rms_norm": lambda s: kda.kda_rms_norm(x, residual=r, stream=s)[:2],
        "decode": lambda s: (kda.kda_latent_decode(q, cache, table, lens, stream=s),),
        "prefill": lambda s: (kda.kda_latent_prefill(pq, kv, rope, cu_seqlens_q=cq, cu_seqlens_k=ck, stream=s),),
        "chunk_fwd": lambda s: kda.kda_chunk_fwd(*k, g, beta, stream=s),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["rms_norm", "decode", "prefill", "chunk_fwd"])
def test_work_of_the_current_stream_does_not_reach_a_call_on_another(name):
    kda.load()
    call = gpu_cases()[name]
    want = [v.clone() for v in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # memory that is freed while the current stream has yet to write it
    torch.cuda._sleep(SLEEP)
    held = [torch.empty_like(v).fill_(7) for v in want for _ in range(3)]
    del held
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del got
    # memory (a workspace among it) that the call gave back before it ran
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    got = call(side)
    held = [torch.full((64 << 20 >> k,), 255, dtype=torch.uint8, device="cuda") for k in range(0, 20) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del held


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["rms_norm", "decode", "prefill", "chunk_fwd"])
def test_a_call_on_a_stream_of_a_captured_graph(name):
    kda.load()
    call = gpu_cases()[name]
    want = [v.clone() for v in call(None)]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        after = [v * 1 for v in got]
    for _ in range(2):
        for v in (*got, *after):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(after, want)) and all(torch.equal(a, b) for a, b in zip(got, want))
