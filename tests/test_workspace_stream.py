"""A workspace that a call allocates itself belongs to the stream that the call runs on."""
import contextlib
import types

import pytest
import torch


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Recorder:
    """Stands for the library and the compiled binding: every call is taken."""

    def __init__(self):
        self.calls = []

    def pa_decode_workspace_bytes_for(self, *a):
        return 4096

    def pa_decode_q8_workspace_bytes(self, *a):
        return 4096

    def __getattr__(self, name):
        def call(*a):
            self.calls.append((name, a))
            return 0
        return call


@pytest.mark.parametrize("call", ["pa_decode", "pa_decode_append", "pa_decode_q8"])
@pytest.mark.parametrize("given", ["none", "stream", "handle", "default handle", "wrapper"])
def test_workspace_is_allocated_under_the_launch_stream(monkeypatch, call, given):
    import paged_kv_cache_301_gb300 as pa
    current, side, default = FakeStream(0x10), FakeStream(0x70), FakeStream(0)
    active, allocated = [current], []

    @contextlib.contextmanager
    def under(s):
        active.append(s)
        yield
        active.pop()

    real = torch.empty

    def empty(n, **kw):
        allocated.append((n, active[-1].cuda_stream))
        return real(n, **kw)

    fake = Recorder()
    cuda = types.SimpleNamespace(
        Stream=FakeStream, stream=under, current_stream=lambda *a: active[-1],
        default_stream=lambda *a: default,
        ExternalStream=lambda handle, device=None: FakeStream(handle))
    monkeypatch.setattr(pa, "torch", types.SimpleNamespace(
        cuda=cuda, empty=empty, uint8=torch.uint8, float16=torch.float16))
    monkeypatch.setattr(pa, "lib", lambda: fake)
    monkeypatch.setattr(pa, "_native", fake)
    if given == "wrapper" and call != "pa_decode_q8":
        pytest.skip("the binding alone takes any object with a cuda_stream")
    q, k = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, 4, 64, dtype=torch.float16)
    pool = torch.zeros(6, 16, 4, 64, dtype=torch.float16)
    tables, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    stream = {"none": None, "stream": side, "handle": 0x70, "default handle": 0,
              "wrapper": types.SimpleNamespace(cuda_stream=0x70)}[given]
    want = {"none": 0x10, "default handle": 0}.get(given, 0x70)
    if call == "pa_decode":
        pa.pa_decode(q, q, pool, pool, tables, lens, 0.1, stream=stream)
    elif call == "pa_decode_append":
        pa.pa_decode_append(q, q, pool, pool, k, k, tables, lens, 0.1, stream=stream)
    else:
        pa.pa_decode_q8(q, q, pool, pool, lens, lens, tables, lens, 0.1, stream=stream)
    assert allocated == [(4096, want)]
    assert len(fake.calls) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["pa_decode", "pa_decode_append", "pa_decode_q8"])
@pytest.mark.parametrize("raw", [False, True])
def test_memory_of_a_running_call_is_not_handed_out(call, raw):
    """A call on a busy side stream without a workspace; meanwhile the current stream
    allocates and fills as much as it likes."""
    from tests.gpu_helpers import i32, lib
    pa = lib()
    B, H, G, D, bs, n = 2, 2, 4, 128, 16, 6000
    g = torch.Generator("cuda").manual_seed(2)
    NB = B * n // bs
    tables = torch.randperm(NB, generator=g, device="cuda").to(torch.int32).view(B, -1)
    lens = i32([n, n - 7])
    q = torch.randn(B, H * G, D, generator=g, device="cuda").to(torch.bfloat16)
    if call == "pa_decode_q8":
        pools = pa.alloc_cache_q8(NB, H, bs, D)
        for p in pools[:2]:
            p.copy_(torch.randn(NB, H, bs, D, generator=g, device="cuda").to(pa.E4M3))
        more = ()
        size = pa.workspace_for_q8(q, pools[0], n).numel()
    else:
        pools = [torch.randn(NB, bs, H, D, generator=g, device="cuda").to(torch.bfloat16)
                 for _ in "kv"]
        more = [torch.randn(B, H, D, generator=g, device="cuda").to(torch.bfloat16)
                for _ in "kv"] if call == "pa_decode_append" else ()
        size = pa.workspace_for(q, *pools[:1], tables, n).numel()
    f = getattr(pa, call)

    def run(out, **kw):
        return f(out, q, *pools, *more, tables, lens, D ** -0.5, max_seq_len=n, **kw)

    want = run(torch.empty_like(q), workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)              # about 10 ms
    run(out, stream=side.cuda_stream if raw else side)
    held = []
    for _ in range(50):
        held.append(torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert all(bool((t == 0xFF).all()) for t in held)
