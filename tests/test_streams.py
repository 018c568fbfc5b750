"""Tensors that the binding allocates belong to the stream of the call: memory that torch's
caching allocator hands out for another stream may still be in use by that stream's work, and
is handed out again while this call's kernels use it.  On the CPU, with every allocation
and the stream of every call recorded."""
import contextlib

import pytest
import torch

from gated_delta_rule_35_amd import binding

HERE = 11   # handle of the current stream


class FakeStream:
    def __init__(self, handle=55, index=0):
        self.cuda_stream, self.device = handle, torch.device("cuda", index)


class OnGpu:
    """A tensor's host-side view that says it lies on GPU 0 and records what it allocates."""
    is_cuda, device = True, torch.device("cuda", 0)
    allocated = None   # the handles that were current when something was allocated

    def __init__(self, x):
        self.x = x

    def get_device(self):
        return 0

    def new_empty(self, shape, dtype=None):
        return made(torch.empty(shape, dtype=dtype or self.x.dtype))

    def __getattr__(self, name):
        return getattr(self.x, name)


def made(x):
    OnGpu.allocated.append(OnGpu.current[-1])
    return OnGpu(x)


@pytest.fixture
def calls(monkeypatch):
    """The stream handles that the library was called with."""
    seen = []
    OnGpu.allocated, OnGpu.current = [], [HERE]
    real_empty, real_like = torch.empty, torch.empty_like

    @contextlib.contextmanager
    def on(stream):
        OnGpu.current.append(stream.cuda_stream)
        yield
        OnGpu.current.pop()

    def empty(*a, device=None, **kw):
        x = real_empty(*a, **kw)
        return made(x) if device is not None else x

    def empty_like(like, **kw):
        return made(real_like(like.x, **kw)) if isinstance(like, OnGpu) else real_like(like, **kw)

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 4096
            return lambda *a: seen.append(a[-1].value or 0) or 0   # c_void_p(0).value is None

    def call(entry, dev, stream, workspace, scalars, tensors):
        seen.append(stream)
        return 0

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: FakeStream(HERE))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: OnGpu.current[-1], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", empty_like)
    monkeypatch.setattr(binding, "load_library", lambda path=None: Lib())
    monkeypatch.setattr(binding, "_call_entry", call)
    return seen


def inputs(channels=False):
    b = lambda *s: OnGpu(torch.zeros(*s, dtype=torch.bfloat16))  # noqa: E731
    f = lambda *s: OnGpu(torch.zeros(*s))  # noqa: E731
    g = f(1, 8, 2, 128) if channels else f(1, 8, 2)
    return [b(1, 8, 1, 128), b(1, 8, 1, 128), b(1, 8, 2, 128), g, f(1, 8, 2)], b, f


def gdr_fwd(stream):
    x, b, f = inputs()
    binding.kda_gdr_fwd(*x, 1.0, final_state=True, stream=stream)


def gdr_bwd(stream):
    x, b, f = inputs()
    binding.kda_gdr_bwd(*x, 1.0, b(1, 8, 2, 128), d_initial_state=True, stream=stream)


def gdr_decode(stream):
    x, b, f = inputs()
    binding.kda_gdr_decode(b(8, 1, 128), b(8, 1, 128), b(8, 2, 128), f(8, 2), f(8, 2), 1.0, None, stream=stream)


def qk_norm(stream):
    x, b, f = inputs()
    binding.kda_qk_norm(x[0], x[1], stream=stream)


def qk_norm_bwd(stream):
    x, b, f = inputs()
    binding.kda_qk_norm_bwd(x[0], x[1], x[0], x[1], q_weight=f(128), k_weight=f(128), stream=stream)


PER_HEAD = [gdr_fwd, gdr_bwd, gdr_decode, qk_norm, qk_norm_bwd]
STREAMS = [77, 0, "stream", None]


def check_allocations(calls, call, stream):
    s = FakeStream(55) if stream == "stream" else stream
    call(s)
    want = HERE if s is None else getattr(s, "cuda_stream", s)
    assert calls == [want]
    assert len(OnGpu.allocated) >= 2 and set(OnGpu.allocated) == {want}
    assert OnGpu.current == [HERE]


@pytest.mark.parametrize("call", PER_HEAD)
@pytest.mark.parametrize("stream", STREAMS)
def test_allocations_belong_to_the_stream_of_the_call(calls, call, stream):
    check_allocations(calls, call, stream)


@pytest.mark.parametrize("call", PER_HEAD)
def test_a_stream_of_another_device_is_refused(calls, call):
    with pytest.raises(ValueError):
        call(FakeStream(55, index=1))
    assert calls == [] and OnGpu.allocated == []


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["stream", "handle"])
def test_unfinished_calls_on_two_streams_share_nothing(how, monkeypatch):
    """A call on the current stream, which is kept busy, and calls on another one meanwhile, on
    inputs of their own: no workspace or output of theirs overlaps one that an unfinished call
    on the other stream uses, and every result is what the call gives alone."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from tests import gdr_ref as ref
    print(f"[gpu] kda_gdr_fwd, kda_gdr_bwd, kda_qk_norm_bwd on two streams, {how}", flush=True)
    real, used = binding._load_caller(), []

    def call(entry, dev, stream, workspace, scalars, tensors):
        keep = [t for t in (workspace,) if t is not None]
        used.append((stream, [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in keep]))
        return real(entry, dev, stream, workspace, scalars, tensors)

    monkeypatch.setattr(binding, "_call_entry", call)
    w = torch.rand(128, device="cuda") + 0.5

    def steps(x, do, stream):
        a = (x["q"], x["k"], x["v"], x["g"], x["beta"], 128 ** -0.5)
        o, hT = binding.kda_gdr_fwd(*a, initial_state=x["h0"], final_state=True, stream=stream)
        d = binding.kda_gdr_bwd(*a, do, initial_state=x["h0"], d_initial_state=True, stream=stream)
        n = binding.kda_qk_norm_bwd(x["q"], x["k"], x["k"], x["q"], q_weight=w, k_weight=w, stream=stream)
        return [o, hT] + [d[m] for m in sorted(d)] + [n[m] for m in sorted(n)]

    data = []
    for seed in range(4):
        x = ref.cuda(ref.make(1, 300, 2, 4, h0=True, seed=seed))
        data.append((x, torch.randn(x["v"].shape, device="cuda").bfloat16()))
    torch.cuda.synchronize()
    want = [[t.clone() for t in steps(x, do, None)] for x, do in data]
    torch.cuda.synchronize()
    used.clear()
    s = torch.cuda.Stream()
    other = s if how == "stream" else s.cuda_stream
    torch.cuda._sleep(100_000_000)   # the current stream is busy: its calls below are not finished
    got = []
    for i, (x, do) in enumerate(data):
        got.append(steps(x, do, other if i % 2 else None))
    torch.cuda.synchronize()
    assert {h for h, _ in used} == {s.cuda_stream, torch.cuda.current_stream().cuda_stream} and len(used) == 12
    for h, spans in used:
        for h2, others in used:
            if h != h2:
                assert all(a >= f or e >= b for a, b in spans for e, f in others)
    for g, r in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, r))


def fwd(name, **kw):
    def call(stream):
        x, b, f = inputs(channels=True)
        getattr(binding, name)(*x, 1.0, final_state=True, stream=stream, **kw)
    call.__name__ = name
    return call


def fwd_trace(stream):
    x, b, f = inputs(channels=True)
    binding.kda_fwd_trace(*x, 1.0, {}, final_state=True, stream=stream)


def bwd(stream):
    x, b, f = inputs(channels=True)
    binding.kda_bwd(*x, 1.0, b(1, 8, 2, 128), d_initial_state=True, stream=stream)


def decode(stream):
    x, b, f = inputs(channels=True)
    binding.kda_decode(b(8, 1, 128), b(8, 1, 128), b(8, 2, 128), f(8, 2, 128), f(8, 2), 1.0, None, stream=stream)


PER_CHANNEL = [fwd(n) for n in ("kda_fwd", "kda_fwd_fused", "kda_fwd_ws", "kda_fwd_qg", "kda_fwd_noalloc")] + \
    [fwd("kda_fwd_cp", segment_chunks=2), fwd_trace, bwd, decode]


@pytest.mark.parametrize("call", PER_CHANNEL)
@pytest.mark.parametrize("stream", STREAMS)
def test_allocations_of_the_per_channel_rule(calls, call, stream):
    check_allocations(calls, call, stream)


@pytest.mark.parametrize("call", PER_CHANNEL)
def test_a_stream_of_another_device_is_refused_by_the_per_channel_rule(calls, call):
    with pytest.raises(ValueError):
        call(FakeStream(55, index=1))
    assert calls == [] and OnGpu.allocated == []
