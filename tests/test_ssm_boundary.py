"""Refusals of the selective state space scan: every bad argument is turned away on the host before any HIP call
and before anything is allocated, and what a call allocates belongs to its stream.  On the CPU; the data pointers
are never dereferenced."""
import ctypes

import pytest
import torch

from gated_delta_rule_35_amd import binding
from tests.test_boundary import FAKE, T
from tests.test_streams import STREAMS, FakeStream, OnGpu, calls, check_allocations  # noqa: F401

F32, BF16, F16, I32 = binding.KDA_F32, binding.KDA_BF16, binding.KDA_F16, binding.KDA_I32
STEP = 1 << 42   # distinct, far apart addresses
WS = FAKE + 90 * STEP


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def at(i, shape, dtype=BF16, **kw):
    return T(shape, dtype, data=FAKE + i * STEP, **kw)


def addr(d):
    return None if d is None else ctypes.addressof(d)


def name(status):
    return binding.STATUS_NAMES[status].replace("KDA_ERR_", "").replace("KDA_", "")


def good(B=1, T_=100, H=4, P=64, G=2, S=128, N=None, dt=F32):
    n = B if N is None else N
    st = [n, H, S, P]
    return dict(x=at(1, [B, T_, H, P]), dt=at(2, [B, T_, H], dt), A=at(3, [H], F32), B=at(4, [B, T_, G, S]), C=at(5, [B, T_, G, S]),
                D=at(6, [H], F32), bias=at(7, [H], F32), sp=1, cu=None if N is None else at(8, [N + 1], I32), h0=at(9, st, F32),
                out=at(10, [B, T_, H, P]), hT=at(11, st, F32), do=at(12, [B, T_, H, P]), dhT=at(13, st, F32),
                dx=at(14, [B, T_, H, P]), ddt=at(15, [B, T_, H], F32), dA=at(16, [H], F32), dB=at(17, [B, T_, G, S]),
                dC=at(18, [B, T_, G, S]), dD=at(19, [H], F32), db=at(20, [H], F32), dh0=at(21, st, F32))


def call(f, a, first, rest, *tail):
    return name(f(*(addr(a[n]) for n in first), a["sp"], *(addr(a[n]) for n in rest), *tail, None))


SHARED = ("x", "dt", "A", "B", "C", "D", "bias")


def fwd(lib, a, ws=WS, size=1 << 50):
    return call(lib.kda_ssm_fwd, a, SHARED, ("cu", "h0", "out", "hT"), ws, size)


def bwd(lib, a, ws=WS, size=1 << 50):
    return call(lib.kda_ssm_bwd, a, SHARED, ("cu", "h0", "do", "dhT", "dx", "ddt", "dA", "dB", "dC", "dD", "db", "dh0"), ws, size)


BAD = [
    ("NULL", dict(x=None)), ("NULL", dict(dt=None)), ("NULL", dict(A=None)), ("NULL", dict(B=None)), ("NULL", dict(C=None)),
    ("NULL", dict(x=T([1, 100, 4, 64], data=None))),
    ("DTYPE", dict(x=at(1, [1, 100, 4, 64], F16))), ("DTYPE", dict(dt=at(2, [1, 100, 4], F16))), ("DTYPE", dict(A=at(3, [4], BF16))),
    ("DTYPE", dict(D=at(6, [4], BF16))), ("DTYPE", dict(h0=at(9, [1, 4, 128, 64], BF16))), ("DTYPE", dict(B=at(4, [1, 100, 2, 128], F32))),
    ("SHAPE", dict(x=at(1, [100, 4, 64]))), ("SHAPE", dict(dt=at(2, [1, 100, 2], F32))), ("SHAPE", dict(dt=at(2, [1, 100], F32))),
    ("SHAPE", dict(A=at(3, [2], F32))), ("SHAPE", dict(C=at(5, [1, 100, 1, 128]))), ("SHAPE", dict(C=at(5, [1, 100, 2, 64]))),
    ("SHAPE", dict(B=at(4, [1, 99, 2, 128]), C=at(5, [1, 99, 2, 128]))), ("SHAPE", dict(bias=at(7, [3], F32))),
    ("SHAPE", dict(h0=at(9, [1, 4, 64, 128], F32))), ("SHAPE", dict(h0=at(9, [2, 4, 128, 64], F32))),
    ("SHAPE", dict(B=at(4, [1, 100, 0, 128]), C=at(5, [1, 100, 0, 128]))),
    ("UNSUPPORTED", dict(x=at(1, [1, 100, 4, 96]))), ("UNSUPPORTED", dict(B=at(4, [1, 100, 2, 256]))),
    ("UNSUPPORTED", dict(B=at(4, [1, 100, 3, 128]), C=at(5, [1, 100, 3, 128]))),
    ("LAYOUT", dict(x=T([1, 100, 4, 64], data=FAKE + STEP + 8))), ("LAYOUT", dict(x=at(1, [1, 100, 4, 64], strides=[25600, 256, 64, 2]))),
    ("LAYOUT", dict(B=at(4, [1, 100, 2, 128], strides=[25600, 260, 128, 1]))),
    ("LAYOUT", dict(C=at(5, [1, 100, 2, 128], strides=[25600, -256, 128, 1]))),
    ("LAYOUT", dict(x=at(1, [1, 100, 4, 64], strides=[0, 0, 64, 1]))), ("LAYOUT", dict(x=at(1, [1, 100, 4, 64], strides=[0, 56, 64, 1]))),
    ("LAYOUT", dict(x=at(1, [1, 100, 4, 64], strides=[1 << 40, 1 << 24, 64, 1]))),
    ("LAYOUT", dict(dt=at(2, [1, 100, 4], F32, strides=[800, 8, 2]))), ("LAYOUT", dict(dt=at(2, [1, 100, 4], F32, strides=[800, -4, 1]))),
    ("LAYOUT", dict(dt=T([1, 100, 4], F32, data=FAKE + 2 * STEP + 2))), ("LAYOUT", dict(A=at(3, [4], F32, strides=[2]))),
    ("VALUE", dict(sp=2)), ("VALUE", dict(sp=-1)),
]


@pytest.mark.parametrize("err,change", BAD)
def test_inputs(lib, err, change):
    assert fwd(lib, {**good(), **change}) == err
    assert bwd(lib, {**good(), **change}) == err


def test_packed_and_sizes(lib):
    assert fwd(lib, {**good(B=2), "cu": at(8, [3], I32)}) == "UNSUPPORTED"
    assert fwd(lib, {**good(N=2), "cu": at(8, [3], F32)}) == "DTYPE"
    assert fwd(lib, {**good(N=2), "cu": at(8, [0], I32)}) == "SHAPE"
    assert bwd(lib, {**good(N=2), "cu": at(8, [4], I32)}) == "SHAPE"   # states of two sequences
    assert fwd(lib, good(T_=1 << 30, H=64, G=1)) == "UNSUPPORTED"
    assert bwd(lib, good(B=1 << 20, T_=1, H=8)) == "UNSUPPORTED"


def test_outputs(lib):
    a = good()
    for change, err in ((dict(out=None), "NULL"), (dict(out=at(10, [1, 100, 4, 64], F32)), "DTYPE"), (dict(out=at(10, [1, 100, 2, 64])), "SHAPE"),
                        (dict(out=at(10, [1, 100, 4, 64], strides=[51200, 512, 64, 1])), "LAYOUT"),
                        (dict(out=T([1, 100, 4, 64], data=a["x"].data)), "LAYOUT"), (dict(hT=T([1, 4, 128, 64], F32, data=a["h0"].data + 64)), "LAYOUT"),
                        (dict(hT=T([1, 4, 128, 64], F32, data=a["out"].data)), "LAYOUT"), (dict(h0=T([1, 4, 128, 64], F32, data=a["out"].data)), "LAYOUT")):
        assert fwd(lib, {**a, **change}) == err, change
    for n in ("dx", "ddt", "dA", "dB", "dC", "do"):
        assert bwd(lib, {**a, n: None}) == "NULL", n
    for change, err in ((dict(D=None), "NULL"), (dict(bias=None), "NULL"), (dict(ddt=at(15, [1, 100, 4])), "DTYPE"),
                        (dict(dB=at(17, [1, 100, 2, 128], F32)), "DTYPE"), (dict(dC=at(18, [1, 100, 1, 128])), "SHAPE"),
                        (dict(do=at(12, [1, 100, 2, 64])), "SHAPE"), (dict(dh0=at(21, [2, 4, 128, 64], F32)), "SHAPE"),
                        (dict(dx=a["do"]), "LAYOUT"), (dict(dh0=a["dhT"]), "LAYOUT"), (dict(dC=T([1, 100, 2, 128], data=a["dB"].data)), "LAYOUT"),
                        (dict(dD=T([4], F32, data=a["dA"].data)), "LAYOUT")):
        assert bwd(lib, {**a, **change}) == err, change


def test_workspaces(lib):
    for f, size in ((fwd, lib.kda_ssm_fwd_workspace_size), (bwd, lib.kda_ssm_bwd_workspace_size)):
        need = size(100, 1, 4, 2, 64, 128)
        assert need > 0 and f(lib, good(), ws=WS + 16) == "WORKSPACE" and f(lib, good(), size=2 * 4 * 2048 - 1) == "WORKSPACE"
        assert size(-1, 1, 4, 2, 64, 128) == size(100, -1, 4, 2, 64, 128) == size(100, 1, 4, 3, 64, 128) == -1
        assert size(100, 1, 4, 2, 96, 128) == size(100, 1, 4, 2, 64, 256) == size(100, 1, 0, 1, 64, 128) == -1
    # the states entering every chunk and the gradients leaving it
    assert lib.kda_ssm_bwd_workspace_size(128, 1, 4, 2, 64, 128) >= 2 * 4 * 2 * 64 * 128 * 4


def test_empty_problems_launch_nothing(lib):
    assert fwd(lib, good(B=0)) == "OK" and fwd(lib, good(N=0)) == "OK"
    assert fwd(lib, {**good(T_=0), "hT": None}) == "OK"


def decode(lib, change=(), N=5, slots=9, indices=True):
    a = dict(x=at(1, [N, 4, 64]), dt=at(2, [N, 4]), A=at(3, [4], F32), B=at(4, [N, 2, 128]), C=at(5, [N, 2, 128]), D=None, bias=None, sp=1,
             s_in=at(9, [slots, 4, 128, 64], F32), s_out=at(9, [slots, 4, 128, 64], F32), idx=at(8, [N], I32) if indices else None,
             out=at(10, [N, 4, 64]))
    a.update(change)
    return call(lib.kda_ssm_decode, a, SHARED, ("s_in", "s_out", "idx", "out"))


def test_decode(lib):
    for change, err in ((dict(s_out=None), "NULL"), (dict(idx=at(8, [4], I32)), "SHAPE"), (dict(idx=at(8, [5], F32)), "DTYPE"),
                        (dict(s_out=at(9, [9, 4, 128, 64])), "DTYPE"), (dict(s_in=at(11, [8, 4, 128, 64], F32)), "SHAPE"),
                        (dict(s_in=T([9, 4, 128, 64], F32, data=FAKE + 9 * STEP + 256)), "LAYOUT"), (dict(out=at(1, [5, 4, 64])), "LAYOUT"),
                        (dict(out=T([5, 4, 64], data=FAKE + 9 * STEP)), "LAYOUT"), (dict(x=at(1, [5, 1, 4, 64])), "SHAPE"), (dict(sp=3), "VALUE"),
                        (dict(out=None), "NULL"), (dict(B=at(4, [5, 3, 128]), C=at(5, [5, 3, 128])), "UNSUPPORTED"),
                        (dict(dt=at(2, [5, 4], strides=[8, 2])), "LAYOUT")):
        assert decode(lib, change) == err, change
    assert decode(lib, indices=False) == "SHAPE"   # nine states for five rows
    assert decode(lib, N=0) == "OK" and decode(lib, slots=0) == "OK"


def gpu(*s, dtype=torch.bfloat16):
    return OnGpu(torch.zeros(*s, dtype=dtype))


def f32(*s):
    return gpu(*s, dtype=torch.float32)


def run_fwd(stream):
    binding.kda_ssm_fwd(gpu(1, 8, 2, 64), f32(1, 8, 2), f32(2), gpu(1, 8, 1, 64), gpu(1, 8, 1, 64), final_state=True, stream=stream)


def run_bwd(stream):
    binding.kda_ssm_bwd(gpu(1, 8, 2, 64), f32(1, 8, 2), f32(2), gpu(1, 8, 1, 64), gpu(1, 8, 1, 64), gpu(1, 8, 2, 64), D=f32(2),
                        dt_bias=f32(2), d_initial_state=True, stream=stream)


def run_decode(stream):
    binding.kda_ssm_decode(gpu(8, 2, 64), f32(8, 2), f32(2), gpu(8, 1, 64), gpu(8, 1, 64), None, stream=stream)


RUNS = [run_fwd, run_bwd, run_decode]


@pytest.mark.parametrize("run", RUNS)
@pytest.mark.parametrize("stream", STREAMS)
def test_allocations_belong_to_the_stream_of_the_call(calls, run, stream):  # noqa: F811
    check_allocations(calls, run, stream)


@pytest.mark.parametrize("run", RUNS)
def test_a_stream_of_another_device_is_refused(calls, run):  # noqa: F811
    with pytest.raises(ValueError):
        run(FakeStream(55, index=1))
    assert calls == [] and OnGpu.allocated == []


x, dt, A, b = torch.zeros(1, 4, 2, 64), torch.zeros(1, 4, 2), torch.zeros(2), torch.zeros(1, 4, 1, 64)
HOST = [lambda: binding.kda_ssm_fwd(x, dt, A, b, b, final_state=True), lambda: binding.kda_ssm_bwd(x, dt, A, b, b, x, D=A),
        lambda: binding.kda_ssm_decode(x[0], dt[0], A, b[0], b[0], None)]


@pytest.mark.parametrize("i", range(len(HOST)))
def test_host_tensors_are_refused_before_anything_is_allocated(i, monkeypatch):
    def no(*a, **kw):
        raise AssertionError("allocated before the refusal")

    monkeypatch.setattr(binding, "_new", no)
    monkeypatch.setattr(binding, "_scratch", no)
    with pytest.raises(ValueError, match="on the GPU"):
        HOST[i]()


def test_a_pool_is_needed_for_its_slots():
    with pytest.raises(ValueError, match="pool"):
        binding.kda_ssm_decode(x[0], dt[0], A, b[0], b[0], None, state_indices=torch.zeros(4, dtype=torch.int32))
