"""Refusals of the short convolution and of the norms around a block: every bad argument is turned away
on the host before any HIP call and before anything is allocated, and what a call allocates belongs to its
stream.  On the CPU; the data pointers are never dereferenced."""
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


# ---- the convolution

def conv_args(B=1, T_=100, C=64, W=4, N=None, dtype=BF16):
    n = B if N is None else N
    return dict(x=at(1, [B, T_, C], dtype), w=at(2, [C, W], F32), bias=at(3, [C], F32), act=1,
                cu=None if N is None else at(4, [N + 1], I32), s0=at(5, [n, W - 1, C], dtype), out=at(6, [B, T_, C], dtype),
                sT=at(7, [n, W - 1, C], dtype), do=at(8, [B, T_, C], dtype), dsT=at(9, [n, W - 1, C], dtype),
                dx=at(10, [B, T_, C], dtype), dw=at(11, [C, W], F32), db=at(12, [C], F32), ds0=at(13, [n, W - 1, C], dtype))


def conv(lib, a):
    return name(lib.kda_conv(addr(a["x"]), addr(a["w"]), addr(a["bias"]), a["act"],
                             *(addr(a[n]) for n in ("cu", "s0", "out", "sT")), None))


def conv_bwd(lib, a, ws=WS, size=1 << 40):
    return name(lib.kda_conv_bwd(addr(a["x"]), addr(a["w"]), addr(a["bias"]), a["act"],
                                 *(addr(a[n]) for n in ("cu", "s0", "do", "dsT", "dx", "dw", "db", "ds0")), ws, size, None))


BAD_CONV = [
    ("NULL", dict(x=None)), ("NULL", dict(w=None)), ("NULL", dict(x=T([1, 100, 64], data=None))),
    ("DTYPE", dict(x=at(1, [1, 100, 64], I32))), ("DTYPE", dict(w=at(2, [64, 4], BF16))), ("DTYPE", dict(bias=at(3, [64], BF16))),
    ("DTYPE", dict(s0=at(5, [1, 3, 64], F32))),
    ("SHAPE", dict(x=at(1, [100, 64]))), ("SHAPE", dict(w=at(2, [65, 4], F32))), ("SHAPE", dict(w=at(2, [64], F32))),
    ("SHAPE", dict(bias=at(3, [63], F32))), ("SHAPE", dict(s0=at(5, [1, 4, 64]))), ("SHAPE", dict(s0=at(5, [2, 3, 64]))),
    ("SHAPE", dict(x=at(1, [1, 100, 0]), w=at(2, [0, 4], F32))),
    ("UNSUPPORTED", dict(w=at(2, [64, 5], F32))), ("UNSUPPORTED", dict(w=at(2, [64, 1], F32))),
    ("UNSUPPORTED", dict(x=at(1, [1, 100, 60]), w=at(2, [60, 4], F32))),
    ("UNSUPPORTED", dict(x=at(1, [1, 100, 1 << 21]), w=at(2, [1 << 21, 4], F32))),
    ("LAYOUT", dict(x=T([1, 100, 64], data=FAKE + 8))), ("LAYOUT", dict(x=at(1, [1, 100, 64], strides=[12800, 128, 2]))),
    ("LAYOUT", dict(x=at(1, [1, 100, 64], strides=[6400, 68, 1]))), ("LAYOUT", dict(x=at(1, [1, 100, 64], strides=[6400, -64, 1]))),
    ("LAYOUT", dict(w=at(2, [64, 4], F32, strides=[8, 1]))), ("LAYOUT", dict(w=T([64, 4], F32, data=FAKE + 2 * STEP + 4))),
    ("LAYOUT", dict(s0=at(5, [1, 3, 64], strides=[384, 128, 1]))),
    ("VALUE", dict(act=2)), ("VALUE", dict(act=-1)),
]


@pytest.mark.parametrize("err,change", BAD_CONV)
def test_conv_inputs(lib, err, change):
    assert conv(lib, {**conv_args(), **change}) == err
    assert conv_bwd(lib, {**conv_args(), **change}) == err


def test_conv_packed_and_sizes(lib):
    assert conv(lib, {**conv_args(B=2), "cu": at(4, [3], I32)}) == "UNSUPPORTED"
    assert conv(lib, {**conv_args(N=2), "cu": at(4, [3], F32)}) == "DTYPE"
    assert conv(lib, {**conv_args(N=2), "cu": at(4, [0], I32)}) == "SHAPE"
    assert conv_bwd(lib, {**conv_args(N=2), "cu": at(4, [4], I32)}) == "SHAPE"   # states of two sequences
    assert conv(lib, conv_args(B=1 << 16, T_=1 << 16, C=8)) == "UNSUPPORTED"
    assert conv(lib, conv_args(T_=1 << 30, C=8192)) == "UNSUPPORTED"


def test_conv_outputs(lib):
    a = conv_args()
    for change, err in ((dict(out=None), "NULL"), (dict(out=at(6, [1, 100, 64], F32)), "DTYPE"), (dict(out=at(6, [1, 99, 64])), "SHAPE"),
                        (dict(out=at(6, [1, 100, 64], strides=[12800, 128, 1])), "LAYOUT"), (dict(out=a["x"]), "LAYOUT"),
                        (dict(sT=a["s0"]), "LAYOUT"), (dict(sT=T([1, 3, 64], data=a["x"].data + 64)), "LAYOUT")):
        assert conv(lib, {**a, **change}) == err, change
    for change, err in ((dict(dx=None), "NULL"), (dict(dw=None), "NULL"), (dict(do=None), "NULL"), (dict(dw=at(11, [64, 4])), "DTYPE"),
                        (dict(dw=at(11, [4, 64], F32)), "SHAPE"), (dict(do=at(8, [1, 100, 64], F32)), "DTYPE"),
                        (dict(bias=None), "NULL"), (dict(dx=a["do"]), "LAYOUT"), (dict(ds0=a["dsT"]), "LAYOUT"),
                        (dict(do=at(8, [1, 100, 64], strides=[12800, 128, 1])), "LAYOUT")):
        assert conv_bwd(lib, {**a, **change}) == err, change
    need = lib.kda_conv_bwd_workspace_size(100, 64, 4)
    assert need > 0 and conv_bwd(lib, a, size=need - 1) == "WORKSPACE" and conv_bwd(lib, a, ws=WS + 8) == "WORKSPACE"
    assert lib.kda_conv_bwd_workspace_size(-1, 64, 4) == lib.kda_conv_bwd_workspace_size(1, -8, 4) == -1
    assert lib.kda_conv_bwd_workspace_size(0, 64, 4) == 0


def conv_decode(lib, change=(), N=5, C=64, slots=9, indices=True):
    a = dict(x=at(1, [N, C]), w=at(2, [C, 4], F32), bias=None, act=1, s_in=at(5, [slots, 3, C]), s_out=at(5, [slots, 3, C]),
             idx=at(4, [N], I32) if indices else None, out=at(6, [N, C]))
    a.update(change)
    return name(lib.kda_conv_decode(addr(a["x"]), addr(a["w"]), addr(a["bias"]), a["act"], addr(a["s_in"]), addr(a["s_out"]),
                                    addr(a["idx"]), addr(a["out"]), None))


def test_conv_decode(lib):
    for change, err in ((dict(s_out=None), "NULL"), (dict(idx=at(4, [4], I32)), "SHAPE"), (dict(idx=at(4, [5], F32)), "DTYPE"),
                        (dict(s_out=at(5, [9, 3, 64], F32)), "DTYPE"), (dict(s_in=at(7, [8, 3, 64])), "SHAPE"),
                        (dict(s_in=T([9, 3, 64], data=FAKE + 5 * STEP + 32)), "LAYOUT"), (dict(out=at(1, [5, 64])), "LAYOUT"),
                        (dict(out=at(5, [5, 64])), "LAYOUT"), (dict(x=at(1, [5, 1, 64])), "SHAPE"), (dict(act=3), "VALUE"),
                        (dict(out=None), "NULL")):
        assert conv_decode(lib, change) == err, change
    assert conv_decode(lib, indices=False) == "SHAPE"   # nine states for five rows
    assert conv_decode(lib, N=0) == "OK" and conv_decode(lib, slots=0) == "OK"


# ---- the norms

def gated_args(B=1, T_=10, H=4, D=128, dtype=BF16, heads=False):
    s = [B, T_, H, D]
    return dict(x=at(1, s, dtype), gate=at(2, s, dtype), w=at(3, [H, D] if heads else [D], F32), act=1, first=0, eps=1e-6,
                out=at(4, s, dtype), do=at(5, s, dtype), dx=at(6, s, dtype), dg=at(7, s, dtype),
                dw=at(8, [H, D] if heads else [D], F32))


def gated(lib, a):
    return name(lib.kda_gated_norm(addr(a["x"]), addr(a["gate"]), addr(a["w"]), a["act"], a["first"], a["eps"], addr(a["out"]), None))


def gated_bwd(lib, a, ws=WS, size=1 << 40):
    return name(lib.kda_gated_norm_bwd(addr(a["x"]), addr(a["gate"]), addr(a["w"]), a["act"], a["first"], a["eps"],
                                       *(addr(a[n]) for n in ("do", "dx", "dg", "dw")), ws, size, None))


S = [1, 10, 4, 128]
BAD_GATED = [
    ("NULL", dict(x=None)), ("NULL", dict(gate=None)), ("DTYPE", dict(gate=at(2, S, F32))), ("DTYPE", dict(x=at(1, S, I32))),
    ("DTYPE", dict(w=at(3, [128], BF16))), ("SHAPE", dict(gate=at(2, [1, 10, 2, 128]))), ("SHAPE", dict(w=at(3, [64], F32))),
    ("SHAPE", dict(w=at(3, [2, 128], F32))), ("SHAPE", dict(x=at(1, [1, 10, 512]))),
    ("UNSUPPORTED", dict(x=at(1, [1, 10, 4, 124]))), ("UNSUPPORTED", dict(x=at(1, [1, 10, 4, 8200]))),
    ("LAYOUT", dict(x=at(1, S, strides=[5120, 512, 128, 2]))), ("LAYOUT", dict(gate=at(2, S, strides=[5120, 516, 128, 1]))),
    ("LAYOUT", dict(gate=T(S, data=FAKE + 2 * STEP + 2))), ("LAYOUT", dict(w=T([128], F32, data=FAKE + 3 * STEP + 4))),
    ("VALUE", dict(act=0)), ("VALUE", dict(act=3)), ("VALUE", dict(eps=0.0)), ("VALUE", dict(eps=float("nan"))),
    ("VALUE", dict(eps=float("inf"))),
]


@pytest.mark.parametrize("err,change", BAD_GATED)
def test_gated_inputs(lib, err, change):
    assert gated(lib, {**gated_args(), **change}) == err
    assert gated_bwd(lib, {**gated_args(), **change}) == err


def test_gated_outputs(lib):
    a = gated_args()
    for change, err in ((dict(out=None), "NULL"), (dict(out=at(4, S, F32)), "DTYPE"), (dict(out=at(4, [1, 10, 4, 64])), "SHAPE"),
                        (dict(out=a["gate"]), "LAYOUT"), (dict(out=T(S, data=a["x"].data + 16)), "LAYOUT"),
                        (dict(x=at(1, S, strides=[10240, 1024, 128, 1]), out=at(1, S)), "LAYOUT")):
        assert gated(lib, {**a, **change}) == err, change
    for change, err in ((dict(do=None), "NULL"), (dict(dx=None), "NULL"), (dict(dg=None), "NULL"), (dict(do=at(5, S, F32)), "DTYPE"),
                        (dict(w=None), "NULL"), (dict(dw=at(8, [4, 128], F32)), "SHAPE"), (dict(dx=a["do"]), "LAYOUT"),
                        (dict(dx=a["x"]), "LAYOUT"), (dict(dg=a["dx"]), "LAYOUT")):
        assert gated_bwd(lib, {**a, **change}) == err, change
    need = lib.kda_norm_bwd_workspace_size(1, 128)
    assert gated_bwd(lib, a, size=need - 1) == "WORKSPACE" and gated_bwd(lib, a, ws=WS + 8) == "WORKSPACE"
    assert lib.kda_norm_bwd_workspace_size(2000, 128) == 2000 * 512
    assert lib.kda_norm_bwd_workspace_size(-1, 128) == lib.kda_norm_bwd_workspace_size(1, 8200) == -1
    assert gated(lib, gated_args(B=1 << 16, T_=1 << 16)) == "UNSUPPORTED"


def add_args(B=1, T_=10, D=256, dtype=BF16, res=F32):
    s = [B, T_, D]
    return dict(x=at(1, s, dtype), res=at(2, s, res), w=at(3, [D], F32), scale=0.5, eps=1e-6, out=at(4, s, dtype), sum=at(5, s, res),
                do=at(6, s, dtype), ds=at(7, s, res), dx=at(8, s, dtype), dr=at(9, s, res), dw=at(10, [D], F32))


def add(lib, a):
    return name(lib.kda_add_norm(addr(a["x"]), addr(a["res"]), addr(a["w"]), a["scale"], a["eps"], addr(a["out"]), addr(a["sum"]), None))


def add_bwd(lib, a, ws=WS, size=1 << 40):
    return name(lib.kda_add_norm_bwd(addr(a["sum"]), addr(a["w"]), a["scale"], a["eps"],
                                     *(addr(a[n]) for n in ("do", "ds", "dx", "dr", "dw")), ws, size, None))


def test_add(lib):
    a, s = add_args(), [1, 10, 256]
    for change, err in ((dict(x=None), "NULL"), (dict(res=None), "NULL"), (dict(out=None), "NULL"), (dict(sum=None), "NULL"),
                        (dict(res=at(2, s, F16), sum=at(5, s, F16)), "DTYPE"), (dict(sum=at(5, s)), "DTYPE"),
                        (dict(res=at(2, [1, 9, 256], F32)), "SHAPE"), (dict(w=at(3, [1, 256], F32)), "SHAPE"),
                        (dict(scale=float("nan")), "VALUE"), (dict(scale=float("inf")), "VALUE"), (dict(eps=-1.0), "VALUE"),
                        (dict(out=T(s, data=a["res"].data)), "LAYOUT"), (dict(sum=T(s, F32, data=a["res"].data + 16)), "LAYOUT"),
                        (dict(sum=T(s, F32, data=a["x"].data)), "LAYOUT"), (dict(out=T(s, data=a["sum"].data)), "LAYOUT"),
                        (dict(res=at(2, s, F32, strides=[1 << 20, 512, 1]), sum=at(2, s, F32)), "LAYOUT"),
                        (dict(x=at(1, [1, 10, 252])), "UNSUPPORTED"), (dict(x=at(1, [10, 256])), "SHAPE")):
        assert add(lib, {**a, **change}) == err, change
    for change, err in ((dict(sum=None), "NULL"), (dict(do=None), "NULL"), (dict(dx=None), "NULL"), (dict(dr=None), "NULL"),
                        (dict(w=None), "NULL"), (dict(do=at(6, s, I32)), "DTYPE"), (dict(sum=at(5, s, F16)), "DTYPE"),
                        (dict(ds=at(7, s)), "DTYPE"), (dict(dr=at(9, s)), "DTYPE"), (dict(ds=at(7, [1, 9, 256], F32)), "SHAPE"),
                        (dict(dr=a["ds"]), "LAYOUT"), (dict(dx=a["do"]), "LAYOUT"), (dict(scale=float("nan")), "VALUE")):
        assert add_bwd(lib, {**a, **change}) == err, change
    assert add_bwd(lib, a, size=lib.kda_norm_bwd_workspace_size(1, 256) - 1) == "WORKSPACE"


# ---- the binding

def gpu(*s, dtype=torch.bfloat16):
    return OnGpu(torch.zeros(*s, dtype=dtype))


def f32(*s):
    return gpu(*s, dtype=torch.float32)


def run_conv(stream):
    binding.kda_conv(gpu(1, 8, 16), f32(16, 4), final_state=True, stream=stream)


def run_conv_bwd(stream):
    binding.kda_conv_bwd(gpu(1, 8, 16), f32(16, 4), gpu(1, 8, 16), f32(16), d_initial_state=True, stream=stream)


def run_conv_decode(stream):
    binding.kda_conv_decode(gpu(8, 16), f32(16, 4), None, stream=stream)


def run_gated_bwd(stream):
    binding.kda_gated_norm_bwd(gpu(1, 8, 2, 64), gpu(1, 8, 2, 64), gpu(1, 8, 2, 64), f32(64), stream=stream)


def run_add(stream):
    binding.kda_add_norm(gpu(1, 8, 64), gpu(1, 8, 64), f32(64), stream=stream)


def run_add_bwd(stream):
    binding.kda_add_norm_bwd(gpu(1, 8, 64), gpu(1, 8, 64), f32(64), stream=stream)


RUNS = [run_conv, run_conv_bwd, run_conv_decode, run_gated_bwd, run_add, run_add_bwd]


@pytest.mark.parametrize("call", RUNS)
@pytest.mark.parametrize("stream", STREAMS)
def test_allocations_belong_to_the_stream_of_the_call(calls, call, stream):  # noqa: F811
    check_allocations(calls, call, stream)


def test_the_gated_norm_allocates_on_the_stream_of_the_call(calls):  # noqa: F811
    binding.kda_gated_norm(gpu(1, 8, 2, 64), gpu(1, 8, 2, 64), f32(64), stream=77)
    assert calls == [77] and OnGpu.allocated == [77]


@pytest.mark.parametrize("call", RUNS)
def test_a_stream_of_another_device_is_refused(calls, call):  # noqa: F811
    with pytest.raises(ValueError):
        call(FakeStream(55, index=1))
    assert calls == [] and OnGpu.allocated == []


x3, x4, w = torch.zeros(1, 4, 64), torch.zeros(1, 4, 2, 64), torch.ones(64)
HOST = [
    lambda: binding.kda_conv(x3, torch.ones(64, 4), final_state=True),
    lambda: binding.kda_conv_bwd(x3, torch.ones(64, 4), x3, w, d_initial_state=True),
    lambda: binding.kda_conv_decode(x3[0], torch.ones(64, 4), None),
    lambda: binding.kda_gated_norm(x4, x4, w),
    lambda: binding.kda_gated_norm_bwd(x4, x4, x4, w),
    lambda: binding.kda_add_norm(x3, x3, w),
    lambda: binding.kda_add_norm_bwd(x3, x3, w),
]


@pytest.mark.parametrize("i", range(len(HOST)))
def test_host_tensors_are_refused_before_anything_is_allocated(i, monkeypatch):
    def no(*a, **kw):
        raise AssertionError("allocated before the refusal")

    monkeypatch.setattr(binding, "_new", no)
    monkeypatch.setattr(binding, "_scratch", no)
    with pytest.raises(ValueError, match="on the GPU"):
        HOST[i]()


@pytest.mark.parametrize("call", [lambda: binding.kda_conv(x3, torch.ones(64, 4), activation="tanh"),
                                  lambda: binding.kda_conv_bwd(x3, torch.ones(64, 4), x3, activation="sigmoid"),
                                  lambda: binding.kda_conv_decode(x3[0], torch.ones(64, 4), None, activation="relu"),
                                  lambda: binding.kda_gated_norm(x4, x4, activation=None),
                                  lambda: binding.kda_gated_norm_bwd(x4, x4, x4, activation="none")])
def test_unknown_activations_are_refused(call):
    with pytest.raises(ValueError, match="activation"):
        call()


def test_a_pool_is_needed_for_its_slots():
    with pytest.raises(ValueError, match="pool"):
        binding.kda_conv_decode(x3[0], torch.ones(64, 4), None, state_indices=torch.zeros(4, dtype=torch.int32))
