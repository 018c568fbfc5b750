"""Host-side refusals of the per-head-decay delta rule and the q/k norm: every bad
argument is turned away before any HIP call (the data pointers are never
dereferenced), and the 64-bit reference's gradients match differences."""
import ctypes

import pytest
import torch

from gated_delta_rule_35_amd import binding
from tests import gdr_ref as ref
from tests.test_boundary import FAKE, T

F32, BF16, F16, I32 = binding.KDA_F32, binding.KDA_BF16, binding.KDA_F16, binding.KDA_I32
STEP = 1 << 42   # distinct, far apart addresses


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def at(i, shape, dtype=BF16, **kw):
    return T(shape, dtype, data=FAKE + i * STEP, **kw)


def addr(d):
    return None if d is None else ctypes.addressof(d)


def good(B=1, T_=100, Hq=2, Hv=4, N=None, beta=F32):
    n = B if N is None else N
    a = dict(q=at(1, [B, T_, Hq, 128]), k=at(2, [B, T_, Hq, 128]), v=at(3, [B, T_, Hv, 128]), g=at(4, [B, T_, Hv], F32),
             beta=at(5, [B, T_, Hv], beta), cu=None if N is None else at(6, [N + 1], I32),
             h0=at(7, [n, Hv, 128, 128], F32), out=at(8, [B, T_, Hv, 128]), hT=at(9, [n, Hv, 128, 128], F32),
             do=at(10, [B, T_, Hv, 128]), dhT=at(11, [n, Hv, 128, 128], F32), dq=at(12, [B, T_, Hq, 128]),
             dk=at(13, [B, T_, Hq, 128]), dv=at(14, [B, T_, Hv, 128]), dg=at(15, [B, T_, Hv], F32),
             dbeta=at(16, [B, T_, Hv], F32), dh0=at(17, [n, Hv, 128, 128], F32))
    return a


def fwd(lib, a, scale=0.088, ws=FAKE, size=1 << 40):
    return binding.STATUS_NAMES[lib.kda_gdr_fwd(*(addr(a[n]) for n in ("q", "k", "v", "g", "beta")), scale,
                                                *(addr(a[n]) for n in ("cu", "h0", "out", "hT")), ws, size, None)]


def bwd(lib, a, scale=0.088, ws=FAKE, size=1 << 40):
    return binding.STATUS_NAMES[lib.kda_gdr_bwd(
        *(addr(a[n]) for n in ("q", "k", "v", "g", "beta")), scale,
        *(addr(a[n]) for n in ("cu", "h0", "do", "dhT", "dq", "dk", "dv", "dg", "dbeta", "dh0")), ws, size, None)]


BAD = [
    ("NULL", dict(q=None)), ("NULL", dict(v=None)), ("NULL", dict(beta=None)), ("NULL", dict(g=None)),
    ("NULL", dict(k=T([1, 100, 2, 128], data=None))),
    ("DTYPE", dict(q=at(1, [1, 100, 2, 128], F16))), ("DTYPE", dict(g=at(4, [1, 100, 4], BF16))),
    ("DTYPE", dict(beta=at(5, [1, 100, 4], F16))), ("DTYPE", dict(h0=at(7, [1, 4, 128, 128], BF16))),
    ("SHAPE", dict(k=at(2, [1, 99, 2, 128]))), ("SHAPE", dict(v=at(3, [1, 101, 4, 128]))),
    ("SHAPE", dict(g=at(4, [1, 100, 4, 128], F32))), ("SHAPE", dict(beta=at(5, [1, 100, 2], F32))),
    ("SHAPE", dict(h0=at(7, [2, 4, 128, 128], F32))), ("SHAPE", dict(q=at(1, [100, 2, 128]))),
    ("UNSUPPORTED", dict(q=at(1, [1, 100, 2, 64]))), ("UNSUPPORTED", dict(v=at(3, [1, 100, 4, 256]))),
    ("UNSUPPORTED", dict(q=at(1, [1, 100, 3, 128]), k=at(2, [1, 100, 3, 128]))),
    ("LAYOUT", dict(q=T([1, 100, 2, 128], data=FAKE + 8))),
    ("LAYOUT", dict(q=at(1, [1, 100, 2, 128], strides=[25600, 256, 128, 2]))),
    ("LAYOUT", dict(q=at(1, [1, 100, 2, 128], strides=[25600, 260, 128, 1]))),
    ("LAYOUT", dict(v=at(3, [1, 100, 4, 128], strides=[51200, -512, 128, 1]))),
    ("LAYOUT", dict(v=at(3, [1, 100, 4, 128], strides=[51200, 0, 128, 1]))),
    ("LAYOUT", dict(v=at(3, [1, 100, 4, 128], strides=[51200, 64, 128, 1]))),
    ("LAYOUT", dict(v=at(3, [1, 100, 4, 128], strides=[1 << 40, 1 << 24, 128, 1]))),
    ("LAYOUT", dict(g=at(4, [1, 100, 4], F32, strides=[800, 8, 1]))),
]


@pytest.mark.parametrize("name,change", BAD)
def test_inputs(lib, name, change):
    assert fwd(lib, {**good(), **change}) == "KDA_ERR_" + name
    assert bwd(lib, {**good(), **change}) == "KDA_ERR_" + name


def test_packed(lib):
    assert fwd(lib, {**good(B=2), "cu": at(6, [3], I32)}) == "KDA_ERR_UNSUPPORTED"
    assert fwd(lib, {**good(N=2), "cu": at(6, [3], F32)}) == "KDA_ERR_DTYPE"
    assert fwd(lib, {**good(N=2), "cu": at(6, [0], I32)}) == "KDA_ERR_SHAPE"
    assert fwd(lib, {**good(N=2), "cu": at(6, [4], I32)}) == "KDA_ERR_SHAPE"   # states of two sequences


def test_scale_and_sizes(lib):
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert fwd(lib, good(), scale=s) == "KDA_ERR_VALUE"
        assert bwd(lib, good(), scale=s) == "KDA_ERR_VALUE"
    a = good(B=1, T_=1 << 30, Hq=4, Hv=4)
    assert fwd(lib, a) == "KDA_ERR_UNSUPPORTED"
    a = good(B=1 << 20, T_=1, Hq=4, Hv=4)
    assert bwd(lib, a) == "KDA_ERR_UNSUPPORTED"


def test_outputs(lib):
    assert fwd(lib, {**good(), "out": None}) == "KDA_ERR_NULL"
    assert fwd(lib, {**good(), "out": at(8, [1, 100, 4, 128], F32)}) == "KDA_ERR_DTYPE"
    assert fwd(lib, {**good(), "out": at(8, [1, 100, 2, 128])}) == "KDA_ERR_SHAPE"
    assert fwd(lib, {**good(), "out": at(8, [1, 100, 4, 128], strides=[1 << 20, 1024, 128, 1])}) == "KDA_ERR_LAYOUT"
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert bwd(lib, {**good(), n: None}) == "KDA_ERR_NULL"
    assert bwd(lib, {**good(), "dq": at(12, [1, 100, 2, 128], F32)}) == "KDA_ERR_DTYPE"
    assert bwd(lib, {**good(), "dg": at(15, [1, 100, 2], F32)}) == "KDA_ERR_SHAPE"
    assert bwd(lib, {**good(), "do": at(10, [1, 100, 2, 128])}) == "KDA_ERR_SHAPE"
    assert bwd(lib, {**good(), "dh0": at(17, [2, 4, 128, 128], F32)}) == "KDA_ERR_SHAPE"


def test_overlaps(lib):
    a = good()
    assert fwd(lib, {**a, "out": T([1, 100, 4, 128], data=a["v"].data)}) == "KDA_ERR_LAYOUT"
    assert fwd(lib, {**a, "out": T([1, 100, 4, 128], data=a["q"].data + 100 * 256 * 2 - 16)}) == "KDA_ERR_LAYOUT"
    assert fwd(lib, {**a, "hT": T([1, 4, 128, 128], F32, data=a["h0"].data + 65536)}) == "KDA_ERR_LAYOUT"
    assert fwd(lib, {**a, "hT": T([1, 4, 128, 128], F32, data=a["out"].data)}) == "KDA_ERR_LAYOUT"
    assert fwd(lib, {**a, "h0": T([1, 4, 128, 128], F32, data=a["out"].data)}) == "KDA_ERR_LAYOUT"
    # the span of a strided view covers what lies between its rows
    q = at(1, [1, 100, 2, 128], strides=[1 << 20, 4096, 128, 1])
    assert fwd(lib, {**a, "q": q, "out": T([1, 100, 4, 128], data=q.data + 4096)}) == "KDA_ERR_LAYOUT"
    assert bwd(lib, {**a, "dk": T([1, 100, 2, 128], data=a["dq"].data)}) == "KDA_ERR_LAYOUT"
    assert bwd(lib, {**a, "dv": T([1, 100, 4, 128], data=a["do"].data)}) == "KDA_ERR_LAYOUT"
    assert bwd(lib, {**a, "dh0": T([1, 4, 128, 128], F32, data=a["dhT"].data)}) == "KDA_ERR_LAYOUT"


def test_workspaces(lib):
    need = lib.kda_gdr_fwd_workspace_size(100, 1, 4)
    assert need == (2 + 1) * 4 * 20480
    assert fwd(lib, good(), size=need - 1) == "KDA_ERR_WORKSPACE"
    assert fwd(lib, good(), ws=FAKE + 8) == "KDA_ERR_WORKSPACE"
    need = lib.kda_gdr_bwd_workspace_size(100, 1, 4)
    assert need >= 3 * 4 * (37888 + 3 * 65536)
    assert bwd(lib, good(), size=need - 1) == "KDA_ERR_WORKSPACE"
    assert bwd(lib, good(), ws=FAKE + 16) == "KDA_ERR_WORKSPACE"
    assert lib.kda_gdr_fwd_workspace_size(-1, 1, 1) == lib.kda_gdr_bwd_workspace_size(1, -1, 1) == -1
    assert lib.kda_gdr_fwd_workspace_size(0, 5, 4) == lib.kda_gdr_bwd_workspace_size(0, 5, 4) == 0


def test_empty_problems_launch_nothing(lib):
    assert fwd(lib, good(B=0)) == "KDA_OK" and bwd(lib, good(B=0)) == "KDA_OK"
    assert fwd(lib, good(N=0)) == "KDA_OK" and bwd(lib, good(N=0)) == "KDA_OK"
    assert fwd(lib, {**good(T_=0), "hT": None}) == "KDA_OK"
    assert bwd(lib, {**good(T_=0), "dh0": None}) == "KDA_OK"


def decode(lib, scale=0.088, **change):
    a = dict(q=at(1, [3, 2, 128]), k=at(2, [3, 2, 128]), v=at(3, [3, 4, 128]), g=at(4, [3, 4], F32), beta=at(5, [3, 4], F32),
             s_in=at(6, [9, 4, 128, 128], F32), s_out=at(6, [9, 4, 128, 128], F32), idx=at(7, [3], I32),
             out=at(8, [3, 4, 128]))
    a.update(change)
    return binding.STATUS_NAMES[lib.kda_gdr_decode(*(addr(a[n]) for n in ("q", "k", "v", "g", "beta")), scale,
                                                   *(addr(a[n]) for n in ("s_in", "s_out", "idx", "out")), None)]


@pytest.mark.parametrize("name,change", [
    ("NULL", dict(q=None)), ("NULL", dict(s_out=None)), ("NULL", dict(out=None)), ("NULL", dict(beta=None)),
    ("DTYPE", dict(idx=at(7, [3], F32))), ("DTYPE", dict(s_out=at(6, [9, 4, 128, 128]))), ("DTYPE", dict(g=at(4, [3, 4]))),
    ("SHAPE", dict(idx=at(7, [4], I32))), ("SHAPE", dict(idx=None)), ("SHAPE", dict(v=at(3, [2, 4, 128]))),
    ("SHAPE", dict(s_in=at(10, [8, 4, 128, 128], F32))), ("SHAPE", dict(out=at(8, [3, 2, 128]))),
    ("SHAPE", dict(g=at(4, [3, 2], F32))), ("SHAPE", dict(q=at(1, [3, 1, 2, 128]))),
    ("UNSUPPORTED", dict(q=at(1, [3, 3, 128]), k=at(2, [3, 3, 128]))), ("UNSUPPORTED", dict(q=at(1, [3, 2, 64]))),
    ("LAYOUT", dict(s_in=at(6, [9, 4, 128, 128], F32), s_out=T([9, 4, 128, 128], F32, data=FAKE + 6 * STEP + 4096))),
    ("LAYOUT", dict(out=T([3, 4, 128], data=FAKE + 3 * STEP))), ("LAYOUT", dict(out=T([3, 4, 128], data=FAKE + 6 * STEP))),
    ("LAYOUT", dict(q=at(1, [3, 2, 128], strides=[516, 128, 1]))),
    ("VALUE", dict(scale=0.0)),
])
def test_decode(lib, name, change):
    assert decode(lib, **change) == "KDA_ERR_" + name


def test_decode_empty(lib):
    e = dict(q=at(1, [0, 2, 128]), k=at(2, [0, 2, 128]), v=at(3, [0, 4, 128]), g=at(4, [0, 4], F32),
             beta=at(5, [0, 4], F32), idx=at(7, [0], I32), out=at(8, [0, 4, 128]))
    assert decode(lib, **e) == "KDA_OK"
    pool = dict(s_in=at(6, [0, 4, 128, 128], F32), s_out=at(6, [0, 4, 128, 128], F32))
    assert decode(lib, **pool) == "KDA_OK"


def norm(lib, backward=False, mode=0, eps=1e-6, ws=FAKE, size=1 << 30, **change):
    a = dict(q=at(1, [2, 5, 4, 128]), k=at(2, [2, 5, 2, 128]), wq=at(3, [128], F32), wk=at(4, [128], F32),
             cos=at(5, [9, 32], F32), sin=at(6, [9, 32], F32), pos=at(7, [2, 5], I32), qo=at(8, [2, 5, 4, 128]),
             ko=at(9, [2, 5, 2, 128]), dq=at(10, [2, 5, 4, 128]), dk=at(11, [2, 5, 2, 128]), dwq=at(12, [128], F32),
             dwk=at(13, [128], F32))
    a.update(change)
    g = lambda *n: [addr(a[i]) for i in n]  # noqa: E731
    if backward:
        st = lib.kda_qk_norm_bwd(*g("q", "k", "qo", "ko", "wq", "wk"), mode, eps, *g("cos", "sin", "pos"), 0,
                                 *g("dq", "dk", "dwq", "dwk"), ws, size, None)
    else:
        st = lib.kda_qk_norm(*g("q", "k", "wq", "wk"), mode, eps, *g("cos", "sin", "pos"), 0, *g("qo", "ko"), None)
    return binding.STATUS_NAMES[st]


@pytest.mark.parametrize("name,change", [
    ("NULL", dict(q=None)), ("NULL", dict(sin=None)), ("NULL", dict(cos=None)), ("NULL", dict(cos=None, sin=None)),
    ("NULL", dict(qo=None)),
    ("DTYPE", dict(k=at(2, [2, 5, 2, 128], F32))), ("DTYPE", dict(wq=at(3, [128]))), ("DTYPE", dict(pos=at(7, [2, 5], F32))),
    ("DTYPE", dict(q=at(1, [2, 5, 4, 128], I32))), ("DTYPE", dict(cos=at(5, [9, 32]), sin=at(6, [9, 32]))),
    ("SHAPE", dict(k=at(2, [2, 6, 2, 128]))), ("SHAPE", dict(wk=at(4, [64], F32))), ("SHAPE", dict(sin=at(6, [9, 16], F32))),
    ("SHAPE", dict(pos=at(7, [2, 6], I32))), ("SHAPE", dict(qo=at(8, [2, 5, 2, 128]))),
    ("SHAPE", dict(cos=at(5, [0, 32], F32), sin=at(6, [0, 32], F32))),
    ("UNSUPPORTED", dict(q=at(1, [2, 5, 4, 64]))),
    ("UNSUPPORTED", dict(cos=at(5, [9, 20], F32), sin=at(6, [9, 20], F32))),
    ("UNSUPPORTED", dict(cos=at(5, [9, 72], F32), sin=at(6, [9, 72], F32))),
    ("LAYOUT", dict(q=at(1, [2, 5, 4, 128], strides=[4096, 516, 128, 1]))),
    ("LAYOUT", dict(sin=T([9, 32], F32, data=FAKE + 6 * STEP + 4))),
    ("UNSUPPORTED", dict(q=at(1, [2, 1 << 29, 4, 128]), k=at(2, [2, 1 << 29, 2, 128]), pos=None,
                         qo=at(8, [2, 1 << 29, 4, 128]), ko=at(9, [2, 1 << 29, 2, 128]),
                         dq=at(10, [2, 1 << 29, 4, 128]), dk=at(11, [2, 1 << 29, 2, 128]))),
    ("VALUE", dict(mode=2)), ("VALUE", dict(eps=0.0)), ("VALUE", dict(eps=float("nan"))),
])
def test_norm(lib, name, change):
    assert norm(lib, **change) == "KDA_ERR_" + name
    assert norm(lib, backward=True, **change) == "KDA_ERR_" + name


def test_norm_outputs(lib):
    q = at(1, [2, 5, 4, 128])
    assert norm(lib, qo=at(8, [2, 5, 4, 128], F32)) == "KDA_ERR_DTYPE"
    assert norm(lib, qo=T([2, 5, 4, 128], data=q.data + 256)) == "KDA_ERR_LAYOUT"
    assert norm(lib, ko=T([2, 5, 2, 128], data=q.data)) == "KDA_ERR_LAYOUT"
    assert norm(lib, ko=T([2, 5, 2, 128], data=FAKE + 8 * STEP)) == "KDA_ERR_LAYOUT"
    # a strided or fp32 input is never written over
    assert norm(lib, q=at(1, [2, 5, 4, 128], strides=[8192, 1024, 128, 1]), qo=T([2, 5, 4, 128], data=q.data)) == \
        "KDA_ERR_LAYOUT"
    assert norm(lib, q=at(1, [2, 5, 4, 128], F32), k=at(2, [2, 5, 2, 128], F32), qo=T([2, 5, 4, 128], data=q.data)) == \
        "KDA_ERR_LAYOUT"
    b = dict(backward=True)
    assert norm(lib, dwq=at(12, [128], F32), wq=None, **b) == "KDA_ERR_NULL"
    assert norm(lib, dq=at(10, [2, 5, 4, 128], F32), **b) == "KDA_ERR_DTYPE"
    assert norm(lib, qo=at(8, [2, 5, 4, 128], F32), **b) == "KDA_ERR_DTYPE"     # both gradients of one type
    assert norm(lib, dk=T([2, 5, 2, 128], data=FAKE + 10 * STEP), **b) == "KDA_ERR_LAYOUT"
    assert norm(lib, dq=T([2, 5, 4, 128], data=FAKE + 8 * STEP), **b) == "KDA_ERR_LAYOUT"
    need = lib.kda_qk_norm_bwd_workspace_size()
    assert norm(lib, size=need - 1, **b) == "KDA_ERR_WORKSPACE"
    assert norm(lib, ws=FAKE + 4, **b) == "KDA_ERR_WORKSPACE"


def test_binding_refuses_host_tensors_and_modes():
    x = torch.zeros(1, 4, 1, 128, dtype=torch.bfloat16)
    g = torch.zeros(1, 4, 1)
    with pytest.raises(ValueError):
        binding.kda_gdr_fwd(x, x, x, g, g, 1.0)
    with pytest.raises(ValueError):
        binding.kda_gdr_bwd(x, x, x, g, g, 1.0, x)
    with pytest.raises(ValueError):
        binding.kda_gdr_decode(x[0], x[0], x[0], g[0], g[0], 1.0, None)
    with pytest.raises(ValueError):
        binding.kda_gdr_decode(x[0], x[0], x[0], g[0], g[0], 1.0, None, state_indices=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.kda_qk_norm(x, x)
    with pytest.raises(ValueError):
        binding.kda_qk_norm(x, x, mode="max")


class _On:
    """A tensor's host-side view that says it lies on a GPU."""

    def __init__(self, index):
        self.index, self.x = index, torch.zeros(1, 4, 1, 128, dtype=torch.bfloat16)

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.x, name)


@pytest.mark.parametrize("other", [-1, 1])
@pytest.mark.parametrize("place", range(9))
def test_binding_refuses_mixed_places(place, other):
    """Nothing is launched unless every tensor is on the GPU of the call."""
    call = binding._load_caller()
    tensors = tuple(_On(other if i == place else 0) for i in range(9))
    with pytest.raises(ValueError):
        call(binding._GDR_DECODE, 0, 0, None, (1.0,), tensors)
    with pytest.raises(ValueError):
        call(binding._GDR_FWD, 0, 0, _On(other), (1.0,), (_On(0),) * 9)
    with pytest.raises(ValueError):
        call(binding._GDR_FWD, -1, 0, None, (1.0,), (_On(-1),) * 9)


def test_caller_checks_its_own_arguments():
    call = binding._load_caller()
    ok = (_On(0),) * 9
    for args in ((9, 0, 0, None, (1.0,), ok), (binding._GDR_FWD, 0, 0, None, (1.0,), ok[:8]),
                 (binding._GDR_FWD, 0, 0, None, (), ok), (binding._GDR_FWD, 0, 0, None, ("x",), ok),
                 (binding._GDR_FWD, 0, 0, None, (1.0,), ok[:8] + (3,)), (binding._GDR_FWD, 0, 0, None, (1.0,))):
        with pytest.raises((TypeError, RuntimeError, AttributeError)):
            call(*args)
    deep = _On(0)
    deep.x = torch.zeros(1, 1, 1, 1, 128)
    with pytest.raises(ValueError):
        call(binding._GDR_FWD, 0, 0, None, (1.0,), (deep,) * 9)
    # what it hands over is what the library checks: an fp32 q is refused by its dtype
    wrong = _On(0)
    wrong.x = torch.zeros(1, 4, 1, 128)
    st = call(binding._GDR_FWD, 0, 0, None, (1.0,), (wrong,) + (_On(0),) * 8)
    assert binding.STATUS_NAMES[st] == "KDA_ERR_DTYPE"


def test_reference_gradients_match_differences():
    """The tests' own 64-bit forms, by finite differences."""
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64).requires_grad_()  # noqa: E731
    q, k, v, g, b, h = r(5, 1, 3), r(5, 1, 3), r(5, 2, 4), r(5, 2), r(5, 2), r(2, 3, 4)
    assert torch.autograd.gradcheck(lambda q, k, v, g, b, h: ref.recurrence(q, k, v, -g.abs(), b, 0.3, h), (q, k, v, g, b, h))
    x, w = r(1, 2, 1, 128), r(128)
    ang = torch.arange(4, dtype=torch.float64)[:, None] * torch.arange(1, 9)
    for inter in (False, True):
        assert torch.autograd.gradcheck(
            lambda x, w: ref.norm(x, w, "rms", 1e-6, ang.cos(), ang.sin(), None, inter), (x, w), fast_mode=True)
