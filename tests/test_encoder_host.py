"""Linear attention, group norm and AdamW without a GPU: argument checks of the C ABI
(nothing is launched: every call below fails its checks) and of the Python package."""
import ctypes

import pytest
import torch

import semi_markov_crf_prefix_b200 as sc
from semi_markov_crf_prefix_b200 import _lib
from semi_markov_crf_prefix_b200 import build as build_mod

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced
OK, ARG, SHAPE, WS = (_lib.SEMICRF_OK, _lib.SEMICRF_ERR_INVALID_ARG, _lib.SEMICRF_ERR_UNSUPPORTED_SHAPE,
                      _lib.SEMICRF_ERR_WORKSPACE_TOO_SMALL)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _lib.load()


def att(B=2, T=64, H=4, dk=32, dv=48, dtype=_lib.F32, reverse=0, scale=1.0, strides=None):
    st = strides or [T * H * dk, H * dk, dk] * 2 + [T * H * dv, H * dv, dv] * 2
    return _lib.ATTENTION_DIMS.pack(B, T, H, dk, dv, dtype, reverse, scale, *st)


BAD_ATTENTION = [
    (dict(B=0), ARG), (dict(T=0), ARG), (dict(H=0), ARG), (dict(dk=0), ARG), (dict(dv=0), ARG), (dict(B=-1), ARG),
    (dict(dtype=3), ARG), (dict(dtype=-1), ARG), (dict(reverse=2), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (dict(strides=[-1] * 12), ARG), (dict(dk=_lib.MAX_HEAD + 1), SHAPE),
    (dict(dv=_lib.MAX_HEAD + 1), SHAPE), (dict(B=1 << 20, H=1 << 10), SHAPE),
]


@pytest.mark.parametrize("kw,status", BAD_ATTENTION)
def test_attention_dims_are_checked(lib, kw, status):
    d = att(**kw)
    assert lib.semicrf_linear_attention_workspace_bytes(d, 0) == 0
    assert lib.semicrf_linear_attention(d, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, 1 << 30, None) == status
    assert lib.semicrf_linear_attention_backward(d, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, FAKE, FAKE,
                                                 None, FAKE, 1 << 30, None) == status
    assert lib.semicrf_linear_attention_step(d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == status


def test_attention_pointers_and_workspace_are_checked(lib):
    d = att()
    need = lib.semicrf_linear_attention_workspace_bytes(d, 0)
    back = lib.semicrf_linear_attention_workspace_bytes(d, 1)
    assert need >= 16 and need % 256 == 0 and back >= need
    assert lib.semicrf_linear_attention_workspace_bytes(d, 2) == 0
    fwd = lib.semicrf_linear_attention
    for hole in (1, 2, 3, 4, 7):
        a = [d, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, need, None]
        a[hole] = None
        assert fwd(*a) == ARG, hole
    assert fwd(d, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, None, need, None) == ARG
    assert fwd(d, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, ctypes.c_void_p((1 << 20) + 8), need, None) == ARG
    assert fwd(d, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, need - 1, None) == WS
    assert fwd(None, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, need, None) == ARG
    step = lib.semicrf_linear_attention_step
    assert step(att(T=2), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == ARG       # one position only
    assert step(att(T=1), FAKE, FAKE, FAKE, FAKE, None, FAKE, None) == ARG
    # few long sequences are walked in segments, whose states take workspace; many are not
    long = lib.semicrf_linear_attention_workspace_bytes(att(B=1, T=100_000, H=8, dk=64, dv=64, dtype=_lib.BF16), 0)
    many = lib.semicrf_linear_attention_workspace_bytes(att(B=64, T=100_000, H=8, dk=64, dv=64, dtype=_lib.BF16), 0)
    assert long > 8 * 64 * 64 * 4 and many == 256


def norm(N=2, S=64, C=32, G=4, dtype=_lib.F32, wtype=_lib.F32, act=1, eps=1e-5):
    return _lib.NORM_DIMS.pack(N, S, C, G, dtype, wtype, act, eps)


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), ARG), (dict(S=0), ARG), (dict(C=0), ARG), (dict(G=0), ARG), (dict(G=3), ARG), (dict(G=64), ARG),
    (dict(dtype=3), ARG), (dict(wtype=_lib.BF16), ARG), (dict(act=3), ARG), (dict(act=-1), ARG),
    (dict(eps=-1e-5), ARG), (dict(eps=float("nan")), ARG), (dict(S=(1 << 30) + 1), SHAPE),
    (dict(N=1 << 29, G=4), SHAPE)])
def test_norm_dims_are_checked(lib, kw, status):
    d = norm(**kw)
    assert lib.semicrf_group_norm_workspace_bytes(d, 0) == 0
    assert lib.semicrf_group_norm(d, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, 1 << 30, None) == status
    assert lib.semicrf_group_norm_backward(d, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30,
                                           None) == status


def test_norm_pointers_and_workspace_are_checked(lib):
    d = norm(N=4, S=200_000, C=256, G=32, dtype=_lib.BF16)
    need = lib.semicrf_group_norm_workspace_bytes(d, 0)
    assert need > 256 and need % 256 == 0
    f = lib.semicrf_group_norm
    assert f(d, None, FAKE, FAKE, None, FAKE, FAKE, FAKE, need, None) == ARG
    assert f(d, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, need, None) == ARG
    assert f(d, FAKE, FAKE, FAKE, None, FAKE, None, FAKE, need, None) == ARG
    assert f(d, FAKE, FAKE, FAKE, None, FAKE, ctypes.c_void_p((1 << 20) + 4), FAKE, need, None) == ARG
    assert f(d, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, need - 1, None) == WS
    assert f(d, FAKE, FAKE, FAKE, None, FAKE, FAKE, ctypes.c_void_p((1 << 20) + 16), need, None) == ARG
    b = lib.semicrf_group_norm_backward
    need = lib.semicrf_group_norm_workspace_bytes(d, 1)
    assert b(d, None, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, need, None) == ARG
    assert b(d, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, need - 1, None) == WS


class Entry(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("ms", ctypes.c_void_p), ("vs", ctypes.c_void_p), ("n", ctypes.c_int64), ("pt", ctypes.c_int32),
                ("gt", ctypes.c_int32)]


def config(**kw):
    c = _lib.AdamWConfig(1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0, 1, None, None)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def entries(*rows):
    return (Entry * max(1, len(rows)))(*[Entry(*r) for r in rows])


@pytest.mark.parametrize("kw", [dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")),
                                dict(eps=-1.0), dict(weight_decay=-1.0), dict(lr=-1.0), dict(lr=float("nan")),
                                dict(step=0), dict(grad_scale=float("inf"))])
def test_adamw_config_is_checked(lib, kw):
    e = entries((8, 8, 8, 8, None, None, 10, 0, 0))
    assert lib.semicrf_adamw(e, 1, config(**kw), None) == ARG


def test_adamw_tensors_are_checked(lib):
    good = (8, 8, 8, 8, None, None, 10, _lib.F32, _lib.F64)
    bad = [(0, None), (1, None), (2, None), (3, None), (6, -1), (7, _lib.F64), (7, -1), (8, 4), (4, 8), (5, 8)]
    for at, value in bad:
        row = list(good)
        row[at] = value
        assert lib.semicrf_adamw(entries(row), 1, config(), None) == ARG, (at, value)
    mixed = entries(good, (8, 8, 8, 8, 8, 8, 10, 0, 0))   # 32- and 8-bit states in one call
    assert lib.semicrf_adamw(mixed, 2, config(), None) == ARG
    assert lib.semicrf_adamw(None, 1, config(), None) == ARG
    assert lib.semicrf_adamw(entries(good), -1, config(), None) == ARG
    assert lib.semicrf_adamw(entries(good), 1, None, None) == ARG
    # nothing to do is no error
    assert lib.semicrf_adamw(None, 0, config(), None) == OK
    assert lib.semicrf_adamw(entries((None, None, None, None, None, None, 0, 0, 0)), 1, config(), None) == OK
    assert lib.semicrf_adamw_state_values(entries(good), 1, 0, None) == ARG       # no scales
    assert lib.semicrf_adamw_state_values(entries((8, None, 8, None, 8, None, 10, 0, 0)), 1, 2, None) == ARG


def test_package_refuses_cpu_tensors(lib):
    q = torch.zeros(1, 4, 2, 8)
    with pytest.raises(TypeError):
        sc.linear_attention(q, q, q, torch.zeros(2))
    with pytest.raises(TypeError):
        sc.linear_attention_step(q[:, 0], q[:, 0], q[:, 0], torch.zeros(2), torch.zeros(1, 2, 8, 8))
    with pytest.raises(TypeError):
        sc.group_norm(torch.zeros(2, 8), 2)
    with pytest.raises(TypeError):
        sc.adamw_step([torch.zeros(3)], [torch.zeros(3)], [torch.zeros(3)], [torch.zeros(3)], 1)
    with pytest.raises(TypeError):
        sc.adamw_state_values([torch.zeros(3, dtype=torch.uint8)], [torch.zeros(1)], "exp_avg")
    with pytest.raises(ValueError):
        sc.adamw_state_values([], [], "exp")
    assert sc.adamw_state_values([], [], "exp_avg") == []
    assert sc.adamw_step([], [], [], [], 1) is None


def test_new_states():
    p = [torch.zeros(300, 2), torch.zeros(0), torch.zeros(256)]
    m, v, ms, vs = sc.new_adamw_state(p)
    assert ms is None and vs is None and [t.dtype for t in m + v] == [torch.float32] * 6
    m, v, ms, vs = sc.new_adamw_state(p, bits=8)
    assert [t.shape for t in m] == [t.shape for t in p] and {t.dtype for t in m + v} == {torch.uint8}
    assert [t.numel() for t in ms] == [3, 0, 1] == [t.numel() for t in vs]
    with pytest.raises(ValueError):
        sc.new_adamw_state(p, bits=4)


def test_unknown_name():
    with pytest.raises(AttributeError):
        sc.no_such_function
