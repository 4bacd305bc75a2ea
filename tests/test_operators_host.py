"""The operators around the loss without a GPU, beside test_encoder_host.py: arguments that are
refused, and what needs no device."""
import ctypes

import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import semi_markov_crf_prefix_b200 as sc
from semi_markov_crf_prefix_b200 import _lib
from semi_markov_crf_prefix_b200 import build as build_mod

ARG = _lib.SEMICRF_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _lib.load()


class Entry(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("ms", ctypes.c_void_p), ("vs", ctypes.c_void_p), ("n", ctypes.c_int64), ("pt", ctypes.c_int32),
                ("gt", ctypes.c_int32)]


@pytest.mark.parametrize("grad_scale,eps", [(1e39, 1e-8), (-1e39, 1e-8), (1e-39, 1e-8), (1e-300, 1e-8), (1.0, 1e-39),
                                            (1.0, 1e-60), (float("nan"), 1e-8)])
def test_what_float32_cannot_hold_is_refused(lib, grad_scale, eps):
    # nothing is launched: the addresses are never used
    e = (Entry * 1)(Entry(8, 8, 8, 8, None, None, 10, _lib.F32, _lib.BF16))
    c = _lib.AdamWConfig(1e-3, 0.9, 0.999, eps, 0.01, grad_scale, 1, None, None)
    assert lib.semicrf_adamw(e, 1, ctypes.byref(c), None) == ARG


def test_overlapping_tensors_are_refused(lib):
    # what a step writes against everything else; fake addresses, and every call is refused
    base, n, cfg = 1 << 30, 300, _lib.AdamWConfig(1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0, 1, None, None)
    at = lambda i: base + (i << 16)  # noqa: E731
    good = [at(i) for i in range(6)]
    for eight in (False, True):
        row = lambda ptrs, k=0: Entry(*[p + (k << 24) for p in ptrs[:4]],  # noqa: E731
                                      *([p + (k << 24) for p in ptrs[4:]] if eight else [None, None]), n, _lib.F32, _lib.F32)
        for i in range(6 if eight else 4):
            for j in range(6 if eight else 4):
                size = [4 * n, 4 * n, n if eight else 4 * n, n if eight else 4 * n, 8, 8][j]
                if i == j:
                    continue
                bad = list(good)
                bad[i] = good[j] + size - 1                # the last byte of the other one
                assert lib.semicrf_adamw((Entry * 1)(row(bad)), 1, ctypes.byref(cfg), None) == ARG, (i, j)
                two = (Entry * 2)(row(good), row(good, 1))
                if i != 1:
                    setattr(two[1], Entry._fields_[i][0], good[i] + 4)     # another tensor's own kind
                    assert lib.semicrf_adamw(two, 2, ctypes.byref(cfg), None) == ARG, i


@pytest.mark.parametrize("which", range(5))
def test_forward_mode_tangents_are_refused(lib, which):
    # before anything else is looked at, so that no device is needed
    args = [torch.ones(1, 3, 2, 8) for _ in range(3)] + [torch.zeros(2), torch.zeros(1, 2, 8, 8)]
    norm = [torch.ones(2, 3, 8), torch.ones(8), torch.zeros(8)]
    with forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        given = [dual(t) if i == which else t for i, t in enumerate(args)]
        with pytest.raises(NotImplementedError):
            sc.linear_attention(*given[:4], initial_state=given[4])
        with pytest.raises(NotImplementedError):
            sc.linear_attention_step(*[t[:, 0] for t in given[:3]], *given[3:])
        if which < 3:
            with pytest.raises(NotImplementedError):
                sc.group_norm(*[dual(t) if i == which else t for i, t in enumerate(norm[:1])] if which == 0 else norm[:1], 2,
                              *[dual(t) if i + 1 == which else t for i, t in enumerate(norm[1:])])
        # a level without tangents is no reason
        with pytest.raises(TypeError):
            sc.linear_attention(*args[:4])


@pytest.mark.parametrize("N,S,C,G", [(64_000, 1, 520, 8), (64_000, 1, 8192, 8), (1 << 20, 1, 8192, 8), (1 << 20, 4, 1000, 8),
                                     (1 << 30, 1, 8, 1), (3, 1 << 30, 513, 1)])
def test_workspace_of_many_row_blocks_stays_small(lib, N, S, C, G):
    # (sizes of calls that nobody makes are still numbers)
    for dtype in (_lib.F32, _lib.BF16):
        for backward in (0, 1):
            need = lib.semicrf_group_norm_workspace_bytes(_lib.NORM_DIMS.pack(N, S, C, G, dtype, _lib.F32, 0, 1e-5), backward)
            assert 0 < need <= max(72 << 20, N * S * C // 8)


def test_repeated_outputs_are_refused(lib):
    # an output axis of stride 0 would be written many times; an input's may repeat
    fake = ctypes.c_void_p(1 << 20)
    for axis in range(3):
        for B, T, H in ((2, 1, 2), (2, 5, 2)):
            st = [[T * H * 8, H * 8, 8] for _ in range(4)]
            if (B, T, H)[axis] == 1:
                continue
            st[3][axis] = 0
            d = _lib.ATTENTION_DIMS.pack(B, T, H, 8, 8, _lib.F32, 0, 1.0, *[x for s in st for x in s])
            assert lib.semicrf_linear_attention(d, fake, fake, fake, fake, None, None, fake, None, fake, 1 << 30, None) == ARG
            if T == 1:
                assert lib.semicrf_linear_attention_step(d, fake, fake, fake, fake, fake, fake, None) == ARG
