"""Limits of the selective layer's calls (CPU): every call below is refused before anything is launched."""
from __future__ import annotations

import ctypes

import pytest
import torch

import bwd_mamba2_scan_amd as m2
from bwd_mamba2_scan_amd import layer
from bwd_mamba2_scan_amd.layer import Rows, Seqs, SsmDims

P, MUCH = 0x100000, 1 << 62


@pytest.fixture(scope="module")
def L():
    return m2.lib()


def test_convolutions_of_too_many_threads(L):
    # 2^27 sequences of one token: a work-group of 64 (256) threads each
    q, r = Seqs(1 << 27, 1, None), Rows(P, 8, 8)
    assert L.mamba2_conv_fwd(1, q, 8, 4, 1, r, P, None, None, r, None, None) == m2.EBADDIM
    q = Seqs(1 << 25, 1, None)
    assert L.mamba2_conv_bwd(1, q, 8, 4, 1, r, P, None, None, r, None, r, P, None, None, P, MUCH, None) == m2.EBADDIM
    # 2^30 tokens of 1024 channels one at a time, their rows not aligned
    q, r = Seqs(1, 1 << 30, None), Rows(P + 4, 0, 1025)
    assert L.mamba2_conv_fwd(0, q, 1024, 4, 1, r, P, None, None, r, None, None) == m2.EBADDIM


def test_scans_of_too_many_threads(L):
    def call(q, d, bwd):
        r, s, t = Rows(P, d.heads * d.width, 0), Rows(P, d.groups * d.states, 0), Rows(P, d.heads, 0)
        head = (q, d, r, t, P, s, s, None, None, None, r)
        if bwd:
            return L.mamba2_ssm_bwd(*head, None, r, t, P, s, s, None, None, None, P, MUCH, None)
        return L.mamba2_ssm_fwd(*head, None, P, MUCH, None)

    q, d = Seqs(65535, 1, None), SsmDims(0, 0, 1100, 8, 1, 8, 1)            # one wave per sequence and head
    assert call(q, d, False) == m2.EBADDIM == call(q, d, True)
    assert L.mamba2_ssm_bwd_workspace_bytes(q, d) == 0 == L.mamba2_ssm_fwd_workspace_bytes(q, d)
    d = SsmDims(0, 0, 200, 8, 200, 8, 1)                                     # 512 threads per step and group
    assert call(q, d, True) == m2.EBADDIM and L.mamba2_ssm_bwd_workspace_bytes(q, d) == 0
    assert L.mamba2_ssm_bwd_workspace_bytes(q, SsmDims(0, 0, 100, 8, 100, 8, 1)) > 0


@pytest.mark.parametrize("shape", [(1, (1 << 32) + 8, 8), ((1 << 32) + 1, 4, 8), (1, 1 << 31, 1)])
def test_sizes_beyond_an_int_are_not_cut_off(shape):
    layer._load()
    with pytest.raises(ValueError, match="too large"):
        layer._seqs(torch.empty(shape, device="meta"), None, 1, torch.device("meta"))
    with pytest.raises(ValueError, match="too large"):
        layer._ssm_dims(0, *_Sizes.of((2, 8), ((1 << 32) + 1, 8)), True)
    with pytest.raises(ValueError, match="too large"):
        layer._ssm_dims(0, *_Sizes.of(((1 << 32) + 2, 8), (1, 8)), True)


class _Sizes(torch.Tensor):
    """A tensor without memory that passes for one on a GPU."""
    is_cuda = True

    @classmethod
    def of(cls, x, B):
        make = lambda *s: torch.empty(s, device="meta").as_subclass(cls)
        return make(1, 4, *x), make(1, 4, x[0]), make(1, 4, *B)


def test_a_refused_stream_leaves_the_current_device(monkeypatch):
    """Tensors on a device that is not the current one, a stream of a third: refused, and the device stays."""
    import types

    current = [0]

    class Guard:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    fake = types.SimpleNamespace(cuda=types.SimpleNamespace(device=Guard),
                                 _C=types.SimpleNamespace(_cuda_getDevice=lambda: current[0]))
    monkeypatch.setattr(layer, "torch", fake)
    with pytest.raises(ValueError, match="stream is on"):
        with layer._On(torch.device("cuda:1"), types.SimpleNamespace(device=torch.device("cuda:2"))):
            pass
    assert current[0] == 0


class Grad(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_longlong), ("type", ctypes.c_int)]


def test_norm_and_workspace_over_a_gradient(L):
    t = (Grad * 3)(Grad(P, None, 100, 0), Grad(None, None, 0, 0), Grad(P + 4096, None, 8, 1))     # 400 and 16 bytes
    need = L.mamba2_grad_workspace_bytes(t, 3)
    call = lambda norm, ws, n=need: L.mamba2_grad_norm(t, 3, norm, ws, n, None)
    far = P + (1 << 20)
    for norm in (P, P + 396, P + 4096, P + 4108):
        assert call(norm, far) == -8, norm - P
    for ws, n in ((P, need), (P + 384, need), (P - need + 16, need), (P + 4096, need), (P - 4096, 4112), (P - 64, 8192)):
        assert call(far, ws, n) == -8, ws - P
    assert call(far, far) == -8 == call(far + need - 4, far)
