"""Refusals of the gated block and of the gradients before any HIP call, through the C ABI and the
binding, and the tests' own derivative against differences (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import post_weight_quantization_channel_amd as awq
from post_weight_quantization_channel_amd import _lib
from tests import blocks_ref as ref

P = 0x10000        # aligned, never dereferenced
NULL, SHAPE, CONFIG, WORKSPACE = (_lib.AWQ_ERR_NULL, _lib.AWQ_ERR_SHAPE, _lib.AWQ_ERR_CONFIG,
                                  _lib.AWQ_ERR_WORKSPACE)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def pk(q=P, s=P, z=None):
    return _lib.AwqPacked(q, s, z)


def refused(fn, good, cases):
    for at, value, status in cases:
        args = list(good)
        args[at] = value
        assert fn(*args) == status, (at, value)


WEIGHTS = [(pk(q=None), NULL), (pk(s=None), NULL), (pk(z=P), CONFIG), (pk(q=P + 8), SHAPE),
           (pk(s=P + 1), SHAPE), (None, NULL)]


def sizes(m, n, k):
    """Refused values of the arguments at m, n, k."""
    return [(m, 0, SHAPE), (m, -3, SHAPE), (m, (1 << 24) + 1, SHAPE), (n, 0, SHAPE),
            (n, (1 << 24) + 16, SHAPE), (k, 0, SHAPE), (k, 64, SHAPE), (k, 200, SHAPE),
            (k, 32768 + 128, SHAPE)]


def test_gated_refuses(lib):
    good = [P, 4, 64, 256, 128, 0, pk(), pk(), P, P, BIG, None]
    refused(lib.w4a16_gated, good, [(0, None, NULL), (8, None, NULL), (4, 32, CONFIG),
                                    (5, 2, CONFIG), (5, -1, CONFIG), (0, P + 8, SHAPE),
                                    (8, P + 2, SHAPE)] + sizes(1, 2, 3) +
            [(6, w, s) for w, s in WEIGHTS] + [(7, w, s) for w, s in WEIGHTS])
    for bad in (pk(s=P + 2), pk(z=P + 1)):       # groups of 64 are read two at a time
        other = pk(z=P if bad.zeros else None)
        assert lib.w4a16_gated(P, 4, 64, 256, 64, 0, bad, other, P, P, BIG, None) == SHAPE
        assert lib.w4a16_gated(P, 4, 64, 256, 64, 0, other, bad, P, P, BIG, None) == SHAPE
    need = lib.w4a16_gated_workspace_bytes(64, 256, 4096, 0)
    assert need > 0
    split = [P, 64, 256, 4096, 128, 0, pk(), pk(), P, P, need - 1, None]
    assert lib.w4a16_gated(*split) == WORKSPACE
    split[9], split[10] = None, need
    assert lib.w4a16_gated(*split) == WORKSPACE
    split[9] = P + 4
    assert lib.w4a16_gated(*split) == WORKSPACE


def test_gated_ckpt_refuses(lib):
    good = [P, 4, 64, 256, 128, 0, pk(), pk(), P, P, P, P, P, P, P, BIG, None]
    refused(lib.w4a16_gated_ckpt, good,
            [(i, None, NULL) for i in (0, 8, 9, 10, 11, 12)] +
            [(2, 60, SHAPE), (9, P + 8, SHAPE), (11, P + 4, SHAPE), (10, P + 2, SHAPE),
             (12, P + 1, SHAPE), (4, 256, CONFIG), (5, 7, CONFIG)] + sizes(1, 2, 3) +
            [(7, w, s) for w, s in WEIGHTS])
    assert lib.w4a16_gated_workspace_bytes(4, 60, 256, 1) == 0
    need = lib.w4a16_gated_workspace_bytes(4, 64, 4096, 1)
    assert need > 0
    good[3], good[15] = 4096, need - 1
    assert lib.w4a16_gated_ckpt(*good) == WORKSPACE


def test_gated_backward_refuses(lib):
    good = [P, P, P, P, P, 4, 64, 256, 128, 0, pk(), pk(), P, P, BIG, None]
    refused(lib.w4a16_gated_backward, good,
            [(i, None, NULL) for i in (0, 1, 2, 3, 4, 12)] +
            [(13, None, WORKSPACE), (14, 0, WORKSPACE), (13, P + 8, WORKSPACE), (6, 72, SHAPE),
             (0, P + 2, SHAPE), (1, P + 8, SHAPE), (3, P + 1, SHAPE), (2, P + 2, SHAPE),
             (12, P + 8, SHAPE), (8, 96, CONFIG), (9, 2, CONFIG)] + sizes(5, 6, 7) +
            [(10, w, s) for w, s in WEIGHTS])
    rows = (1 << 22) + 1
    assert lib.w4a16_gated_backward_workspace_bytes(rows, 16, 128, 128, 0) == 0
    assert lib.w4a16_gated_backward(P, P, P, P, P, rows, 16, 128, 128, 0, pk(), pk(), P, P, BIG,
                                    None) == SHAPE
    need = lib.w4a16_gated_backward_workspace_bytes(4, 64, 256, 128, 0)
    good[14] = need - 1
    assert need > 0 and lib.w4a16_gated_backward(*good) == WORKSPACE
    assert lib.w4a16_gated_backward_workspace_bytes(4, 72, 256, 128, 0) == 0
    assert lib.w4a16_gated_backward_workspace_bytes(4, 64, 256, 32, 0) == 0


def test_gemm_backward_refuses(lib):
    good = [P, 4, 64, 256, 128, P, P, None, P, P, P, BIG, None]
    refused(lib.w4a16_gemm_backward, good,
            [(i, None, NULL) for i in (0, 5, 6, 9)] +
            [(10, None, WORKSPACE), (11, 16, WORKSPACE), (10, P + 4, WORKSPACE), (0, P + 1, SHAPE),
             (5, P + 8, SHAPE), (6, P + 1, SHAPE), (8, P + 1, SHAPE), (9, P + 8, SHAPE),
             (4, 0, CONFIG)] + sizes(1, 2, 3))
    assert lib.w4a16_gemm_backward_workspace_bytes(4, 64, 250, 128, 0) == 0
    rows = (1 << 22) + 1
    assert lib.w4a16_gemm_backward_workspace_bytes(rows, 16, 128, 128, 0) == 0
    assert lib.w4a16_gemm_backward(P, rows, 16, 128, 128, P, P, None, P, P, P, BIG, None) == SHAPE
    assert lib.w4a16_gated(P, 1 << 19, (1 << 17) + 1, 128, 128, 0, pk(), pk(), P, P, BIG, None) == SHAPE


def test_binding_refuses_before_the_call():
    a, q, s = torch.zeros(4, 256).half(), torch.zeros(64, 32, dtype=torch.int32), torch.zeros(64, 2).half()
    f8 = torch.zeros(4, 64, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        awq.w4a16_gated(a, q, s, q, s)
    with pytest.raises(ValueError):
        awq.w4a16_gated_ckpt(a, q, s, q, s)
    with pytest.raises(ValueError):
        awq.w4a16_gemm_backward(torch.zeros(4, 64).half(), q, s, None)
    with pytest.raises(ValueError):
        awq.w4a16_gated_backward(torch.zeros(4, 64).half(), f8, torch.ones(4, 1), f8,
                                 torch.ones(4, 1), q, s, q, s)


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_derivative_of_the_reference(name):
    g = np.linspace(-9, 9, 2001)
    h = 1e-5
    diff = (ref.act(g + h, name)[0] - ref.act(g - h, name)[0]) / (2 * h)
    assert np.abs(diff - ref.act(g, name)[1]).max() < 1e-8
    t = torch.from_numpy(g)
    want = torch.nn.functional.silu(t) if name == "silu" else \
        torch.nn.functional.gelu(t, approximate="tanh")
    assert np.abs(want.numpy() - ref.act(g, name)[0]).max() < 1e-12
