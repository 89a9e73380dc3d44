"""Refusals of the 8-bit calls before any HIP call, through the C ABI and the binding (no GPU)."""
import numpy as np
import pytest
import torch

from tests import blocks_ref as ref
import post_weight_quantization_channel_amd as awq
from post_weight_quantization_channel_amd import _lib

P = 0x10000        # aligned, never dereferenced
NULL, SHAPE, DTYPE, CONFIG, WORKSPACE = (_lib.AWQ_ERR_NULL, _lib.AWQ_ERR_SHAPE, _lib.AWQ_ERR_DTYPE,
                                         _lib.AWQ_ERR_CONFIG, _lib.AWQ_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def refused(fn, good, cases):
    for at, value, status in cases:
        args = list(good)
        args[at] = value
        assert fn(*args) == status, (at, value)


def test_quantize_refuses(lib):
    good = [P, 1, 4, 256, 256, 1, P, P, P, None]
    refused(lib.awq_fp8_quantize, good, [
        (0, None, NULL), (6, None, NULL), (7, None, NULL), (1, 3, DTYPE),
        (1, -1, DTYPE), (2, 0, SHAPE), (2, -1, SHAPE), (2, (1 << 24) + 1, SHAPE), (3, 0, SHAPE),
        (3, 8, SHAPE), (3, 250, SHAPE), (4, 248, SHAPE), (4, 257, SHAPE), (5, 0, CONFIG),
        (5, 64, CONFIG), (0, P + 8, SHAPE), (6, P + 4, SHAPE), (7, P + 2, SHAPE)])
    big = [P, 1, 1 << 24, 1 << 16, 1 << 16, 1, P, P, P, None]      # more than 2^28 blocks
    assert lib.awq_fp8_quantize(*big) == SHAPE
    big[2] = (1 << 19) + 1
    assert lib.awq_fp8_quantize(*big) == SHAPE
    assert lib.awq_fp8_dequantize(P, P, (1 << 19) + 1, 1 << 16, 1, 1, P, None) == SHAPE


def test_dequantize_refuses(lib):
    good = [P, P, 4, 256, 1, 1, P, None]
    refused(lib.awq_fp8_dequantize, good, [
        (0, None, NULL), (1, None, NULL), (6, None, NULL), (5, 3, DTYPE), (2, 0, SHAPE),
        (3, 24, SHAPE), (4, 2, CONFIG), (0, P + 1, SHAPE), (1, P + 1, SHAPE), (6, P + 8, SHAPE)])


def test_gemm_refuses(lib):
    good = [P, P, P, P, 4, 64, 256, 1, P, None, 0, None]
    refused(lib.awq_fp8_gemm, good, [
        (0, None, NULL), (1, None, NULL), (2, None, NULL), (3, None, NULL), (8, None, NULL),
        (7, 0, DTYPE), (7, 5, DTYPE), (4, 0, SHAPE), (5, 0, SHAPE), (6, 0, SHAPE), (6, 40, SHAPE),
        (6, (1 << 20) + 16, SHAPE), (4, (1 << 24) + 1, SHAPE), (0, P + 8, SHAPE),
        (2, P + 4, SHAPE), (8, P + 2, SHAPE), (1, P + 1, SHAPE), (3, P + 2, SHAPE)])
    assert lib.awq_fp8_gemm(P, P, P, P, 1 << 19, (1 << 17) + 1, 256, 1, P, None, 0, None) == SHAPE
    need = lib.awq_fp8_gemm_workspace_bytes(100, 256, 4096)
    assert need > 0
    split = [P, P, P, P, 100, 256, 4096, 1, P, P, need - 1, None]
    assert lib.awq_fp8_gemm(*split) == WORKSPACE
    split[9], split[10] = None, need
    assert lib.awq_fp8_gemm(*split) == WORKSPACE
    split[9] = P + 8
    assert lib.awq_fp8_gemm(*split) == WORKSPACE
    assert lib.awq_fp8_gemm_workspace_bytes(100, 256, 4090) == 0


def test_binding_refuses_before_the_call():
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError):
        awq.fp8_quantize(x)
    q, s = torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.ones(4, 2)
    with pytest.raises(ValueError):
        awq.fp8_dequantize(q, s)
    with pytest.raises(ValueError):
        awq.fp8_gemm(q, s, q, s)


def test_reference_rounding_agrees_with_torch():
    """The tests' own e4m3 rounding against torch's conversion, on every midpoint and beside it."""
    v = ref.E4M3
    pts = np.concatenate([v, (v[1:] + v[:-1]) / 2]).astype(np.float32)
    pts = np.concatenate([pts, np.nextafter(pts, np.float32(1e9)), np.nextafter(pts, np.float32(-1e9))])
    pts = pts[np.abs(pts) <= 448]
    pts = np.concatenate([pts, -pts])
    want = torch.from_numpy(pts).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_codes(pts.astype(np.float64)), want)
