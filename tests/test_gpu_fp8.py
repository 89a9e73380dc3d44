"""The 8-bit block quantizer, its inverse and the 8-bit product on the GPU against float64.

Quantizer: bit for bit. Product: one rounding of the output, plus two terms inside.
(a) The 8-bit MFMA adds 8 consecutive channels at a time: it cuts each of their products (toward
zero) at 2^-13 times 2^(e_a + e_w), the largest sum of the two operands' exponents in the eight,
with exponents of zeros and subnormals counted as -6. (Measured by adding one product to a known
larger one: against 256 * 256 = 2^16, 7.5 adds 0, 8 to 15 add 8, 16 to 20 add 16.) A product of two
4-bit significands ends at 2^-6 of its own 2^(e_a + e_w), so the one that sets the cut is exact and
the other seven lose less than 7 2^-13 2^(e_a + e_w); 2^(e_a + e_w) is at most the largest product
of the magnitudes raised to 2^-6.
(b) What is left is fp32 sums: K additions at most, and the scale product and the fma of each block,
each within 2^-24 of the sum of magnitudes: (K + 2 ceil(K / 128) + 4) 2^-24 sum |a w|.
"""
import numpy as np
import pytest
import torch

from tests import blocks_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU in this process")
    import post_weight_quantization_channel_amd as m
    from post_weight_quantization_channel_amd import _lib
    _lib.load()
    return m


def say(*a):
    print("  ", *a, flush=True)


def host(t):
    torch.cuda.synchronize()
    return t.cpu()


def same(r, codes, scales):
    q, s = host(r.q).view(torch.uint8).numpy(), host(r.scales).numpy().astype(np.float64)
    assert s.shape == scales.shape and not (s != scales).any()
    at = np.argwhere(q != codes)
    assert len(at) == 0, (len(at), at[0], q[tuple(at[0])], codes[tuple(at[0])])


def wide(m, k, dtype, seed):
    """Values over many binades, with zeros, a block of zeros and a block of tiny values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * torch.exp(2 * torch.randn(m, k, generator=g))
    x[torch.rand(m, k, generator=g) < 0.1] = 0.0
    x = x.to(dtype)
    x[0, :128] = 0.0
    if k > 128:
        x[:, 128:256] *= torch.finfo(dtype).tiny
    return x


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("m,k", [(1, 16), (1, 4096), (3, 144), (127, 128), (129, 272), (300, 1040)])
def test_quantize_bit_exact(awq, dtype, rows, m, k):
    x = wide(m, k, dtype, m + k)
    say("fp8_quantize", dtype, (m, k), "rows", rows)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = awq.fp8_quantize(x.cuda(), block_rows=rows, flags=flags)
    codes, scales = ref.quantize(x.float().numpy(), rows)
    same(r, codes, scales)
    assert int(flags.item()) == 0


def test_quantize_every_rounding_of_e4m3(awq):
    """All values, all midpoints and their fp32 neighbours, in blocks whose scale is 1, and the
    magnitudes around the border between two scales."""
    v = ref.E4M3
    mid = (v[1:] + v[:-1]) / 2
    pts = np.concatenate([v, mid]).astype(np.float32)
    pts = np.concatenate([pts, np.nextafter(pts, np.float32(1e9)), np.nextafter(pts, np.float32(-1))])
    pts = pts[(pts >= 0) & (pts <= 448)]
    pts = np.concatenate([pts, -pts])
    rows = -(-len(pts) // 127)
    x = np.zeros((rows, 128), np.float32)
    x[:, 127] = 448
    x[:, :127].flat[: len(pts)] = pts
    edge = np.full((6, 128), 0.25, np.float32)
    for i, e in enumerate([-126, -3, 100]):
        edge[2 * i, 0] = np.float32(448 * 2.0 ** e)
        edge[2 * i + 1, 0] = np.nextafter(edge[2 * i, 0], np.float32(np.inf))
    edge[:, 1:] *= edge[:, :1]
    x = np.concatenate([x, edge])
    say("fp8_quantize roundings", x.shape)
    r = awq.fp8_quantize(torch.from_numpy(x).cuda())
    codes, scales = ref.quantize(x, 1)
    same(r, codes, scales)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_nonfinite_and_extremes(awq, dtype, rows):
    x = wide(140, 400, dtype, 7)
    x[3, 5], x[3, 200], x[131, 399] = float("nan"), float("inf"), float("-inf")
    x[5, :128] = float("inf")                      # a row block with nothing finite
    x[6, 0] = torch.finfo(dtype).max
    x[7, 130] = -torch.finfo(dtype).max
    say("fp8_quantize nonfinite", dtype, rows)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = awq.fp8_quantize(x.cuda(), block_rows=rows, flags=flags)
    codes, scales = ref.quantize(x.float().numpy(), rows)
    same(r, codes, scales)
    assert int(flags.item()) == 1               # AWQ_FLAG_NONFINITE_X


def test_quantize_strided_view_and_stream(awq):
    base = wide(70, 512, torch.float16, 9).cuda()
    x = base[::2, :272]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("fp8_quantize strided, side stream")
    with torch.cuda.stream(side):
        r = awq.fp8_quantize(x)
    side.synchronize()
    codes, scales = ref.quantize(host(x).float().numpy(), 1)
    same(r, codes, scales)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("m,k", [(1, 16), (131, 272), (64, 1024)])
def test_dequantize(awq, dtype, rows, m, k):
    """Every code; a scale that is no power of two: one fp32 product (exact within 2^-24), rounded
    once to the output type."""
    g = np.random.default_rng(m + k)
    codes = g.integers(0, 256, (m, k)).astype(np.uint8)
    shape = (-(-m // rows), -(-k // 128))
    scales = np.exp(g.standard_normal(shape)).astype(np.float32)
    say("fp8_dequantize", dtype, (m, k), rows)
    y = awq.fp8_dequantize(torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn),
                           torch.from_numpy(scales).cuda(), block_rows=rows, dtype=dtype)
    want = ref.e4m3_values(codes) * ref.spread(scales.astype(np.float64), rows, m, k)
    y = host(y).double().numpy()
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(y), nan)
    ok, used = ref.within(y[~nan], want[~nan], dtype, ref.U32 * np.abs(want[~nan]))
    assert ok, used


def test_round_trip_is_exact_in_bf16(awq):
    x = wide(37, 656, torch.float32, 3)
    r = awq.fp8_quantize(x.cuda())
    v32 = awq.fp8_dequantize(r.q, r.scales, dtype=torch.float32)
    v16 = awq.fp8_dequantize(r.q, r.scales, dtype=torch.bfloat16)
    big = v32.abs() > 1e-30                       # the smallest scales leave bf16's normal range
    assert torch.equal(v32[big], v16.float()[big])
    again = awq.fp8_quantize(v32)
    assert torch.equal(awq.fp8_dequantize(again.q, again.scales, dtype=torch.float32), v32)


def _operands(m, n, k, seed, scale_mult=1.0):
    g = np.random.default_rng(seed)
    a = g.integers(0, 256, (m, k)).astype(np.uint8)
    w = g.integers(0, 256, (n, k)).astype(np.uint8)
    a[(a & 0x7F) == 0x7F] = 0x38
    w[(w & 0x7F) == 0x7F] = 0x30
    kb = -(-k // 128)
    sa = (scale_mult * 1e-3 * np.exp(g.standard_normal((m, kb)))).astype(np.float32)
    sw = (1e-3 * np.exp(g.standard_normal((-(-n // 128), kb)))).astype(np.float32)
    return a, sa, w, sw


def _reference(a, sa, w, sw):
    m, k = a.shape
    n = w.shape[0]
    av = ref.e4m3_values(a) * ref.spread(sa.astype(np.float64), 1, m, k)
    wv = ref.e4m3_values(w) * ref.spread(sw.astype(np.float64), 128, n, k)
    slack = (k + 2 * (-(-k // 128)) + 4) * ref.U32 * (np.abs(av) @ np.abs(wv).T)
    # (a), block by block: the largest raised products of each group of 8, times the scales
    ra = np.maximum(np.abs(ref.e4m3_values(a)), 2.0 ** -6).reshape(m, k // 8, 8)
    rw = np.maximum(np.abs(ref.e4m3_values(w)), 2.0 ** -6).reshape(n, k // 8, 8)
    sae = np.repeat(sa.astype(np.float64), 16, 1)[:, : k // 8]
    swe = np.repeat(np.repeat(sw.astype(np.float64), 128, 0)[:n], 16, 1)[:, : k // 8]
    for g in range(k // 8):
        top = np.zeros((m, n))
        for c in range(8):
            np.maximum(top, ra[:, g, c, None] * rw[None, :, g, c], out=top)
        slack += 7 * 2.0 ** -13 * top * sae[:, g, None] * swe[None, :, g]
    return av @ wv.T, slack


def _dev(codes):
    return torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)


# one row to two tiles; N and K off every tile; one and several K slices; the 256-row tile
GEMM = [(1, 16, 16), (1, 1, 128), (2, 130, 144), (16, 128, 256), (17, 33, 1040), (33, 100, 2064),
        (64, 257, 4112), (65, 130, 144), (100, 1000, 4112), (128, 128, 128), (129, 385, 1168),
        (200, 64, 8192), (300, 260, 16), (1, 4096, 4096), (4097, 4100, 144),
        (8, 4112, 4112), (9, 4112, 4112), (50, 4111, 4112), (49, 130, 144), (64, 128, 1040)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", GEMM)
def test_fp8_gemm(awq, dtype, m, n, k):
    a, sa, w, sw = _operands(m, n, k, m + n + k)
    say("fp8_gemm", (m, n, k), dtype, "workspace", awq.fp8_gemm_workspace_bytes(m, n, k))
    y = awq.fp8_gemm(_dev(a), torch.from_numpy(sa).cuda(), _dev(w), torch.from_numpy(sw).cuda(),
                     out_dtype=dtype)
    want, slack = _reference(a, sa, w, sw)
    ok, used = ref.within(host(y).double().numpy(), want, dtype, slack)
    say("share of the bound", used)
    assert ok, used


@pytest.mark.parametrize("m,n,k", [(3, 40, 256), (70, 140, 1024), (300, 300, 512)])
def test_fp8_gemm_exact_integers(awq, m, n, k):
    """Codes of 0, 1, 2 with either sign and scales of powers of two: every sum is exact."""
    g = np.random.default_rng(5)
    codes = np.array([0x00, 0x38, 0x40, 0xB8, 0xC0], np.uint8)
    a, w = codes[g.integers(0, 5, (m, k))], codes[g.integers(0, 5, (n, k))]
    kb = -(-k // 128)
    sa = (2.0 ** g.integers(-2, 3, (m, kb))).astype(np.float32)
    sw = (2.0 ** g.integers(-2, 1, (-(-n // 128), kb))).astype(np.float32)
    y = awq.fp8_gemm(_dev(a), torch.from_numpy(sa).cuda(), _dev(w), torch.from_numpy(sw).cuda())
    want, _ = _reference(a, sa, w, sw)
    assert np.array_equal(host(y).numpy(), want.astype(np.float16))


@pytest.mark.parametrize("m", [1, 40, 70])
def test_fp8_gemm_rows_are_independent(awq, m):
    """A NaN row, and what lies behind the last row of the outputs, stay where they are; repeated
    calls and a workspace with old contents give the same bits."""
    n, k = 200, 1040
    a, sa, w, sw = _operands(m, n, k, 11)
    a[0, 3] = 0x7F
    t = [_dev(a), torch.from_numpy(sa).cuda(), _dev(w), torch.from_numpy(sw).cuda()]
    buf = torch.full((m + 2, n), 7.0, dtype=torch.float16, device="cuda")
    ws = torch.full((awq.fp8_gemm_workspace_bytes(m, n, k) + 16,), 255, dtype=torch.uint8, device="cuda")
    y = awq.fp8_gemm(*t, out=buf[:m], workspace=ws)
    assert bool((buf[m:] == 7.0).all())
    assert bool(torch.isnan(y[0]).all()) and not bool(torch.isnan(y[1:]).any())
    z = awq.fp8_gemm(*t)
    assert torch.equal(y[1:], z[1:])


@pytest.mark.parametrize("m", [2, 100])
def test_fp8_gemm_streams_and_graph(awq, m):
    """Quantizer and product captured together; replays follow new inputs, with eager calls on the
    same stream and on another one between them."""
    n, k = 384, 1040
    g = torch.Generator().manual_seed(1)
    x = torch.randn(m, k, generator=g).to(torch.bfloat16).cuda()
    w = awq.fp8_quantize((0.1 * torch.randn(n, k, generator=g)).cuda(), block_rows=128)

    def pair():
        r = awq.fp8_quantize(x)
        return awq.fp8_gemm(r.q, r.scales, w.q, w.scales, out_dtype=torch.bfloat16)

    pair()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = pair()
    for i in range(4):
        x.copy_(torch.randn(m, k, generator=g).to(torch.bfloat16))
        graph.replay()
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            e2 = pair()
        e1 = pair()
        torch.cuda.synchronize()
        assert torch.equal(y, e1) and torch.equal(e1, e2), i


def test_output_apart_from_inputs(awq):
    """An output in the memory of an operand is refused."""
    a, w = awq.fp8_quantize(torch.randn(4, 256, device="cuda")), \
        awq.fp8_quantize(torch.randn(128, 256, device="cuda"), block_rows=128)
    with pytest.raises(ValueError, match="share memory"):
        awq.fp8_gemm(a.q, a.scales, w.q, w.scales, out=a.q.view(torch.float16))
    with pytest.raises(ValueError, match="share memory"):
        awq.fp8_gemm(a.q, a.scales, w.q, w.scales, out=w.q[:4].view(torch.float16))
