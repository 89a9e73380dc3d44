"""The gated feed-forward block on packed weights, its 8-bit activations, and the gradients through
packed weights on the GPU, against float64 (bounds: tests/blocks_ref.py)."""
import numpy as np
import pytest
import torch

from tests import blocks_ref as ref

pytestmark = pytest.mark.gpu


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


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().double().numpy()


def packed(n, k, group, zp, seed, step=0.01):
    """Random codes, steps over a factor of a hundred with a few zero ones, zero points."""
    g = np.random.default_rng(seed)
    q = g.integers(0, 2 ** 32, (n, k // 8), dtype=np.uint64).astype(np.uint32).view(np.int32)
    s = (step * np.exp(g.standard_normal((n, k // group)))).astype(np.float16)
    s[g.random(s.shape) < 0.02] = 0
    z = g.integers(0, 16, (n, k // group)).astype(np.uint8) if zp else None
    return q, s, z


def on_gpu(gate, up):
    return [dev(gate[0]), dev(gate[1]), dev(up[0]), dev(up[1])], \
        {"gate_zeros": dev(gate[2]), "up_zeros": dev(up[2])}


def check(y, want, slack, dtype=torch.float16):
    ok, used = ref.within(y, want, dtype, slack)
    say("share of the bound", used)
    assert ok, used


# one row; two; the MFMA paths at their edges; tiles; odd N; one and several K slices
FORWARD = [(1, 1, 128), (1, 130, 4224), (1, 64, 8320), (2, 257, 1024), (2, 40, 8192), (3, 16, 128),
           (16, 100, 1152), (17, 31, 2048), (32, 128, 640), (33, 1, 128), (64, 250, 4096),
           (65, 129, 1024), (128, 384, 256), (300, 200, 512), (300, 1100, 2048), (700, 4112, 128),
           (17, 4200, 4096), (32, 4104, 4224), (300, 3000, 1024), (9, 200, 8192)]


@pytest.mark.parametrize("group,zp,act", [(128, False, "silu"), (64, True, "gelu"),
                                          (128, True, "gelu"), (64, False, "silu")])
@pytest.mark.parametrize("m,n,k", FORWARD)
def test_gated(awq, m, n, k, group, zp, act):
    gate, up = (packed(n, k, group, zp, s + m) for s in (1, 2))
    a = np.random.default_rng(m + n + k).standard_normal((m, k)).astype(np.float16)
    w, z = on_gpu(gate, up)
    say("w4a16_gated", (m, n, k), group, zp, act, awq.w4a16_gated_workspace_bytes(m, n, k))
    h = awq.w4a16_gated(dev(a), *w, group=group, act=act, **z)
    r = ref.gated(a.astype(np.float64), ref.unpack(*gate, group), ref.unpack(*up, group), group, act)
    check(host(h), r[4], r[5])


@pytest.mark.parametrize("group,zp,act", [(128, False, "silu"), (64, True, "gelu")])
@pytest.mark.parametrize("m,n,k", [(1, 16, 128), (3, 144, 4096), (64, 128, 256), (70, 272, 1024),
                                   (300, 4112, 512), (300, 1104, 1024), (300, 3008, 1024),
                                   (1000, 4096, 128)])
def test_gated_ckpt(awq, m, n, k, group, zp, act):
    gate, up = (packed(n, k, group, zp, s + m) for s in (1, 2))
    a = np.random.default_rng(m + n + k).standard_normal((m, k)).astype(np.float16)
    w, z = on_gpu(gate, up)
    say("w4a16_gated_ckpt", (m, n, k), group, zp, act, awq.w4a16_gated_workspace_bytes(m, n, k, True))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = awq.w4a16_gated_ckpt(dev(a), *w, group=group, act=act, flags=flags, **z)
    g, eg, u, eu, h, eh = ref.gated(a.astype(np.float64), ref.unpack(*gate, group),
                                    ref.unpack(*up, group), group, act)
    check(host(r.H), h, eh)
    assert int(flags.item()) == 0
    for q, s, x, ex in ((r.g8, r.g_scales, g, eg), (r.u8, r.u_scales, u, eu)):
        s = host(s)
        pad = ((0, 0), (0, -n % 128))
        lo = np.pad(np.abs(x) - ex, pad).reshape(m, -1, 128).max(2)
        hi = np.pad(np.abs(x) + ex, pad).reshape(m, -1, 128).max(2)
        assert s.shape == lo.shape and np.all(np.log2(s) % 1 == 0)
        # the smallest 2^e that holds the block, up to the error of its largest value
        assert np.all(lo <= 448 * s) and np.all((hi > 224 * s) | (s == 1))
        sp = ref.spread(s, 1, m, n)
        v = host(q.float()) * sp
        # half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale below 2^-6
        tol = 2.0 ** -4 * (np.abs(x) + ex) + ex + 2.0 ** -10 * sp
        assert np.all(np.abs(v - x) <= tol)


@pytest.mark.parametrize("m", [5, 200])
def test_gated_ckpt_exact(awq, m):
    """Small whole numbers and steps of 1: g and u are exact, so their blocks are bit for bit those
    of the quantizer, whichever path (K slices or not) made them."""
    n, k, g = 272, 1024, np.random.default_rng(3)
    a = g.integers(-2, 3, (m, k)).astype(np.float16)
    w = [(q, np.ones_like(s), None) for q, s, _ in (packed(n, k, 128, False, s) for s in (5, 6))]
    wd, z = on_gpu(*w)
    r = awq.w4a16_gated_ckpt(dev(a), *wd, **z)
    for q, s, p in ((r.g8, r.g_scales, w[0]), (r.u8, r.u_scales, w[1])):
        c, _ = ref.unpack(*p, 128)
        codes, scales = ref.quantize(a.astype(np.float64) @ c.T, 1)
        assert np.array_equal(host(s), scales)
        assert np.array_equal(q.cpu().view(torch.uint8).numpy(), codes)


@pytest.mark.parametrize("m", [1, 20, 100])
def test_gated_nonfinite_rows(awq, m):
    """An infinite or NaN activation changes its own row only; the 8-bit form flags it."""
    n, k = 144, 1024
    gate, up = packed(n, k, 128, False, 1), packed(n, k, 128, False, 2)
    a = np.random.default_rng(1).standard_normal((m, k)).astype(np.float16)
    a[0, 77] = np.nan
    w, z = on_gpu(gate, up)
    h = host(awq.w4a16_gated(dev(a), *w, **z))
    assert np.isnan(h[0]).all() and np.isfinite(h[1:]).all()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = awq.w4a16_gated_ckpt(dev(a), *w, flags=flags, **z)
    assert int(flags.item()) == 1 << 11
    awq.w4a16_gated_ckpt(dev(a), *w, **z)          # unflagged
    assert np.isnan(host(r.g8.float())[0]).all() and np.isfinite(host(r.g8.float())[1:]).all()
    assert np.all(host(r.g_scales)[0] == 1)


def saved(m, n, seed):
    """Projections in 8 bits with scales that are no powers of two."""
    g = np.random.default_rng(seed)
    codes = g.integers(0, 256, (m, n)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x30
    scales = (0.004 * np.exp(g.standard_normal((m, -(-n // 128))))).astype(np.float32)
    return codes, scales, ref.e4m3_values(codes) * ref.spread(scales.astype(np.float64), 1, m, n)


BACKWARD = [(1, 16, 128), (3, 144, 384), (45, 2000, 1024), (64, 128, 256), (65, 272, 640),
            (129, 304, 128), (300, 1040, 384), (1100, 48, 256)]


@pytest.mark.parametrize("group,zp,act", [(128, False, "silu"), (64, True, "gelu"),
                                          (128, True, "gelu"), (64, False, "silu")])
@pytest.mark.parametrize("m,n,k", BACKWARD)
def test_gated_backward(awq, m, n, k, group, zp, act):
    gate, up = (packed(n, k, group, zp, s + m) for s in (1, 2))
    dh = (0.01 * np.random.default_rng(m).standard_normal((m, n))).astype(np.float16)
    g8, gs, g = saved(m, n, 7)
    u8, us, u = saved(m, n, 8)
    w, z = on_gpu(gate, up)
    f8 = torch.float8_e4m3fn
    say("w4a16_gated_backward", (m, n, k), group, zp, act)
    da = awq.w4a16_gated_backward(dev(dh), dev(g8).view(f8), dev(gs), dev(u8).view(f8), dev(us), *w,
                                  group=group, act=act, **z)
    dg, du, eg, eu = ref.grads(dh.astype(np.float64), g, u, act)
    want, slack = ref.backward([(dg, eg, ref.unpack(*gate, group)), (du, eu, ref.unpack(*up, group))],
                               group)
    check(host(da), want, slack)


@pytest.mark.parametrize("group,zp,with_s", [(128, False, True), (64, True, False), (128, True, True),
                                             (64, False, True)])
@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (2, 33, 256), (16, 1001, 512), (64, 64, 1152),
                                   (100, 4099, 128), (257, 300, 384), (1030, 77, 256)])
def test_gemm_backward(awq, m, n, k, group, zp, with_s):
    w = packed(n, k, group, zp, m)
    r = np.random.default_rng(m + n)
    dy = (1e-3 * np.exp(2 * r.standard_normal((m, 1))) * r.standard_normal((m, n))).astype(np.float16)
    s = np.exp(r.standard_normal(k)).astype(np.float16) if with_s else None
    say("w4a16_gemm_backward", (m, n, k), group, zp, with_s)
    da = awq.w4a16_gemm_backward(dev(dy), dev(w[0]), dev(w[1]), dev(s), group=group, zeros=dev(w[2]))
    d = dy.astype(np.float64)
    want, slack = ref.backward([(d, 0 * d, ref.unpack(*w, group))], group)
    if with_s:
        want, slack = want / s.astype(np.float64), slack / s.astype(np.float64)
    check(host(da), want, slack + 2.0 ** -22 * np.abs(want))


def test_gemm_backward_wide_ranges(awq):
    """Rows from 2^-20 to 2^15 and column groups whose steps differ by 2^16: nothing overflows or
    vanishes; a row of zeros gives zeros."""
    m, n, k = 40, 96, 512
    q, s, _ = packed(n, k, 128, False, 1)
    s = (np.abs(s) + np.float16(0.01)) * np.array([2.0 ** -12, 1, 16, 2.0 ** -8], np.float16)
    r = np.random.default_rng(2)
    dy = (r.standard_normal((m, n)) * 2.0 ** r.integers(-20, 13, (m, 1))).astype(np.float16)
    dy[5] = 0
    da = host(awq.w4a16_gemm_backward(dev(dy), dev(q), dev(s.astype(np.float16)), None))
    assert np.all(da[5] == 0)
    d = dy.astype(np.float64)
    want, slack = ref.backward([(d, 0 * d, ref.unpack(q, s.astype(np.float16), None, 128))], 128)
    fits = np.abs(want) + slack < 65504
    assert np.isinf(da[np.abs(want) - slack > 65536]).all()
    ok, used = ref.within(da[fits], want[fits], torch.float16, slack[fits])
    assert ok, used


@pytest.mark.parametrize("m", [3, 300])
def test_backward_nonfinite_rows(awq, m):
    n, k = 160, 256
    w = packed(n, k, 128, False, 1)
    dy = np.random.default_rng(1).standard_normal((m, n)).astype(np.float16)
    dy[1, 3] = np.nan
    da = host(awq.w4a16_gemm_backward(dev(dy), dev(w[0]), dev(w[1]), None))
    assert not np.isfinite(da[1]).any()
    assert np.isfinite(np.delete(da, 1, 0)).all()


def test_gradient_against_differences(awq):
    """g and u that e4m3 holds exactly (small whole numbers), so the kept activations are the true
    ones: dA against central differences of the block's float64 value along random directions."""
    m, n, k, g = 6, 32, 128, np.random.default_rng(9)
    a = np.zeros((m, k))
    a[:, :2] = g.integers(-1, 2, (m, 2))
    gate, up = ((q, np.ones_like(s), None) for q, s, _ in (packed(n, k, 128, False, s) for s in (5, 6)))
    dh = g.integers(-2, 3, (m, n)).astype(np.float16)
    w, z = on_gpu(gate, up)
    r = awq.w4a16_gated_ckpt(dev(a.astype(np.float16)), *w, **z)
    cg, cu = ref.unpack(*gate, 128)[0], ref.unpack(*up, 128)[0]
    assert np.array_equal(host(awq.fp8_dequantize(r.g8, r.g_scales)), a @ cg.T)
    da = host(awq.w4a16_gated_backward(dev(dh), r.g8, r.g_scales, r.u8, r.u_scales, *w, **z))

    def loss(x):
        return (ref.act(x @ cg.T, "silu")[0] * (x @ cu.T) * dh).sum(1)

    _, _, eg, eu = ref.grads(dh.astype(np.float64), a @ cg.T, a @ cu.T, "silu")
    dg, du, _, _ = ref.grads(dh.astype(np.float64), a @ cg.T, a @ cu.T, "silu")
    want, slack = ref.backward([(dg, eg, (cg, np.ones_like(cg))), (du, eu, (cu, np.ones_like(cu)))], 128)
    step = 1e-5
    for _ in range(8):
        v = g.standard_normal((m, k))
        diff = (loss(a + step * v) - loss(a - step * v)) / (2 * step)
        # central differences: third derivatives times step^2 (far below), rounding of the losses
        tol = (np.abs(v) * (slack + 2.0 ** -11 * np.abs(want) + 2.0 ** -25)).sum(1) + 1e-5 * (1 + np.abs(diff))
        assert np.all(np.abs((da * v).sum(1) - diff) <= tol)


def test_whole_block_forward_and_backward(awq):
    """Packing, the gated block, the down projection and both gradients as a training step over
    frozen weights makes them, through the package's own artefacts."""
    m, hidden, inter, g = 96, 256, 384, torch.Generator().manual_seed(4)

    def pack(n, k):
        wt = (0.05 * torch.randn(n, k, generator=g)).cuda()
        return awq.pack_int4(wt, torch.ones(k, device="cuda"))

    gate, up, down = pack(inter, hidden), pack(inter, hidden), pack(hidden, inter)
    x = torch.randn(m, hidden, generator=g).half().cuda()
    dy = (0.1 * torch.randn(m, hidden, generator=g)).half().cuda()
    w = (gate.qweight, gate.scales16, up.qweight, up.scales16)
    r = awq.w4a16_gated_ckpt(x, *w)
    assert torch.equal(r.H, awq.w4a16_gated(x, *w))
    y = awq.w4a16_gemm(r.H, down.qweight, down.scales16, down.s16)
    dh = awq.w4a16_gemm_backward(dy, down.qweight, down.scales16, down.s16)
    dx = awq.w4a16_gated_backward(dh, r.g8, r.g_scales, r.u8, r.u_scales, *w)
    cpu = [ref.unpack(p.qweight.cpu().numpy(), p.scales16.cpu().numpy(), None, 128)
           for p in (gate, up, down)]
    wg, wu, wd = (c * s for c, s in cpu)
    xd = host(x)
    f, df = ref.act(xd @ wg.T, "silu")
    u = xd @ wu.T
    want_y, want_dh = (f * u) @ wd.T, host(dy) @ wd
    want_dx = (want_dh * u * df) @ wg + (want_dh * f) @ wu
    rel = lambda p, q: np.linalg.norm(host(p) - q) / np.linalg.norm(q)
    # fp16 roundings of H and of the outputs, 2^-11 each and the norm of their sum below it
    assert rel(y, want_y) < 2 * 2.0 ** -11 and rel(dh, want_dh) < 2 * 2.0 ** -11
    # the kept g and u are off by up to 2^-4 each; act' and act have slopes below 1.2 in g
    assert rel(dx, want_dx) < 2.0 ** -4


def _ckpt_call(awq, x, w):
    r = awq.w4a16_gated_ckpt(x, *w)
    return awq.w4a16_gated_backward(r.H, r.g8, r.g_scales, r.u8, r.u_scales, *w)


@pytest.mark.parametrize("m,k", [(4, 1024), (150, 2048)])
def test_graph_replays_and_streams(awq, m, k):
    """Forward and backward captured together; replays follow new inputs, with eager calls on the
    same and on another stream between them; a second graph of its own runs in between too."""
    n = 208
    gate, up = packed(n, k, 128, False, 1), packed(n, k, 128, False, 2)
    w, _ = on_gpu(gate, up)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(m, k, generator=g).half().cuda()
    x2 = x.flip(0).contiguous()
    _ckpt_call(awq, x, w)
    torch.cuda.synchronize()
    graphs = []
    for src in (x, x2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = _ckpt_call(awq, src, w)
        graphs.append((gr, src, out))
    for i in range(4):
        x.copy_(torch.randn(m, k, generator=g).half())
        x2.copy_(x.flip(0))
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(s1):
            graphs[0][0].replay()
        with torch.cuda.stream(s2):
            graphs[1][0].replay()
        eager = _ckpt_call(awq, x, w)
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][2], eager), i
        assert torch.equal(graphs[1][2], _ckpt_call(awq, x2, w)), i


@pytest.mark.parametrize("m", [1, 20, 70, 200])
def test_outputs_end_where_they_should(awq, m):
    """What lies behind the last row of the outputs stays; an old workspace's contents do not
    matter; repeated calls give the same bits."""
    n, k = 176, 2048
    gate, up = packed(n, k, 64, True, 1), packed(n, k, 64, True, 2)
    w, z = on_gpu(gate, up)
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(2)).half().cuda()
    buf = torch.full((m + 1, n), 5.0, dtype=torch.float16, device="cuda")
    ws = torch.full((awq.w4a16_gated_workspace_bytes(m, n, k) + 64,), 255, dtype=torch.uint8,
                    device="cuda")
    h = awq.w4a16_gated(x, *w, group=64, out=buf[:m], workspace=ws, **z)
    assert bool((buf[m:] == 5).all())
    assert torch.equal(h, awq.w4a16_gated(x, *w, group=64, **z))
    r = awq.w4a16_gated_ckpt(x, *w, group=64, **z)
    need = awq.w4a16_gated_backward_workspace_bytes(m, n, k, 64, True)
    buf = torch.full((m + 1, k), 5.0, dtype=torch.float16, device="cuda")
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    args = (r.H, r.g8, r.g_scales, r.u8, r.u_scales, *w)
    d = awq.w4a16_gated_backward(*args, group=64, out=buf[:m], workspace=ws, **z)
    assert bool((buf[m:] == 5).all())
    assert bool((ws[need:] == 255).all())
    assert torch.equal(d, awq.w4a16_gated_backward(*args, group=64, **z))


def test_output_apart_from_inputs(awq):
    """An output that shares memory with an input, whole or in part, is refused; one that starts
    where the input ends is not."""
    n = k = 256
    gate, up = packed(n, k, 128, False, 1), packed(n, k, 128, False, 2)
    w, _ = on_gpu(gate, up)
    buf = torch.randn(12, k, generator=torch.Generator().manual_seed(3)).half().cuda()
    x = buf[4:8]
    r = awq.w4a16_gated_ckpt(x, *w)
    saved8 = (r.g8, r.g_scales, r.u8, r.u_scales)
    for out in (buf[4:8], buf[3:7], buf[7:11]):
        with pytest.raises(ValueError, match="share memory"):
            awq.w4a16_gated(x, *w, out=out)
        with pytest.raises(ValueError, match="share memory"):
            awq.w4a16_gemm_backward(x, w[0], w[1], None, out=out)
        with pytest.raises(ValueError, match="share memory"):
            awq.w4a16_gated_backward(x, *saved8, *w, out=out)
    want = awq.w4a16_gated(x, *w)
    for out in (buf[:4], buf[8:]):
        assert torch.equal(awq.w4a16_gated(x, *w, out=out), want)
