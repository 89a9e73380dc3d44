"""Python face of libawq: the four C-ABI calls on torch tensors.

Argument marshalling only -- torch supplies device memory and the current HIP stream; every step
of the computation runs in the library's HIP kernels. Names follow the C ABI (include/awq.h).
Nothing here synchronises: results are ready when the current stream reaches them.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _lib
from ._lib import AwqCfg, check

_DT = {torch.float32: _lib.AWQ_F32, torch.float16: _lib.AWQ_F16, torch.bfloat16: _lib.AWQ_BF16}


@dataclasses.dataclass(frozen=True)
class AwqConfig:
    """bits in {3, 4}; group = 128 input channels per step; n_grid alpha points i/(n_grid-1);
    s = max(s_X, s_floor)^alpha; form "direct" (contract X with every error matrix) or "gram"
    (form H = X^T X once, then contract each error matrix with H); the clipping search tries
    n_clip ratios from 1 down to clip_min; zero_point selects unsigned codes with a zero point
    per (row, group) instead of symmetric ones; group 128 or 64."""
    bits: int = 4
    group: int = 128
    n_grid: int = 20
    s_floor: float = 1e-5
    form: str = "direct"
    n_clip: int = 11
    clip_min: float = 0.5
    zero_point: bool = False

    def c(self) -> AwqCfg:
        forms = {"direct": _lib.AWQ_FORM_DIRECT, "gram": _lib.AWQ_FORM_GRAM}
        if self.form not in forms:
            raise ValueError(f"form must be one of {sorted(forms)}, got {self.form!r}")
        return AwqCfg(self.bits, self.group, self.n_grid, self.s_floor, forms[self.form],
                      self.n_clip, self.clip_min, int(bool(self.zero_point)))


def _dev(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _flags(device, flags):
    if flags is None:
        return torch.zeros(1, dtype=torch.int32, device=device)
    return flags


@dataclasses.dataclass
class SearchResult:
    losses: torch.Tensor   # fp64 [n_grid]
    best: torch.Tensor     # int32 [1]
    s_best: torch.Tensor   # fp32 [K]
    flags: torch.Tensor    # int32 [1] holding the uint32 flag bits


@dataclasses.dataclass
class PackResult:
    qweight: torch.Tensor   # int32 [N, K/8] holding the uint32 words
    scales16: torch.Tensor  # fp16 [N, K/group]
    s16: torch.Tensor       # fp16 [K]
    codes: torch.Tensor | None
    flags: torch.Tensor
    zeros: torch.Tensor | None = None   # uint8 [N, K/group] for zero-point codes


def act_stats_workspace_bytes(M: int, K: int) -> int:
    return int(_lib.load().awq_act_stats_workspace_bytes(M, K))


def search_workspace_bytes(M: int, N: int, K: int, x_dtype: torch.dtype, cfg: AwqConfig) -> int:
    c = cfg.c()
    return int(_lib.load().awq_search_workspace_bytes(M, N, K, _DT[x_dtype], c))


def act_stats(X: torch.Tensor, flags: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """s_X = mean over tokens of |X| per input channel (fp32 [K]). X may be a row-strided view
    (unit column stride, row stride a multiple of 8 elements)."""
    lib = _lib.load()
    if not X.is_cuda or X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a 2-D device tensor with unit column stride")
    M, K = X.shape
    ldx = X.stride(0) if M > 1 else K
    flags = _flags(X.device, flags)
    nbytes = lib.awq_act_stats_workspace_bytes(M, K)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=X.device)
    sx = torch.empty(K, dtype=torch.float32, device=X.device)
    check("awq_act_stats", lib.awq_act_stats(X.data_ptr(), _DT[X.dtype], M, K, ldx, sx.data_ptr(),
                                             flags.data_ptr(), workspace.data_ptr(),
                                             workspace.numel(), _stream(X)))
    return sx, flags


def act_stats_noalloc(X: torch.Tensor, sx: torch.Tensor,
                      flags: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """act_stats into caller-provided sx (fp32 [K]) and flags (int32 [1]) with the library's
    static scratch instead of a workspace: the C call allocates nothing, and neither does this
    binding (usable under graph capture). Overlapping calls on one GPU race."""
    lib = _lib.load()
    if not X.is_cuda or X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a 2-D device tensor with unit column stride")
    M, K = X.shape
    _dev(sx, "sx")
    _dev(flags, "flags")
    if sx.shape != (K,) or sx.dtype != torch.float32 or flags.numel() != 1 or \
            flags.dtype != torch.int32:
        raise ValueError("sx must be fp32 [K] and flags int32 [1]")
    ldx = X.stride(0) if M > 1 else K
    check("awq_act_stats_noalloc", lib.awq_act_stats_noalloc(
        X.data_ptr(), _DT[X.dtype], M, K, ldx, sx.data_ptr(), flags.data_ptr(), _stream(X)))
    return sx, flags


def search_layer(W: torch.Tensor, X: torch.Tensor, sx: torch.Tensor,
                 cfg: AwqConfig = AwqConfig(), flags: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None,
                 stage_ms: dict | None = None) -> SearchResult:
    """Grid search over alpha: losses L_i, best index, s_best = s_{i*}.

    With a dict as `stage_ms` the profiled C call is used: it fills the dict with the duration
    of each kernel of the search (HIP events on the current stream) and blocks until done."""
    lib = _lib.load()
    for t, nm in ((W, "W"), (X, "X"), (sx, "sx")):
        _dev(t, nm)
    N, K = W.shape
    M = X.shape[0]
    if X.shape[1] != K or sx.shape != (K,) or sx.dtype != torch.float32:
        raise ValueError("shape mismatch: W [N,K], X [M,K], sx fp32 [K]")
    c = cfg.c()
    flags = _flags(W.device, flags)
    nbytes = lib.awq_search_workspace_bytes(M, N, K, _DT[X.dtype], c)
    if nbytes == 0:
        raise ValueError("invalid shape or config for the search")
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    losses = torch.empty(cfg.n_grid, dtype=torch.float64, device=W.device)
    best = torch.empty(1, dtype=torch.int32, device=W.device)
    s_best = torch.empty(K, dtype=torch.float32, device=W.device)
    args = (W.data_ptr(), _DT[W.dtype], N, K, X.data_ptr(), _DT[X.dtype], M, sx.data_ptr(), c,
            losses.data_ptr(), best.data_ptr(), s_best.data_ptr(), flags.data_ptr(),
            workspace.data_ptr(), workspace.numel(), _stream(W))
    if stage_ms is None:
        check("awq_search_layer", lib.awq_search_layer(*args))
    else:
        ms = (ctypes.c_float * len(_lib.SEARCH_STAGES))()
        check("awq_search_layer_profiled", lib.awq_search_layer_profiled(*args, ms))
        stage_ms.update({k: float(v) for k, v in zip(_lib.SEARCH_STAGES, ms)})
    return SearchResult(losses, best, s_best, flags)


def stats_search_layer(W: torch.Tensor, X: torch.Tensor, cfg: AwqConfig = AwqConfig(),
                       flags: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       stage_ms: dict | None = None) -> tuple[torch.Tensor, SearchResult]:
    """act_stats and search_layer in one call: returns (s_X, result), s_X identical to what
    act_stats gives for this X. `stage_ms` as in search_layer, with the statistics counted in the
    X preparation stage."""
    lib = _lib.load()
    for t, nm in ((W, "W"), (X, "X")):
        _dev(t, nm)
    N, K = W.shape
    M = X.shape[0]
    if X.shape[1] != K:
        raise ValueError("shape mismatch: W [N,K], X [M,K]")
    c = cfg.c()
    flags = _flags(W.device, flags)
    nbytes = lib.awq_search_workspace_bytes(M, N, K, _DT[X.dtype], c)
    if nbytes == 0:
        raise ValueError("invalid shape or config for the search")
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    sx = torch.empty(K, dtype=torch.float32, device=W.device)
    losses = torch.empty(cfg.n_grid, dtype=torch.float64, device=W.device)
    best = torch.empty(1, dtype=torch.int32, device=W.device)
    s_best = torch.empty(K, dtype=torch.float32, device=W.device)
    ms = (ctypes.c_float * len(_lib.SEARCH_STAGES))() if stage_ms is not None else None
    check("awq_stats_search_layer", lib.awq_stats_search_layer(
        W.data_ptr(), _DT[W.dtype], N, K, X.data_ptr(), _DT[X.dtype], M, c, sx.data_ptr(),
        losses.data_ptr(), best.data_ptr(), s_best.data_ptr(), flags.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _stream(W), ms))
    if stage_ms is not None:
        stage_ms.update({k: float(v) for k, v in zip(_lib.SEARCH_STAGES, ms)})
    return sx, SearchResult(losses, best, s_best, flags)


@dataclasses.dataclass
class ClipResult:
    clip: torch.Tensor               # fp32 [N, K/group]: the chosen ratios
    err: torch.Tensor | None         # fp32 [n_clip, N, K/group]: group error of every ratio
    flags: torch.Tensor


def clip_workspace_bytes(M: int, N: int, K: int, x_dtype: torch.dtype, cfg: AwqConfig) -> int:
    return int(_lib.load().awq_clip_workspace_bytes(M, N, K, _DT[x_dtype], cfg.c()))


def clip_search(W: torch.Tensor, X: torch.Tensor, s: torch.Tensor, cfg: AwqConfig = AwqConfig(),
                with_err: bool = False, flags: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> ClipResult:
    """Per (row, group), the clip ratio of the grid whose clipped quantization of W s gives the
    smallest group output error."""
    lib = _lib.load()
    for t, nm in ((W, "W"), (X, "X"), (s, "s")):
        _dev(t, nm)
    N, K = W.shape
    M = X.shape[0]
    if X.shape[1] != K or s.shape != (K,) or s.dtype != torch.float32:
        raise ValueError("shape mismatch: W [N,K], X [M,K], s fp32 [K]")
    c = cfg.c()
    flags = _flags(W.device, flags)
    nbytes = lib.awq_clip_workspace_bytes(M, N, K, _DT[X.dtype], c)
    if nbytes == 0:
        raise ValueError("invalid shape or config for the clipping search")
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    G = K // cfg.group
    clip = torch.empty((N, G), dtype=torch.float32, device=W.device)
    err = torch.empty((cfg.n_clip, N, G), dtype=torch.float32, device=W.device) \
        if with_err else None
    check("awq_clip_search", lib.awq_clip_search(
        W.data_ptr(), _DT[W.dtype], N, K, X.data_ptr(), _DT[X.dtype], M, s.data_ptr(), c,
        clip.data_ptr(), err.data_ptr() if err is not None else None, flags.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _stream(W)))
    return ClipResult(clip, err, flags)


def clip_search_gram(W: torch.Tensor, s: torch.Tensor, search_workspace: torch.Tensor,
                     cfg: AwqConfig = AwqConfig(form="gram"), with_err: bool = False,
                     flags: torch.Tensor | None = None) -> ClipResult:
    """The clipping search of clip_search, with H_gg and d taken from the workspace of the
    Gram-form search (search_layer / search_layers with this `cfg` and an explicit workspace)
    that just ran on the same X, instead of being formed from X again."""
    lib = _lib.load()
    _dev(W, "W")
    _dev(s, "s")
    _dev(search_workspace, "search_workspace")
    N, K = W.shape
    if s.shape != (K,) or s.dtype != torch.float32:
        raise ValueError("shape mismatch: W [N,K], s fp32 [K]")
    if cfg.form != "gram":
        raise ValueError("clip_search_gram needs the configuration of a Gram-form search")
    c = cfg.c()
    if lib.awq_clip_search_gram_ws_bytes(K, c) == 0:
        raise ValueError("invalid shape or config for the clipping search")
    flags = _flags(W.device, flags)
    G = K // cfg.group
    clip = torch.empty((N, G), dtype=torch.float32, device=W.device)
    err = torch.empty((cfg.n_clip, N, G), dtype=torch.float32, device=W.device) \
        if with_err else None
    check("awq_clip_search_gram", lib.awq_clip_search_gram(
        W.data_ptr(), _DT[W.dtype], N, K, s.data_ptr(), c, search_workspace.data_ptr(),
        search_workspace.numel() * search_workspace.element_size(), clip.data_ptr(),
        err.data_ptr() if err is not None else None, flags.data_ptr(), _stream(W)))
    return ClipResult(clip, err, flags)


def search_layers(Ws: list, X: torch.Tensor, sx: torch.Tensor | None,
                  cfg: AwqConfig = AwqConfig(), flags: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None):
    """One alpha for several weights that read the same X (rows stacked, no copy). With
    sx = None, s_X is taken in the same call (awq_stats_search_layers) and (s_X, result) is
    returned; otherwise the result."""
    lib = _lib.load()
    for i, W in enumerate(Ws):
        _dev(W, f"W[{i}]")
    _dev(X, "X")
    if sx is not None:
        _dev(sx, "sx")
    K = X.shape[1]
    if any(W.shape[1] != K or W.dtype != Ws[0].dtype for W in Ws):
        raise ValueError("every W must be [N_l, K] with the dtype of W[0]")
    Ns = [int(W.shape[0]) for W in Ws]
    M, N = X.shape[0], sum(Ns)
    c = cfg.c()
    flags = _flags(X.device, flags)
    nbytes = lib.awq_search_workspace_bytes(M, N, K, _DT[X.dtype], c)
    if nbytes == 0:
        raise ValueError("invalid shape or config for the search")
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
    losses = torch.empty(cfg.n_grid, dtype=torch.float64, device=X.device)
    best = torch.empty(1, dtype=torch.int32, device=X.device)
    s_best = torch.empty(K, dtype=torch.float32, device=X.device)
    ptrs = (ctypes.c_void_p * len(Ws))(*[W.data_ptr() for W in Ws])
    rows = (ctypes.c_int64 * len(Ws))(*Ns)
    if sx is None:
        sx_out = torch.empty(K, dtype=torch.float32, device=X.device)
        check("awq_stats_search_layers", lib.awq_stats_search_layers(
            ptrs, rows, len(Ws), _DT[Ws[0].dtype], K, X.data_ptr(), _DT[X.dtype], M, c,
            sx_out.data_ptr(), losses.data_ptr(), best.data_ptr(), s_best.data_ptr(),
            flags.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(X)))
        return sx_out, SearchResult(losses, best, s_best, flags)
    if sx.shape != (K,) or sx.dtype != torch.float32:
        raise ValueError("sx must be fp32 [K]")
    check("awq_search_layers", lib.awq_search_layers(
        ptrs, rows, len(Ws), _DT[Ws[0].dtype], K, X.data_ptr(), _DT[X.dtype], M, sx.data_ptr(),
        c, losses.data_ptr(), best.data_ptr(), s_best.data_ptr(), flags.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _stream(X)))
    return SearchResult(losses, best, s_best, flags)


def fold_scale(prev: torch.Tensor, s: torch.Tensor, axis: int,
               flags: torch.Tensor | None = None) -> torch.Tensor:
    """In place: prev /= s along `axis` (1: columns of a [rows, K] parameter such as a norm
    weight [1, K]; 0: rows, e.g. a previous linear layer's output channels). Returns flags."""
    lib = _lib.load()
    _dev(s, "s")
    if not prev.is_cuda or prev.dim() != 2 or prev.stride(1) != 1:
        raise ValueError("prev must be a 2-D device tensor with unit column stride")
    rows, cols = prev.shape
    if s.dtype != torch.float32 or s.shape != ((cols,) if axis == 1 else (rows,)):
        raise ValueError("s must be fp32 with one entry per folded channel")
    flags = _flags(prev.device, flags)
    check("awq_fold_scale", lib.awq_fold_scale(prev.data_ptr(), _DT[prev.dtype], rows, cols,
                                               prev.stride(0) if rows > 1 else cols,
                                               s.data_ptr(), axis, flags.data_ptr(),
                                               _stream(prev)))
    return flags


def pack_int4(W: torch.Tensor, s: torch.Tensor, cfg: AwqConfig = AwqConfig(),
              with_codes: bool = False, flags: torch.Tensor | None = None,
              clip: torch.Tensor | None = None) -> PackResult:
    """Packed codes of Q(W s) (clipped by the per-group ratios `clip`, if given), fp16 group
    steps and fp16 s."""
    lib = _lib.load()
    _dev(W, "W")
    _dev(s, "s")
    N, K = W.shape
    if s.shape != (K,) or s.dtype != torch.float32:
        raise ValueError("s must be fp32 [K]")
    if clip is not None:
        _dev(clip, "clip")
        if clip.shape != (N, K // cfg.group) or clip.dtype != torch.float32:
            raise ValueError("clip must be fp32 [N, K/group]")
    c = cfg.c()
    flags = _flags(W.device, flags)
    qweight = torch.empty((N, K // 8), dtype=torch.int32, device=W.device)
    scales16 = torch.empty((N, K // cfg.group), dtype=torch.float16, device=W.device)
    s16 = torch.empty(K, dtype=torch.float16, device=W.device)
    codes = torch.empty((N, K), dtype=torch.int8, device=W.device) if with_codes else None
    zeros = torch.empty((N, K // cfg.group), dtype=torch.uint8, device=W.device) \
        if cfg.zero_point else None
    check("awq_pack_int4", lib.awq_pack_int4(
        W.data_ptr(), _DT[W.dtype], N, K, s.data_ptr(),
        clip.data_ptr() if clip is not None else None, c, qweight.data_ptr(),
        scales16.data_ptr(), zeros.data_ptr() if zeros is not None else None, s16.data_ptr(),
        codes.data_ptr() if codes is not None else None, flags.data_ptr(), _stream(W)))
    return PackResult(qweight, scales16, s16, codes, flags, zeros)


def _w4a16_check(A, qweight, scales16, s16, group, zeros):
    for t, nm in ((A, "A"), (qweight, "qweight"), (scales16, "scales16")):
        _dev(t, nm)
    if s16 is not None:
        _dev(s16, "s16")
    M, K = A.shape
    N = qweight.shape[0]
    if A.dtype != torch.float16 or scales16.dtype != torch.float16 or \
            (s16 is not None and s16.dtype != torch.float16):
        raise ValueError("A, scales16 and s16 must be fp16")
    if qweight.shape != (N, K // 8) or scales16.shape != (N, K // group) or \
            (s16 is not None and s16.shape != (K,)):
        raise ValueError("packed artefact shapes do not match A")
    if zeros is not None:
        _dev(zeros, "zeros")
        if zeros.shape != (N, K // group) or zeros.dtype != torch.uint8:
            raise ValueError("zeros must be uint8 [N, K/group]")
    return M, N, K


def w4a16_gemm(A: torch.Tensor, qweight: torch.Tensor, scales16: torch.Tensor,
               s16: torch.Tensor | None, group: int = 128, out: torch.Tensor | None = None,
               zeros: torch.Tensor | None = None) -> torch.Tensor:
    """Y = (A / s) (c(q) * step)^T, fp16 [M, N], c(q) = q (symmetric) or q - z (zeros given);
    s16 = None when s^-1 is folded into A's producer."""
    lib = _lib.load()
    M, N, K = _w4a16_check(A, qweight, scales16, s16, group, zeros)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=A.device)
    check("w4a16_gemm", lib.w4a16_gemm(A.data_ptr(), M, N, K, group, qweight.data_ptr(),
                                       scales16.data_ptr(),
                                       zeros.data_ptr() if zeros is not None else None,
                                       s16.data_ptr() if s16 is not None else None, out.data_ptr(),
                                       _stream(A)))
    return out


def w4a16_gemm_workspace_bytes(M: int, N: int, K: int, group: int = 128) -> int:
    """Bytes of the w4a16_gemm_ws workspace for these sizes (0: none needed)."""
    return int(_lib.load().w4a16_gemm_workspace_bytes(M, N, K, group))


# w4a16_gemm_ws workspaces kept per (device, stream), so that calls on one stream share one
_W4A16_WS: dict = {}


def w4a16_gemm_workspace(device: torch.device, nbytes: int) -> torch.Tensor:
    """The cached w4a16_gemm_ws workspace of the current stream on `device`, at least `nbytes`
    bytes (a larger one replaces a smaller one)."""
    key = (device.index, torch.cuda.current_stream(device).cuda_stream)
    ws = _W4A16_WS.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
        _W4A16_WS[key] = ws
    return ws


def w4a16_gemm_ws(A: torch.Tensor, qweight: torch.Tensor, scales16: torch.Tensor,
                  s16: torch.Tensor | None, group: int = 128, out: torch.Tensor | None = None,
                  zeros: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """w4a16_gemm with a workspace (K split over workgroups for M <= 64). workspace: a uint8
    device tensor of at least w4a16_gemm_workspace_bytes bytes, or None for the cached one of
    the current stream."""
    lib = _lib.load()
    M, N, K = _w4a16_check(A, qweight, scales16, s16, group, zeros)
    need = w4a16_gemm_workspace_bytes(M, N, K, group)
    if workspace is None:
        workspace = w4a16_gemm_workspace(A.device, need)
    else:
        _dev(workspace, "workspace")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=A.device)
    check("w4a16_gemm_ws", lib.w4a16_gemm_ws(
        A.data_ptr(), M, N, K, group, qweight.data_ptr(), scales16.data_ptr(),
        zeros.data_ptr() if zeros is not None else None,
        s16.data_ptr() if s16 is not None else None, out.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(A)))
    return out


FP8 = torch.float8_e4m3fn


@dataclasses.dataclass
class Fp8Result:
    q: torch.Tensor        # float8_e4m3fn [M, K]
    scales: torch.Tensor   # fp32 [ceil(M / block_rows), ceil(K / 128)], powers of two
    flags: torch.Tensor | None = None   # the tensor given to the call


def _same_device(ref: torch.Tensor, *named) -> None:
    device = ref.device
    for t, nm in named:
        if t is not None and t.device != device:
            raise ValueError(f"{nm} must be on {device}")


def _flags_arg(flags, device):
    """The pointer of an optional flag word."""
    if flags is None:
        return None
    _dev(flags, "flags")
    if flags.dtype != torch.int32 or flags.numel() != 1 or flags.device != device:
        raise ValueError(f"flags must be int32 [1] on {device}")
    return flags.data_ptr()


def _launch(call: str, fn, device: torch.device, *args) -> None:
    """fn(*args, stream) on the current stream of `device`, with that device current. (The raw
    stream handle and the check before the device guard keep a small call's host time near the
    launch itself.)"""
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if torch.cuda.current_device() == device.index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status:
        check(call, status)


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two contiguous tensors share memory."""
    pa, pb = a.data_ptr(), b.data_ptr()
    return pa < pb + b.numel() * b.element_size() and pb < pa + a.numel() * a.element_size()


def _out(out, shape, dtype, device, *inputs) -> torch.Tensor:
    """The caller's output (checked), or a new one. Workgroups read the inputs while others write,
    so the output must be apart from them."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _dev(out, "out")
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype or out.device != device:
        raise ValueError(f"out must be {dtype} {tuple(shape)} on {device}")
    if any(t is not None and _overlap(out, t) for t in inputs):
        raise ValueError("out must not share memory with an input")
    return out


def _scratch(workspace, nbytes: int, device):
    """A workspace of `nbytes`: the caller's (checked), or one of this call's own from torch's
    allocator, which orders its reuse by stream and keeps a captured graph's apart."""
    if workspace is not None:
        _dev(workspace, "workspace")
        if workspace.device != device or workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace must hold {nbytes} bytes on {device}")
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _blocks_shape(M: int, K: int, block_rows: int):
    return ((M + block_rows - 1) // block_rows, (K + 127) // 128)


def _fp8_check(q, scales, block_rows, name):
    _dev(q, name)
    _dev(scales, "the scales of " + name)
    if q.dim() != 2 or q.dtype != FP8:
        raise ValueError(f"{name} must be float8_e4m3fn [rows, columns]")
    M, K = q.shape
    if scales.dtype != torch.float32 or scales.shape != _blocks_shape(M, K, block_rows):
        raise ValueError(f"{name}: the scales must be fp32, one per block of {block_rows} x 128")
    return M, K


def fp8_quantize(X: torch.Tensor, block_rows: int = 1,
                 flags: torch.Tensor | None = None) -> Fp8Result:
    """X in 8 bits: e4m3 codes with one power-of-two scale per block of 128 columns by 1 row
    (activations) or 128 rows (weights). X may be a row-strided view (unit column stride, row
    stride a multiple of 8 elements); its columns are a multiple of 16. flags: an int32 [1] tensor
    that collects the library's flag bits, or None for none."""
    lib = _lib.load()
    if not X.is_cuda or X.dim() != 2 or (X.stride(1) != 1 and X.shape[1] > 1):
        raise ValueError("X must be a 2-D device tensor with unit column stride")
    if X.dtype not in _DT:
        raise ValueError("X must be fp16, bf16 or fp32")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    M, K = X.shape
    dev = X.device
    fl = _flags_arg(flags, dev)
    q = torch.empty((M, K), dtype=FP8, device=dev)
    scales = torch.empty(_blocks_shape(M, K, block_rows), dtype=torch.float32, device=dev)
    _launch("awq_fp8_quantize", lib.awq_fp8_quantize, dev,
            X.data_ptr(), _DT[X.dtype], M, K, X.stride(0) if M > 1 else K, block_rows,
            q.data_ptr(), scales.data_ptr(), fl)
    return Fp8Result(q, scales, flags)


def fp8_dequantize(q: torch.Tensor, scales: torch.Tensor, block_rows: int = 1,
                   dtype: torch.dtype = torch.float16,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """The values code * scale of fp8_quantize's result, in `dtype`."""
    lib = _lib.load()
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    _fp8_check(q, scales, block_rows, "q")
    if dtype not in _DT:
        raise ValueError("dtype must be fp16, bf16 or fp32")
    _same_device(q, (scales, "scales"))
    M, K = q.shape
    out = _out(out, (M, K), dtype, q.device, q, scales)
    _launch("awq_fp8_dequantize", lib.awq_fp8_dequantize, q.device,
            q.data_ptr(), scales.data_ptr(), M, K, block_rows, _DT[dtype], out.data_ptr())
    return out


def fp8_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    """Bytes of the fp8_gemm workspace for these sizes (0: none needed)."""
    return int(_lib.load().awq_fp8_gemm_workspace_bytes(M, N, K))


def fp8_gemm(A8: torch.Tensor, a_scales: torch.Tensor, W8: torch.Tensor, w_scales: torch.Tensor,
             out_dtype: torch.dtype = torch.float16, out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Y = (A8 a_scales) (W8 w_scales)^T, fp16 or bf16 [M, N], from fp8_quantize's formats: A8 in
    blocks of 1 x 128, W8 [N, K] in blocks of 128 x 128."""
    lib = _lib.load()
    M, K = _fp8_check(A8, a_scales, 1, "A8")
    N, KW = _fp8_check(W8, w_scales, 128, "W8")
    if KW != K:
        raise ValueError("A8 and W8 must have the same number of columns")
    if out_dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("out_dtype must be fp16 or bf16")
    dev = A8.device
    _same_device(A8, (a_scales, "a_scales"), (W8, "W8"), (w_scales, "w_scales"))
    out = _out(out, (M, N), out_dtype, dev, A8, a_scales, W8, w_scales)
    ws = _scratch(workspace, lib.awq_fp8_gemm_workspace_bytes(M, N, K), dev)
    _launch("awq_fp8_gemm", lib.awq_fp8_gemm, dev,
            A8.data_ptr(), a_scales.data_ptr(), W8.data_ptr(), w_scales.data_ptr(), M, N, K,
            _DT[out_dtype], out.data_ptr(), ws.data_ptr() if ws is not None else None,
            ws.numel() * ws.element_size() if ws is not None else 0)
    return out


_ACTS = {"silu": _lib.AWQ_ACT_SILU, "gelu": _lib.AWQ_ACT_GELU}


def _packed_check(x, K, qweight, scales16, zeros, group, name):
    """Checks one packed weight that goes with x on its device; returns N."""
    _dev(qweight, f"{name} qweight")
    _dev(scales16, f"{name} scales16")
    if group not in (64, 128):
        raise ValueError("group must be 64 or 128")
    N = qweight.shape[0] if qweight.dim() == 2 else -1
    if qweight.dtype != torch.int32 or tuple(qweight.shape) != (N, K // 8):
        raise ValueError(f"{name} qweight must be int32 [N, K/8]")
    if scales16.dtype != torch.float16 or tuple(scales16.shape) != (N, K // group):
        raise ValueError(f"{name} scales16 must be fp16 [N, K/group]")
    if zeros is not None:
        _dev(zeros, f"{name} zeros")
        if zeros.dtype != torch.uint8 or tuple(zeros.shape) != (N, K // group):
            raise ValueError(f"{name} zeros must be uint8 [N, K/group]")
    _same_device(x, (qweight, f"{name} qweight"), (scales16, f"{name} scales16"),
                 (zeros, f"{name} zeros"))
    return N


def _in_channels(qweight, name):
    if qweight.dim() != 2:
        raise ValueError(f"{name} must be int32 [N, K/8]")
    return qweight.shape[1] * 8


def _packed_arg(qweight, scales16, zeros):
    return _lib.AwqPacked(qweight.data_ptr(), scales16.data_ptr(),
                          zeros.data_ptr() if zeros is not None else None)


def _gated_check(x, K, gate, up, group, act):
    N = _packed_check(x, K, *gate, group, "gate")
    if _packed_check(x, K, *up, group, "up") != N:
        raise ValueError("gate and up must have the same number of rows")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    if (gate[2] is None) != (up[2] is None):
        raise ValueError("zeros must be given for both gate and up, or for neither")
    return N


def _halves(t, name):
    _dev(t, name)
    if t.dim() != 2 or t.dtype != torch.float16:
        raise ValueError(f"{name} must be fp16 [rows, columns]")


def _ws_args(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def w4a16_gated_workspace_bytes(M: int, N: int, K: int, keep: bool = False) -> int:
    """Bytes of the w4a16_gated (keep: w4a16_gated_ckpt) workspace (0: none needed)."""
    return int(_lib.load().w4a16_gated_workspace_bytes(M, N, K, int(keep)))


def w4a16_gated(A: torch.Tensor, gate_qweight: torch.Tensor, gate_scales16: torch.Tensor,
                up_qweight: torch.Tensor, up_scales16: torch.Tensor, group: int = 128,
                act: str = "silu", out: torch.Tensor | None = None,
                gate_zeros: torch.Tensor | None = None, up_zeros: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """H = act(A Wg^T) * (A Wu^T), fp16 [M, N], on two packed weights (pack_int4's artefacts) whose
    s is folded into A's producer; act "silu" or "gelu" (tanh form)."""
    lib = _lib.load()
    _halves(A, "A")
    M, K = A.shape
    gate = (gate_qweight, gate_scales16, gate_zeros)
    up = (up_qweight, up_scales16, up_zeros)
    N = _gated_check(A, K, gate, up, group, act)
    out = _out(out, (M, N), torch.float16, A.device, A, *gate, *up)
    ws = _scratch(workspace, lib.w4a16_gated_workspace_bytes(M, N, K, 0), A.device)
    _launch("w4a16_gated", lib.w4a16_gated, A.device,
            A.data_ptr(), M, N, K, group, _ACTS[act], _packed_arg(*gate), _packed_arg(*up),
            out.data_ptr(), *_ws_args(ws))
    return out


@dataclasses.dataclass
class GatedResult:
    H: torch.Tensor          # fp16 [M, N]
    g8: torch.Tensor         # float8_e4m3fn [M, N]: A Wg^T
    g_scales: torch.Tensor   # fp32 [M, ceil(N / 128)]
    u8: torch.Tensor         # float8_e4m3fn [M, N]: A Wu^T
    u_scales: torch.Tensor
    flags: torch.Tensor | None = None


def w4a16_gated_ckpt(A: torch.Tensor, gate_qweight: torch.Tensor, gate_scales16: torch.Tensor,
                     up_qweight: torch.Tensor, up_scales16: torch.Tensor, group: int = 128,
                     act: str = "silu", gate_zeros: torch.Tensor | None = None,
                     up_zeros: torch.Tensor | None = None, flags: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None) -> GatedResult:
    """w4a16_gated that also keeps both projections in 8 bits (fp8_quantize's format, blocks of
    1 x 128) for w4a16_gated_backward; N a multiple of 16. flags as in fp8_quantize."""
    lib = _lib.load()
    _halves(A, "A")
    M, K = A.shape
    gate = (gate_qweight, gate_scales16, gate_zeros)
    up = (up_qweight, up_scales16, up_zeros)
    N = _gated_check(A, K, gate, up, group, act)
    dev = A.device
    fl = _flags_arg(flags, dev)
    H = torch.empty((M, N), dtype=torch.float16, device=dev)
    g8, u8 = (torch.empty((M, N), dtype=FP8, device=dev) for _ in range(2))
    gs, us = (torch.empty(_blocks_shape(M, N, 1), dtype=torch.float32, device=dev)
              for _ in range(2))
    ws = _scratch(workspace, lib.w4a16_gated_workspace_bytes(M, N, K, 1), dev)
    _launch("w4a16_gated_ckpt", lib.w4a16_gated_ckpt, dev,
            A.data_ptr(), M, N, K, group, _ACTS[act], _packed_arg(*gate), _packed_arg(*up),
            H.data_ptr(), g8.data_ptr(), gs.data_ptr(), u8.data_ptr(), us.data_ptr(),
            fl, *_ws_args(ws))
    return GatedResult(H, g8, gs, u8, us, flags)


def w4a16_gated_backward_workspace_bytes(M: int, N: int, K: int, group: int = 128,
                                         zero_point: bool = False) -> int:
    return int(_lib.load().w4a16_gated_backward_workspace_bytes(M, N, K, group, int(zero_point)))


def w4a16_gated_backward(dH: torch.Tensor, g8: torch.Tensor, g_scales: torch.Tensor,
                         u8: torch.Tensor, u_scales: torch.Tensor, gate_qweight: torch.Tensor,
                         gate_scales16: torch.Tensor, up_qweight: torch.Tensor,
                         up_scales16: torch.Tensor, group: int = 128, act: str = "silu",
                         out: torch.Tensor | None = None, gate_zeros: torch.Tensor | None = None,
                         up_zeros: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None) -> torch.Tensor:
    """dA, fp16 [M, K]: the gradient of w4a16_gated's input from dH and the kept projections
    (dg = dH u act'(g), du = dH act(g), dA = dg Wg + du Wu); the packed weights are constants."""
    lib = _lib.load()
    _halves(dH, "dH")
    M, N = dH.shape
    for q, s, nm in ((g8, g_scales, "g8"), (u8, u_scales, "u8")):
        _fp8_check(q, s, 1, nm)
        if tuple(q.shape) != (M, N):
            raise ValueError(f"{nm} must have dH's shape")
    K = _in_channels(gate_qweight, "gate qweight")
    gate = (gate_qweight, gate_scales16, gate_zeros)
    up = (up_qweight, up_scales16, up_zeros)
    if _gated_check(dH, K, gate, up, group, act) != N:
        raise ValueError("the weights' rows must be dH's columns")
    _same_device(dH, (g8, "g8"), (g_scales, "g_scales"), (u8, "u8"), (u_scales, "u_scales"))
    out = _out(out, (M, K), torch.float16, dH.device, dH, g8, g_scales, u8, u_scales, *gate, *up)
    ws = _scratch(workspace, lib.w4a16_gated_backward_workspace_bytes(
        M, N, K, group, int(gate_zeros is not None)), dH.device)
    _launch("w4a16_gated_backward", lib.w4a16_gated_backward, dH.device,
            dH.data_ptr(), g8.data_ptr(), g_scales.data_ptr(), u8.data_ptr(), u_scales.data_ptr(),
            M, N, K, group, _ACTS[act], _packed_arg(*gate), _packed_arg(*up), out.data_ptr(),
            *_ws_args(ws))
    return out


def w4a16_gemm_backward_workspace_bytes(M: int, N: int, K: int, group: int = 128,
                                        zero_point: bool = False) -> int:
    return int(_lib.load().w4a16_gemm_backward_workspace_bytes(M, N, K, group, int(zero_point)))


def w4a16_gemm_backward(dY: torch.Tensor, qweight: torch.Tensor, scales16: torch.Tensor,
                        s16: torch.Tensor | None, group: int = 128,
                        out: torch.Tensor | None = None, zeros: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None) -> torch.Tensor:
    """dA = (dY (c(q) * step)) / s, fp16 [M, K]: the gradient of w4a16_gemm's input; s16 = None
    when s^-1 is folded into A's producer."""
    lib = _lib.load()
    _halves(dY, "dY")
    M, N = dY.shape
    K = _in_channels(qweight, "qweight")
    if _packed_check(dY, K, qweight, scales16, zeros, group, "the weight's") != N:
        raise ValueError("the weight's rows must be dY's columns")
    if s16 is not None:
        _dev(s16, "s16")
        if s16.dtype != torch.float16 or tuple(s16.shape) != (K,):
            raise ValueError("s16 must be fp16 [K]")
        _same_device(dY, (s16, "s16"))
    out = _out(out, (M, K), torch.float16, dY.device, dY, qweight, scales16, zeros, s16)
    ws = _scratch(workspace, lib.w4a16_gemm_backward_workspace_bytes(
        M, N, K, group, int(zeros is not None)), dY.device)
    _launch("w4a16_gemm_backward", lib.w4a16_gemm_backward, dY.device,
            dY.data_ptr(), M, N, K, group, qweight.data_ptr(), scales16.data_ptr(),
            zeros.data_ptr() if zeros is not None else None,
            s16.data_ptr() if s16 is not None else None, out.data_ptr(), *_ws_args(ws))
    return out
