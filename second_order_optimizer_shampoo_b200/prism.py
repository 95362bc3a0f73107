"""Python binding of the C ABI (argument marshalling only).

Each function takes CUDA tensors, allocates the scratch buffer the library
asks for through PyTorch's allocator, and calls the entry point of the same
name on the current stream.  Every arithmetic step runs in the library's
kernels; there is no CPU path.
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi as A

_PREC = {"tf32": A.SHP_TF32, "3xtf32": A.SHP_3XTF32, "bf16": A.SHP_BF16, "ozaki": A.SHP_OZAKI}
_POW = {"inv4": A.SHP_POW_INV4, "inv2": A.SHP_POW_INV2, "sqrt": A.SHP_POW_SQRT}


def status_string(code: int) -> str:
    return A.lib().shp_status_string(int(code)).decode()


def version() -> str:
    return A.lib().shp_version().decode()


def _check(code: int, name: str):
    if code != A.SHP_OK:
        extra = ""
        if code == A.SHP_ECUDA:
            extra = f", {A.lib().shp_last_cuda_error().decode()}"
        raise RuntimeError(f"{name} failed: {status_string(code)} ({code}{extra})")


def _dev(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device (the library has no CPU path)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def make_opts(d=2, p=8, lo=None, hi=1.0, tol=1e-3, max_iter=40, prec="3xtf32",
              fixed_alpha=False, stall_below=0.05, stall_ratio=0.75, adaptive_degree=False,
              raise_above=0.9, host_loop=False) -> A.PrismOpts:
    if lo is None:
        lo = 0.5 if d == 1 else 0.375
    return A.PrismOpts(d, p, lo, hi, tol, max_iter, _PREC[prec] if isinstance(prec, str) else prec,
                       int(bool(fixed_alpha)), stall_below, stall_ratio,
                       int(bool(adaptive_degree)), raise_above, int(bool(host_loop)))


def shp_workspace_bytes(op: int, m: int, n: int, batch: int, opts: A.PrismOpts | None = None) -> int:
    return int(A.lib().shp_workspace_bytes(op, m, n, batch,
                                           ctypes.byref(opts) if opts is not None else None))


def _ws(nbytes: int, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _as3(t, rows, cols):
    return t.reshape(-1, rows, cols)


def shampoo_gram_ema(G, L, R, beta: float, eps: float, prec: str = "tf32", ws=None):
    """L <- beta L + (1-beta) G G^T + eps I ; R <- beta R + (1-beta) G^T G + eps I (in place)."""
    _dev(G, L, R)
    m, n = G.shape[-2], G.shape[-1]
    batch = G.numel() // (m * n)
    o = make_opts(prec=prec)
    need = shp_workspace_bytes(A.SHP_OP_GRAM_EMA, m, n, batch, o)
    ws = _ws(need, G.device) if ws is None else ws
    _check(A.lib().shampoo_gram_ema(_p(G), m, n, batch, _p(L), _p(R), beta, eps, _PREC[prec],
                                    _p(ws), ws.numel(), _stream()), "shampoo_gram_ema")


def shampoo_gram_ema_steps(G, L, R, beta: float, eps: float, prec: str = "tf32", ws=None):
    """count successive EMA steps, one per gradient of G: [count][batch][m][n]
    (or [count][m][n]): L <- beta L + (1-beta) G_t G_t^T + eps I and
    R <- beta R + (1-beta) G_t^T G_t + eps I for t = 1..count (in place)."""
    _dev(G, L, R)
    m, n = G.shape[-2], G.shape[-1]
    count = G.shape[0]
    batch = G.numel() // (count * m * n)
    o = make_opts(prec=prec)
    need = shp_workspace_bytes(A.SHP_OP_GRAM_EMA_STEPS, m, n, count * batch, o)
    ws = _ws(need, G.device) if ws is None else ws
    _check(A.lib().shampoo_gram_ema_steps(_p(G), count, m, n, batch, _p(L), _p(R), beta, eps,
                                          _PREC[prec], _p(ws), ws.numel(), _stream()),
           "shampoo_gram_ema_steps")


def shampoo_apply(W, G, Lroot, Rroot, lr: float, prec: str = "tf32", ws=None):
    """W <- W - lr * Lroot G Rroot (in place)."""
    _dev(W, G, Lroot, Rroot)
    m, n = W.shape[-2], W.shape[-1]
    batch = W.numel() // (m * n)
    o = make_opts(prec=prec)
    need = shp_workspace_bytes(A.SHP_OP_APPLY, m, n, batch, o)
    ws = _ws(need, W.device) if ws is None else ws
    _check(A.lib().shampoo_apply(_p(W), _p(G), _p(Lroot), _p(Rroot), m, n, batch, lr, _PREC[prec],
                                 _p(ws), ws.numel(), _stream()), "shampoo_apply")


def shampoo_apply_ex(W, G, Lroot, Rroot, lr: float, prec: str = "tf32", M=None, gamma=0.0,
                     gnorm2_acc=None, ws=None):
    """Update variants (in place): with gnorm2_acc (float64 [batch]) the step is
    lr / sqrt(1 + acc) after acc += ||G||_F^2; with M (momentum buffer)
    M <- gamma M + P and W <- W - eta M; P = Lroot G Rroot."""
    _dev(W, G, Lroot, Rroot, M, gnorm2_acc)
    if gnorm2_acc is not None and gnorm2_acc.dtype != torch.float64:
        raise ValueError("gnorm2_acc must be float64")
    m, n = W.shape[-2], W.shape[-1]
    batch = W.numel() // (m * n)
    o = make_opts(prec=prec)
    need = shp_workspace_bytes(A.SHP_OP_APPLY, m, n, batch, o)
    ws = _ws(need, W.device) if ws is None else ws
    _check(A.lib().shampoo_apply_ex(_p(W), _p(M), _p(gnorm2_acc), _p(G), _p(Lroot), _p(Rroot),
                                    m, n, batch, lr, gamma, _PREC[prec], _p(ws), ws.numel(),
                                    _stream()), "shampoo_apply_ex")


def _report(batch, max_iter, device):
    return {
        "status": torch.full((batch,), -1, dtype=torch.int32, device=device),
        "iters": torch.full((batch, 2), -1, dtype=torch.int32, device=device),
        "resid": torch.full((batch, 2, max_iter + 1), float("nan"), dtype=torch.float32, device=device),
        "alpha": torch.full((batch, 2, max_iter), float("nan"), dtype=torch.float32, device=device),
        "degree": torch.full((batch, 2, max_iter), -1, dtype=torch.int32, device=device),
    }


def _report_struct(rep):
    if rep is None:
        return None
    deg = rep.get("degree")
    return ctypes.byref(A.PrismReport(rep["status"].data_ptr(), rep["iters"].data_ptr(),
                                      rep["resid"].data_ptr(), rep["alpha"].data_ptr(),
                                      deg.data_ptr() if deg is not None else None))


def make_report(batch, max_iter, device):
    """Device tensors for the per-block trajectory (status, iters, resid, alpha,
    degree)."""
    return _report(batch, max_iter, device)


def matfn_inv_root(Amat, power="inv4", opts: A.PrismOpts | None = None, S=None, out=None,
                   report=True, ws=None):
    """A^(-1/4) (or A^(-1/2), A^(1/2)) of a batch of SPD matrices.

    report: True (fresh tensors), False, or a dict from make_report() to reuse;
    the library caches one CUDA graph per distinct set of pointers and sizes,
    so reusing out/ws/report buffers keeps repeated calls on the cached graph."""
    opts = opts or make_opts()
    _dev(Amat, S, out)
    n = Amat.shape[-1]
    batch = Amat.numel() // (n * n)
    out = torch.empty_like(Amat) if out is None else out
    rep = report if isinstance(report, dict) else (
        _report(batch, opts.max_iter, Amat.device) if report else None)
    need = shp_workspace_bytes(A.SHP_OP_INV_ROOT, n, n, batch, opts)
    ws = _ws(need, Amat.device) if ws is None else ws
    s_count = 0 if S is None else S.shape[0]
    _check(A.lib().matfn_inv_root(_p(Amat), n, batch, _POW[power], ctypes.byref(opts), _p(S),
                                  s_count, _p(out), _report_struct(rep), _p(ws), ws.numel(),
                                  _stream()), "matfn_inv_root")
    return out, rep


def matfn_polar(G, opts: A.PrismOpts | None = None, S=None, out=None, report=True, ws=None):
    """Polar factor of a batch of m x n matrices; bf16 input keeps bf16 storage."""
    opts = opts or make_opts()
    _dev(G, S, out)
    m, n = G.shape[-2], G.shape[-1]
    batch = G.numel() // (m * n)
    if G.dtype == torch.bfloat16:
        storage = A.SHP_BF16
    elif G.dtype == torch.float32:
        storage = opts.prec if opts.prec in (A.SHP_TF32, A.SHP_3XTF32) else A.SHP_TF32
    else:
        raise ValueError("G must be float32 or bfloat16")
    out = torch.empty_like(G) if out is None else out
    rep = report if isinstance(report, dict) else (
        _report(batch, opts.max_iter, G.device) if report else None)
    o2 = A.PrismOpts.from_buffer_copy(opts)
    o2.prec = storage
    need = shp_workspace_bytes(A.SHP_OP_POLAR, m, n, batch, o2)
    ws = _ws(need, G.device) if ws is None else ws
    s_count = 0 if S is None else S.shape[0]
    _check(A.lib().matfn_polar(_p(G), storage, m, n, batch, ctypes.byref(opts), _p(S), s_count,
                               _p(out), _report_struct(rep), _p(ws), ws.numel(), _stream()),
           "matfn_polar")
    return out, rep


def matfn_polar_varsize(G, dims, offsets, opts: A.PrismOpts | None = None, S=None, out=None,
                        report=True):
    """Polar factors of small blocks of different shapes packed in the fp32
    tensor G: block b is dims[b] = (m_b, n_b) at element offsets[b] (dims int32
    [batch, 2], offsets int64 [batch], both on the device)."""
    opts = opts or make_opts()
    _dev(G, dims, offsets, S, out)
    if G.dtype != torch.float32 or dims.dtype != torch.int32 or offsets.dtype != torch.int64:
        raise ValueError("G float32, dims int32, offsets int64")
    batch = dims.shape[0]
    out = torch.empty_like(G) if out is None else out
    rep = report if isinstance(report, dict) else (
        _report(batch, opts.max_iter, G.device) if report else None)
    s_count = 0 if S is None else S.shape[0]
    _check(A.lib().matfn_polar_varsize(_p(G), _p(dims), _p(offsets), batch, ctypes.byref(opts),
                                       _p(S), s_count, _p(out), _report_struct(rep), _stream()),
           "matfn_polar_varsize")
    return out, rep


def matfn_sign(Amat, opts: A.PrismOpts | None = None, S=None, out=None, report=True, ws=None):
    """Matrix sign function of a batch of symmetric n x n matrices (bf16 input
    keeps bf16 storage)."""
    opts = opts or make_opts()
    _dev(Amat, S, out)
    n = Amat.shape[-1]
    if Amat.shape[-2] != n:
        raise ValueError("matfn_sign needs square matrices")
    batch = Amat.numel() // (n * n)
    if Amat.dtype == torch.bfloat16:
        storage = A.SHP_BF16
    elif Amat.dtype == torch.float32:
        storage = opts.prec if opts.prec in (A.SHP_TF32, A.SHP_3XTF32) else A.SHP_TF32
    else:
        raise ValueError("A must be float32 or bfloat16")
    out = torch.empty_like(Amat) if out is None else out
    rep = report if isinstance(report, dict) else (
        _report(batch, opts.max_iter, Amat.device) if report else None)
    o2 = A.PrismOpts.from_buffer_copy(opts)
    o2.prec = storage
    need = shp_workspace_bytes(A.SHP_OP_POLAR, n, n, batch, o2)
    ws = _ws(need, Amat.device) if ws is None else ws
    s_count = 0 if S is None else S.shape[0]
    _check(A.lib().matfn_sign(_p(Amat), storage, n, batch, ctypes.byref(opts), _p(S), s_count,
                              _p(out), _report_struct(rep), _p(ws), ws.numel(), _stream()),
           "matfn_sign")
    return out, rep


def prism_alpha_fit(R, S, d: int, lo: float, hi: float, ws=None):
    """alpha* on [lo, hi] for each residual in the batch, plus J's coefficients."""
    _dev(R, S)
    n = R.shape[-1]
    batch = R.numel() // (n * n)
    p = S.shape[-1]
    alpha = torch.empty(batch, dtype=torch.float32, device=R.device)
    J = torch.empty(batch, 5, dtype=torch.float64, device=R.device)
    need = shp_workspace_bytes(A.SHP_OP_ALPHA_FIT, n, n, batch, make_opts(d=d, p=p))
    ws = _ws(need, R.device) if ws is None else ws
    _check(A.lib().prism_alpha_fit(_p(R), n, batch, _p(S), p, d, lo, hi, _p(alpha), _p(J), _p(ws),
                                   ws.numel(), _stream()), "prism_alpha_fit")
    return alpha, J


def kernel_launches() -> int:
    """Kernels the library has launched in this process so far."""
    return int(A.lib().shp_kernel_launches())


def shp_split_tf32(X, hi=None, lo=None):
    """(hi, lo) with hi = TF32(X), lo = TF32(X - hi)."""
    _dev(X)
    hi = torch.empty_like(X) if hi is None else hi
    lo = torch.empty_like(X) if lo is None else lo
    _check(A.lib().shp_split_tf32(_p(X), X.numel(), _p(hi), _p(lo), _stream()), "shp_split_tf32")
    return hi, lo


def shp_matmul(Amat, B, prec="tf32", a_trans=False, b_trans=False, A_lo=None, B_lo=None, out=None):
    """Batched C = op(A) op(B) on the tensor cores (one kernel launch).

    A: [batch][M][K] (or [batch][K][M] with a_trans), B: [batch][K][N] (or
    [batch][N][K] with b_trans).  For prec='3xtf32' pass the high parts as
    A/B and the low parts as A_lo/B_lo (see shp_split_tf32)."""
    _dev(Amat, B, A_lo, B_lo, out)
    M, K = (Amat.shape[-1], Amat.shape[-2]) if a_trans else (Amat.shape[-2], Amat.shape[-1])
    N = B.shape[-2] if b_trans else B.shape[-1]
    batch = Amat.numel() // (M * K)
    dt = torch.bfloat16 if prec == "bf16" else torch.float32
    out = torch.empty(batch, M, N, dtype=dt, device=Amat.device) if out is None else out
    _check(A.lib().shp_matmul(_p(Amat), _p(A_lo), int(a_trans), _p(B), _p(B_lo), int(b_trans),
                              _p(out), M, N, K, batch, _PREC[prec], _stream()), "shp_matmul")
    return out


# The current stream's handle without building a Stream object (1 us per call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _ready(*ts):
    """Checks that the tensors (None is skipped) are contiguous and on the
    current CUDA device; returns the handle of its current stream."""
    if not ts[0].is_cuda:
        _dev(*ts)
    dev = torch.cuda.current_device()
    for t in ts:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            _dev(t)
            raise ValueError(f"tensor on {t.device}, but the current device is cuda:{dev}")
    return _raw_stream(dev)


def _want(name, t, dtype, shape):
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


_BF16 = torch.bfloat16
_STORAGE = {torch.bfloat16: A.SHP_BF16, torch.float32: A.SHP_TF32}


def _storage(dtype):
    if dtype not in _STORAGE:
        raise ValueError(f"bfloat16 or float32, not {dtype}")
    return _STORAGE[dtype]


def _result(out, shape, dtype, device):
    """`out`, checked, or a new tensor; and its storage code."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device), _storage(dtype)
    _want("out", out, out.dtype, shape)
    return out, _storage(out.dtype)


def shp_grouped_matmul(X, offsets, W, w_trans=False, out=None, dtype=torch.bfloat16):
    """Y[t] = X[t] W[e] (or X[t] W[e]^T with w_trans) for the rows t in
    offsets[e] .. offsets[e+1]-1 of each group e: the forward product of an
    expert layer, or the gradient of its input.

    X: [T, K] bf16, rows sorted by group; offsets: [groups + 1] int64 on the
    device; W: [groups, K, N] bf16 ([groups, N, K] with w_trans).  Y: `out`, or
    a new [T, N] tensor of `dtype` (bf16 or float32) whose rows outside every
    group are uninitialised; in `out`, which may not share memory with X or W,
    those rows are left as they were."""
    st = _ready(X, offsets, W, out)
    if X.dim() != 2 or W.dim() != 3:
        raise ValueError("X is [T, K] and W [groups, K, N]")
    T, K = X.shape
    groups, N, k = W.shape
    if not w_trans:
        N, k = k, N
    if k != K or X.dtype != _BF16 or W.dtype != _BF16:
        _want("X", X, _BF16, (T, K))
        _want("W", W, _BF16, (groups, N, K) if w_trans else (groups, K, N))
    _want("offsets", offsets, torch.int64, (groups + 1,))
    out, storage = _result(out, (T, N), dtype, X.device)
    _check(A.lib().shp_grouped_matmul(X.data_ptr(), offsets.data_ptr(), W.data_ptr(),
                                      1 if w_trans else 0, out.data_ptr(), storage, T, K, N,
                                      groups, st), "shp_grouped_matmul")
    return out


def shp_grouped_wgrad(Amat, B, offsets, out=None, accumulate=False):
    """G[e] = A_e^T B_e over the rows of each group: the gradient of an expert
    layer's weight blocks, in the fp32 layout shampoo_gram_ema takes.

    A: [T, m], B: [T, n] bf16; offsets as in shp_grouped_matmul; G: `out`, or a
    new [groups, m, n] float32 tensor.  accumulate adds to `out` (which must
    then be given).  An empty group gives zeros, or leaves `out` as it is."""
    st = _ready(Amat, B, offsets, out)
    if Amat.dim() != 2 or B.dim() != 2 or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("A is [T, m], B [T, n] and offsets [groups + 1]")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    T, m = Amat.shape
    n, groups = B.shape[1], offsets.shape[0] - 1
    _want("A", Amat, _BF16, (T, m))
    _want("B", B, _BF16, (T, n))
    _want("offsets", offsets, torch.int64, (groups + 1,))
    if out is None:
        out = torch.empty((groups, m, n), dtype=torch.float32, device=B.device)
    else:
        _want("out", out, torch.float32, (groups, m, n))
    _check(A.lib().shp_grouped_wgrad(Amat.data_ptr(), B.data_ptr(), offsets.data_ptr(),
                                     out.data_ptr(), T, m, n, groups, 1 if accumulate else 0, st),
           "shp_grouped_wgrad")
    return out


def _mx4_shapes(batch, rows, cols):
    """Shapes of the codes and of the scale tiles."""
    return ((batch, rows, (cols + 31) // 32 * 16),
            (batch, (rows + 127) // 128, (cols + 127) // 128, 512))


def _mx4_new(batch, rows, cols, device):
    q, s = _mx4_shapes(batch, rows, cols)
    return (torch.empty(q, dtype=torch.uint8, device=device),
            torch.empty(s, dtype=torch.uint8, device=device))


def shp_mx4_quantize(X, along="cols"):
    """MXFP4 codes and scales of X ([batch, rows, cols] or [rows, cols], bf16 or
    float32), in blocks of 32 along the columns: (Q, S); along="rows" gives
    those of X^T, blocks along X's rows: (Qt, St); along="both" gives (Q, S,
    Qt, St) from one read of X.  Q: uint8 [batch, rows, Cp / 2], S: uint8
    [batch, rows / 128, cols / 128, 512] tiles (rounded up); layouts in the C
    header."""
    st = _ready(X)
    if along not in ("cols", "rows", "both") or X.dim() not in (2, 3):
        raise ValueError("X is [batch, rows, cols] or [rows, cols]; along is cols, rows or both")
    rows, cols = X.shape[-2:]
    batch = X.shape[0] if X.dim() == 3 else 1
    storage = _storage(X.dtype)
    res = () if along == "rows" else _mx4_new(batch, rows, cols, X.device)
    if along != "cols":
        res += _mx4_new(batch, cols, rows, X.device)
    ptrs = [t.data_ptr() for t in res]
    if along != "both":
        ptrs = ptrs + [None, None] if along == "cols" else [None, None] + ptrs
    _check(A.lib().shp_mx4_quantize(X.data_ptr(), storage, rows, cols, batch, *ptrs, st),
           "shp_mx4_quantize")
    return res


def shp_mx4_dequantize(Q, S, cols, dtype=torch.float32, out=None):
    """The values [batch, rows, cols] of MXFP4 codes and scales."""
    st = _ready(Q, S, out)
    if Q.dim() != 3:
        raise ValueError("Q is [batch, rows, Cp / 2]")
    batch, rows = Q.shape[:2]
    q, s = _mx4_shapes(batch, rows, cols)
    _want("Q", Q, torch.uint8, q)
    _want("S", S, torch.uint8, s)
    out, storage = _result(out, (batch, rows, cols), dtype, Q.device)
    _check(A.lib().shp_mx4_dequantize(Q.data_ptr(), S.data_ptr(), rows, cols, batch,
                                      out.data_ptr(), storage, st), "shp_mx4_dequantize")
    return out


def shp_mx4_matmul(Amat, A_scales, B, B_scales, dtype=torch.bfloat16, out=None):
    """C[b] = A[b] B[b]^T of two MXFP4 operands quantised along the contraction:
    A [batch, M, K / 2] and B [batch, N, K / 2] with their scale tiles.  C:
    `out`, or a new [batch, M, N] tensor of `dtype` (bf16 or float32)."""
    st = _ready(Amat, A_scales, B, B_scales, out)
    if Amat.dim() != 3 or B.dim() != 3:
        raise ValueError("A is [batch, M, K / 2] and B [batch, N, K / 2]")
    batch, M, half = Amat.shape
    N, K = B.shape[1], 2 * half
    q, s = _mx4_shapes(batch, M, K)
    _want("A", Amat, torch.uint8, q)
    _want("A_scales", A_scales, torch.uint8, s)
    q, s = _mx4_shapes(batch, N, K)
    _want("B", B, torch.uint8, q)
    _want("B_scales", B_scales, torch.uint8, s)
    out, storage = _result(out, (batch, M, N), dtype, B.device)
    _check(A.lib().shp_mx4_matmul(Amat.data_ptr(), A_scales.data_ptr(), B.data_ptr(),
                                  B_scales.data_ptr(), out.data_ptr(), storage, M, N, K, batch, st),
           "shp_mx4_matmul")
    return out


def shp_matmul_f64(Amat, B, out=None, ws=None, reuse_a=False, reuse_b=False, accumulate=False):
    """Batched C = A B in fp64-grade arithmetic on the int8 tensor cores (the
    Ozaki scheme); A [batch][M][K], B [batch][K][N] float64.  reuse_a /
    reuse_b take that operand's digit slices from `ws` as the previous call
    with the same operand and workspace left them; accumulate adds the
    product to `out` (which must then be given)."""
    _dev(Amat, B, out)
    if Amat.dtype != torch.float64 or B.dtype != torch.float64:
        raise ValueError("shp_matmul_f64 takes float64 tensors")
    M, K = Amat.shape[-2], Amat.shape[-1]
    N = B.shape[-1]
    batch = Amat.numel() // (M * K)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    out = torch.empty(batch, M, N, dtype=torch.float64, device=Amat.device) if out is None else out
    need = int(A.lib().shp_matmul_f64_workspace_bytes(M, N, K, batch))
    if ws is None:
        if reuse_a or reuse_b:
            raise ValueError("reusing slices needs the workspace of the previous call")
        ws = _ws(need, Amat.device)
    flags = ((A.SHP_MATMUL_REUSE_A if reuse_a else 0) | (A.SHP_MATMUL_REUSE_B if reuse_b else 0)
             | (A.SHP_MATMUL_ACCUMULATE if accumulate else 0))
    _check(A.lib().shp_matmul_f64_ex(_p(Amat), _p(B), _p(out), M, N, K, batch, flags, _p(ws),
                                     ws.numel(), _stream()), "shp_matmul_f64")
    return out


def selftest_bounded_wait(which: str, device=None):
    """Make one bounded pipeline wait run out on purpose ("gemm", "ozaki",
    "sketch", "sketch_alpha" -- the last sketch pass with the fit folded in --
    or "sketch_chain", the few-block sketch's grid barrier -- or "grouped",
    "wgrad", "mx4_quantize", "mx4_matmul"); returns (status
    the kernel recorded, alpha of the sketch's fit) -- SHP_ETIMEOUT and, for
    the sketch cases, NaN are expected.  "grouped_long", "wgrad_long" and
    "mx4_matmul_long" are launches much longer than the limit of a wait, in
    which none may run out: SHP_OK is expected."""
    code = {"gemm": A.SHP_SELFTEST_GEMM, "ozaki": A.SHP_SELFTEST_OZAKI,
            "sketch": A.SHP_SELFTEST_SKETCH, "sketch_alpha": A.SHP_SELFTEST_SKETCH_ALPHA,
            "sketch_chain": A.SHP_SELFTEST_SKETCH_CHAIN, "grouped": A.SHP_SELFTEST_GROUPED,
            "wgrad": A.SHP_SELFTEST_WGRAD, "mx4_quantize": A.SHP_SELFTEST_MX4_QUANTIZE,
            "mx4_matmul": A.SHP_SELFTEST_MX4_MATMUL,
            "grouped_long": A.SHP_SELFTEST_GROUPED_LONG,
            "wgrad_long": A.SHP_SELFTEST_WGRAD_LONG,
            "mx4_matmul_long": A.SHP_SELFTEST_MX4_MATMUL_LONG}[which]
    device = device or torch.device("cuda", torch.cuda.current_device())
    status = torch.full((1,), -1, dtype=torch.int32, device=device)
    alpha = torch.zeros(1, dtype=torch.float32, device=device)
    size = A.SHP_SELFTEST_LONG_WS_BYTES if which.endswith("_long") else A.SHP_SELFTEST_WS_BYTES
    ws = torch.empty(size, dtype=torch.uint8, device=device)
    _check(A.lib().shp_selftest_bounded_wait(code, _p(status), _p(alpha), _p(ws), ws.numel(),
                                             _stream()), "shp_selftest_bounded_wait")
    return int(status.item()), float(alpha.item())
