"""User-facing calls of the W4A4 rotated linear layer, one per C-ABI entry point
(same names), plus :class:`W4A4Linear`, which holds a prepared layer.

Every function takes and returns PyTorch CUDA tensors, checks nothing beyond
shapes and dtypes needed to size its outputs (the C ABI validates the rest and
its status is raised as :class:`HQError`), and enqueues on the current stream.

Sources (page title, section): the rotation and quantiser follow "OffQ:
Taming Structured Outliers in LLM Quantization by Offsetting", Methodology 2-3,
and "SERQ: Saliency-Aware Low-Rank Error Reconstruction for LLM Quantization",
technical summary sections 1-3; the salient channels are those with the
largest activation L2 norm ("CMPQ", Methodology A).
"""
import torch

from . import _lib
from ._lib import HQError, check, dtype_code, lib, ptr, stream_handle

__all__ = [
    "HQError", "hq_rotate_quant", "hq_rotate", "hq_channel_sqnorm", "hq_select_salient", "w4_pack",
    "serq_prepare", "w4a4_linear", "hq_linear_workspace_size", "hq_debug_accum", "hq_last_device_status",
    "hq_debug_wait_probe", "hq_packed_weight_bytes", "wq_tile", "wq_untile", "W4A4Linear",
    "hq_rotate_quant8", "w4a8_linear", "hq_debug_accum8", "hq_rotate_quant_asym", "w4a4_linear_asym",
    "hq_debug_accum_asym", "hq_calib_extreme_tokens", "hq_calib_top1_pca", "hq_calib_householder",
    "hq_calib_channel_absmax", "hq_calib_sorted_perm", "hq_calib_flatten_scales", "hq_permute_channels",
    "calibrate_rotation_and_grouping", "hq_quant_mxfp4", "hq_mxfp4_linear", "hq_residual_norm",
    "hq_norm_rotate_quant", "hq_lora_max_tiles", "hq_lora_plan", "hq_lora_workspace_size", "hq_lora_apply",
]


def _signs_arg(H_signs):
    if H_signs is None:
        return None
    assert H_signs.dtype == torch.int8 and H_signs.is_cuda
    return ptr(H_signs)


def hq_rotate_quant(X, group, H_signs=None, Xq=None, sx=None):
    """(Xq uint8 [M, K/2], sx float32 [M]): grouped Hadamard rotation with H[0,:] = 1,
    per-token symmetric int4 codes packed two per byte."""
    M, K = X.shape
    if Xq is None:
        Xq = torch.empty((M, K // 2), dtype=torch.uint8, device=X.device)
    if sx is None:
        sx = torch.empty((M,), dtype=torch.float32, device=X.device)
    check(lib.hq_rotate_quant(ptr(X), dtype_code(X.dtype), M, K, X.stride(0), group, _signs_arg(H_signs),
                              ptr(Xq), ptr(sx), stream_handle()), "hq_rotate_quant")
    return Xq, sx


def hq_rotate_quant_asym(X, group, H_signs=None, Xq=None, sx=None, zx=None):
    """OffQ per-group asymmetric codes: (Xq uint8 [M, K/2] unsigned nibbles,
    sx float32 [M, K/group], zx int32 [M, K/group])."""
    M, K = X.shape
    Xq = torch.empty((M, K // 2), dtype=torch.uint8, device=X.device) if Xq is None else Xq
    sx = torch.empty((M, K // group), dtype=torch.float32, device=X.device) if sx is None else sx
    zx = torch.empty((M, K // group), dtype=torch.int32, device=X.device) if zx is None else zx
    check(lib.hq_rotate_quant_asym(ptr(X), dtype_code(X.dtype), M, K, X.stride(0), group, _signs_arg(H_signs),
                                   ptr(Xq), ptr(sx), ptr(zx), stream_handle()), "hq_rotate_quant_asym")
    return Xq, sx, zx


def hq_rotate_quant8(X, group, H_signs=None, Xq8=None, sx=None):
    """(Xq8 int8 [M, K], sx float32 [M]): the same rotation with per-token
    symmetric 8-bit codes in [-127, 127] (the W4A8 activations)."""
    M, K = X.shape
    if Xq8 is None:
        Xq8 = torch.empty((M, K), dtype=torch.int8, device=X.device)
    if sx is None:
        sx = torch.empty((M,), dtype=torch.float32, device=X.device)
    check(lib.hq_rotate_quant8(ptr(X), dtype_code(X.dtype), M, K, X.stride(0), group, _signs_arg(H_signs),
                               ptr(Xq8), ptr(sx), stream_handle()), "hq_rotate_quant8")
    return Xq8, sx


def hq_rotate(X, group, H_signs=None, out=None):
    """fp32 X * blockdiag(H) / sqrt(group) (the rotation folded into weights)."""
    M, K = X.shape
    X = X.contiguous()
    if out is None:
        out = torch.empty((M, K), dtype=torch.float32, device=X.device)
    check(lib.hq_rotate(ptr(X), dtype_code(X.dtype), M, K, group, _signs_arg(H_signs), ptr(out), stream_handle()),
          "hq_rotate")
    return out


def hq_channel_sqnorm(X, group, H_signs=None, norm2=None):
    """Accumulates the per-channel sum of squares of the rotated rows into norm2 [K]."""
    M, K = X.shape
    X = X.contiguous()
    if norm2 is None:
        norm2 = torch.zeros((K,), dtype=torch.float32, device=X.device)
    check(lib.hq_channel_sqnorm(ptr(X), dtype_code(X.dtype), M, K, group, _signs_arg(H_signs), ptr(norm2),
                                stream_handle()), "hq_channel_sqnorm")
    return norm2


def hq_select_salient(norm2, r):
    """Indices of the r largest entries (ascending), as an int32 CPU tensor."""
    n = norm2.detach().to("cpu", torch.float32).contiguous()
    out = torch.empty((r,), dtype=torch.int32)
    check(lib.hq_select_salient(ptr(n), n.numel(), r, ptr(out)), "hq_select_salient")
    return out


def hq_packed_weight_bytes(N, K):
    return int(lib.hq_packed_weight_bytes(N, K))


def wq_tile(Wq_rows):
    """Row-major packed weights [N, K/2] -> the tile-major layout of the C ABI,
    shaped [ceil(N/128), K/128, 128, 64] (padding rows are zero)."""
    N, Kh = Wq_rows.shape
    T = (N + 127) // 128
    pad = torch.zeros((T * 128, Kh), dtype=torch.uint8, device=Wq_rows.device)
    pad[:N] = Wq_rows
    return pad.view(T, 128, Kh // 64, 64).permute(0, 2, 1, 3).contiguous()


def wq_untile(Wq, N):
    """Tile-major packed weights -> row-major [N, K/2]."""
    T, KB = Wq.shape[0], Wq.shape[1]
    return Wq.permute(0, 2, 1, 3).reshape(T * 128, KB * 64)[:N]


def w4_pack(W, group):
    """(Wq uint8 tile-major [ceil(N/128), K/128, 128, 64], sw fp16 [N] or [K/group, N],
    zw fp16 [K/group, N] or None)."""
    N, K = W.shape
    W = W.contiguous()
    Wq = torch.empty(((N + 127) // 128, K // 128, 128, 64), dtype=torch.uint8, device=W.device)
    if group:
        sw = torch.empty((K // group, N), dtype=torch.float16, device=W.device)
        zw = torch.empty((K // group, N), dtype=torch.float16, device=W.device)
    else:
        sw = torch.empty((N,), dtype=torch.float16, device=W.device)
        zw = None
    check(lib.w4_pack(ptr(W), dtype_code(W.dtype), N, K, group, ptr(Wq), ptr(sw), ptr(zw), stream_handle()),
          "w4_pack")
    return Wq, sw, zw


def serq_prepare(W_rot, Wq, sw, zw, group, sal_idx):
    """(Rq uint8 [N, ceil(r/2)], sr fp16 [N]): SERQ's single error matrix on the salient inputs."""
    N, K = W_rot.shape
    r = int(sal_idx.numel())
    Rq = torch.empty((N, (r + 1) // 2), dtype=torch.uint8, device=W_rot.device)
    sr = torch.empty((N,), dtype=torch.float16, device=W_rot.device)
    check(lib.serq_prepare(ptr(W_rot), N, K, ptr(Wq), ptr(sw), ptr(zw), group, ptr(sal_idx), r, ptr(Rq), ptr(sr),
                           stream_handle()), "serq_prepare")
    return Rq, sr


def hq_linear_workspace_size(M, N, K, group):
    return int(lib.hq_linear_workspace_size(M, N, K, group))


def w4a4_linear(Xq, sx, Wq, sw, zw, group, A, B, sal_idx, out_dtype=torch.bfloat16, Y=None, workspace=None):
    """Y [M, N] = sx * (sum_b sw * acc_b + sr * acc_c), one fused launch.
    N is taken from the scales (sw [N] or [K/group, N])."""
    M = Xq.shape[0]
    K = Xq.shape[1] * 2
    N = sw.shape[-1]
    r = 0 if sal_idx is None else int(sal_idx.numel())
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=Xq.device)
    need = hq_linear_workspace_size(M, N, K, group)
    if need and workspace is None:
        workspace = torch.zeros((need,), dtype=torch.uint8, device=Xq.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib.w4a4_linear(ptr(Xq), ptr(sx), M, K, ptr(Wq), ptr(sw), ptr(zw), N, group,
                          ptr(A) if r else None, ptr(B) if r else None, ptr(sal_idx) if r else None, r,
                          ptr(Y), dtype_code(Y.dtype), ptr(workspace), ws_bytes, stream_handle()), "w4a4_linear")
    return Y


def w4a8_linear(Xq8, sx, Wq, sw, zw, group, A, B, sal_idx, out_dtype=torch.bfloat16, Y=None, workspace=None):
    """w4a4_linear on 8-bit activation codes Xq8 int8 [M, K]."""
    M, K = Xq8.shape
    N = sw.shape[-1]
    r = 0 if sal_idx is None else int(sal_idx.numel())
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=Xq8.device)
    need = hq_linear_workspace_size(M, N, K, group)
    if need and workspace is None:
        workspace = torch.zeros((need,), dtype=torch.uint8, device=Xq8.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib.w4a8_linear(ptr(Xq8), ptr(sx), M, K, ptr(Wq), ptr(sw), ptr(zw), N, group,
                          ptr(A) if r else None, ptr(B) if r else None, ptr(sal_idx) if r else None, r,
                          ptr(Y), dtype_code(Y.dtype), ptr(workspace), ws_bytes, stream_handle()), "w4a8_linear")
    return Y


def w4a4_linear_asym(Xq, sx, zx, Wq, sw, zw, group, A, B, sal_idx, out_dtype=torch.bfloat16, Y=None):
    """Y [M, N] from OffQ per-group asymmetric codes (hq_rotate_quant_asym with
    group 128)."""
    M, K = Xq.shape[0], Xq.shape[1] * 2
    N = sw.shape[-1]
    r = 0 if sal_idx is None else sal_idx.numel()
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=Xq.device)
    check(lib.w4a4_linear_asym(ptr(Xq), ptr(sx), ptr(zx), M, K, ptr(Wq), ptr(sw), ptr(zw), N, group, ptr(A), ptr(B),
                               ptr(sal_idx), r, ptr(Y), dtype_code(Y.dtype), stream_handle()), "w4a4_linear_asym")
    return Y


def hq_debug_accum_asym(Xq, zx, Wq, zw, group, N):
    """Integer accumulators [M, N, K/128] of w4a4_linear_asym (test hook)."""
    M, K = Xq.shape[0], Xq.shape[1] * 2
    acc = torch.empty((M, N, K // 128), dtype=torch.int32, device=Xq.device)
    check(lib.hq_debug_accum_asym(ptr(Xq), ptr(zx), M, K, ptr(Wq), ptr(zw), N, group, ptr(acc), stream_handle()),
          "hq_debug_accum_asym")
    return acc


def hq_debug_accum8(Xq8, Wq, zw, group, A, sal_idx, N, decode=False, workspace=None):
    """Exact int32 accumulators of the W4A8 GEMM kernel: (acc [M, N, G], acc_c [M, N])."""
    M, K = Xq8.shape
    r = 0 if sal_idx is None else int(sal_idx.numel())
    G = K // group if group else 1
    acc = torch.zeros((M, N, G), dtype=torch.int32, device=Xq8.device)
    acc_c = torch.zeros((M, N), dtype=torch.int32, device=Xq8.device)
    need = hq_linear_workspace_size(M, N, K, group) if decode else 0
    if need and workspace is None:
        workspace = torch.zeros((need,), dtype=torch.uint8, device=Xq8.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib.hq_debug_accum8(ptr(Xq8), M, K, ptr(Wq), ptr(zw), N, group, ptr(A) if r else None,
                              ptr(sal_idx) if r else None, r, ptr(acc), ptr(acc_c), 1 if decode else 0,
                              ptr(workspace), ws_bytes, stream_handle()), "hq_debug_accum8")
    return acc, acc_c


def hq_debug_accum(Xq, Wq, zw, group, A, sal_idx, N, decode=False, workspace=None):
    """Exact int32 accumulators of the GEMM kernel: (acc [M, N, G], acc_c [M, N])."""
    M = Xq.shape[0]
    K = Xq.shape[1] * 2
    r = 0 if sal_idx is None else int(sal_idx.numel())
    G = K // group if group else 1
    acc = torch.zeros((M, N, G), dtype=torch.int32, device=Xq.device)
    acc_c = torch.zeros((M, N), dtype=torch.int32, device=Xq.device)
    need = hq_linear_workspace_size(M, N, K, group) if decode else 0
    if need and workspace is None:
        workspace = torch.zeros((need,), dtype=torch.uint8, device=Xq.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib.hq_debug_accum(ptr(Xq), M, K, ptr(Wq), ptr(zw), N, group, ptr(A) if r else None,
                             ptr(sal_idx) if r else None, r, ptr(acc), ptr(acc_c), 1 if decode else 0,
                             ptr(workspace), ws_bytes, stream_handle()), "hq_debug_accum")
    return acc, acc_c


# ------------------------------------------------------------ offline calibration
# OffQ, Methodology 1 (Top-1 PCA) and 3 (sorted grouping); SERQ sections 1
# (static flattening) and 3 (offline permutation).

def hq_calib_extreme_tokens(X, S, L, tok=None, T=None):
    """(tok int32 [S], T float32 [S, K]): per calibration sequence (L rows of
    X each) the token of largest max |x| and its values."""
    K = X.shape[1]
    assert X.shape[0] == S * L
    tok = torch.empty((S,), dtype=torch.int32, device=X.device) if tok is None else tok
    T = torch.empty((S, K), dtype=torch.float32, device=X.device) if T is None else T
    check(lib.hq_calib_extreme_tokens(ptr(X), dtype_code(X.dtype), S, L, K, X.stride(0), ptr(tok), ptr(T),
                                      stream_handle()), "hq_calib_extreme_tokens")
    return tok, T


def hq_calib_top1_pca(T, iters=100, v=None, lam=None):
    """(v float32 [K] unit, lam float32 [1]): principal eigenvector of T^T T / S."""
    S, K = T.shape
    assert T.dtype == torch.float32 and T.is_contiguous()
    v = torch.empty((K,), dtype=torch.float32, device=T.device) if v is None else v
    lam = torch.empty((1,), dtype=torch.float32, device=T.device) if lam is None else lam
    check(lib.hq_calib_top1_pca(ptr(T), S, K, iters, ptr(v), ptr(lam), stream_handle()), "hq_calib_top1_pca")
    return v, lam


def hq_calib_householder(X, v, Y=None):
    """Y float32 [M, K] = X Q, Q the reflection that sends +-v to e0."""
    M, K = X.shape
    Y = torch.empty((M, K), dtype=torch.float32, device=X.device) if Y is None else Y
    check(lib.hq_calib_householder(ptr(X), dtype_code(X.dtype), M, K, X.stride(0), ptr(v), ptr(Y),
                                   stream_handle()), "hq_calib_householder")
    return Y


def hq_calib_channel_absmax(X, amax=None):
    """amax float32 [K] = max over rows of |X|."""
    M, K = X.shape
    amax = torch.empty((K,), dtype=torch.float32, device=X.device) if amax is None else amax
    check(lib.hq_calib_channel_absmax(ptr(X), dtype_code(X.dtype), M, K, max(X.stride(0), K), ptr(amax),
                                      stream_handle()), "hq_calib_channel_absmax")
    return amax


def hq_calib_sorted_perm(stat, perm=None):
    """perm int32 [K]: channels in decreasing stat (ties to the lower index)."""
    K = stat.shape[0]
    perm = torch.empty((K,), dtype=torch.int32, device=stat.device) if perm is None else perm
    check(lib.hq_calib_sorted_perm(ptr(stat), K, ptr(perm), stream_handle()), "hq_calib_sorted_perm")
    return perm


def hq_calib_flatten_scales(xmax, wmax, alpha=0.5, s=None):
    """s float32 [K] = xmax^alpha / wmax^(1-alpha)."""
    K = xmax.shape[0]
    s = torch.empty((K,), dtype=torch.float32, device=xmax.device) if s is None else s
    check(lib.hq_calib_flatten_scales(ptr(xmax), ptr(wmax), K, float(alpha), ptr(s), stream_handle()),
          "hq_calib_flatten_scales")
    return s


def hq_permute_channels(X, perm=None, s=None, op=0, Y=None):
    """Y float32 [M, K]: Y[:, j] = X[:, perm[j]] (op 1: / s, op 2: * s, taken at perm[j])."""
    M, K = X.shape
    Y = torch.empty((M, K), dtype=torch.float32, device=X.device) if Y is None else Y
    check(lib.hq_permute_channels(ptr(X), dtype_code(X.dtype), M, K, max(X.stride(0), K),
                                  None if perm is None else ptr(perm), None if s is None else ptr(s), op, ptr(Y),
                                  stream_handle()), "hq_permute_channels")
    return Y


def calibrate_rotation_and_grouping(X_calib, S, L, W, iters=100):
    """The offline OffQ calibration of one layer, every step on the GPU:
    extreme tokens -> Top-1 PCA direction v -> Householder rotation of the
    calibration activations and of the weight rows -> per-channel max |x| ->
    sorted-grouping permutation.  Returns (v, perm, W_cal) with W_cal float32
    [N, K] = (W Q)[:, perm]: activations that arrive as (X Q)[:, perm] give
    the same product X W^T."""
    _, T = hq_calib_extreme_tokens(X_calib, S, L)
    v, _ = hq_calib_top1_pca(T, iters)
    Xr = hq_calib_householder(X_calib, v)
    perm = hq_calib_sorted_perm(hq_calib_channel_absmax(Xr))
    W_cal = hq_permute_channels(hq_calib_householder(W, v), perm)
    return v, perm, W_cal


def hq_quant_mxfp4(X, Xq=None, scales=None):
    """(codes uint8 [M, K/2], scale bytes uint8 [M, K/32]): MXFP4 blocks of 32
    values (E2M1 codes, UE8M0 shared exponent) of the rows of X."""
    M, K = X.shape
    Xq = torch.empty((M, K // 2), dtype=torch.uint8, device=X.device) if Xq is None else Xq
    scales = torch.empty((M, K // 32), dtype=torch.uint8, device=X.device) if scales is None else scales
    check(lib.hq_quant_mxfp4(ptr(X), dtype_code(X.dtype), M, K, X.stride(0), ptr(Xq), ptr(scales),
                             stream_handle()), "hq_quant_mxfp4")
    return Xq, scales


def hq_mxfp4_linear(Xq, sx, Wq, sw, Y=None, accumulate=False):
    """Y float32 [M, N] (+)= X^ W^T for MXFP4 codes and scale bytes."""
    M, N, K = Xq.shape[0], Wq.shape[0], 2 * Xq.shape[1]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=Xq.device)
        accumulate = False
    check(lib.hq_mxfp4_linear(ptr(Xq), ptr(sx), M, K, ptr(Wq), ptr(sw), N, ptr(Y), 1 if accumulate else 0,
                              stream_handle()), "hq_mxfp4_linear")
    return Y


# ------------------------------------------------- between two layers of a decoder
# These calls check devices, types and shapes themselves (ValueError) and run
# on the device of their first tensor, on its current stream.  A single-token
# call takes a few microseconds on the GPU, less than plain Python marshalling:
# the checks are one comparison each, pointers and the stream are passed as
# integers, and the device is switched only where it is not the current one.

def _device(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be on a CUDA device" % name)
    return dev


def _rows(t, name, dev, shape, dtype):
    """Row stride in elements of a matrix of `shape` whose rows are contiguous."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        raise ValueError("%s must be a %s tensor of shape %s on the device of the first argument"
                         % (name, dtype, tuple(shape)))
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1 and shape[0] > 0:
        raise ValueError("%s must have contiguous rows" % name)
    # the stride of a single row (or of none) says nothing
    return s0 if shape[0] > 1 else max(shape[1] + 7 & ~7, s0 & ~7)


def _whole(t, name, dev, shape, dtype):
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on the device of the first argument"
                         % (name, dtype, tuple(shape)))


def _launch(dev, fn, where, args):
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        raise HQError(status, where)


def _gate_args(gate, dev, shape, dtype):
    """(address, row stride) of the gate: one row [K] for all (stride 0) or [M, K]."""
    if gate.dim() == 1:
        _whole(gate, "gate", dev, shape[1:], dtype)
        return gate.data_ptr(), 0
    return gate.data_ptr(), _rows(gate, "gate", dev, shape, dtype)


def _new_rows(like, M, K):
    """Empty [M, K] rows that start on 16 bytes."""
    per = 16 // like.element_size()
    pad = -(-K // per) * per
    t = torch.empty((M, pad), dtype=like.dtype, device=like.device)
    return t if pad == K else t[:, :K]


def hq_residual_norm(H, w, eps, Y=None, w_post=None, gate=None, alpha=1.0, w_offset=0.0, H_out=None, X=None):
    """(H_out, X): the residual stream H [M, K] plus alpha * gate * (norm of) the
    block's output Y, and its RMS norm with weights w (None: no second norm, X is
    None).  gate is [K] or [M, K]; w_offset is added to w and w_post.  H_out may
    be H (in place) and X may be Y; without Y there is no H_out unless one is given."""
    dev = _device(H, "H")
    dt, shape = H.dtype, H.shape
    M, K = shape
    wt = dt
    p_y = p_post = p_gate = p_w = p_ho = p_x = None
    ld_h = _rows(H, "H", dev, shape, dt)
    ld_y = ld_g = ld_ho = ld_x = 0
    if Y is not None:
        ld_y, p_y = _rows(Y, "Y", dev, shape, dt), Y.data_ptr()
        if H_out is None:
            H_out = _new_rows(H, M, K)
    if w is not None:
        wt = w.dtype
        _whole(w, "w", dev, (K,), wt)
        p_w = w.data_ptr()
        if X is None:
            X = _new_rows(H, M, K)
    if w_post is not None:
        wt = w_post.dtype if w is None else wt
        _whole(w_post, "w_post", dev, (K,), wt)
        p_post = w_post.data_ptr()
    if gate is not None:
        p_gate, ld_g = _gate_args(gate, dev, shape, dt)
    if H_out is not None:
        ld_ho, p_ho = _rows(H_out, "H_out", dev, shape, dt), H_out.data_ptr()
    if X is not None:
        ld_x, p_x = _rows(X, "X", dev, shape, dt), X.data_ptr()
    _launch(dev, lib.hq_residual_norm, "hq_residual_norm",
            (H.data_ptr(), ld_h, p_y, ld_y, dtype_code(dt), M, K, p_post, p_gate, ld_g, alpha, p_w, dtype_code(wt),
             w_offset, eps, p_ho, ld_ho, p_x, ld_x))
    return H_out, X


def hq_norm_rotate_quant(H, w, eps, group, H_signs=None, Y=None, gate=None, alpha=1.0, w_offset=0.0, bits=4,
                         H_out=None, X=None, Xq=None, sx=None, want_x=False):
    """(Xq, sx, H_out, X): hq_residual_norm (no norm after the block) with
    hq_rotate_quant (bits=4) or hq_rotate_quant8 (bits=8) in one pass; the
    normed rows X only with want_x or an X to write."""
    dev = _device(H, "H")
    dt, shape = H.dtype, H.shape
    M, K = shape
    wt = dt
    p_w = p_y = p_gate = p_ho = p_x = p_d = None
    ld_h = _rows(H, "H", dev, shape, dt)
    ld_y = ld_g = ld_ho = ld_x = 0
    if w is not None:
        wt = w.dtype
        _whole(w, "w", dev, (K,), wt)
        p_w = w.data_ptr()
    if Y is not None:
        ld_y, p_y = _rows(Y, "Y", dev, shape, dt), Y.data_ptr()
        if H_out is None:
            H_out = _new_rows(H, M, K)
    if gate is not None:
        p_gate, ld_g = _gate_args(gate, dev, shape, dt)
    if H_out is not None:
        ld_ho, p_ho = _rows(H_out, "H_out", dev, shape, dt), H_out.data_ptr()
    if X is None and want_x:
        X = _new_rows(H, M, K)
    if X is not None:
        ld_x, p_x = _rows(X, "X", dev, shape, dt), X.data_ptr()
    if H_signs is not None:
        _whole(H_signs, "H_signs", dev, (group,), torch.int8)
        p_d = H_signs.data_ptr()
    codes, ct = ((M, K), torch.int8) if bits == 8 else ((M, K // 2), torch.uint8)
    if Xq is None:
        Xq = torch.empty(codes, dtype=ct, device=H.device)
    else:
        _whole(Xq, "Xq", dev, codes, ct)
    if sx is None:
        sx = torch.empty((M,), dtype=torch.float32, device=H.device)
    else:
        _whole(sx, "sx", dev, (M,), torch.float32)
    _launch(dev, lib.hq_norm_rotate_quant, "hq_norm_rotate_quant",
            (H.data_ptr(), ld_h, p_y, ld_y, dtype_code(dt), M, K, p_gate, ld_g, alpha, p_w, dtype_code(wt),
             w_offset, eps, group, p_d, bits, p_ho, ld_ho, p_x, ld_x, Xq.data_ptr(), sx.data_ptr()))
    return Xq, sx, H_out, X


def hq_lora_max_tiles(M, n):
    return M // 64 + min(n + 1, M) if M > 0 and n >= 0 else 0     # as the C call


def hq_lora_plan(ids, n, order=None, tiles=None):
    """(order int32 [M], tiles int32 [hq_lora_max_tiles(M, n), 3]): the tokens of a
    batch grouped by their adapter ids int32 [M] in [0, n), -1 for none.  One
    plan serves every adapted layer of the step."""
    dev = _device(ids, "ids")
    shape = ids.shape
    M = shape[0]
    _whole(ids, "ids", dev, (M,), torch.int32)
    rows = hq_lora_max_tiles(M, n)
    if order is None:
        order = torch.empty((M,), dtype=torch.int32, device=ids.device)
    else:
        _whole(order, "order", dev, shape, torch.int32)
    if tiles is None:
        tiles = torch.empty((rows, 3), dtype=torch.int32, device=ids.device)
    else:
        _whole(tiles, "tiles", dev, (rows, 3), torch.int32)
    _launch(dev, lib.hq_lora_plan, "hq_lora_plan", (ids.data_ptr(), M, n, order.data_ptr(), tiles.data_ptr()))
    return order, tiles


def hq_lora_workspace_size(M, r_max):
    return int(lib.hq_lora_workspace_size(M, r_max))


def hq_lora_apply(X, A, B, order, tiles, ranks=None, scales=None, base=None, Y=None, out_dtype=None, workspace=None):
    """Y [M, N] = base + scales[a] (X A[a]^T) B[a]^T with a the token's adapter, base
    alone (zero if None) for a token without one.  A [n, r_max, K] and B
    [n, N, r_max] have X's type; order and tiles come from hq_lora_plan.  Y may be
    base (in place); it has base's type, or out_dtype (X's by default)."""
    dev = _device(X, "X")
    dt, shape = X.dtype, X.shape
    M, K = shape
    n, r, _ = A.shape
    N = B.shape[1]
    if Y is None:
        yt = base.dtype if base is not None else dt if out_dtype is None else out_dtype
        Y = torch.empty((M, N), dtype=yt, device=X.device)
    yt = Y.dtype
    out = (M, N)
    ld_x, ld_y = _rows(X, "X", dev, shape, dt), _rows(Y, "Y", dev, out, yt)
    p_base = p_ranks = p_scales = None
    ld_b = 0
    if base is not None:
        ld_b, p_base = ld_y if base is Y else _rows(base, "base", dev, out, yt), base.data_ptr()
    _whole(A, "A", dev, (n, r, K), dt)
    _whole(B, "B", dev, (n, N, r), dt)
    _whole(order, "order", dev, (M,), torch.int32)
    _whole(tiles, "tiles", dev, (hq_lora_max_tiles(M, n), 3), torch.int32)
    if ranks is not None:
        _whole(ranks, "ranks", dev, (n,), torch.int32)
        p_ranks = ranks.data_ptr()
    if scales is not None:
        _whole(scales, "scales", dev, (n,), torch.float32)
        p_scales = scales.data_ptr()
    if workspace is None:
        workspace = torch.empty((M, r), dtype=torch.float32, device=X.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of X")
    _launch(dev, lib.hq_lora_apply, "hq_lora_apply",
            (X.data_ptr(), dtype_code(dt), M, K, ld_x, A.data_ptr(), B.data_ptr(), N, n, r, p_ranks, p_scales,
             order.data_ptr(), tiles.data_ptr(), p_base, ld_b, Y.data_ptr(), dtype_code(yt), ld_y,
             workspace.data_ptr(), workspace.numel() * workspace.element_size()))
    return Y


def hq_last_device_status():
    return int(lib.hq_last_device_status(stream_handle()))


def hq_debug_wait_probe(limit_ns):
    check(lib.hq_debug_wait_probe(int(limit_ns), stream_handle()), "hq_debug_wait_probe")


class W4A4Linear:
    """A prepared W4A4 layer (W4A8 with act_bits=8; OffQ per-group asymmetric
    4-bit activations with offq=True): rotation signs, packed weights, SERQ
    term, workspace.

    ``prepare`` runs the offline steps on the GPU: fold the rotation into W,
    pack to int4, pick the r salient input channels from calibration
    activations (largest rotated L2 norm), build SERQ's error matrix.
    ``forward`` is the online path: one rotate/quant launch and one GEMM launch.
    ``forward_normed`` takes the residual stream instead of the layer's input.
    ``set_adapters`` puts low-rank adapters beside the layer; a batch's plan
    (hq_lora_plan) then adds each token's adapter to the output.
    """

    def __init__(self, group, gw, H_signs, Wq, sw, zw, Rq, sr, sal_idx, K, N, out_dtype, act_bits=4, offq=False):
        self.group, self.gw, self.H_signs = group, gw, H_signs
        self.Wq, self.sw, self.zw, self.Rq, self.sr, self.sal_idx = Wq, sw, zw, Rq, sr, sal_idx
        self.K, self.N, self.out_dtype = K, N, out_dtype
        if act_bits not in (4, 8):
            raise ValueError("act_bits must be 4 (W4A4) or 8 (W4A8)")
        if offq and (act_bits != 4 or group != 128):
            raise ValueError("OffQ activations are 4-bit with groups of 128 channels")
        self.act_bits = act_bits
        self.offq = offq
        self.adapters = None
        self._ws = {}

    @staticmethod
    def check_inputs(K, group, r, H_signs=None, sal_idx=None):
        """Host-side checks of the caller-supplied Hadamard signs and salient
        channels (ValueError): H_signs is `group` entries in {+1, -1} with
        H_signs[0] = +1 (the first row of H all ones); sal_idx is r strictly
        ascending indices in [0, K)."""
        if H_signs is not None:
            d = H_signs.detach().to("cpu")
            if d.dim() != 1 or d.numel() != group:
                raise ValueError("H_signs must hold one sign per channel of a group (%d)" % group)
            if not bool(((d == 1) | (d == -1)).all()):
                raise ValueError("H_signs entries must be +1 or -1")
            if int(d[0]) != 1:
                raise ValueError("H_signs[0] must be +1 (the first row of H is all ones)")
        if sal_idx is not None:
            s = sal_idx.detach().to("cpu").to(torch.int64).reshape(-1)
            if s.numel() != r:
                raise ValueError("sal_idx holds %d indices, r = %d" % (s.numel(), r))
            if r and (int(s.min()) < 0 or int(s.max()) >= K):
                raise ValueError("sal_idx entries must lie in [0, K)")
            if r > 1 and not bool((s[1:] > s[:-1]).all()):
                raise ValueError("sal_idx must be strictly ascending")

    @classmethod
    def prepare(cls, W, group, gw, r, H_signs=None, X_calib=None, sal_idx=None, out_dtype=torch.bfloat16,
                act_bits=4, offq=False):
        N, K = W.shape
        cls.check_inputs(K, group, r, H_signs, sal_idx)
        W_rot = hq_rotate(W, group, H_signs)
        Wq, sw, zw = w4_pack(W_rot, gw)
        if sal_idx is None and r > 0:
            norm2 = hq_channel_sqnorm(X_calib, group, H_signs)
            sal_idx = hq_select_salient(norm2, r).to(W.device)
        if r > 0:
            sal_idx = sal_idx.to(device=W.device, dtype=torch.int32).contiguous()
            Rq, sr = serq_prepare(W_rot, Wq, sw, zw, gw, sal_idx)
        else:
            sal_idx, Rq, sr = None, None, None
        del W_rot
        return cls(group, gw, H_signs, Wq, sw, zw, Rq, sr, sal_idx, K, N, out_dtype, act_bits, offq)

    def reset_workspaces(self):
        """Zero the cached workspaces (none is allocated while
        hq_linear_workspace_size reports 0, as it does for every shape)."""
        for ws in self._ws.values():
            ws.zero_()

    def workspace(self, M, device):
        need = hq_linear_workspace_size(M, self.N, self.K, self.gw)
        if need == 0:
            return None
        ws = self._ws.get(need)
        if ws is None:
            ws = torch.zeros((need,), dtype=torch.uint8, device=device)
            self._ws[need] = ws
        return ws

    def set_adapters(self, A, B, ranks=None, scales=None):
        """Low-rank adapters beside the layer (hq_lora_apply): A [n, r_max, K] on the
        layer's input, B [n, N, r_max], 16-bit; None takes them away.  What no call
        could use is refused here."""
        if A is None:
            self.adapters = None
            return
        if A.dim() != 3 or A.shape[2] != self.K or B.shape != (A.shape[0], self.N, A.shape[1]):
            raise ValueError("A must be [n, r_max, %d] and B [n, %d, r_max]" % (self.K, self.N))
        n, r, _ = A.shape
        if A.dtype not in (torch.float16, torch.bfloat16) or r % 8 or not 0 < r <= 256 or n > 1022:
            raise ValueError("A and B must be 16-bit, r_max a multiple of 8 up to 256, n at most 1022")
        dev = A.get_device()
        _whole(A, "A", dev, A.shape, A.dtype)
        _whole(B, "B", dev, B.shape, A.dtype)
        if ranks is not None:
            _whole(ranks, "ranks", dev, (n,), torch.int32)
        if scales is not None:
            _whole(scales, "scales", dev, (n,), torch.float32)
        if A.data_ptr() % 16 or B.data_ptr() % 16:
            raise ValueError("A and B must be 16-byte aligned")
        self.adapters = (A, B, ranks, scales)

    def _check(self, X, plan):
        """Refuses rows and plans before anything runs on them; the device they are on."""
        dev = _device(X, "the layer's input")
        if X.dim() != 2 or X.shape[1] != self.K:
            raise ValueError("the layer's input must be [M, %d]" % self.K)
        if plan is not None:
            if self.adapters is None:
                raise ValueError("the layer has no adapters (set_adapters)")
            A, M = self.adapters[0], X.shape[0]
            if A.get_device() != dev or A.dtype is not X.dtype:
                raise ValueError("the adapters must have the type and device of the layer's input")
            order, tiles = plan
            _whole(order, "the plan's order", dev, (M,), torch.int32)
            _whole(tiles, "the plan's tiles", dev, (hq_lora_max_tiles(M, A.shape[0]), 3), torch.int32)
        return dev

    def _adapted(self, X, plan, Y):
        if plan is None:
            return Y
        A, B, ranks, scales = self.adapters
        dev, M = X.get_device(), X.shape[0]      # adapters and plan are checked (set_adapters, _check)
        n, r, K = A.shape
        ld_x, ld_y = _rows(X, "X", dev, X.shape, A.dtype), _rows(Y, "Y", dev, (M, self.N), Y.dtype)
        work = torch.empty((M, r), dtype=torch.float32, device=X.device)
        p_y = Y.data_ptr()
        _launch(dev, lib.hq_lora_apply, "hq_lora_apply",
                (X.data_ptr(), dtype_code(A.dtype), M, K, ld_x, A.data_ptr(), B.data_ptr(), self.N, n, r,
                 ranks.data_ptr() if ranks is not None else None, scales.data_ptr() if scales is not None else None,
                 plan[0].data_ptr(), plan[1].data_ptr(), p_y, ld_y, p_y, dtype_code(Y.dtype), ld_y,
                 work.data_ptr(), 4 * M * r))
        return Y

    def _linear(self, Xq, sx, Y):
        gemm = w4a8_linear if self.act_bits == 8 else w4a4_linear
        return gemm(Xq, sx, self.Wq, self.sw, self.zw, self.gw, self.Rq, self.sr, self.sal_idx, self.out_dtype, Y,
                    self.workspace(Xq.shape[0], Xq.device))

    def forward(self, X, Y=None, Xq=None, sx=None, plan=None):
        """Y [M, N] of the rows X.  plan = hq_lora_plan(ids, n) adds the adapters of
        the tokens."""
        dev = self._check(X, plan)
        if torch._C._cuda_getDevice() != dev:        # every launch is on the device of X
            with torch.cuda.device(dev):
                return self.forward(X, Y, Xq, sx, plan)
        if self.offq:
            Xq, sx, zx = hq_rotate_quant_asym(X, self.group, self.H_signs, Xq, sx)
            Y = w4a4_linear_asym(Xq, sx, zx, self.Wq, self.sw, self.zw, self.gw, self.Rq, self.sr,
                                 self.sal_idx, self.out_dtype, Y)
        else:
            quant = hq_rotate_quant8 if self.act_bits == 8 else hq_rotate_quant
            Xq, sx = quant(X, self.group, self.H_signs, Xq, sx)
            Y = self._linear(Xq, sx, Y)
        return self._adapted(X, plan, Y)

    def forward_normed(self, H, w, eps, block=None, w_post=None, gate=None, alpha=1.0, w_offset=0.0, Y=None,
                       H_out=None, plan=None):
        """(Y, H_out): the layer on the RMS norm (weights w) of the residual stream H
        updated with the previous block's output, and that stream
        (hq_residual_norm; H itself without a block).  One launch makes the codes
        from the stream (hq_norm_rotate_quant); with a norm after the block, or
        OffQ activations, the normed rows are written and quantised from memory.
        A refused call leaves the stream as it was."""
        dev = self._check(H, plan)
        if torch._C._cuda_getDevice() != dev:
            with torch.cuda.device(dev):
                return self.forward_normed(H, w, eps, block, w_post, gate, alpha, w_offset, Y, H_out, plan)
        if H.dtype not in (torch.float16, torch.bfloat16):
            raise ValueError("the residual stream must be 16-bit")
        if self.Wq.get_device() != dev:
            raise ValueError("the layer and the residual stream must be on one device")
        if Y is not None:
            _whole(Y, "Y", dev, (H.shape[0], self.N), Y.dtype)
            if Y.data_ptr() % 16:
                raise ValueError("Y must be 16-byte aligned")
            dtype_code(Y.dtype)
        if self.offq or w_post is not None:
            H_out, X = hq_residual_norm(H, w, eps, block, w_post, gate, alpha, w_offset, H_out)
            Y = self.forward(X, Y, plan=plan)
        else:
            Xq, sx, H_out, X = hq_norm_rotate_quant(H, w, eps, self.group, self.H_signs, block, gate, alpha, w_offset,
                                                    self.act_bits, H_out, want_x=plan is not None)
            Y = self._adapted(X, plan, self._linear(Xq, sx, Y))
        return Y, H if H_out is None else H_out

    __call__ = forward
