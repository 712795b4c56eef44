"""A MoE block's operators in bf16: the experts' products in both directions, the combine's gradient, and the norm
before the experts, in bf16 and FP8.

Binding of ``include/moe_block.h`` in the manner of the package: the functions named like the C entry points only check
and marshal arguments; :func:`rmsnorm`, :func:`rmsnorm_backward` and :class:`BF16MoELayer` allocate with torch. All names
are reachable from the package itself.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import (MOE_MODE_MASKED, MOE_QUANT_FP8_G128, MOE_QUANT_FP8_G128_UE8M0, MOE_QUANT_NONE, _check, _need, _ptr,
               check_status, load_library, moe_combine_ex, moe_dispatch_ex, moe_route_meta_ex, new_status, new_workspace)
from .experts import MOE_LAYER_MAX_TOKENS, _current, _mode, _on, moe_layer_few_tokens, new_layer_workspace

__all__ = [
    "MOE_WEIGHTS_NK", "MOE_WEIGHTS_KN", "MOE_GRAD_BF16", "MOE_GRAD_FP32", "MOE_NORM_MAX_HIDDEN", "NormOutput",
    "LayerGradients", "BF16MoELayer", "moe_expert_gemm_bf16", "moe_expert_gemm_swiglu_bf16",
    "moe_expert_gemm_dswiglu_bf16", "moe_expert_wgrad_bf16", "moe_combine_backward", "moe_rmsnorm",
    "moe_rmsnorm_backward_workspace_size", "moe_rmsnorm_backward", "rmsnorm", "rmsnorm_backward",
]

MOE_WEIGHTS_NK = 0
MOE_WEIGHTS_KN = 1
MOE_GRAD_BF16 = 0
MOE_GRAD_FP32 = 1
MOE_NORM_MAX_HIDDEN = 32768

NORM_QUANTS = {"none": MOE_QUANT_NONE, "fp8g128": MOE_QUANT_FP8_G128, "fp8g128_ue8m0": MOE_QUANT_FP8_G128_UE8M0}
_BF16, _I32, _I64, _F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


# ---------------------------------------------------------------------------
# thin wrappers with the C names
# ---------------------------------------------------------------------------

def _pointers(*specs):
    """The data pointers of (tensor or None, bytes needed, name, dtype), checked as the expert operators' are, and that all
    are tensors of the current device, where the kernels run. In one pass: a second one is 1 us of a call's 20."""
    out, wrong, device = [], None, None
    for t, nbytes, name, dtype in specs:
        if t is None:
            out.append(None)
            continue
        if t.dtype is not dtype or t.nbytes < nbytes:
            _need(t, nbytes, name, dtype)
        if not (t.is_cuda and t.is_contiguous()):
            wrong = t if wrong is None else wrong
        elif device is None:
            device = t.get_device()
        elif t.get_device() != device:
            device = -1                                 # of several
        out.append(t.data_ptr())
    if wrong is not None:
        _ptr(wrong)
    if device is not None:
        current = torch._C._cuda_getDevice()
        if device != current:
            names = [spec[2] for spec in specs if spec[0] is not None and spec[0].get_device() != current]
            raise ValueError(f"{', '.join(names)}: tensors of the current device expected")
    return out


def _rows(mode: str, a: torch.Tensor, K: int, E: int, M: int, seg_indptr, name: str = "a") -> int:
    """Rows of a layout whose row buffer `a` has K columns."""
    masked = _mode(mode) == MOE_MODE_MASKED
    if a.dim() < 2:
        raise ValueError(f"{name}: rows of {K} values needed, got shape {tuple(a.shape)}")
    _row_buffer(mode, a, K, M, name)
    if masked:
        return E * M
    if seg_indptr is None:
        raise ValueError("seg_indptr: needed in normal mode")
    return a.shape[:-1].numel()


def _row_buffer(mode: str, t: Optional[torch.Tensor], K: int, M: int, name: str) -> None:
    """Refuses a buffer whose rows have another length or stride than the kernels' K columns and M rows an expert; one
    without a shape that says (one dimension) is theirs to lay out."""
    if t is None:
        return
    shape = t.shape
    if len(shape) < 2:
        return
    if mode == "masked" and len(shape) == 3 and (shape[1] != M or shape[2] != K):
        raise ValueError(f"{name}: [E, {M}, {K}] expected in masked mode, got shape {tuple(shape)}")
    if shape[-1] != K:
        raise ValueError(f"{name}: rows of {K} values needed, got shape {tuple(shape)}")


def _layout(mode: str, E: int, masked_m, seg_indptr, dev_status):
    return ((masked_m, 4 * E, "masked_m", _I32),
            (seg_indptr, 8 * (E + 1) if mode == "normal" else 0, "seg_indptr", _I64),
            (dev_status, 4, "dev_status", _I32))


def moe_expert_gemm_bf16(mode: str, a: torch.Tensor, masked_m: torch.Tensor, w: torch.Tensor, out: torch.Tensor,
                         dev_status: torch.Tensor, transposed: bool = False, seg_indptr: Optional[torch.Tensor] = None,
                         max_tokens_per_expert: int = 0, stream=None) -> None:
    """out[r] = w[e] a[r] for the rows of every expert e of a dispatched layout, w [E, n, k]; with `transposed`
    w[e]^T a[r], w [E, k, n]: the gradient with respect to the rows of a product with these weights.

    a [rows, k] (normal) or [E, M, k] (masked, M = max_tokens_per_expert), out alike with n columns; all bf16."""
    E, N, K = w.shape
    if transposed:
        N, K = K, N
    rows = _rows(mode, a, K, E, max_tokens_per_expert, seg_indptr)
    _row_buffer(mode, out, N, max_tokens_per_expert, "out")
    pm, pseg, pst, pa, pw, po = _pointers(
        *_layout(mode, E, masked_m, seg_indptr, dev_status), (a, 2 * rows * K, "a", _BF16), (w, 0, "w", _BF16),
        (out, 2 * rows * N, "out", _BF16))
    st = load_library().moe_expert_gemm_bf16(_mode(mode), pa, E, max_tokens_per_expert, rows, N, K, pseg, pm,
                                             MOE_WEIGHTS_KN if transposed else MOE_WEIGHTS_NK, pw, po, pst, _on(stream))
    _check(st, "moe_expert_gemm_bf16")


def moe_expert_gemm_swiglu_bf16(mode: str, a: torch.Tensor, masked_m: torch.Tensor, w13: torch.Tensor, h: torch.Tensor,
                                dev_status: torch.Tensor, gate_up: Optional[torch.Tensor] = None,
                                seg_indptr: Optional[torch.Tensor] = None, max_tokens_per_expert: int = 0,
                                stream=None) -> None:
    """h[r] = up * silu(gate) of the products with w13 [E, 2*inter, k] (gate rows, then up rows), in one kernel; gate_up
    [rows, 2*inter], if given, receives their values for :func:`moe_expert_gemm_dswiglu_bf16`."""
    E, N, K = w13.shape
    if N % 2:
        raise ValueError(f"w13: gate and up rows do not fit {N} rows")
    N //= 2
    rows = _rows(mode, a, K, E, max_tokens_per_expert, seg_indptr)
    _row_buffer(mode, h, N, max_tokens_per_expert, "h")
    _row_buffer(mode, gate_up, 2 * N, max_tokens_per_expert, "gate_up")
    pm, pseg, pst, pa, pw, ph, pg = _pointers(
        *_layout(mode, E, masked_m, seg_indptr, dev_status), (a, 2 * rows * K, "a", _BF16), (w13, 0, "w13", _BF16),
        (h, 2 * rows * N, "h", _BF16), (gate_up, 4 * rows * N, "gate_up", _BF16))
    st = load_library().moe_expert_gemm_swiglu_bf16(_mode(mode), pa, E, max_tokens_per_expert, rows, N, K, pseg, pm, pw,
                                                    ph, pg, pst, _on(stream))
    _check(st, "moe_expert_gemm_swiglu_bf16")


def moe_expert_gemm_dswiglu_bf16(mode: str, grad_out: torch.Tensor, masked_m: torch.Tensor, w2: torch.Tensor,
                                 gate_up: torch.Tensor, grad_gate_up: torch.Tensor, dev_status: torch.Tensor,
                                 seg_indptr: Optional[torch.Tensor] = None, max_tokens_per_expert: int = 0,
                                 stream=None) -> None:
    """The gradient of gate and up from that of the rows h w2[e]^T: w2 [E, k, inter], grad_out [rows, k], gate_up and
    grad_gate_up [rows, 2*inter] (grad_gate_up may be gate_up)."""
    E, K, N = w2.shape
    rows = _rows(mode, grad_out, K, E, max_tokens_per_expert, seg_indptr, "grad_out")
    _row_buffer(mode, gate_up, 2 * N, max_tokens_per_expert, "gate_up")
    _row_buffer(mode, grad_gate_up, 2 * N, max_tokens_per_expert, "grad_gate_up")
    pm, pseg, pst, pa, pw, pg, po = _pointers(
        *_layout(mode, E, masked_m, seg_indptr, dev_status), (grad_out, 2 * rows * K, "grad_out", _BF16),
        (w2, 0, "w2", _BF16), (gate_up, 4 * rows * N, "gate_up", _BF16),
        (grad_gate_up, 4 * rows * N, "grad_gate_up", _BF16))
    st = load_library().moe_expert_gemm_dswiglu_bf16(_mode(mode), pa, E, max_tokens_per_expert, rows, N, K, pseg, pm, pw,
                                                     pg, po, pst, _on(stream))
    _check(st, "moe_expert_gemm_dswiglu_bf16")


def moe_expert_wgrad_bf16(mode: str, a: torch.Tensor, b: torch.Tensor, masked_m: torch.Tensor, out: torch.Tensor,
                          dev_status: torch.Tensor, accumulate: bool = False,
                          seg_indptr: Optional[torch.Tensor] = None, max_tokens_per_expert: int = 0,
                          stream=None) -> None:
    """out[e] = sum over the rows r of expert e of a[r]^T b[r], or added to out with `accumulate`: out [E, m, n] fp32 or
    bf16, a [rows, m] and b [rows, n] bf16."""
    E, Ma, N = out.shape
    if out.dtype not in (_F32, _BF16):
        raise ValueError(f"out: torch.float32 or torch.bfloat16 expected, got {out.dtype}")
    rows = _rows(mode, a, Ma, E, max_tokens_per_expert, seg_indptr)
    if _rows(mode, b, N, E, max_tokens_per_expert, seg_indptr, "b") != rows:
        raise ValueError(f"b: {rows} rows needed, got shape {tuple(b.shape)}")
    pm, pseg, pst, pa, pb, po = _pointers(
        *_layout(mode, E, masked_m, seg_indptr, dev_status), (a, 2 * rows * Ma, "a", _BF16),
        (b, 2 * rows * N, "b", _BF16), (out, 0, "out", out.dtype))
    st = load_library().moe_expert_wgrad_bf16(_mode(mode), pa, pb, E, max_tokens_per_expert, rows, Ma, N, pseg, pm,
                                              MOE_GRAD_FP32 if out.dtype is _F32 else MOE_GRAD_BF16, int(bool(accumulate)),
                                              po, pst, _on(stream))
    _check(st, "moe_expert_wgrad_bf16")


def moe_combine_backward(mode: str, grad_out: torch.Tensor, expert_out: Optional[torch.Tensor], topk_ids: torch.Tensor,
                         topk_weights: torch.Tensor, num_experts: int, src2dst: torch.Tensor, seg_indptr: torch.Tensor,
                         grad_expert_out: Optional[torch.Tensor], grad_topk_weights: Optional[torch.Tensor],
                         dev_status: torch.Tensor, max_tokens_per_expert: int = 0, expert_out_rows: int = 0,
                         stream=None) -> None:
    """The gradient of :func:`moe_combine_ex`: of its rows into grad_expert_out, of its weights into grad_topk_weights
    [T, K] fp32 (either may be None)."""
    T, K = topk_ids.shape
    H = grad_out.shape[-1]
    if tuple(grad_out.shape) != (T, H):
        raise ValueError(f"grad_out: [{T}, hidden] expected, got {tuple(grad_out.shape)}")
    if grad_topk_weights is not None and expert_out is None:
        raise ValueError("expert_out: needed for grad_topk_weights")
    masked = _mode(mode) == MOE_MODE_MASKED
    # normal layout: a declared capacity; 0: N rows, known only on the device
    rows = num_experts * max_tokens_per_expert if masked else int(expert_out_rows)
    _row_buffer(mode, expert_out, H, max_tokens_per_expert, "expert_out")
    _row_buffer(mode, grad_expert_out, H, max_tokens_per_expert, "grad_expert_out")
    pg, pe, pi, pw, ps, pseg, pge, pgw, pst = _pointers(
        (grad_out, 0, "grad_out", _BF16), (expert_out, 2 * rows * H, "expert_out", _BF16),
        (topk_ids, 0, "topk_ids", _I32), (topk_weights, 4 * T * K, "topk_weights", _F32),
        (src2dst, 4 * T * K, "src2dst", _I32), (seg_indptr, 8 * (num_experts + 1) if masked else 0, "seg_indptr", _I64),
        (grad_expert_out, 2 * rows * H, "grad_expert_out", _BF16),
        (grad_topk_weights, 4 * T * K, "grad_topk_weights", _F32), (dev_status, 4, "dev_status", _I32))
    st = load_library().moe_combine_backward(_mode(mode), pg, pe, T, H, K, num_experts, max_tokens_per_expert,
                                             int(expert_out_rows), pi, ps, pseg, pw, pge, pgw, pst, _on(stream))
    _check(st, "moe_combine_backward")


def _norm_quant(quant: str) -> int:
    if quant not in NORM_QUANTS:
        raise ValueError(f"quant: one of {sorted(NORM_QUANTS)} expected, got {quant!r}")
    return NORM_QUANTS[quant]


def moe_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, out: Optional[torch.Tensor] = None,
                residual: Optional[torch.Tensor] = None, sum: Optional[torch.Tensor] = None,
                rstd: Optional[torch.Tensor] = None, quant: str = "none", codes: Optional[torch.Tensor] = None,
                scales: Optional[torch.Tensor] = None, stream=None) -> None:
    """Root-mean-square norm of x + residual [T, hidden]: into out in bf16 and, with `quant`, into codes [T, hidden] uint8
    and scales [T, hidden/128] (fp32, or uint8 for fp8g128_ue8m0); the sum into sum (only with a residual), 1/rms into rstd
    [T] fp32."""
    T, H = x.shape
    if sum is not None and residual is None:
        raise ValueError("sum: without a residual it is x, and not written")
    q = _norm_quant(quant)
    if not q and (codes is not None or scales is not None):
        raise ValueError("codes, scales: not written without quant")
    for t, name, width in ((out, "out", H), (residual, "residual", H), (sum, "sum", H), (codes, "codes", H),
                           (scales, "scales", H // 128)):
        _row_buffer("normal", t, width, 0, name)
    n = 2 * T * H
    sdtype = _F32 if q == MOE_QUANT_FP8_G128 else torch.uint8
    px, pw, po, pr, psum, prs, pc, psc = _pointers(
        (x, 0, "x", _BF16), (weight, 2 * H, "weight", _BF16), (out, n, "out", _BF16), (residual, n, "residual", _BF16),
        (sum, n, "sum", _BF16), (rstd, 4 * T, "rstd", _F32), (codes, T * H, "codes", torch.uint8),
        (scales, T * (H // 128) * sdtype.itemsize if q else 0, "scales", sdtype if q else None))
    st = load_library().moe_rmsnorm(px, pr, pw, float(eps), T, H, q, po, pc, psc, psum, prs, _on(stream))
    _check(st, "moe_rmsnorm")


def moe_rmsnorm_backward_workspace_size(num_tokens: int, hidden: int) -> int:
    return int(load_library().moe_rmsnorm_backward_workspace_size(int(num_tokens), int(hidden)))


def moe_rmsnorm_backward(grad_out: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                         grad_x: torch.Tensor, grad_weight: torch.Tensor, workspace: Optional[torch.Tensor],
                         grad_sum: Optional[torch.Tensor] = None, stream=None) -> None:
    """The gradient of :func:`moe_rmsnorm`, from its sum (x without a residual) and rstd: grad_x [T, hidden] bf16 of x and
    of the residual alike, grad_sum being what else flows into their sum, and grad_weight [hidden] fp32."""
    T, H = s.shape
    n = 2 * T * H
    for t, name in ((grad_out, "grad_out"), (grad_sum, "grad_sum"), (grad_x, "grad_x")):
        _row_buffer("normal", t, H, 0, name)
    pg, ps, pw, pr, pgs, pgx, pgw, pws = _pointers(
        (grad_out, n, "grad_out", _BF16), (s, 0, "s", _BF16), (weight, 2 * H, "weight", _BF16), (rstd, 4 * T, "rstd", _F32),
        (grad_sum, n, "grad_sum", _BF16), (grad_x, n, "grad_x", _BF16), (grad_weight, 4 * H, "grad_weight", _F32),
        (workspace, 0, "workspace", None))
    st = load_library().moe_rmsnorm_backward(pg, ps, pw, pr, pgs, T, H, pgx, pgw, pws,
                                             workspace.nbytes if workspace is not None else 0, _on(stream))
    _check(st, "moe_rmsnorm_backward")


# ---------------------------------------------------------------------------
# convenience layer
# ---------------------------------------------------------------------------

class NormOutput(NamedTuple):
    out: Optional[torch.Tensor]      # bf16 [T, hidden]
    codes: Optional[torch.Tensor]    # uint8 [T, hidden]: e4m3
    scales: Optional[torch.Tensor]   # [T, hidden/128], fp32 or UE8M0 bytes
    sum: Optional[torch.Tensor]      # bf16 [T, hidden]: x + residual; x itself without a residual
    rstd: Optional[torch.Tensor]     # fp32 [T], with keep


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
            quant: str = "none", bf16: Optional[bool] = None, keep: bool = False, stream=None) -> NormOutput:
    """Root-mean-square norm of x + residual [T, hidden], as bf16 rows, as FP8 rows with the dispatch's scales (`quant`),
    or both (`bf16`: by default the rows are bf16 where they are not FP8). `keep` also returns what
    :func:`rmsnorm_backward` needs. The result is allocated on `stream`.

    Codes go through the dispatch as they are (quant="fp8_passthrough"); it moves rows of a multiple of 32 bytes. So do scale
    rows, as bytes, where they are such rows (fp32: hidden a multiple of 1024; UE8M0: of 4096), and else padded to 32."""
    if stream is not None:
        with _current(stream):
            return rmsnorm(x, weight, eps, residual, quant, bf16, keep)
    T, H = x.shape
    q, n = _norm_quant(quant), 2 * T * H
    _row_buffer("normal", residual, H, 0, "residual")
    px, pw, pr = _pointers((x, 0, "x", _BF16), (weight, 2 * H, "weight", _BF16), (residual, n, "residual", _BF16))
    if bf16 is None:
        bf16 = not q
    out = codes = scales = rstd = None
    total = x
    if bf16:
        out = torch.empty_like(x)
    if residual is not None:
        total = torch.empty_like(x)
    if q:
        codes = torch.empty_like(x, dtype=torch.uint8)
        scales = torch.empty((T, H // 128), dtype=_F32 if q == MOE_QUANT_FP8_G128 else torch.uint8, device=x.device)
    if keep:
        rstd = torch.empty(T, dtype=_F32, device=x.device)
    # what is allocated here needs no checks
    st = load_library().moe_rmsnorm(px, pr, pw, float(eps), T, H, q, out.data_ptr() if bf16 else None,
                                    codes.data_ptr() if q else None, scales.data_ptr() if q else None,
                                    total.data_ptr() if total is not x else None, rstd.data_ptr() if keep else None,
                                    _on(None))
    _check(st, "moe_rmsnorm")
    return NormOutput(out, codes, scales, total, rstd)


def rmsnorm_backward(grad_out: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     grad_residual: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(grad_x, grad_weight) of :func:`rmsnorm` from its sum and rstd: grad_x is the gradient of x and of the residual
    alike; `grad_residual` is what flows into their sum by other ways. Allocated on `stream`."""
    if stream is not None:
        with _current(stream):
            return rmsnorm_backward(grad_out, s, weight, rstd, grad_residual)
    T, H = s.shape
    n = 2 * T * H
    _row_buffer("normal", grad_out, H, 0, "grad_out")
    _row_buffer("normal", grad_residual, H, 0, "grad_residual")
    pg, ps, pw, pr, pgs = _pointers((grad_out, n, "grad_out", _BF16), (s, 0, "s", _BF16), (weight, 2 * H, "weight", _BF16),
                                    (rstd, 4 * T, "rstd", _F32), (grad_residual, n, "grad_residual", _BF16))
    lib = load_library()
    size = lib.moe_rmsnorm_backward_workspace_size(T, H)
    # what is allocated here needs no checks
    grad_x, grad_weight = torch.empty_like(s), torch.empty(H, dtype=_F32, device=s.device)
    workspace = torch.empty(size, dtype=torch.uint8, device=s.device)
    st = lib.moe_rmsnorm_backward(pg, ps, pw, pr, pgs, T, H, grad_x.data_ptr(), grad_weight.data_ptr(),
                                  workspace.data_ptr(), size, _on(None))
    _check(st, "moe_rmsnorm_backward")
    return grad_x, grad_weight


class LayerGradients(NamedTuple):
    x: torch.Tensor              # bf16 [T, hidden]
    topk_weights: torch.Tensor   # fp32 [T, K]
    w13: torch.Tensor            # fp32 or bf16 [E, 2*inter, hidden]
    w2: torch.Tensor             # [E, hidden, inter]


class BF16MoELayer:
    """A layer's experts with bf16 weights and pre-allocated buffers, for training and for serving: token rows and their
    routing in, the weighted sum out, and the gradients of all of them.

    Route metadata, dispatch of bf16 rows, the two products and the combine; for up to ``few_tokens`` tokens (at most
    MOE_LAYER_MAX_TOKENS, never with ``train``) :func:`moe_layer_few_tokens` instead. It defaults to four pairs an expert, as
    in :class:`MoELayer`: below that the few-token kernels are ahead (16 experts of 4096 x 1024, top-2, 8 tokens: 51 us
    against 68; 256 experts of 7168 x 512, top-8, 64 tokens: 699 against 724), there both are about as fast (64 tokens, 128
    experts, top-8, of 2048 x 768: 201 against 193; of 4096 x 768: 355 against 362). With few experts they stay 4 to 11 %
    ahead up to 64 tokens (16 experts as above: 76 against 81). With ``train`` a call keeps what
    :meth:`backward` needs until the next call. Weight gradients are ``grad_dtype`` (fp32 or bf16), in kept buffers that
    ``accumulate`` adds to. No call allocates, so a call of a fixed size can be captured in a CUDA graph. All calls share
    the layer's buffers: one at a time, a backward pass after its own forward pass, which reads that call's topk_ids and
    topk_weights again: they have to hold what they held.
    """

    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, topk: int, max_tokens: int, *, train: bool = False,
                 grad_dtype: torch.dtype = torch.float32, few_tokens: Optional[int] = None):
        if w13.dim() != 3 or w2.dim() != 3 or w13.shape[1] % 2 or \
                tuple(w2.shape) != (w13.shape[0], w13.shape[2], w13.shape[1] // 2):
            raise ValueError(f"w13 [E, 2*inter, hidden] and w2 [E, hidden, inter] expected, got {tuple(w13.shape)} and "
                             f"{tuple(w2.shape)}")
        if w13.dtype is not _BF16 or w2.dtype is not _BF16:
            raise ValueError(f"w13, w2: bf16 weights expected, got {w13.dtype} and {w2.dtype}")
        if max_tokens < 1 or topk < 1:
            raise ValueError(f"max_tokens and topk: 1 or more expected, got {max_tokens} and {topk}")
        if grad_dtype not in (_F32, _BF16):
            raise ValueError(f"grad_dtype: torch.float32 or torch.bfloat16 expected, got {grad_dtype}")
        self.w13, self.w2, self.K, self.T, self.train = w13, w2, topk, max_tokens, train
        self.E, self.H, self.I = w2.shape
        if self.H % 16 or self.I % 8:
            raise ValueError(f"hidden a multiple of 16 and inter one of 8 expected, got {self.H} and {self.I}")
        few = 4 * self.E // topk if few_tokens is None else few_tokens
        self.few = 0 if train or self.I % 16 else min(few, MOE_LAYER_MAX_TOKENS, max_tokens)
        dev = w13.device
        rows = max_tokens * topk
        bf16, i32 = dict(dtype=_BF16, device=dev), dict(dtype=_I32, device=dev)
        self.status = new_status(dev)
        self.out = torch.empty((max_tokens, self.H), **bf16)
        self.few_workspace = new_layer_workspace(self.few, topk, self.H, self.I, self.E, dev) if self.few else None
        # fewer pairs can need more blocks of the count kernel (its blocks grow by 131072 pairs at a time)
        sizes = [max_tokens] + [131072 * r // topk for r in range(1, 17) if 131072 * r // topk < max_tokens]
        self.workspace = max((new_workspace(t, topk, self.E, dev) for t in sizes),
                             key=lambda w: 0 if w is None else w.numel())
        self.seg_indptr = torch.zeros(self.E + 1, dtype=_I64, device=dev)
        self.src2dst = torch.empty(rows, **i32)
        self.reorder_topk_ids = torch.empty(rows, **i32)
        self.masked_m = torch.zeros(self.E, **i32)
        self.rows_x = torch.empty((rows, self.H), **bf16)
        self.rows_h = torch.empty((rows, self.I), **bf16)
        self.rows_out = torch.empty((rows, self.H), **bf16)
        self.seen = None
        if not train:
            return
        self.gate_up = torch.empty((rows, 2 * self.I), **bf16)
        self.ones = torch.ones((max_tokens, topk), dtype=_F32, device=dev)
        self.grad_x = torch.empty((max_tokens, self.H), **bf16)
        self.grad_topk_weights = torch.empty((max_tokens, topk), dtype=_F32, device=dev)
        self.grad_w13 = torch.zeros(w13.shape, dtype=grad_dtype, device=dev)
        self.grad_w2 = torch.zeros(w2.shape, dtype=grad_dtype, device=dev)

    def __call__(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                 stream=None) -> torch.Tensor:
        """x [T, hidden] bf16, T <= max_tokens: the layer's output [T, hidden], a view of a kept buffer."""
        T = x.shape[0]
        if T > self.T:
            raise ValueError(f"{T} tokens: the layer was made for {self.T}")
        if x.shape != (T, self.H) or topk_ids.shape != (T, self.K) or topk_weights.shape != (T, self.K):
            raise ValueError(f"x, topk_ids, topk_weights: [T, {self.H}], [T, {self.K}] and [T, {self.K}] expected, got "
                             f"{tuple(x.shape)}, {tuple(topk_ids.shape)} and {tuple(topk_weights.shape)}")
        # all of them before the first launch: the route metadata and the few-token kernels do not ask for the device
        _pointers((x, 0, "x", _BF16), (topk_ids, 0, "topk_ids", _I32), (topk_weights, 0, "topk_weights", _F32),
                  (self.w13, 0, "w13", _BF16), (self.w2, 0, "w2", _BF16))
        out = self.out[:T]
        self.seen = None
        if self.few and T <= self.few:
            moe_layer_few_tokens(x, topk_ids, topk_weights, self.w13, self.w2, out, self.few_workspace, self.status,
                                 stream=stream)
            return out
        n, seg = T * self.K, self.seg_indptr
        moe_route_meta_ex(topk_ids, self.E, seg, self.src2dst, self.reorder_topk_ids, self.masked_m, self.status,
                          self.workspace, stream=stream)
        moe_dispatch_ex("normal", "none", "row", x, topk_ids, self.E, self.src2dst, seg, self.rows_x, None, self.status,
                        out_rows=n, stream=stream)
        moe_expert_gemm_swiglu_bf16("normal", self.rows_x[:n], self.masked_m, self.w13, self.rows_h, self.status,
                                    self.gate_up if self.train else None, seg, stream=stream)
        moe_expert_gemm_bf16("normal", self.rows_h[:n], self.masked_m, self.w2, self.rows_out, self.status,
                             seg_indptr=seg, stream=stream)
        moe_combine_ex("normal", self.rows_out, topk_ids, topk_weights, self.E, self.src2dst, seg, out, self.status,
                       expert_out_rows=n, stream=stream)
        if self.train:
            self.seen = (topk_ids, topk_weights)
        return out

    def backward(self, grad_out: torch.Tensor, accumulate: bool = False, stream=None) -> LayerGradients:
        """The gradients of the last call's x, topk_weights and of the weights, from that of its output [T, hidden]. They
        are views of kept buffers; with `accumulate` the weights' gradients are added to what these hold."""
        if self.seen is None:
            raise RuntimeError("backward: no forward pass of a layer made with train=True to go back through")
        ids, weights = self.seen
        T, seg = ids.shape[0], self.seg_indptr
        if grad_out.shape != (T, self.H):
            raise ValueError(f"grad_out: [{T}, {self.H}] expected, got {tuple(grad_out.shape)}")
        n = T * self.K
        where = dict(seg_indptr=seg, stream=stream)
        grad_rows = self.rows_out[:n]          # the experts' outputs become their gradients
        moe_combine_backward("normal", grad_out, grad_rows, ids, weights, self.E, self.src2dst, seg, grad_rows,
                             self.grad_topk_weights, self.status, expert_out_rows=n, stream=stream)
        self.seen = None                       # the rows are gone, but not if that call was refused
        moe_expert_wgrad_bf16("normal", grad_rows, self.rows_h[:n], self.masked_m, self.grad_w2, self.status, accumulate,
                              **where)
        gate_up = self.gate_up[:n]             # and gate and up theirs
        moe_expert_gemm_dswiglu_bf16("normal", grad_rows, self.masked_m, self.w2, gate_up, gate_up, self.status, **where)
        moe_expert_wgrad_bf16("normal", gate_up, self.rows_x[:n], self.masked_m, self.grad_w13, self.status, accumulate,
                              **where)
        moe_expert_gemm_bf16("normal", gate_up, self.masked_m, self.w13, self.rows_x, self.status, True, **where)
        grad_x = self.grad_x[:T]
        moe_combine_ex("normal", self.rows_x, ids, self.ones, self.E, self.src2dst, seg, grad_x, self.status,
                       expert_out_rows=n, stream=stream)
        return LayerGradients(grad_x, self.grad_topk_weights[:T], self.grad_w13, self.grad_w2)

    def check(self) -> None:
        check_status(self.status, "BF16MoELayer")
