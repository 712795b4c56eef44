"""The expert operators between dispatch and combine: NVFP4 quantisation, the products over a
dispatched layout's experts, and the whole layer for a few tokens.

Binding of ``include/moe_experts.h`` in the manner of the package: the functions named like the C
entry points only check and marshal arguments; :func:`quantize_nvfp4`, :func:`quantize_experts` and
:class:`MoELayer` allocate with torch. All names are reachable from the package itself.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import (MOE_ERR_UNSUPPORTED, MOE_MODE_MASKED, MOE_QUANT_NONE, MOE_QUANT_NVFP4_B16, MOE_SCALES_ROW_MAJOR,
               MOE_SCALES_SWIZZLED_128X4, MODES, SCALE_LAYOUTS, MoEError, _check, _need, _ptr, _stream, check_status,
               load_library, moe_combine_ex, moe_dispatch_ex, moe_route_meta_ex, new_status, new_workspace)

__all__ = [
    "MOE_LAYER_MAX_TOKENS", "NVFP4Rows", "ExpertWeights", "MoELayer", "moe_quantize_nvfp4", "moe_dequantize_nvfp4",
    "moe_expert_gemm", "moe_expert_gemm_swiglu", "moe_layer_workspace_size", "moe_layer_few_tokens",
    "nvfp4_scale_bytes", "quantize_nvfp4", "dequantize_nvfp4", "new_layer_workspace", "quantize_experts",
]

MOE_LAYER_MAX_TOKENS = 64


def _layout(scale_layout: str) -> int:
    if scale_layout not in SCALE_LAYOUTS:
        raise ValueError(f"scale_layout: one of {sorted(SCALE_LAYOUTS)} expected, got {scale_layout!r}")
    return SCALE_LAYOUTS[scale_layout]


def nvfp4_scale_bytes(rows: int, hidden: int, scale_layout: str) -> int:
    """Bytes of the block scales of one [rows, hidden] matrix."""
    if _layout(scale_layout) == MOE_SCALES_SWIZZLED_128X4:
        rows = (rows + 127) // 128 * 128
    return rows * (hidden // 16)


def _mode(mode: str) -> int:
    if mode not in MODES:
        raise ValueError(f"mode: one of {sorted(MODES)} expected, got {mode!r}")
    return MODES[mode]


def _pointers(*specs):
    """Checks (tensor or None, bytes needed, name, dtype) and returns the data pointers: element types and sizes of all of
    them first, then that they are contiguous device tensors."""
    out, wrong = [], None
    for t, nbytes, name, dtype in specs:
        if t is None:
            out.append(None)
            continue
        if t.dtype is not dtype or t.nbytes < nbytes:
            _need(t, nbytes, name, dtype)
        if wrong is None and not (t.is_cuda and t.is_contiguous()):
            wrong = t
        out.append(t.data_ptr())
    if wrong is not None:
        _ptr(wrong)
    return out


def _on(stream):
    """The handle of `stream`, or of torch's current one (the tensors are on the device: torch has its context)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return _stream(stream)


def _current(stream):
    """A context with `stream` (a torch stream or a raw handle) current, so that what is allocated in it is its own."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)))
    return torch.cuda.stream(stream)


# ---------------------------------------------------------------------------
# thin wrappers with the C names
# ---------------------------------------------------------------------------

def moe_quantize_nvfp4(x: torch.Tensor, global_scales: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                       scale_layout: str = "swizzled", stream=None) -> None:
    """x [groups, rows, hidden] bf16 -> codes [groups, rows, hidden/2] and the groups' block scales."""
    G, R, H = x.shape
    layout = _layout(scale_layout)
    px, pg, pc, ps = _pointers((x, 0, "x", torch.bfloat16), (global_scales, 4 * G, "global_scales", torch.float32),
                               (codes, G * R * (H // 2), "codes", torch.uint8),
                               (scales, G * nvfp4_scale_bytes(R, H, scale_layout), "scales", torch.uint8))
    st = load_library().moe_quantize_nvfp4(px, G, R, H, pg, layout, pc, ps, _on(stream))
    _check(st, "moe_quantize_nvfp4")


def moe_dequantize_nvfp4(codes: torch.Tensor, scales: torch.Tensor, global_scales: torch.Tensor, out: torch.Tensor,
                         scale_layout: str = "swizzled", stream=None) -> None:
    """The reverse of :func:`moe_quantize_nvfp4`, into out [groups, rows, hidden] bf16."""
    G, R, H = out.shape
    layout = _layout(scale_layout)
    pc, ps, pg, po = _pointers((codes, G * R * (H // 2), "codes", torch.uint8),
                               (scales, G * nvfp4_scale_bytes(R, H, scale_layout), "scales", torch.uint8),
                               (global_scales, 4 * G, "global_scales", torch.float32),
                               (out, 0, "out", torch.bfloat16))
    st = load_library().moe_dequantize_nvfp4(pc, ps, G, R, H, pg, layout, po, _on(stream))
    _check(st, "moe_dequantize_nvfp4")


def _rows(mode: str, a_codes: torch.Tensor, K: int, E: int, M: int, seg_indptr) -> int:
    if a_codes.shape[-1] != K // 2:
        raise ValueError(f"a_codes: rows of {K // 2} bytes needed, got {a_codes.shape[-1]}")
    if _mode(mode) == MOE_MODE_MASKED:
        return E * M
    if seg_indptr is None:
        raise ValueError("seg_indptr: needed in normal mode")
    return a_codes.shape[:-1].numel()


def moe_expert_gemm(mode: str, a_codes: torch.Tensor, a_scales: torch.Tensor, masked_m: torch.Tensor,
                    w_codes: torch.Tensor, w_scales: torch.Tensor, out: torch.Tensor, dev_status: torch.Tensor,
                    alpha: Optional[torch.Tensor] = None, seg_indptr: Optional[torch.Tensor] = None,
                    max_tokens_per_expert: int = 0, scale_layout: str = "swizzled", stream=None) -> None:
    """out[r] = alpha[e] * w[e] a[r] for the rows of every expert e of a dispatched layout.

    w_codes [E, n, k/2]; a_codes [rows, k/2] (normal) or [E, M, k/2] (masked, M = max_tokens_per_expert)."""
    E, N, K = w_codes.shape
    K *= 2
    rows = _rows(mode, a_codes, K, E, max_tokens_per_expert, seg_indptr)
    layout = _layout(scale_layout)
    pa, pas, pm, pseg, pal, pw, pws, po, pst = _pointers(
        (a_codes, rows * (K // 2), "a_codes", torch.uint8),
        (a_scales, nvfp4_scale_bytes(rows, K, scale_layout), "a_scales", torch.uint8),
        (masked_m, 4 * E, "masked_m", torch.int32),
        (seg_indptr, 8 * (E + 1) if mode == "normal" else 0, "seg_indptr", torch.int64),
        (alpha, 4 * E, "alpha", torch.float32),
        (w_codes, 0, "w_codes", torch.uint8),
        (w_scales, E * ((N + 127) // 128 * 128) * (K // 16), "w_scales", torch.uint8),
        (out, 2 * rows * N, "out", torch.bfloat16), (dev_status, 4, "dev_status", torch.int32))
    st = load_library().moe_expert_gemm(MODES[mode], pa, pas, layout, E, max_tokens_per_expert, rows, N, K, pseg, pm, pw,
                                        pws, pal, po, pst, _on(stream))
    _check(st, "moe_expert_gemm")


def moe_expert_gemm_swiglu(mode: str, a_codes: torch.Tensor, a_scales: torch.Tensor, masked_m: torch.Tensor,
                           w13_codes: torch.Tensor, w13_scales: torch.Tensor, out_codes: torch.Tensor,
                           out_scales: torch.Tensor, dev_status: torch.Tensor, out_global_scale: float,
                           alpha: Optional[torch.Tensor] = None, seg_indptr: Optional[torch.Tensor] = None,
                           max_tokens_per_expert: int = 0, scale_layout: str = "swizzled", stream=None) -> None:
    """The gate and up products (w13_codes [E, 2*inter, k/2]), SwiGLU and quantisation of its result in one kernel."""
    E, N, K = w13_codes.shape
    if N % 2:
        raise ValueError(f"w13_codes: gate and up rows do not fit {N} rows")
    N, K = N // 2, 2 * K
    rows = _rows(mode, a_codes, K, E, max_tokens_per_expert, seg_indptr)
    layout = _layout(scale_layout)
    pa, pas, pm, pseg, pal, pw, pws, po, pos, pst = _pointers(
        (a_codes, rows * (K // 2), "a_codes", torch.uint8),
        (a_scales, nvfp4_scale_bytes(rows, K, scale_layout), "a_scales", torch.uint8),
        (masked_m, 4 * E, "masked_m", torch.int32),
        (seg_indptr, 8 * (E + 1) if mode == "normal" else 0, "seg_indptr", torch.int64),
        (alpha, 4 * E, "alpha", torch.float32),
        (w13_codes, 0, "w13_codes", torch.uint8),
        (w13_scales, 2 * E * ((N + 127) // 128 * 128) * (K // 16), "w13_scales", torch.uint8),
        (out_codes, rows * (N // 2), "out_codes", torch.uint8),
        (out_scales, nvfp4_scale_bytes(rows, N, scale_layout), "out_scales", torch.uint8),
        (dev_status, 4, "dev_status", torch.int32))
    st = load_library().moe_expert_gemm_swiglu(MODES[mode], pa, pas, layout, E, max_tokens_per_expert, rows, N, K, pseg,
                                               pm, pw, pws, pal, float(out_global_scale), po, pos, pst, _on(stream))
    _check(st, "moe_expert_gemm_swiglu")


def moe_layer_workspace_size(num_tokens: int, topk: int, hidden: int, inter: int, num_experts: int) -> int:
    return int(load_library().moe_layer_workspace_size(int(num_tokens), int(topk), int(hidden), int(inter),
                                                       int(num_experts)))


def moe_layer_few_tokens(x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor, w13: torch.Tensor,
                         w2: torch.Tensor, out: torch.Tensor, workspace: Optional[torch.Tensor],
                         dev_status: torch.Tensor, w13_scales: Optional[torch.Tensor] = None,
                         w2_scales: Optional[torch.Tensor] = None, alpha13: Optional[torch.Tensor] = None,
                         alpha2: Optional[torch.Tensor] = None, stream=None) -> None:
    """The layer's experts and their weighted sum for up to MOE_LAYER_MAX_TOKENS tokens.

    Weights bf16 (w13 [E, 2*inter, hidden], w2 [E, hidden, inter]) or, as uint8, NVFP4 codes with their scales."""
    T, H = x.shape
    K = topk_ids.shape[1]
    E, I2, W = w13.shape
    I = I2 // 2
    nvfp4 = w13.dtype is torch.uint8
    dtype, per = (torch.uint8, 2) if nvfp4 else (torch.bfloat16, 1)
    if I2 % 2 or W != H // per or tuple(w2.shape) != (E, H, I // per):
        raise ValueError(f"w13 {tuple(w13.shape)} and w2 {tuple(w2.shape)} do not fit hidden {H}")
    if nvfp4 and (w13_scales is None or w2_scales is None):
        raise ValueError("w13_scales, w2_scales: needed with NVFP4 weights")
    if not nvfp4:
        w13_scales = w2_scales = None
    px, pi, pt, p13, p2, ps13, ps2, pa13, pa2, po, pws, pst = _pointers(
        (x, 0, "x", torch.bfloat16), (topk_ids, 0, "topk_ids", torch.int32),
        (topk_weights, 4 * T * K, "topk_weights", torch.float32), (w13, 0, "w13", dtype), (w2, 0, "w2", dtype),
        (w13_scales, 2 * E * ((I + 127) // 128 * 128) * (H // 16), "w13_scales", torch.uint8),
        (w2_scales, E * ((H + 127) // 128 * 128) * (I // 16), "w2_scales", torch.uint8),
        (alpha13, 4 * E, "alpha13", torch.float32), (alpha2, 4 * E, "alpha2", torch.float32),
        (out, 2 * T * H, "out", torch.bfloat16), (workspace, 0, "workspace", torch.uint8),
        (dev_status, 4, "dev_status", torch.int32))
    if topk_ids.shape[0] != T:
        raise ValueError(f"topk_ids: {T} rows needed, got {topk_ids.shape[0]}")
    st = load_library().moe_layer_few_tokens(
        px, T, H, I, pi, pt, K, E, MOE_QUANT_NVFP4_B16 if nvfp4 else MOE_QUANT_NONE, p13, ps13, pa13, p2, ps2, pa2, po,
        pws, workspace.nbytes if workspace is not None else 0, pst, _on(stream))
    _check(st, "moe_layer_few_tokens")


# ---------------------------------------------------------------------------
# convenience layer
# ---------------------------------------------------------------------------

class NVFP4Rows(NamedTuple):
    codes: torch.Tensor    # uint8 [.., rows, hidden/2]
    scales: torch.Tensor   # uint8, one matrix's scales per group: [.., rows, hidden/16] or [.., tile bytes]
    scale_layout: str


def quantize_nvfp4(x: torch.Tensor, global_scales: torch.Tensor, scale_layout: str = "swizzled",
                   stream=None) -> NVFP4Rows:
    """Quantise x [groups, rows, hidden], or one matrix [rows, hidden], with one global scale per group. The result is
    allocated on `stream`."""
    if stream is not None:
        with _current(stream):
            return quantize_nvfp4(x, global_scales, scale_layout)
    shape = x.shape
    if len(shape) == 2:
        q = quantize_nvfp4(x.unsqueeze(0), global_scales, scale_layout)
        return NVFP4Rows(q.codes[0], q.scales[0], scale_layout)
    G, R, H = shape
    layout = _layout(scale_layout)
    px, pg = _pointers((x, 0, "x", torch.bfloat16), (global_scales, 4 * G, "global_scales", torch.float32))
    dev = x.device
    codes = torch.empty((G, R, H // 2), dtype=torch.uint8, device=dev)
    tail = (R, H // 16) if layout == MOE_SCALES_ROW_MAJOR else ((R + 127) // 128 * 128 * (H // 16),)
    scales = torch.empty((G, *tail), dtype=torch.uint8, device=dev)
    st = load_library().moe_quantize_nvfp4(px, G, R, H, pg, layout, codes.data_ptr(), scales.data_ptr(), _on(None))
    _check(st, "moe_quantize_nvfp4")
    return NVFP4Rows(codes, scales, scale_layout)


def dequantize_nvfp4(q: NVFP4Rows, global_scales: torch.Tensor, stream=None) -> torch.Tensor:
    """The bf16 values that q stands for, allocated on `stream`."""
    if stream is not None:
        with _current(stream):
            return dequantize_nvfp4(q, global_scales)
    codes, scales, scale_layout = q
    shape = codes.shape
    if len(shape) == 2:
        return dequantize_nvfp4(NVFP4Rows(codes.unsqueeze(0), scales, scale_layout), global_scales)[0]
    G, R, C = shape
    layout = _layout(scale_layout)
    pc, ps, pg = _pointers((codes, 0, "codes", torch.uint8),
                           (scales, G * nvfp4_scale_bytes(R, 2 * C, scale_layout), "scales", torch.uint8),
                           (global_scales, 4 * G, "global_scales", torch.float32))
    out = torch.empty((G, R, 2 * C), dtype=torch.bfloat16, device=codes.device)
    st = load_library().moe_dequantize_nvfp4(pc, ps, G, R, 2 * C, pg, layout, out.data_ptr(), _on(None))
    _check(st, "moe_dequantize_nvfp4")
    return out


def new_layer_workspace(num_tokens: int, topk: int, hidden: int, inter: int, num_experts: int,
                        device=None) -> Optional[torch.Tensor]:
    n = moe_layer_workspace_size(num_tokens, topk, hidden, inter, num_experts)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda") if n else None


class ExpertWeights(NamedTuple):
    """A layer's expert weights: bf16 (scales and alphas None) or NVFP4."""
    w13: torch.Tensor                      # [E, 2*inter, hidden] bf16, or codes [E, 2*inter, hidden/2]
    w2: torch.Tensor                       # [E, hidden, inter] bf16, or codes [E, hidden, inter/2]
    w13_scales: Optional[torch.Tensor] = None
    w2_scales: Optional[torch.Tensor] = None
    alpha13: Optional[torch.Tensor] = None  # [E] fp32: 1 / global scale of w13[e]; None: 1
    alpha2: Optional[torch.Tensor] = None

    @property
    def quantised(self) -> bool:
        return self.w13.dtype == torch.uint8


def quantize_experts(w13: torch.Tensor, w2: torch.Tensor) -> ExpertWeights:
    """NVFP4 weights of bf16 ones, one global scale (448 * 6 / max|w|) per expert and matrix."""
    E, I2, H = w13.shape
    g13 = (2688.0 / w13.abs().amax(dim=(1, 2)).float().clamp(min=1e-30)).contiguous()
    g2 = (2688.0 / w2.abs().amax(dim=(1, 2)).float().clamp(min=1e-30)).contiguous()
    q13 = quantize_nvfp4(w13.view(2 * E, I2 // 2, H), g13.repeat_interleave(2))
    q2 = quantize_nvfp4(w2, g2)
    return ExpertWeights(q13.codes.view(E, I2, H // 2), q2.codes, q13.scales, q2.scales, 1 / g13, 1 / g2)


class MoELayer:
    """A layer's experts with pre-allocated buffers: token rows and their routing in, the weighted sum out.

    Up to ``few_tokens`` tokens (at most MOE_LAYER_MAX_TOKENS) take :func:`moe_layer_few_tokens`, which
    quantises weights only. More take route metadata, NVFP4 dispatch into 128-row segments, the two
    products and the combine, which quantise activations too: by ``input_scale`` (448 * 6 over the largest
    |x| to expect) and ``inter_scale`` (the same of the SwiGLU outputs). Without these scales, or with bf16
    weights, the layer serves few tokens only. ``few_tokens`` defaults to four pairs an expert, about where the
    two ways take the same time: between three pairs (128 experts of 2048 x 768, top-8, 48 tokens: 82 us against
    82) and eight (16 experts of 4096 x 1024, top-2, 64 tokens: 49 against 47); 64 experts of 4096 x 1024, top-8
    take 43 us against 60 with 4 tokens, 91 against 101 with 32 and 122 against 102 with 64. No call allocates, so
    a call of a fixed size can be captured in a CUDA graph. All calls share the layer's buffers: one at a time.
    """

    ALIGN = 128

    def __init__(self, weights: ExpertWeights, topk: int, max_tokens: int, *, input_scale: float = 0.0,
                 inter_scale: float = 0.0, few_tokens: Optional[int] = None):
        self.weights = weights
        self.E, self.H = weights.w2.shape[0], weights.w2.shape[1]
        self.I, self.K, self.T = weights.w13.shape[1] // 2, topk, max_tokens
        if few_tokens is None:
            scaled = weights.quantised and input_scale > 0 and inter_scale > 0
            few_tokens = 4 * self.E // topk if scaled else MOE_LAYER_MAX_TOKENS
        self.few = min(few_tokens, MOE_LAYER_MAX_TOKENS, max_tokens)
        dev = weights.w13.device
        self.status = new_status(dev)
        self.out = torch.empty((max_tokens, self.H), dtype=torch.bfloat16, device=dev)
        self.few_workspace = new_layer_workspace(self.few, topk, self.H, self.I, self.E, dev)
        if max_tokens <= self.few:
            return
        if not weights.quantised:
            raise MoEError(MOE_ERR_UNSUPPORTED, f"MoELayer: bf16 weights serve at most {self.few} tokens")
        if not (input_scale > 0 and inter_scale > 0):
            raise ValueError("input_scale, inter_scale: positive scales needed to quantise activations")
        self.input_scale, self.inter_scale = float(input_scale), float(inter_scale)
        one = torch.ones(self.E, dtype=torch.float32, device=dev)
        self.alpha13 = (one if weights.alpha13 is None else weights.alpha13) / self.input_scale
        self.alpha2 = (one if weights.alpha2 is None else weights.alpha2) / self.inter_scale
        rows = max_tokens * topk + self.E * (self.ALIGN - 1)
        byte = dict(dtype=torch.uint8, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        # fewer pairs can need more blocks of the count kernel (its blocks grow by 131072 pairs at a time)
        sizes = [max_tokens] + [131072 * r // topk for r in range(1, 17) if 131072 * r // topk < max_tokens]
        self.workspace = max((new_workspace(t, topk, self.E, dev) for t in sizes),
                             key=lambda w: 0 if w is None else w.numel())
        self.seg_indptr = torch.zeros(self.E + 1, dtype=torch.int64, device=dev)
        self.src2dst = torch.empty(max_tokens * topk, **i32)
        self.reorder_topk_ids = torch.empty(rows, **i32)
        self.masked_m = torch.zeros(self.E, **i32)
        self.x_codes = torch.empty((rows, self.H // 2), **byte)
        self.x_scales = torch.empty(nvfp4_scale_bytes(rows, self.H, "swizzled"), **byte)
        self.h_codes = torch.empty((rows, self.I // 2), **byte)
        self.h_scales = torch.empty(nvfp4_scale_bytes(rows, self.I, "swizzled"), **byte)
        self.expert_out = torch.empty((rows, self.H), dtype=torch.bfloat16, device=dev)

    def __call__(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                 stream=None) -> torch.Tensor:
        """x [T, hidden] bf16, T <= max_tokens: the layer's output [T, hidden], a view of a kept buffer."""
        T, w = x.shape[0], self.weights
        if T > self.T:
            raise ValueError(f"{T} tokens: the layer was made for {self.T}")
        if x.shape != (T, self.H) or topk_ids.shape != (T, self.K) or topk_weights.shape != (T, self.K):
            raise ValueError(f"x, topk_ids, topk_weights: [T, {self.H}], [T, {self.K}] and [T, {self.K}] expected, got "
                             f"{tuple(x.shape)}, {tuple(topk_ids.shape)} and {tuple(topk_weights.shape)}")
        out = self.out[:T]
        if T <= self.few:
            moe_layer_few_tokens(x, topk_ids, topk_weights, w.w13, w.w2, out, self.few_workspace, self.status,
                                 w.w13_scales, w.w2_scales, w.alpha13, w.alpha2, stream)
            return out
        rows = T * self.K + self.E * (self.ALIGN - 1)
        moe_route_meta_ex(topk_ids, self.E, self.seg_indptr, self.src2dst, self.reorder_topk_ids, self.masked_m,
                          self.status, self.workspace, expert_alignment=self.ALIGN, stream=stream)
        moe_dispatch_ex("normal", "nvfp4b16", "swizzled", x, topk_ids, self.E, self.src2dst, self.seg_indptr,
                        self.x_codes, self.x_scales, self.status, out_rows=rows, input_global_scale=self.input_scale,
                        stream=stream)
        moe_expert_gemm_swiglu("normal", self.x_codes[:rows], self.x_scales, self.masked_m, w.w13, w.w13_scales,
                               self.h_codes, self.h_scales, self.status, self.inter_scale, self.alpha13,
                               self.seg_indptr, stream=stream)
        moe_expert_gemm("normal", self.h_codes[:rows], self.h_scales, self.masked_m, w.w2, w.w2_scales,
                        self.expert_out, self.status, self.alpha2, self.seg_indptr, stream=stream)
        moe_combine_ex("normal", self.expert_out, topk_ids, topk_weights, self.E, self.src2dst, self.seg_indptr, out,
                       self.status, expert_out_rows=rows, stream=stream)
        return out

    def check(self) -> None:
        check_status(self.status, "MoELayer")
