"""A MoE block's bf16 operators refuse bad arguments on the host: the C entry points by their status, the binding before
any launch. CPU only: no call gets as far as a GPU."""
import ctypes

import pytest
import torch

import combine_moe_route_meta_gb300 as moe

P = ctypes.c_void_p
FAKE, ODD, TWO = P(0x1000), P(0x1008), P(0x1002)    # never dereferenced: validation fails first
INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED


def test_header_declares_what_the_library_exports():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "moe_block.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(moe_\w+)\s*\(", text))
    assert len(names) == 8
    lib = moe.load_library()
    for n in names:
        assert getattr(lib, n).argtypes is not None and hasattr(moe, n), n


def _gemm(op, **kw):
    a = dict(mode=1, a=FAKE, E=4, M=8, rows=0, n=64, k=128, seg=None, count=FAKE, weights=0, w=FAKE, out=FAKE, gu=FAKE,
             st=FAKE)
    a.update(kw)
    lib = moe.load_library()
    head = (a["mode"], a["a"], a["E"], a["M"], a["rows"], a["n"], a["k"], a["seg"], a["count"])
    if op == "plain":
        return lib.moe_expert_gemm_bf16(*head, a["weights"], a["w"], a["out"], a["st"], None)
    if op == "swiglu":
        return lib.moe_expert_gemm_swiglu_bf16(*head, a["w"], a["out"], a["gu"], a["st"], None)
    return lib.moe_expert_gemm_dswiglu_bf16(*head, a["w"], a["gu"], a["out"], a["st"], None)


@pytest.mark.parametrize("op", ["plain", "swiglu", "dswiglu"])
def test_product_arguments(op):
    for kw in (dict(mode=2), dict(E=0), dict(M=0), dict(n=0), dict(n=-8), dict(n=12), dict(k=0), dict(k=4), dict(k=100),
               dict(count=None), dict(st=None), dict(a=None), dict(w=None), dict(out=None), dict(a=ODD), dict(w=ODD),
               dict(out=ODD), dict(mode=0, rows=8), dict(mode=0, rows=-1, seg=FAKE), dict(seg=P(0x1004)), dict(count=TWO),
               dict(st=TWO)):
        assert _gemm(op, **kw) == INVALID, kw
    assert _gemm(op, E=1025) == UNSUPPORTED and _gemm(op, M=1 << 30) == UNSUPPORTED
    assert _gemm(op, mode=0, rows=1 << 31, seg=FAKE) == UNSUPPORTED
    assert _gemm(op, n=1 << 25) == UNSUPPORTED and _gemm(op, k=1 << 25) == UNSUPPORTED
    assert _gemm(op, mode=0, rows=(1 << 31) - 1, seg=FAKE, n=1 << 24) == UNSUPPORTED       # tiles beyond 31 bits
    assert _gemm(op, mode=0, rows=0, seg=FAKE) == 0
    if op == "plain":
        assert _gemm(op, weights=2) == INVALID
    elif op == "swiglu":
        assert _gemm(op, gu=ODD) == INVALID and _gemm(op, n=1 << 24) == UNSUPPORTED
    else:
        assert _gemm(op, gu=None) == INVALID and _gemm(op, gu=ODD) == INVALID


def _wgrad(**kw):
    a = dict(mode=1, a=FAKE, b=FAKE, E=4, M=8, rows=0, m=64, n=128, seg=None, count=FAKE, grad=1, acc=0, out=FAKE, st=FAKE)
    a.update(kw)
    return moe.load_library().moe_expert_wgrad_bf16(a["mode"], a["a"], a["b"], a["E"], a["M"], a["rows"], a["m"], a["n"],
                                                    a["seg"], a["count"], a["grad"], a["acc"], a["out"], a["st"], None)


def test_weight_gradient_arguments():
    for kw in (dict(mode=5), dict(E=0), dict(M=0), dict(m=0), dict(m=4), dict(n=0), dict(n=129), dict(count=None),
               dict(st=None), dict(a=None), dict(b=None), dict(out=None), dict(a=ODD), dict(b=ODD), dict(out=ODD),
               dict(grad=2), dict(acc=2), dict(mode=0, rows=4), dict(mode=0, rows=0, seg=FAKE, out=None), dict(st=TWO)):
        assert _wgrad(**kw) == INVALID, kw
    assert _wgrad(E=1025) == UNSUPPORTED and _wgrad(m=1 << 25) == UNSUPPORTED
    assert _wgrad(m=1 << 24, n=1 << 24) == UNSUPPORTED
    assert _wgrad(M=(1 << 26) + 1) == UNSUPPORTED and _wgrad(mode=0, seg=FAKE, rows=(1 << 26) + 1) == UNSUPPORTED


def _combine(**kw):
    a = dict(mode=0, g=FAKE, eo=FAKE, T=4, H=64, K=2, E=4, M=8, rows=0, ids=FAKE, s2d=FAKE, seg=FAKE, w=FAKE, ge=FAKE, gw=FAKE,
             st=FAKE)
    a.update(kw)
    return moe.load_library().moe_combine_backward(a["mode"], a["g"], a["eo"], a["T"], a["H"], a["K"], a["E"], a["M"],
                                                   a["rows"], a["ids"], a["s2d"], a["seg"], a["w"], a["ge"], a["gw"],
                                                   a["st"], None)


def test_combine_gradient_arguments():
    for kw in (dict(mode=3), dict(T=-1), dict(H=0), dict(H=12), dict(K=0), dict(E=0), dict(mode=1, M=0), dict(rows=7),
               dict(rows=-1), dict(st=None), dict(st=TWO), dict(ge=None, gw=None), dict(g=None), dict(eo=None), dict(s2d=None),
               dict(w=None), dict(mode=1, ids=None), dict(mode=1, seg=None), dict(g=ODD), dict(eo=ODD), dict(ge=ODD),
               dict(gw=TWO), dict(w=TWO), dict(s2d=TWO), dict(ids=TWO), dict(seg=P(0x1004))):
        assert _combine(**kw) == INVALID, kw
    assert _combine(K=17) == UNSUPPORTED and _combine(E=1025) == UNSUPPORTED and _combine(T=1 << 31) == UNSUPPORTED
    assert _combine(T=0) == 0 and _combine(T=0, g=None, eo=None, s2d=None, w=None) == 0


def _norm(**kw):
    a = dict(x=FAKE, res=FAKE, w=FAKE, eps=1e-6, T=4, H=256, q=1, out=FAKE, c=FAKE, s=FAKE, sum=FAKE, r=FAKE)
    a.update(kw)
    return moe.load_library().moe_rmsnorm(a["x"], a["res"], a["w"], a["eps"], a["T"], a["H"], a["q"], a["out"], a["c"], a["s"],
                                          a["sum"], a["r"], None)


def _norm_grad(**kw):
    a = dict(g=FAKE, s=FAKE, w=FAKE, r=FAKE, gs=None, T=4, H=256, gx=FAKE, gw=FAKE, ws=FAKE, n=1 << 30)
    a.update(kw)
    return moe.load_library().moe_rmsnorm_backward(a["g"], a["s"], a["w"], a["r"], a["gs"], a["T"], a["H"], a["gx"], a["gw"],
                                                   a["ws"], a["n"], None)


def test_norm_arguments():
    for kw in (dict(T=-1), dict(H=0), dict(H=12), dict(H=136), dict(q=2), dict(q=4), dict(q=9), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(w=None), dict(c=None), dict(s=None),
               dict(q=0, out=None), dict(x=ODD), dict(res=ODD), dict(w=ODD), dict(out=ODD), dict(c=ODD), dict(sum=ODD),
               dict(r=TWO), dict(s=TWO)):
        assert _norm(**kw) == INVALID, kw
    assert _norm(H=32896) == UNSUPPORTED and _norm(T=1 << 31) == UNSUPPORTED
    assert _norm(T=0) == 0


def test_norm_gradient_arguments():
    for kw in (dict(T=-1), dict(H=12), dict(g=None), dict(s=None), dict(w=None), dict(r=None), dict(gx=None), dict(gw=None),
               dict(ws=None), dict(n=moe.moe_rmsnorm_backward_workspace_size(4, 256) - 1), dict(g=ODD), dict(s=ODD), dict(w=ODD), dict(r=TWO), dict(gs=ODD),
               dict(gx=ODD), dict(gw=ODD), dict(ws=ODD)):
        assert _norm_grad(**kw) == INVALID, kw
    assert _norm_grad(H=32776) == UNSUPPORTED
    assert moe.moe_rmsnorm_backward_workspace_size(4, 12) == 0 and moe.moe_rmsnorm_backward_workspace_size(-1, 8) == 0
    assert moe.moe_rmsnorm_backward_workspace_size(0, 8) == 0
    assert moe.moe_rmsnorm_backward_workspace_size(4, 4096) >= 4096 * 4


def _operands():
    bf = dict(dtype=torch.bfloat16)
    return dict(a=torch.zeros((4, 8, 128), **bf), count=torch.zeros(4, dtype=torch.int32), w=torch.zeros((4, 64, 128), **bf),
                out=torch.zeros((4, 8, 64), **bf), st=torch.zeros(1, dtype=torch.int32), gu=torch.zeros((4, 8, 128), **bf))


def test_binding_checks_products():
    def plain(mode="masked", seg=None, M=8, transposed=False, **bad):
        o = _operands() | bad
        moe.moe_expert_gemm_bf16(mode, o["a"], o["count"], o["w"], o["out"], o["st"], transposed=transposed, seg_indptr=seg,
                                 max_tokens_per_expert=M)

    def swiglu(**bad):
        o = _operands() | dict(w=torch.zeros((4, 128, 128), dtype=torch.bfloat16)) | bad
        moe.moe_expert_gemm_swiglu_bf16("masked", o["a"], o["count"], o["w"], o["out"], o["st"], o["gu"],
                                        max_tokens_per_expert=8)

    def dswiglu(**bad):
        o = _operands() | dict(w=torch.zeros((4, 128, 64), dtype=torch.bfloat16),
                               out=torch.zeros((4, 8, 128), dtype=torch.bfloat16)) | bad
        moe.moe_expert_gemm_dswiglu_bf16("masked", o["a"], o["count"], o["w"], o["gu"], o["out"], o["st"],
                                         max_tokens_per_expert=8)

    o = _operands()
    for f in (plain, swiglu, dswiglu):
        for bad in (dict(a=o["a"][:3]), dict(a=o["a"].half()), dict(a=o["a"][..., :64]), dict(count=o["count"][1:]),
                    dict(count=o["count"].long()), dict(w=o["w"].float()), dict(out=o["out"][1:]), dict(out=o["out"].half()),
                    dict(st=o["st"].float())):
            with pytest.raises(ValueError):
                f(**bad)
        with pytest.raises(ValueError, match="no CPU path"):
            f()
    for bad in (dict(M=9), dict(mode="normal"), dict(mode="both"), dict(mode="normal", seg=torch.zeros(4, dtype=torch.int64)),
                dict(transposed=True)):
        with pytest.raises(ValueError):
            plain(**bad)
    for bad in (dict(gu=o["gu"][1:]), dict(w=torch.zeros((4, 127, 128), dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            swiglu(**bad)
    with pytest.raises(ValueError):
        dswiglu(gu=o["gu"][1:])


def test_binding_checks_weight_gradient():
    o = _operands()

    def call(**bad):
        v = o | dict(b=o["gu"], out=torch.zeros(4, 128, 128)) | bad
        moe.moe_expert_wgrad_bf16("masked", v["a"], v["b"], v["count"], v["out"], v["st"], max_tokens_per_expert=8)

    for bad in (dict(a=o["a"][:, :7]), dict(b=o["a"].float()), dict(b=o["out"]), dict(out=torch.zeros(4, 64, 128)),
                dict(out=torch.zeros(4, 128, 128).double()), dict(out=torch.zeros(5, 128, 128)), dict(st=o["st"].long())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError, match="no CPU path"):
        call()
    with pytest.raises(ValueError, match="rows"):
        moe.moe_expert_wgrad_bf16("normal", torch.zeros(8, 128).bfloat16(), torch.zeros(9, 128).bfloat16(), o["count"],
                                  torch.zeros(4, 128, 128), o["st"], seg_indptr=torch.zeros(5, dtype=torch.int64))


def test_binding_checks_combine_gradient():
    T, K, H, E = 3, 2, 64, 4
    good = dict(g=torch.zeros(T, H).bfloat16(), eo=torch.zeros(6, H).bfloat16(), ids=torch.zeros(T, K, dtype=torch.int32),
                w=torch.zeros(T, K), s2d=torch.zeros(6, dtype=torch.int32), seg=torch.zeros(E + 1, dtype=torch.int64),
                ge=torch.zeros(6, H).bfloat16(), gw=torch.zeros(T, K), st=torch.zeros(1, dtype=torch.int32))

    def call(mode="normal", rows=6, M=0, **bad):
        v = good | bad
        moe.moe_combine_backward(mode, v["g"], v["eo"], v["ids"], v["w"], E, v["s2d"], v["seg"], v["ge"], v["gw"], v["st"],
                                 max_tokens_per_expert=M, expert_out_rows=rows)

    for bad in (dict(g=good["g"][1:]), dict(g=good["g"].float()), dict(eo=good["eo"][1:]), dict(eo=None),
                dict(ids=good["ids"].long()), dict(w=good["w"][1:]), dict(s2d=good["s2d"][1:]), dict(ge=good["ge"][1:]),
                dict(gw=good["gw"].double()), dict(st=good["st"].float()), dict(mode="masked", M=2), dict(mode="x"),
                dict(mode="masked", M=1, seg=good["seg"][1:])):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError, match="no CPU path"):
        call()


def test_binding_checks_norm():
    T, H = 3, 256
    x, w = torch.zeros(T, H).bfloat16(), torch.zeros(H).bfloat16()
    for kw in (dict(x=x.float()), dict(w=w[1:]), dict(residual=x[1:]), dict(quant="fp4"), dict(quant="nvfp4b16")):
        a = dict(x=x, w=w) | kw
        with pytest.raises(ValueError):
            moe.rmsnorm(a.pop("x"), a.pop("w"), **a)
    codes, scales = torch.zeros(T, H, dtype=torch.uint8), torch.zeros(T, 2)
    for kw in (dict(codes=codes[1:]), dict(scales=scales[1:]), dict(scales=scales.double()), dict(sum=x[1:]),
               dict(rstd=torch.zeros(2)), dict(out=x[1:])):
        a = dict(codes=codes, scales=scales) | kw
        with pytest.raises(ValueError):
            moe.moe_rmsnorm(x, w, 1e-6, a.pop("out", None), quant="fp8g128", **a)
    with pytest.raises(ValueError, match="no CPU path"):
        moe.moe_rmsnorm(x, w, 1e-6, x)
    r, ws = torch.zeros(T), torch.zeros(1 << 16, dtype=torch.uint8)
    for kw in (dict(g=x[1:]), dict(s=x.half()), dict(w=w[1:]), dict(r=r[1:]), dict(gx=x[1:]), dict(gw=torch.zeros(H - 1)),
               dict(gs=x[1:])):
        a = dict(g=x, s=x, w=w, r=r, gx=x, gw=torch.zeros(H), gs=None) | kw
        with pytest.raises(ValueError):
            moe.moe_rmsnorm_backward(a["g"], a["s"], a["w"], a["r"], a["gx"], a["gw"], ws, a["gs"])
    with pytest.raises(ValueError, match="no CPU path"):
        moe.moe_rmsnorm_backward(x, x, w, r, x, torch.zeros(H), ws)


def test_masked_rows_of_another_stride():
    bf = dict(dtype=torch.bfloat16)
    count, st = torch.ones(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    a, w, out = torch.zeros(4, 9, 64, **bf), torch.zeros(4, 32, 64, **bf), torch.zeros(4, 9, 32, **bf)
    with pytest.raises(ValueError, match=r"a: \[E, 8, 64\] expected"):
        moe.moe_expert_gemm_bf16("masked", a, count, w, out, st, max_tokens_per_expert=8)
    with pytest.raises(ValueError, match=r"grad_out: \[E, 8, 64\] expected"):
        moe.moe_expert_gemm_dswiglu_bf16("masked", a, count, torch.zeros(4, 64, 32, **bf), torch.zeros(36, 64, **bf),
                                         torch.zeros(36, 64, **bf), st, max_tokens_per_expert=8)
    with pytest.raises(ValueError, match=r"b: \[E, 8, 32\] expected"):
        moe.moe_expert_wgrad_bf16("masked", torch.zeros(32, 64, **bf), out, count, torch.zeros(4, 64, 32), st,
                                  max_tokens_per_expert=8)


def test_layer_sizes():
    w13, w2 = torch.zeros(4, 64, 32, dtype=torch.bfloat16), torch.zeros(4, 32, 32, dtype=torch.bfloat16)
    for topk, tokens in ((2, 0), (0, 4), (2, -1)):
        with pytest.raises(ValueError, match="max_tokens and topk"):
            moe.BF16MoELayer(w13, w2, topk, tokens)


def test_longest_sums_of_a_weight_gradient():
    """2^26 rows are the most that are taken (the kernel's waits are bounded for two such sums: it asserts so as it is
    compiled)."""
    most = 1 << 26
    assert _wgrad(E=1, M=most, out=None) == INVALID and _wgrad(E=1, M=most + 1, out=None) == UNSUPPORTED
    assert _wgrad(mode=0, seg=FAKE, rows=most, out=None) == INVALID


class _OnDevice:
    """What the binding asks of a tensor, as one of a GPU's would answer."""

    def __init__(self, device, dtype=torch.bfloat16):
        self.device_index, self.dtype, self.nbytes, self.is_cuda = device, dtype, 64, True

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device_index

    def data_ptr(self):
        return 0x1000


def test_tensors_of_another_device(monkeypatch):
    """The block's operators refuse them; the NVFP4 experts' take them as they did before there was a block, by peer access."""
    from combine_moe_route_meta_gb300 import block, experts
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    mixed = [(_OnDevice(d), 64, f"t{d}", torch.bfloat16) for d in (0, 1)] + [(None, 0, "absent", torch.float32)]
    assert experts._pointers(*mixed) == [0x1000, 0x1000, None]
    assert experts._pointers(mixed[1]) == [0x1000]
    with pytest.raises(ValueError, match="t1: tensors of the current device"):
        block._pointers(*mixed)
    with pytest.raises(ValueError, match="t1: tensors of the current device"):
        block._pointers(mixed[1])
    assert block._pointers(mixed[0], mixed[2]) == [0x1000, None]


class _GpuTensor(torch.Tensor):
    """A host tensor that says it is one of GPU 1."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 1


@pytest.mark.parametrize("few", [0, 4])
def test_layer_refuses_before_its_first_launch(few, monkeypatch):
    from combine_moe_route_meta_gb300 import block

    def launched(*args, **kwargs):
        raise AssertionError("launched")

    for name in ("moe_route_meta_ex", "moe_layer_few_tokens"):
        monkeypatch.setattr(block, name, launched)
    gpu = 0
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: gpu, raising=False)
    w13, w2 = (torch.zeros(s, dtype=torch.bfloat16).as_subclass(_GpuTensor) for s in ((4, 64, 32), (4, 32, 32)))
    layer = block.BF16MoELayer(w13, w2, 2, 4, few_tokens=few)
    good = dict(x=torch.zeros(4, 32, dtype=torch.bfloat16), ids=torch.zeros(4, 2, dtype=torch.int32), w=torch.zeros(4, 2))
    good = {k: t.as_subclass(_GpuTensor) for k, t in good.items()}
    with pytest.raises(ValueError, match="x, .*: tensors of the current device"):
        layer(*good.values())
    gpu = 1
    for bad in (dict(x=good["x"].float()), dict(ids=good["ids"].long()), dict(w=good["w"].double()),
                dict(w=torch.zeros(2, 4).T.as_subclass(_GpuTensor)), dict(x=torch.zeros(4, 32, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            layer(*(good | bad).values())
    with pytest.raises(AssertionError, match="launched"):
        layer(*good.values())


def test_a_refused_backward_pass_can_be_made_again():
    w13, w2 = torch.zeros(4, 64, 32, dtype=torch.bfloat16), torch.zeros(4, 32, 32, dtype=torch.bfloat16)
    layer = moe.BF16MoELayer(w13, w2, 2, 4, train=True)
    layer.seen = (torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))   # as a forward pass leaves it
    for grad in (torch.zeros(3, 32, dtype=torch.bfloat16), torch.zeros(4, 32), torch.zeros(4, 32, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):                                      # shape, type, no GPU
            layer.backward(grad)
        assert layer.seen is not None


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_results_of_another_stride():
    """Outputs and kept values whose shape says another row length or another number of rows an expert than the kernels
    write: large enough, and every expert but the first would find its rows elsewhere."""
    count, st = torch.ones(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    seg, masked = torch.zeros(5, dtype=torch.int64), dict(max_tokens_per_expert=8)
    a, w, w13, w2 = _bf(4, 8, 64), _bf(4, 32, 64), _bf(4, 64, 64), _bf(4, 64, 32)
    for out in (_bf(4, 9, 32), _bf(4, 8, 64), _bf(32, 64)):
        with pytest.raises(ValueError, match="^out: "):
            moe.moe_expert_gemm_bf16("masked", a, count, w, out, st, **masked)
        with pytest.raises(ValueError, match="^h: "):
            moe.moe_expert_gemm_swiglu_bf16("masked", a, count, w13, out, st, **masked)
    for gu in (_bf(4, 9, 64), _bf(4, 16, 32), _bf(64, 32)):
        with pytest.raises(ValueError, match="^gate_up: "):
            moe.moe_expert_gemm_swiglu_bf16("masked", a, count, w13, _bf(4, 8, 32), st, gu, **masked)
        with pytest.raises(ValueError, match="^gate_up: "):
            moe.moe_expert_gemm_dswiglu_bf16("masked", a, count, w2, gu, _bf(4, 8, 64), st, **masked)
        with pytest.raises(ValueError, match="^grad_gate_up: "):
            moe.moe_expert_gemm_dswiglu_bf16("masked", a, count, w2, _bf(4, 8, 64), gu, st, **masked)
    with pytest.raises(ValueError, match="^out: "):
        moe.moe_expert_gemm_bf16("normal", a.view(32, 64), count, w, _bf(32, 40), st, seg_indptr=seg)
    with pytest.raises(ValueError, match="no CPU path"):     # in one dimension
        moe.moe_expert_gemm_bf16("masked", a, count, w, _bf(4 * 8 * 32), st, **masked)
    T, K, H = 3, 2, 64
    ids, s2d = torch.zeros(T, K, dtype=torch.int32), torch.zeros(T * K, dtype=torch.int32)

    def combine(mode, eo, ge, **kw):
        moe.moe_combine_backward(mode, _bf(T, H), eo, ids, torch.zeros(T, K), 4, s2d, seg, ge, torch.zeros(T, K), st, **kw)

    for bad in (_bf(4, 9, H), _bf(4, 8, 2 * H), _bf(32, 72)):
        with pytest.raises(ValueError, match="^expert_out: "):
            combine("masked", bad, _bf(4, 8, H), **masked)
        with pytest.raises(ValueError, match="^grad_expert_out: "):
            combine("masked", _bf(4, 8, H), bad, **masked)
    with pytest.raises(ValueError, match="^grad_expert_out: "):
        combine("normal", _bf(6, H), _bf(6, 72), expert_out_rows=6)


def test_norm_refuses_a_sum_that_it_would_not_write():
    x, w = _bf(3, 256), _bf(256)
    with pytest.raises(ValueError, match="^sum: "):
        moe.moe_rmsnorm(x, w, 1e-6, _bf(3, 256), sum=_bf(3, 256))
    with pytest.raises(ValueError, match="no CPU path"):
        moe.moe_rmsnorm(x, w, 1e-6, _bf(3, 256), residual=x, sum=_bf(3, 256))


def test_norm_refuses_codes_that_it_would_not_write():
    x, w, codes, scales = _bf(3, 256), _bf(256), torch.zeros(3, 256, dtype=torch.uint8), torch.zeros(3, 2)
    for kw in (dict(codes=codes, scales=scales), dict(codes=codes), dict(scales=scales)):
        with pytest.raises(ValueError, match="^codes, scales: "):
            moe.moe_rmsnorm(x, w, 1e-6, _bf(3, 256), **kw)


def test_which_scale_rows_the_dispatch_passes_through():
    """As the norm's documentation says: fp32 scale rows have hidden / 32 bytes, UE8M0 ones hidden / 128."""
    def passes(nbytes):
        return moe.load_library().moe_dispatch_ex(0, moe.MOE_QUANT_FP8_PASSTHROUGH, 0, FAKE, 0, nbytes, FAKE, 2, 4, 0, 0, FAKE,
                                                  FAKE, 0.0, FAKE, None, FAKE, None) == 0

    for hidden in (128, 512, 1024, 2048, 2176, 2560, 4096, 7168, 8192):
        assert passes(hidden)
        assert passes(hidden // 32) == (hidden % 1024 == 0) and passes(hidden // 128) == (hidden % 4096 == 0)
        for nbytes in (hidden // 32, hidden // 128):
            assert passes((nbytes + 31) // 32 * 32)


def test_norms_rows_of_another_length():
    x, w, wide = _bf(3, 256), _bf(256), _bf(3, 264)
    for kw in (dict(out=wide), dict(residual=wide), dict(residual=x, sum=wide)):
        with pytest.raises(ValueError, match=f"^{list(kw)[-1]}: rows of 256"):
            moe.moe_rmsnorm(x, w, 1e-6, **(dict(out=_bf(3, 256)) | kw))
    good = dict(codes=torch.zeros(3, 256, dtype=torch.uint8), scales=torch.zeros(3, 2))
    for bad in (dict(codes=torch.zeros(3, 384, dtype=torch.uint8)), dict(scales=torch.zeros(3, 3))):
        with pytest.raises(ValueError, match=f"^{list(bad)[0]}: rows of"):
            moe.moe_rmsnorm(x, w, 1e-6, quant="fp8g128", **(good | bad))
    with pytest.raises(ValueError, match="^residual: "):
        moe.rmsnorm(x, w, residual=wide)
    r, gw, ws = torch.zeros(3), torch.zeros(256), torch.zeros(1 << 16, dtype=torch.uint8)
    for name, a in (("grad_out", (wide, x, None)), ("grad_x", (x, wide, None)), ("grad_sum", (x, x, wide))):
        with pytest.raises(ValueError, match=f"^{name}: "):
            moe.moe_rmsnorm_backward(a[0], x, w, r, a[1], gw, ws, a[2])
    for name, a in (("grad_out", (wide, None)), ("grad_residual", (x, wide))):
        with pytest.raises(ValueError, match=f"^{name}: "):
            moe.rmsnorm_backward(a[0], x, w, r, a[1])
