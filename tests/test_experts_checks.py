"""The expert operators refuse bad arguments on the host: the C entry points by their status, the binding
before any launch. CPU only: no call gets as far as a GPU."""
import ctypes

import pytest
import torch

import combine_moe_route_meta_gb300 as moe

P = ctypes.c_void_p
FAKE = P(0x1000)                     # never dereferenced: validation fails first
ODD = P(0x1008)
INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED


def _quant(fn, **kw):
    a = dict(x=FAKE, G=1, R=4, H=64, gs=FAKE, layout=2, q=FAKE, s=FAKE)
    a.update(kw)
    lib = moe.load_library()
    if fn == "quantize":
        return lib.moe_quantize_nvfp4(a["x"], a["G"], a["R"], a["H"], a["gs"], a["layout"], a["q"], a["s"], None)
    return lib.moe_dequantize_nvfp4(a["q"], a["s"], a["G"], a["R"], a["H"], a["gs"], a["layout"], a["x"], None)


@pytest.mark.parametrize("fn", ["quantize", "dequantize"])
def test_quantise_arguments(fn):
    for kw in (dict(G=-1), dict(R=-1), dict(H=0), dict(H=24), dict(H=80), dict(layout=1), dict(layout=7), dict(x=None),
               dict(gs=None), dict(q=None), dict(s=None), dict(x=ODD), dict(s=P(0x1002)), dict(gs=P(0x1002)),
               dict(q=P(0x1004))):
        assert _quant(fn, **kw) == INVALID, kw
    assert _quant(fn, H=80, layout=0, x=None) == INVALID          # H % 16 is enough for rows: only x is wrong
    assert _quant(fn, R=1 << 31) == UNSUPPORTED
    assert _quant(fn, G=1 << 30, R=1 << 20) == UNSUPPORTED
    assert _quant(fn, G=0) == 0 and _quant(fn, R=0) == 0


def _gemm(swiglu=False, **kw):
    a = dict(mode=1, a=FAKE, sf=FAKE, layout=2, E=4, M=8, rows=0, n=64, k=128, seg=None, count=FAKE, w=FAKE, wsf=FAKE,
             alpha=None, out=FAKE, osf=FAKE, st=FAKE)
    a.update(kw)
    lib = moe.load_library()
    head = (a["mode"], a["a"], a["sf"], a["layout"], a["E"], a["M"], a["rows"], a["n"], a["k"], a["seg"], a["count"],
            a["w"], a["wsf"], a["alpha"])
    if swiglu:
        return lib.moe_expert_gemm_swiglu(*head, 1.0, a["out"], a["osf"], a["st"], None)
    return lib.moe_expert_gemm(*head, a["out"], a["st"], None)


@pytest.mark.parametrize("swiglu", [False, True])
def test_product_arguments(swiglu):
    for kw in (dict(mode=2), dict(layout=1), dict(layout=5), dict(E=0), dict(M=0), dict(n=0), dict(n=72), dict(k=0),
               dict(k=32), dict(k=96), dict(count=None), dict(st=None), dict(a=None), dict(sf=None), dict(w=None),
               dict(wsf=None), dict(out=None), dict(a=ODD), dict(w=ODD), dict(wsf=ODD), dict(out=ODD),
               dict(sf=P(0x1002)), dict(mode=0, rows=8), dict(mode=0, rows=-1, seg=FAKE), dict(alpha=P(0x1002)),
               dict(seg=P(0x1004)), dict(count=P(0x1002)), dict(st=P(0x1002))):
        assert _gemm(swiglu, **kw) == INVALID, kw
    assert _gemm(swiglu, E=1025) == UNSUPPORTED
    assert _gemm(swiglu, M=1 << 30) == UNSUPPORTED
    assert _gemm(swiglu, mode=0, rows=1 << 31, seg=FAKE) == UNSUPPORTED
    assert _gemm(swiglu, n=1 << 25) == UNSUPPORTED and _gemm(swiglu, k=1 << 25) == UNSUPPORTED
    assert _gemm(swiglu, mode=0, rows=0, seg=FAKE) == 0
    if swiglu:
        assert _gemm(True, n=80) == INVALID and _gemm(True, osf=None) == INVALID and _gemm(True, osf=P(0x1002)) == INVALID


def _layer(**kw):
    a = dict(x=FAKE, T=4, H=128, I=64, ids=FAKE, w=FAKE, K=2, E=8, q=2, w13=FAKE, s13=FAKE, a13=None, w2=FAKE, s2=FAKE,
             a2=None, out=FAKE, ws=FAKE, n=1 << 30, st=FAKE)
    a.update(kw)
    return moe.load_library().moe_layer_few_tokens(
        a["x"], a["T"], a["H"], a["I"], a["ids"], a["w"], a["K"], a["E"], a["q"], a["w13"], a["s13"], a["a13"], a["w2"],
        a["s2"], a["a2"], a["out"], a["ws"], a["n"], a["st"], None)


def test_layer_arguments():
    for kw in (dict(T=-1), dict(H=0), dict(H=72), dict(H=80), dict(I=0), dict(I=72), dict(I=80), dict(K=0), dict(E=0),
               dict(q=1), dict(q=9), dict(x=None), dict(ids=None), dict(w=None), dict(w13=None), dict(w2=None),
               dict(s13=None), dict(s2=None), dict(out=None), dict(ws=None), dict(n=0), dict(st=None), dict(x=ODD),
               dict(w13=ODD), dict(w2=ODD), dict(s13=ODD), dict(s2=ODD), dict(out=ODD), dict(ws=P(0x1010)),
               dict(ids=P(0x1002)), dict(w=P(0x1002)), dict(a13=P(0x1002)), dict(a2=P(0x1002)), dict(st=P(0x1002)),
               dict(q=0, H=72), dict(q=0, I=8)):
        assert _layer(**kw) == INVALID, kw
    assert _layer(T=65) == UNSUPPORTED and _layer(K=17) == UNSUPPORTED and _layer(E=1025) == UNSUPPORTED
    assert _layer(T=0) == 0
    assert moe.moe_layer_workspace_size(65, 8, 128, 64, 8) == 0
    assert moe.moe_layer_workspace_size(4, 8, 100, 64, 8) == 0
    assert moe.moe_layer_workspace_size(4, 8, 128, 64, 8) > 0


def test_binding_checks_quantise():
    x, g = torch.zeros((2, 5, 128), dtype=torch.bfloat16), torch.ones(2)
    q, s = torch.zeros((2, 5, 64), dtype=torch.uint8), torch.zeros(2 * 128 * 8, dtype=torch.uint8)
    for bad in (dict(x=x.float()), dict(g=g[:1]), dict(g=g.double()), dict(q=q[:1]), dict(s=s[1:])):
        a = dict(x=x, g=g, q=q, s=s) | bad
        with pytest.raises(ValueError, match="needed|expected"):
            moe.moe_quantize_nvfp4(a["x"], a["g"], a["q"], a["s"])
        with pytest.raises(ValueError, match="needed|expected"):
            moe.moe_dequantize_nvfp4(a["q"], a["s"], a["g"], a["x"])
    with pytest.raises(ValueError, match="scale_layout"):
        moe.moe_quantize_nvfp4(x, g, q, s, "tiled")
    with pytest.raises(ValueError, match="no CPU path"):
        moe.moe_quantize_nvfp4(x, g, q, s)


def _operands():
    E, M, n, k = 4, 8, 64, 128
    return dict(a=torch.zeros((E, M, k // 2), dtype=torch.uint8), sf=torch.zeros(128 * 8, dtype=torch.uint8),
                count=torch.zeros(E, dtype=torch.int32), w=torch.zeros((E, n, k // 2), dtype=torch.uint8),
                wsf=torch.zeros(E * 128 * 8, dtype=torch.uint8), out=torch.zeros((E, M, n), dtype=torch.bfloat16),
                st=torch.zeros(1, dtype=torch.int32), alpha=torch.ones(E))


def test_binding_checks_product():
    def call(mode="masked", layout="swizzled", seg=None, M=8, **bad):
        o = _operands() | bad
        moe.moe_expert_gemm(mode, o["a"], o["sf"], o["count"], o["w"], o["wsf"], o["out"], o["st"], alpha=o["alpha"],
                            seg_indptr=seg, max_tokens_per_expert=M, scale_layout=layout)
    o = _operands()
    for bad in (dict(a=o["a"][:3]), dict(sf=o["sf"][1:]), dict(count=o["count"][1:]), dict(count=o["count"].long()),
                dict(w=o["w"].float()), dict(wsf=o["wsf"][1:]), dict(out=o["out"][1:]), dict(out=o["out"].half()),
                dict(alpha=o["alpha"][1:]), dict(st=o["st"].float()), dict(M=9), dict(mode="normal"),
                dict(mode="normal", seg=torch.zeros(4, dtype=torch.int64)), dict(layout="x"), dict(mode="both"),
                dict(a=torch.zeros((4, 16, 32), dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError, match="no CPU path"):
        call()


def test_binding_checks_swiglu():
    def call(**bad):
        o = _operands() | dict(out=torch.zeros((4, 8, 32), dtype=torch.uint8), osf=torch.zeros(128 * 4, dtype=torch.uint8),
                               w=torch.zeros((4, 128, 64), dtype=torch.uint8),
                               wsf=torch.zeros(8 * 128 * 8, dtype=torch.uint8)) | bad
        moe.moe_expert_gemm_swiglu("masked", o["a"], o["sf"], o["count"], o["w"], o["wsf"], o["out"], o["osf"], o["st"],
                                   1.0, alpha=o["alpha"], max_tokens_per_expert=8)
    o = _operands()
    for bad in (dict(out=torch.zeros((4, 8, 31), dtype=torch.uint8)), dict(osf=o["sf"][:511]), dict(wsf=o["wsf"]),
                dict(w=torch.zeros((4, 127, 64), dtype=torch.uint8))):
        with pytest.raises(ValueError, match="needed|fit"):
            call(**bad)
    with pytest.raises(ValueError, match="no CPU path"):
        call()


def test_binding_checks_layer():
    T, H, I, E, K = 3, 128, 64, 4, 2
    good = dict(x=torch.zeros((T, H), dtype=torch.bfloat16), ids=torch.zeros((T, K), dtype=torch.int32),
                w=torch.zeros((T, K)), w13=torch.zeros((E, 2 * I, H // 2), dtype=torch.uint8),
                w2=torch.zeros((E, H, I // 2), dtype=torch.uint8), out=torch.zeros((T, H), dtype=torch.bfloat16),
                st=torch.zeros(1, dtype=torch.int32), s13=torch.zeros(2 * E * 128 * 8, dtype=torch.uint8),
                s2=torch.zeros(E * 128 * 4, dtype=torch.uint8))

    def call(**bad):
        o = good | bad
        moe.moe_layer_few_tokens(o["x"], o["ids"], o["w"], o["w13"], o["w2"], o["out"], None, o["st"], o["s13"], o["s2"])
    for bad in (dict(x=good["x"].float()), dict(ids=good["ids"].long()), dict(w=good["w"][:2]), dict(w13=good["w13"][:, 1:]),
                dict(w2=good["w2"][1:]), dict(w2=good["w2"].bfloat16()), dict(out=good["out"][1:]), dict(s13=None),
                dict(s13=good["s13"][1:]), dict(s2=good["s2"][1:]), dict(st=good["st"].float())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError, match="no CPU path"):
        call()
