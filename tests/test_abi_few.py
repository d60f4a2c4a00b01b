"""The 4-bit calls and moe_layer_few refuse bad arguments on the host, before
any launch, in C and in the Python binding.  No call here reaches a kernel."""
import ctypes

import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M

F = ctypes.c_void_p(0x1000)      # never dereferenced
ODD = ctypes.c_void_p(0x1008)    # not 16-byte aligned
F32, BF16, E4M3, E2M1 = M.MOE_F32, M.MOE_BF16, M.MOE_E4M3, M.MOE_E2M1


def call(fn, base, kw):
    assert set(kw) <= set(base)
    return fn(*{**base, **kw}.values())


def quant(**kw):
    return call(M.lib().fp4_quantize_groups, dict(x=F, t=BF16, rows=4, cols=64, q=F, s=F, st=None), kw)


def dequant(**kw):
    return call(M.lib().fp4_dequantize_groups, dict(q=F, s=F, rows=4, cols=64, out=F, t=F32, st=None), kw)


def matvec(**kw):
    return call(M.lib().fp4_matvec, dict(x=F, xt=BF16, q=F, s=F, T=3, N=40, K=64, y=F, yt=F32, ws=F, wsb=1 << 40,
                                         st=None), kw)


def few(**kw):
    return call(M.lib().moe_layer_few, dict(u=F, ut=BF16, e=F, b=F, wt=BF16, w13=F, s13=F, w2=F, s2=F, T=4, d=256,
                                            Nr=16, Ns=1, I=128, K=4, res=F, rt=BF16, idx=F, gate=F, score=F, load=F,
                                            ws=F, wsb=1 << 40, out=F, ot=BF16, st=None), kw)


@pytest.mark.parametrize("kw", [dict(x=None), dict(q=None), dict(s=None), dict(t=E4M3), dict(t=E2M1), dict(cols=48),
                                dict(cols=-32), dict(rows=-1), dict(x=ODD), dict(q=ODD), dict(rows=1 << 40, cols=64)])
def test_quantize_refuses(kw):
    assert quant(**kw) == M.MOE_EINVAL


@pytest.mark.parametrize("kw", [dict(out=None), dict(q=None), dict(s=None), dict(t=E4M3), dict(cols=48),
                                dict(rows=-1), dict(out=ODD), dict(q=ODD)])
def test_dequantize_refuses(kw):
    assert dequant(**kw) == M.MOE_EINVAL


@pytest.mark.parametrize("kw", [dict(x=None), dict(q=None), dict(s=None), dict(y=None), dict(xt=E4M3), dict(yt=E2M1),
                                dict(T=-1), dict(N=-1), dict(K=0), dict(K=48), dict(x=ODD), dict(q=ODD)])
def test_matvec_refuses(kw):
    assert matvec(**kw) == M.MOE_EINVAL


def test_matvec_limits():
    assert matvec(xt=F32) == M.MOE_EUNSUPPORTED
    assert matvec(K=(1 << 20) + 32) == M.MOE_EUNSUPPORTED
    assert matvec(T=16 * 65535 + 1) == M.MOE_EUNSUPPORTED
    assert matvec(N=(1 << 34) + 1) == M.MOE_EUNSUPPORTED
    assert matvec(N=(1 << 27) + 1) == M.MOE_EUNSUPPORTED
    need = M.fp4_matvec_workspace_bytes(3, 40, 64)
    assert need == 0 or matvec(wsb=need - 1) == M.MOE_EWORKSPACE
    assert matvec(T=0, x=None, y=None) == M.MOE_OK and matvec(N=0, y=None) == M.MOE_OK
    assert quant(rows=0, x=None) == M.MOE_OK and dequant(cols=0, q=None) == M.MOE_OK


@pytest.mark.parametrize("kw", [dict(u=None), dict(e=None), dict(b=None), dict(w13=None), dict(w2=None),
                                dict(idx=None), dict(gate=None), dict(out=None), dict(ut=E4M3), dict(wt=4),
                                dict(ot=E4M3), dict(rt=E2M1), dict(T=-1), dict(d=0), dict(d=260), dict(I=132),
                                dict(I=0), dict(Nr=0), dict(Nr=1025), dict(Ns=-1), dict(Nr=1000, Ns=25), dict(K=0),
                                dict(K=17, Nr=32), dict(K=5, Nr=4), dict(wt=E4M3, s13=None), dict(wt=E4M3, s2=None),
                                dict(wt=E2M1, s13=None), dict(wt=E2M1, s2=None), dict(u=ODD), dict(e=ODD),
                                dict(w13=ODD), dict(w2=ODD), dict(res=ODD), dict(ws=ODD), dict(out=ODD)])
def test_few_refuses(kw):
    assert few(**kw) == M.MOE_EINVAL
    assert b"layer_few" in M.lib().moe_last_error()


@pytest.mark.parametrize("kw", [dict(T=33), dict(ut=F32), dict(wt=F32), dict(ut=F32, wt=E4M3),
                                dict(wt=E4M3, d=264), dict(wt=E4M3, I=192), dict(wt=E2M1, d=264),
                                dict(wt=E2M1, I=136), dict(d=1 << 17, I=1 << 13), dict(d=1 << 24)])
def test_few_does_not_support(kw):
    assert few(**kw) == M.MOE_EUNSUPPORTED


@pytest.mark.parametrize("kw", [dict(T=32, I=1 << 18, Nr=1024, Ns=0, K=16),
                                dict(T=32, d=1 << 18, I=128, Nr=1024, Ns=0, K=16)])
def test_few_refuses_more_blocks_than_a_launch_holds(kw):
    assert few(wsb=1 << 60, **kw) == M.MOE_EUNSUPPORTED


def test_few_workspace():
    need = M.moe_layer_few_workspace_bytes(4, 256, 16, 1, 128, 4, BF16)
    assert need > 0
    assert few(wsb=need - 1) == M.MOE_EWORKSPACE and few(ws=None) == M.MOE_EWORKSPACE
    assert M.moe_layer_few_workspace_bytes(4, 256, 16, 1, 128, 4, F32) > need      # h in fp32
    for bad in ((33, 256, 16, 1, 128, 4), (-1, 256, 16, 1, 128, 4), (4, 260, 16, 1, 128, 4), (4, 256, 16, 1, 0, 4),
                (4, 256, 0, 1, 128, 1), (4, 256, 3, 1, 128, 4), (4, 256, 16, -1, 128, 4)):
        assert M.moe_layer_few_workspace_bytes(*bad, BF16) == 0
    assert few(T=0, load=None, u=None, out=None) == M.MOE_OK


def test_other_calls_refuse_4_bit_weights():
    a = [F, BF16, None, E2M1, F, F, F, F, 64, 4, 16, 1, 256, 128, 32, F, F, F, F, F, 1 << 40, F, BF16, None]
    assert M.lib().moe_expert_gemm(*a) == M.MOE_EINVAL


class _NoStream:
    cuda_stream = 0


def test_binding_refuses_shapes():
    st = _NoStream()
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    x = torch.zeros(4, 64)
    for kw in (dict(q=u8(4, 31), scale=u8(4, 2)), dict(q=u8(4, 32), scale=u8(4, 3)),
               dict(q=torch.zeros(4, 32), scale=u8(4, 2)), dict(q=u8(3, 32), scale=u8(4, 2))):
        with pytest.raises(ValueError):
            M.fp4_quantize_groups(x, **kw, stream=st)
        with pytest.raises(ValueError):
            M.fp4_dequantize_groups(**kw, out=x, stream=st)
    xb = x.bfloat16()
    ok = dict(x=xb, q=u8(10, 32), scale=u8(10, 2), y=torch.zeros(4, 10))
    for kw in (dict(q=u8(10, 16)), dict(scale=u8(9, 2)), dict(y=torch.zeros(4, 11)), dict(y=torch.zeros(3, 10)),
               dict(x=torch.zeros(64, 4).bfloat16().t()), dict(y=torch.zeros(10, 4).t())):
        with pytest.raises(ValueError):
            M.fp4_matvec(**(ok | kw), stream=st)


def test_layer_refuses_shapes():
    T, d, Nr, Ns, I, K = 4, 256, 8, 1, 128, 2
    w13, w2 = torch.zeros(9, 256, 256).bfloat16(), torch.zeros(9, 256, 128).bfloat16()
    mk = lambda **kw: M.FewTokenLayer(T, d, Nr, Ns, I, K, torch.bfloat16,  # noqa: E731
                                      M.ExpertWeights(**(dict(w_t=BF16, w13=w13, w2=w2) | kw)), device="cpu")
    for kw in (dict(w13=w13[:8]), dict(w2=w2[:, :, :64].contiguous()), dict(w_t=F32), dict(w_t=E2M1),
               dict(w_t=E4M3, w13=w13.to(torch.uint8), w2=w2.to(torch.uint8))):
        with pytest.raises(ValueError):
            mk(**kw)
    with pytest.raises(ValueError):
        M.FewTokenLayer(33, d, Nr, Ns, I, K, torch.bfloat16, M.ExpertWeights(BF16, w13, w2), device="cpu")
    layer = mk()
    u, e, b = torch.zeros(4, 256).bfloat16(), torch.zeros(8, 256), torch.zeros(8)
    for kw in (dict(u=torch.zeros(5, 256).bfloat16()), dict(u=u.float()), dict(u=u[:, :128].contiguous()),
               dict(centroids=e[:7]), dict(bias=b[:7]), dict(residual=u[:3]), dict(flags=2)):
        with pytest.raises(ValueError):
            layer.forward(**(dict(u=u, centroids=e, bias=b, stream=_NoStream()) | kw))
