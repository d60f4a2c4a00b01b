"""moe_rmsnorm and its backward refuse bad arguments on the host, before any
launch, in C and in the Python binding.  No call here reaches a kernel."""
import ctypes

import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M

F = ctypes.c_void_p(0x1000)      # never dereferenced
ODD = ctypes.c_void_p(0x1008)    # not 16-byte aligned
F32, BF16, E4M3 = M.MOE_F32, M.MOE_BF16, M.MOE_E4M3


def fwd(**kw):
    a = dict(x=F, xt=BF16, r=F, rt=BF16, w=F, wt=F32, eps=1e-6, T=4, d=256, ro=F, u=F, ut=BF16, q=F, qs=F, rstd=F,
             st=None)
    assert set(kw) <= set(a)
    return M.lib().moe_rmsnorm(*{**a, **kw}.values())


def bwd(**kw):
    a = dict(du=F, dut=BF16, r=F, rt=F32, w=F, wt=BF16, rstd=F, dr=F, T=4, d=256, dx=F, dw=F, ws=F, wsb=1 << 30,
             st=None)
    assert set(kw) <= set(a)
    return M.lib().moe_rmsnorm_backward(*{**a, **kw}.values())


@pytest.mark.parametrize("kw", [dict(x=None), dict(w=None), dict(xt=E4M3), dict(rt=E4M3), dict(wt=E4M3), dict(wt=7),
                                dict(ut=E4M3), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                                dict(T=-1), dict(d=0), dict(d=12), dict(d=264), dict(q=None), dict(qs=None),
                                dict(u=None, q=None, qs=None), dict(x=ODD), dict(r=ODD), dict(w=ODD), dict(ro=ODD),
                                dict(u=ODD), dict(q=ODD)])
def test_forward_refuses(kw):
    assert fwd(**kw) == M.MOE_EINVAL
    assert b"rmsnorm" in M.lib().moe_last_error()


@pytest.mark.parametrize("kw", [dict(du=None), dict(r=None), dict(w=None), dict(rstd=None), dict(dx=None),
                                dict(dw=None), dict(dw=None, T=0), dict(dut=E4M3), dict(rt=E4M3), dict(wt=E4M3),
                                dict(T=-1), dict(d=12), dict(d=0), dict(du=ODD), dict(dr=ODD), dict(dx=ODD),
                                dict(ws=ODD)])
def test_backward_refuses(kw):
    assert bwd(**kw) == M.MOE_EINVAL


def test_limits_and_workspace():
    L = M.lib()
    assert fwd(d=M.MOE_NORM_MAX_D + 128) == M.MOE_EUNSUPPORTED
    assert bwd(d=M.MOE_NORM_MAX_D + 8) == M.MOE_EUNSUPPORTED
    need = L.moe_rmsnorm_backward_workspace_bytes(4, 256)
    assert need >= 256 * 4
    assert bwd(wsb=need - 1) == M.MOE_EWORKSPACE
    assert bwd(ws=None) == M.MOE_EWORKSPACE
    for T, d in ((0, 256), (-3, 256), (4, 12), (4, 0), (4, M.MOE_NORM_MAX_D + 8)):
        assert L.moe_rmsnorm_backward_workspace_bytes(T, d) == 0
    assert fwd(T=0) == M.MOE_OK and fwd(T=0, x=None, u=F) == M.MOE_OK      # nothing to do, nothing launched


def test_binding_refuses_shapes():
    x, w = torch.zeros(4, 256), torch.zeros(256)
    u = torch.zeros(4, 256)
    bad = [dict(weight=w[:128]), dict(u=u[:3]), dict(residual=x[:2]), dict(r_out=x[:, :128].contiguous()),
           dict(residual=x, r_out=x.bfloat16()), dict(rstd=torch.zeros(3)), dict(rstd=torch.zeros(4).double()),
           dict(q=torch.zeros(4, 256), q_scale=torch.zeros(4, 2)),
           dict(q=torch.zeros(4, 256, dtype=torch.uint8), q_scale=torch.zeros(4, 3)),
           dict(u=torch.zeros(256, 4).t()), dict(x=x.double())]
    for kw in bad:
        a = dict(x=x, weight=w, eps=1e-6, u=u, stream=_NoStream()) | kw
        with pytest.raises(ValueError):
            M.moe_rmsnorm(**a)
    ok = dict(du=x, r=x, weight=w, rstd=torch.zeros(4), dr=None, dx=x.clone(), dw=torch.zeros(256),
              ws=torch.zeros(1 << 16), stream=_NoStream())
    for kw in (dict(du=x[:3]), dict(dr=x.bfloat16()), dict(dx=x.bfloat16()), dict(rstd=torch.zeros(5)),
               dict(dw=torch.zeros(128)), dict(dw=torch.zeros(256).bfloat16()), dict(weight=w[:8])):
        with pytest.raises(ValueError):
            M.moe_rmsnorm_backward(**(ok | kw))


class _NoStream:
    cuda_stream = 0
