"""moe_layer_few in Python refuses, before the library is called, tensors that
the kernels would read or write past the end of."""
import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M

T, D, NR, NS, I, K = 4, 256, 8, 1, 128, 2
E = NR + NS


class _NoStream:
    cuda_stream = 0


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def weights(wt):
    if wt in (M.MOE_F32, M.MOE_BF16):
        dt = torch.float32 if wt == M.MOE_F32 else torch.bfloat16
        return dict(w_t=wt, w13=torch.zeros(E, 2 * I, D, dtype=dt), w2=torch.zeros(E, D, I, dtype=dt))
    if wt == M.MOE_E4M3:
        return dict(w_t=wt, w13=u8(E, 2 * I, D), w2=u8(E, D, I), w13_scale=torch.zeros(E, 2 * I // 128, D // 128),
                    w2_scale=torch.zeros(E, D // 128, I // 128))
    return dict(w_t=wt, w13=u8(E, 2 * I, D // 2), w2=u8(E, D, I // 2), w13_scale=u8(E, 2 * I, D // 32),
                w2_scale=u8(E, D, I // 32))


def args(wt=M.MOE_BF16, **kw):
    act = torch.float32 if wt == M.MOE_F32 else torch.bfloat16
    a = dict(u=torch.zeros(T, D, dtype=act), centroids=torch.zeros(NR, D), bias=torch.zeros(NR),
             w=M.ExpertWeights(**weights(wt)), Ns=NS, I=I, K=K, resid=torch.zeros(T, D, dtype=act),
             topk_idx=torch.zeros(T, K, dtype=torch.int32), topk_gate=torch.zeros(T, K), topk_score=torch.zeros(T, K),
             expert_load=torch.zeros(NR, dtype=torch.int32), ws=u8(1 << 20), out=torch.zeros(T, D, dtype=act),
             stream=_NoStream())
    assert set(kw) <= set(a)
    return a | kw


@pytest.fixture
def calls(monkeypatch):
    """The arguments of each call that reaches the library, which answers MOE_OK."""
    seen = []

    class Lib:
        def moe_layer_few(self, *a):
            seen.append(a)
            return M.MOE_OK

    monkeypatch.setattr(M, "lib", Lib)
    return seen


@pytest.mark.parametrize("wt", [M.MOE_F32, M.MOE_BF16, M.MOE_E4M3, M.MOE_E2M1])
def test_right_shapes_reach_the_library(calls, wt):
    M.moe_layer_few(**args(wt))
    M.moe_layer_few(**args(wt, resid=None, topk_score=None, expert_load=None))
    more = dict(topk_idx=torch.zeros(T + 3, K, dtype=torch.int32), topk_gate=torch.zeros(T + 3, K),
                topk_score=torch.zeros(T + 3, K))                      # outputs of a layer that holds more tokens
    M.moe_layer_few(**args(wt, **more))
    assert len(calls) == 3


@pytest.mark.parametrize("kw", [dict(out=torch.zeros(T - 1, D)), dict(out=torch.zeros(T, D - 8)),
                                dict(resid=torch.zeros(T - 1, D)), dict(resid=torch.zeros(T, D + 8)),
                                dict(centroids=torch.zeros(NR, D - 8)), dict(centroids=torch.zeros(NR, D).bfloat16()),
                                dict(centroids=torch.zeros(NR + 1, D)), dict(bias=torch.zeros(NR - 1)),
                                dict(bias=torch.zeros(NR).double()), dict(K=3), dict(Ns=2), dict(I=256), dict(I=120),
                                dict(topk_idx=torch.zeros(T - 1, K, dtype=torch.int32)),
                                dict(topk_idx=torch.zeros(T, K)), dict(topk_idx=torch.zeros(T * K, dtype=torch.int32)),
                                dict(topk_gate=torch.zeros(T - 1, K)), dict(topk_gate=torch.zeros(T, K).bfloat16()),
                                dict(topk_gate=torch.zeros(T, K - 1)), dict(topk_score=torch.zeros(T - 1, K)),
                                dict(topk_score=torch.zeros(T, K).half()),
                                dict(expert_load=torch.zeros(NR - 1, dtype=torch.int32)),
                                dict(expert_load=torch.zeros(NR, dtype=torch.int16))])
def test_wrong_shapes_are_refused(calls, kw):
    with pytest.raises(ValueError):
        M.moe_layer_few(**args(**kw))
    assert not calls


@pytest.mark.parametrize("wt", [M.MOE_F32, M.MOE_BF16, M.MOE_E4M3, M.MOE_E2M1])
def test_wrong_weights_are_refused(calls, wt):
    for name, t in weights(wt).items():
        if name == "w_t":
            continue
        for bad in (t[:-1], t[..., :-1].contiguous(), t[:, :-1].contiguous(), t.double()) + \
                   (() if "scale" not in name else (None,)):
            with pytest.raises(ValueError):
                M.moe_layer_few(**args(wt, w=M.ExpertWeights(**(weights(wt) | {name: bad}))))
    with pytest.raises(ValueError):
        M.moe_layer_few(**args(wt, w=M.ExpertWeights(**(weights(wt) | dict(w_t=4)))))
    assert not calls
