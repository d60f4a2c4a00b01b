"""FewTokenLayer.update_bias: the mean load is that of the tokens that the
last forward() had, unless told otherwise."""
import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M


class _NoStream:
    cuda_stream = 0


@pytest.fixture
def layer(monkeypatch):
    """A layer of 8 tokens whose library calls are recorded, not run: totals of the bias steps in order."""
    T, d, Nr, Ns, I, K = 8, 64, 16, 0, 32, 4
    w = M.ExpertWeights(M.MOE_F32, torch.zeros(Nr, 2 * I, d), torch.zeros(Nr, d, I))
    layer = M.FewTokenLayer(T, d, Nr, Ns, I, K, torch.float32, w, device="cpu")
    layer.totals = []
    monkeypatch.setattr(M, "_layer_few", lambda *a: None)
    monkeypatch.setattr(M, "moe_bias_update", lambda load, total, gamma, bias, stream: layer.totals.append(total))
    layer.step = lambda n: layer.forward(torch.zeros(n, d), torch.zeros(Nr, d), torch.zeros(Nr), stream=_NoStream())
    return layer


def test_default_is_the_last_forwards_tokens(layer):
    b = torch.zeros(16)
    for n in (6, 8, 1, 0, 5):
        layer.step(n)
        layer.update_bias(b)
        layer.update_bias(b)
    assert layer.totals == [n * 4 for n in (6, 6, 8, 8, 1, 1, 0, 0, 5, 5)]
    layer.update_bias(b, tokens=3)
    assert layer.totals[-1] == 12


def test_a_refused_forward_changes_nothing(layer):
    layer.step(6)
    with pytest.raises(ValueError):
        layer.step(9)
    layer.update_bias(torch.zeros(16))
    assert layer.totals == [24]


def test_before_any_forward_all_tokens(layer):
    layer.update_bias(torch.zeros(16))
    assert layer.totals == [32]


@pytest.mark.gpu
@pytest.mark.parametrize("n", [8, 6, 1])
def test_bias_after_fewer_tokens_against_the_oracle(n):
    import workloads as W
    from moe_testutil import np_of
    from oracle import moe as O

    T, d, Nr, I, K = 8, 64, 16, 32, 4
    w = M.ExpertWeights(M.MOE_F32, W.make_free((Nr, 2 * I, d), d ** -0.5, 1, "cuda"),
                        W.make_free((Nr, d, I), d ** -0.5, 2, "cuda"))
    layer = M.FewTokenLayer(T, d, Nr, 0, I, K, torch.float32, w)
    u, e, b = W.make_free((T, d), 1.0, 3, "cuda"), W.make_free((Nr, d), d ** -0.5, 4, "cuda"), torch.zeros(Nr, device="cuda")
    layer.forward(u, e, b)
    layer.forward(u[:n], e, b)
    want = O.bias_update(np_of(b), np_of(layer.expert_load), n, K)
    layer.update_bias(b)
    assert (np_of(b).view("uint32") == want.view("uint32")).all()
