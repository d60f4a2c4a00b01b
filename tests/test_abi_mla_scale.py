"""A scale whose product with log2(e) leaves fp32 would turn scores of zero
into NaN: it is refused; those below are taken."""
import pytest

import sparse_expert_routing_sigmoid_amd as M
from test_abi_mla import attention, backward, decode, refused


@pytest.mark.parametrize("scale", [2.0 ** 127 * (1 + 2.0 ** -23), 2.4e38, 3.4e38])
@pytest.mark.parametrize("fn,where", [(decode, "decode"), (attention, "attention"), (backward, "attention_backward")])
def test_refused(fn, where, scale):
    refused(fn(scale=scale), where)


@pytest.mark.parametrize("scale", [2.0 ** 127, 2.0 ** -149])
def test_taken(scale):
    """By calls that end before a launch."""
    for fn in (decode, attention, backward):
        assert fn(scale=scale, B=0) == M.MOE_OK


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.0 ** 127, 2.0 ** -149])
def test_scores_of_zero(scale):
    """Zero queries: every weight is exactly 1, so outputs are means (their sums and the division round by 2^-24 a few
    times, mla_decode's o~ in two bf16 halves by 2^-16), at the largest and the smallest scale."""
    import torch
    import test_gpu_mla_attention as T
    import test_gpu_mla_decode as D
    q, kv, r, cu_q, cu_k = T.make([70], [300], 2, T.WIDE, seed=60)
    q.zero_()
    out, lse = T.forward(q, kv, r, cu_q, cu_k, False, T.WIDE, scale=scale)
    v = kv[:, :, 128:].double()
    assert torch.all((out.double() - v.mean(0)).abs() <= 2.0 ** -20 * v.abs().mean(0))
    assert torch.all((lse.double() - torch.tensor(300.0).double().log()).abs() <= 2.0 ** -20 * 6)
    q, w, cache, table, n, rows = D.make([300], 1, 2, D.WIDE, 16, seed=61)
    out = torch.empty(1, 2, 128, device="cuda")
    ws = torch.empty(M.mla_decode_workspace_bytes(1, 1, 2, *D.WIDE, 400), dtype=torch.uint8, device="cuda")
    M.mla_decode(q.zero_(), w, cache, table, n, 1, 400, scale, out, ws)
    mid = torch.from_numpy(rows[0][:, :512].mean(0)).cuda()
    w = w[:, 128:].double()
    assert torch.all((out[0].double() - w @ mid).abs() <= 2.0 ** -15 * (w.abs() @ mid.abs()))
