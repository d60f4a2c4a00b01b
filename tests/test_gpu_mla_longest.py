"""mla_decode at lengths next to 2^31, which a table that repeats a page can
hold: the tiles' numbers stay in 31 bits, and a length past them makes its own
request NaN and no other."""
import numpy as np
import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M

pytestmark = pytest.mark.gpu

MAX_LEN = 2 ** 31 - 256


# a table of just 2^31 tokens and one of more, whose pages are looked up row by row
@pytest.mark.parametrize("page,W", [(2 ** 20, 2048), (2 ** 20 - 1, 2050)])
@pytest.mark.parametrize("long", [MAX_LEN, MAX_LEN + 1, 2 ** 31 - 1])
def test_lengths_next_to_the_limit(page, W, long):
    """All rows of the one page alike, so every output is W^V c whatever the length.  The weights are 1 and c's values
    small whole numbers: sums of n of them need 26 bits at most, so they and l are off by 2^-24 a few times."""
    c = torch.arange(1, 9, device="cuda")
    cache = torch.cat([c, c.flip(0)]).to(torch.bfloat16).repeat(1, page, 1).contiguous()
    w = torch.randint(-3, 4, (2, 16, 8), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    q = torch.zeros(4, 2, 16, dtype=torch.bfloat16, device="cuda")
    lens = [70, long, 33, 0]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table = torch.zeros(4, W, dtype=torch.int32, device="cuda")
    out = torch.full((4, 2, 8), 7.0, device="cuda")
    ws = torch.empty(M.mla_decode_workspace_bytes(4, 1, 2, 8, 8, 8, 8, MAX_LEN), dtype=torch.uint8, device="cuda")
    M.mla_decode(q, w, cache, table, n, 1, MAX_LEN, 0.125, out, ws)
    got = out.double().cpu().numpy()
    want = np.einsum("hvc,c->hv", w[:, 8:].double().cpu().numpy(), np.arange(1.0, 9.0))
    size = np.einsum("hvc,c->hv", w[:, 8:].double().abs().cpu().numpy(), np.arange(1.0, 9.0))
    for b in (0, 2) if long > MAX_LEN else (0, 1, 2):
        assert np.all(np.abs(got[b] - want) <= 2.0 ** -20 * size), b
    assert np.all(got[3] == 0)
    if long > MAX_LEN:
        assert np.all(np.isnan(got[1]))
