"""LatentCache.write takes the rows of the last extend() and no others: slots
behind them are those of an earlier step, whose cached rows a larger write
would replace."""
import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M
from test_binding_mla import B, DC, DN, DR, DV, H, N, PAGE, PAGES, _NoStream, b16, calls, i32  # noqa: F401


@pytest.fixture
def cache(calls, monkeypatch):  # noqa: F811
    for fn in ("mla_pages_workspace_bytes", "mla_decode_workspace_bytes"):
        monkeypatch.setattr(M, fn, lambda *a: 64)
    c = M.LatentCache(PAGES, PAGE, B, 40, N, H, DN, DR, DV, DC, layers=2, device="cpu")
    c.calls, c.st = calls, _NoStream()
    return c


def refuses(c, n):
    seen = len(c.calls)
    with pytest.raises(ValueError, match="rows"):
        c.write(b16(n, DC), b16(n, DR), stream=c.st)
    assert len(c.calls) == seen


def test_write_takes_the_last_extends_rows(cache):
    c = cache
    refuses(c, 1)                                                  # no rows yet
    c.extend(i32(B), stream=c.st)
    c.write(b16(N, DC), b16(N, DR), stream=c.st)
    c.extend(i32(B), 3, stream=c.st)
    for n in (4, N, N + 1):
        refuses(c, n)
    for layer, n in ((0, 3), (1, 2), (1, 0)):                      # each layer, and fewer
        c.write(b16(n, DC), b16(n, DR), layer, c.st)
    assert [a[5] for name, a in c.calls if name == "mla_cache_write"] == [N, 3, 2, 0]


def test_a_refused_extend_leaves_the_rows(cache):
    c = cache
    c.extend(i32(B), 3, stream=c.st)
    for bad in (lambda: c.extend(i32(B + 1), N, stream=c.st), lambda: c.extend(i32(B), N + 1, stream=c.st)):
        with pytest.raises(ValueError):
            bad()
    refuses(c, 4)
    c.write(b16(3, DC), b16(3, DR), stream=c.st)
    c.extend(i32(B), 0, stream=c.st)
    refuses(c, 1)
