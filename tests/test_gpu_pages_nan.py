"""NaN in stored tokens: every query that sees one gets NaN, and no other query's result changes by a bit, also where
queries that see it share a tile with queries that do not."""
import numpy as np
import pytest
import torch

from pages_common import Cache, queries, visible
from test_gpu_pages import csa, run_prefix, run_window   # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def spoil(cache, b, positions, what):
    for j in positions:
        at = cache.row(b, j)
        if what == "row":
            cache.kv[at] = 0x7F
        elif what == "channel":
            cache.kv[at][(37 * j) % 512] = 0xFF
        else:
            cache.kv_sc[at] = np.nan


def compare(clean, dirty, hit):
    """hit [B, Q]: the queries that see a spoilt token."""
    hit = torch.from_numpy(hit).cuda()
    for c, d in zip(clean, dirty):
        assert d[hit].isnan().all()
        assert torch.equal(c[~hit], d[~hit])
    assert hit.any() and not hit.all()


@pytest.mark.parametrize("what", ["row", "channel", "scale"])
@pytest.mark.parametrize("n,Q,window,sink,bad", [
    (700, 320, 100, 3, [502]),             # four queries a CTA; queries 502 .. 601 see it
    (700, 320, 100, 3, [430, 431, 641]),
    (700, 323, 64, 400, [399, 520]),       # a first token of every later query, and a ragged last block
    (9000, 24, 9000, 0, [8982, 8991]),     # split keys, joined
    (300, 8, 50, 0, [296]),                # a query a CTA
    (3000, 30, 2900, 1, [2976])])
def test_window(csa, n, Q, window, sink, bad, what):   # noqa: F811
    cache = Cache(n + Q, [n], 16)
    q, q_pos = queries(Q, 1, Q), np.arange(n - Q, n, dtype=np.int32)[None]
    clean = run_window(csa, cache, q, q_pos, window, sink)
    hit = np.array([[bool(set(bad) & set(visible(cache, 0, int(i), window, sink))) for i in q_pos[0]]])
    spoil(cache, 0, bad, what)
    compare(clean, run_window(csa, cache, q, q_pos, window, sink), hit)


@pytest.mark.parametrize("what", ["row", "channel", "scale"])
def test_prefix(csa, what):   # noqa: F811
    """Queries inside a shared prefix, on both sides of a spoilt token, and one sequence's own spoilt token."""
    B = 300
    prefix, own = Cache(1, [200], 16), Cache(2, [5] * B, 8, pos0=200)
    q, q_pos = queries(3, B, 1), np.array([[204] if b % 3 else [(7 * b) % 200] for b in range(B)], np.int32)
    clean = run_prefix(csa, prefix, own, q, q_pos)
    hit = np.array([[b % 3 == 1 and b > 150] for b in range(B)])
    for b in np.flatnonzero(hit):
        spoil(own, b, [202], what)
    compare(clean, run_prefix(csa, prefix, own, q, q_pos), hit)
    spoil(prefix, 0, [123], what)
    compare(clean, run_prefix(csa, prefix, own, q, q_pos), hit | (q_pos >= 123))
