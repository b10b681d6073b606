"""The paged attentions where four queries share a CTA and their keys are split over several, with the join behind it:
every number of splits that leads to another form of the join, several blocks, ragged last blocks, mixed key lists."""
import numpy as np
import pytest
import torch

from pages_common import Cache, D, H, check, queries, reference, visible
from test_gpu_pages import csa, run_prefix, run_window, tail_positions   # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def assert_splits(csa, op, B, Q, keys, splits):   # noqa: F811
    """The workspace holds the partial rows of blocks of four queries: one row of 512 fp32 and two numbers for each of
    16 heads x 4 queries, block and split.  Another form of the call would need another size."""
    blocks = -(-B * Q // 4) if op == csa.OP_PREFIX_ATTN else B * -(-Q // 4)
    assert csa.csa2_workspace_bytes(op, B, Q, keys, 0) == 256 + blocks * splits * 4 * H * (4 * D + 8)


def bad_heads(q, q_pos, picks):
    """The queries with NaN or infinity in a few heads, and where these are.  Each pick sees a token."""
    bad, hit = q.clone(), torch.zeros(q.shape[:3], dtype=torch.bool)
    for k, (b, c, h) in enumerate(picks):
        bad[b, c, h, (71 * k) % D] = (float("nan"), float("inf"), -float("inf"))[k % 3]
        hit[b, c, h] = bool(q_pos[b, c] >= 0)
    return bad, hit.cuda()


def same_elsewhere(got, clean, hit):
    for g, c in zip(got, clean):
        assert g[hit].isnan().all() and torch.equal(g[~hit], c[~hit])


@pytest.mark.parametrize("lens,Q,window,sink,page,splits,replay", [
    ([512] * 20 + [511, 3, 0, 129] + [300] * 13, 8, 1 << 30, 0, 16, 2, False),
    ([1500, 40, 1, 1499] * 5, 6, 1 << 30, 0, 64, 3, False),
    ([3000, 0, 2999, 128, 1000], 10, 2990, 5, 32, 9, True),
    ([9000, 5003, 8111], 7, 1 << 30, 0, 64, 24, False),
    ([9000, 5003, 8111], 7, 8900, 40, 16, 24, True),
    ([30000, 17001], 5, 1 << 30, 0, 64, 37, False),
    ([20000], 9, 19000, 7, 64, 49, False),
    ([33001], 4, 1 << 30, 0, 64, 148, False)])
def test_window(csa, lens, Q, window, sink, page, splits, replay):   # noqa: F811
    B = len(lens)
    cache = Cache(Q + splits, lens, page)
    assert_splits(csa, csa.OP_WINDOW_ATTN, B, Q, min(window + sink, cache.table.shape[1] * page), splits)
    q, q_pos = queries(splits, B, Q), tail_positions(lens, Q)
    start = [n // 5 for n in lens] if replay else None
    clean = run_window(csa, cache, q, q_pos, window, sink, start)
    check(*clean, reference(q, q_pos, [(cache, True)], window, sink, start))
    cache.poison_dead({cache.row(b, j) for b in range(B) for i in q_pos[b]
                       for j in visible(cache, b, int(i), window, sink, None if start is None else start[b])})
    bad, hit = bad_heads(q, q_pos, [(0, 0, 3), (0, Q - 1, 15), (B - 1, Q // 2, 0)])
    same_elsewhere(run_window(csa, cache, bad, q_pos, window, sink, start), clean, hit)


@pytest.mark.parametrize("n,own,Q,page_prefix,page,splits", [
    (700, [(37 * b) % 90 for b in range(200)], 1, 64, 16, 2),
    (3001, [5 + (97 * b) % 400 for b in range(30)], 3, 64, 64, 6),
    (4000, [2 + (61 * b) % 70 for b in range(21)], 2, 16, 16, 13),
    (5000, [b for b in range(33)], 1, 64, 8, 16),
    (30000, [300, 0, 7, 64, 129, 1, 2, 600, 9], 1, 64, 64, 49)])
def test_prefix(csa, n, own, Q, page_prefix, page, splits):   # noqa: F811
    B = len(own)
    prefix, mine = Cache(splits, [n], page_prefix), Cache(splits + 1, own, page, pos0=n)
    caps = [c.table.shape[1] * c.page for c in (prefix, mine)]
    assert_splits(csa, csa.OP_PREFIX_ATTN, B, Q, sum(caps), splits)
    q = queries(splits, B, Q)
    q_pos = np.array([[n + m - Q + c for c in range(Q)] for m in own], np.int32)
    q_pos[B // 2, 0], q_pos[B // 3, 0] = n // 3, -1   # one inside the prefix, one none
    clean = run_prefix(csa, prefix, mine, q, q_pos)
    check(*clean, reference(q, q_pos, [(prefix, False), (mine, True)]))
    prefix.poison_dead({prefix.row(0, j) for j in visible(prefix, 0, int(q_pos.max()))})
    mine.poison_dead({mine.row(b, j) for b in range(B) for i in q_pos[b] for j in visible(mine, b, int(i))})
    bad, hit = bad_heads(q, q_pos, [(0, 0, 3), (B - 1, Q - 1, 15), (B // 2, 0, 0)])
    same_elsewhere(run_prefix(csa, prefix, mine, bad, q_pos), clean, hit)


def test_workspace_of_a_large_call_for_a_small_one(csa):   # noqa: F811
    """The size belongs to a call's shape: a workspace of a larger call may be too small for a smaller one, and the call says
    so; one that is large enough for both serves both, whatever it held before."""
    cache = Cache(7, [2000, 600], 64)
    big, small = queries(1, 2, 160), queries(2, 2, 1)
    sizes = [csa.csa2_workspace_bytes(csa.OP_WINDOW_ATTN, 2, Q, cache.table.shape[1] * 64, 0) for Q in (160, 1)]
    assert sizes[0] < sizes[1]
    pages, pos = cache.gpu(), [torch.from_numpy(tail_positions([2000, 600], Q)).cuda() for Q in (160, 1)]
    with pytest.raises(csa.CSA2Error, match="WORKSPACE"):
        csa.csa2_window_attn(small.cuda(), pages, pos[1], window=1 << 30,
                             ws=torch.empty(sizes[0], dtype=torch.uint8, device="cuda"))
    ws = torch.full((max(sizes) // 4 + 1,), float("nan"), device="cuda")
    for _ in range(2):
        for q, p in ((big, pos[0]), (small, pos[1])):
            want = csa.csa2_window_attn(q.cuda(), pages, p, window=1 << 30, lse=True)
            got = csa.csa2_window_attn(q.cuda(), pages, p, window=1 << 30, lse=True, ws=ws)
            assert all(torch.equal(a, b) for a, b in zip(want, got))
    csa.csa2_flag_status()
