"""Paged FP8 cache on the GPU: the append, the sliding-window and the shared-prefix attention against
the 64-bit definition (pages_common), at the sizes, masks and pages where they can go wrong."""
import math

import numpy as np
import pytest
import torch

from pages_common import Cache, D, E4M3, H, check, queries, reference, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def csa():
    import sparse_attention_fp4_quant_b200 as csa
    csa.lib()
    return csa


# ---- append ------------------------------------------------------------------------------------

def append_reference(x, pos, inv_freq, norm_w, eps, normalise):
    y = x.double().cpu().numpy()
    if normalise:
        y = y / np.sqrt((y * y).mean(1, keepdims=True) + eps)
    if norm_w is not None:
        y = y * norm_w.double().cpu().numpy()
    if inv_freq is not None:
        t = pos.astype(np.float64)[:, None] * inv_freq.double().cpu().numpy()
        a, b = y[:, 448::2].copy(), y[:, 449::2].copy()
        y[:, 448::2], y[:, 449::2] = a * np.cos(t) - b * np.sin(t), a * np.sin(t) + b * np.cos(t)
    return y, np.abs(y).max(1) / 448


def inv_freq_table():
    return (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()


@pytest.mark.parametrize("rows,page,stride,normalise,weight,rope,far", [
    (1, 64, 512, True, True, True, 0), (2, 8, 520, True, False, True, 1 << 20), (33, 16, 1024, True, True, True, 262000),
    (257, 128, 512, False, False, True, 0), (130, 24, 640, True, True, False, 5), (1000, 64, 512, False, True, True, 2000000)])
def test_append(csa, rows, page, stride, normalise, weight, rope, far):
    g = torch.Generator().manual_seed(rows)
    x = (torch.randn((rows, stride), generator=g) * 3).to(torch.bfloat16).cuda()[:, :D]
    x[rows // 2] = 0
    seq = torch.randint(0, 3, (rows,), generator=g).to(torch.int32)
    local = torch.zeros(3, dtype=torch.int64)
    pos = torch.empty(rows, dtype=torch.int32)
    for r in range(rows):   # tokens of each sequence in order, from position far
        pos[r] = far + local[seq[r]]
        local[seq[r]] += 1
    if rows > 5:
        seq[3], seq[4] = -1, 3   # dropped: no such sequence
    cache = Cache(rows, [rows] * 3, page, pos0=far)
    cache.table[2, -1] = -1 if rows > 5 else cache.table[2, -1]
    cache.kv_sc[:] = -7.0
    before = cache.kv.copy()
    pages = cache.gpu()
    w = (torch.rand(D, generator=g) + 0.5).cuda() if weight else None
    f = inv_freq_table() if rope else None
    csa.csa2_pages_append(x, pages, seq.cuda(), pos.cuda(), inv_freq=f, norm_w=w, normalise=normalise)
    y, scale = append_reference(x, pos.numpy(), f, w, 1e-6, normalise)
    kv, sc = pages.kv.cpu().numpy(), pages.kv_sc.cpu().numpy()
    touched = np.zeros(sc.shape, bool)
    for r in range(rows):
        at = cache.row(int(seq[r]), int(pos[r])) if 0 <= seq[r] < 3 else None
        if at is None:
            continue
        touched[at] = True
        # fp32 sums and one reciprocal: 2^-18 of the row's largest value is ample; then half an E4M3 step
        assert abs(sc[at] - scale[r]) <= 2.0 ** -18 * scale[r]
        want = y[r] / scale[r] if scale[r] > 0 else y[r] * 0
        tol = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + 448 * 2.0 ** -18
        assert (np.abs(E4M3[kv[at]] - want) <= tol).all(), r
    assert np.array_equal(kv[~touched], before[~touched]) and (sc[~touched] == -7.0).all()


def test_append_tiny_and_huge_values(csa):
    x = torch.zeros((4, D), dtype=torch.bfloat16)
    x[0], x[1, 5], x[2, 500] = 1e-38, 3e38, 2.0 ** -133
    cache = Cache(1, [4], 8)
    pages = cache.gpu()
    csa.csa2_pages_append(x.cuda(), pages, torch.zeros(4, dtype=torch.int32).cuda(),
                          torch.arange(4, dtype=torch.int32).cuda(), normalise=False)
    got = E4M3[pages.kv.cpu().numpy()] * pages.kv_sc.cpu().double().numpy()[..., None]
    for r in range(4):
        want = x[r].double().numpy()
        assert np.isfinite(got[cache.row(0, r)]).all()
        # the scale itself is rounded to the fp32 grid, 2^-149 near zero
        assert (np.abs(got[cache.row(0, r)] - want) <= 2.0 ** -4 * np.abs(want) + 448 * 2.0 ** -149).all()


# ---- sliding window ----------------------------------------------------------------------------

def run_window(csa, cache, q, q_pos, window, sink, start=None, **kw):
    qp = torch.from_numpy(np.asarray(q_pos, np.int32)).cuda()
    st = None if start is None else torch.tensor(start, dtype=torch.int32).cuda()
    r = csa.csa2_window_attn(q.cuda(), cache.gpu() if isinstance(cache, Cache) else cache, qp, window=window, n_sink=sink,
                             replay_start=st, lse=True, **kw)
    csa.csa2_flag_status()
    return r


def tail_positions(lens, Q):
    return np.array([[max(-1, n - Q + i) for i in range(Q)] for n in lens], np.int32)


@pytest.mark.parametrize("lens,Q,window,sink,page", [
    ([1], 1, 1, 0, 64), ([1], 1, 128, 4, 8), ([129], 1, 128, 0, 64), ([130, 5, 300], 1, 128, 4, 16),
    ([1000, 127, 128, 2, 511], 1, 257, 9, 64), ([700, 3], 2, 64, 1, 32), ([90, 400], 3, 33, 0, 8), ([513], 4, 128, 130, 128),
    ([260, 7, 31], 5, 16, 3, 24), ([150], 37, 20, 2, 64), ([200, 64], 64, 128, 4, 64), ([97], 97, 2147483647, 0, 16),
    ([5000], 1, 4096, 7, 64), ([3001, 2999], 2, 1 << 30, 0, 40), ([640], 9, 1, 1, 64), ([2100], 7, 2000, 700, 16)])
def test_window(csa, lens, Q, window, sink, page):
    cache = Cache(sum(lens) + Q, lens, page)
    q, q_pos = queries(Q, len(lens), Q), tail_positions(lens, Q)
    out, lse = run_window(csa, cache, q, q_pos, window, sink)
    check(out, lse, reference(q, q_pos, [(cache, True)], window, sink))


@pytest.mark.parametrize("Q", [1, 2, 4, 11])
def test_window_positions_in_any_order(csa, Q):
    """Queries anywhere (before the first token, behind the last one, none), sequences of no token, tokens without a page."""
    lens = [300, 0, 77, 512]
    cache = Cache(5, lens, 16, max_pages=40)
    cache.table[0, 3] = -1
    cache.table[3, 30] = cache.kv.shape[0]
    cache.table[3, 0] = -5
    cache.n_tokens[3] = 10 ** 6   # clamped to the table, whose pages beyond 512 tokens are absent
    rng = np.random.default_rng(Q)
    q_pos = rng.integers(-3, 700, (4, Q)).astype(np.int32)
    q = queries(9, 4, Q)
    for window, sink in ((64, 0), (200, 20), (5, 600)):
        out, lse = run_window(csa, cache, q, q_pos, window, sink)
        check(out, lse, reference(q, q_pos, [(cache, True)], window, sink))


@pytest.mark.parametrize("Q,page", [(1, 64), (128, 64), (30, 16)])
def test_window_replay(csa, Q, page):
    lens = [400, 260]
    cache = Cache(Q, lens, page)
    start = [300, 259]
    q, q_pos = queries(3, 2, Q), tail_positions(lens, Q)
    for sink in (0, 5):
        out, lse = run_window(csa, cache, q, q_pos, 128, sink, start)
        check(out, lse, reference(q, q_pos, [(cache, True)], 128, sink, start))


@pytest.mark.parametrize("Q,window,sink,page", [(1, 100, 3, 64), (3, 40, 0, 16), (6, 130, 17, 8), (40, 77, 1, 64)])
def test_window_never_reads_a_masked_value(csa, Q, window, sink, page):
    """NaN bytes and scales wherever no query of the call looks: the result is bit-identical to the clean cache's."""
    lens = [533, 290]
    cache = Cache(11, lens, page)
    q, q_pos = queries(4, 2, Q), tail_positions(lens, Q)
    clean = run_window(csa, cache, q, q_pos, window, sink)
    cache.poison_dead({cache.row(b, j) for b in range(2) for i in q_pos[b] for j in visible(cache, b, int(i), window, sink)})
    dirty = run_window(csa, cache, q, q_pos, window, sink)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])
    check(*dirty, reference(q, q_pos, [(cache, True)], window, sink))


@pytest.mark.parametrize("Q", [1, 4, 8])
def test_extreme_keys_and_queries(csa, Q):
    """Zero rows, scales twenty orders apart, one key that takes nearly all the weight with many behind it, large queries."""
    lens = [2000]
    cache = Cache(21, lens, 64)
    order = [cache.row(0, j) for j in range(2000)]
    for j in (0, 5, 1999):
        cache.kv[order[j]], cache.kv_sc[order[j]] = 0, 0.0
    for j in range(100, 200):
        cache.kv_sc[order[j]] *= 1e-20
    for j in range(300, 310):
        cache.kv_sc[order[j]] *= 30.0
    q, q_pos = queries(5, 1, Q), tail_positions(lens, Q)
    q[0, :, 3] = 0
    q[0, :, 4] *= 2.0 ** 100
    q[0, :, 5] *= 2.0 ** -100
    q[0, 0, 6] = torch.from_numpy(E4M3[cache.kv[order[1000]]]).to(torch.bfloat16) * 0.05   # looks straight at token 1000
    q[0, :, 7, 100] = 300.0   # one channel far above the others
    out, lse = run_window(csa, cache, q, q_pos, 1 << 30, 0)
    check(out, lse, reference(q, q_pos, [(cache, True)], None, 0))


def test_weight_behind_one_dominant_key(csa):
    """A first token with half of the weight, the other half spread over 30,000 tokens of about 2^-15 each."""
    n = 30001
    cache = Cache(2, [n], 64)
    q = torch.zeros((1, 1, H, D))
    q[..., 0] = 1.0
    codes = torch.full((n,), 0x38, dtype=torch.uint8).numpy()   # 1.0
    for j in range(n):
        at = cache.row(0, j)
        cache.kv[at][0] = 0
        cache.kv_sc[at] = 0.01
    at = cache.row(0, 0)
    cache.kv[at] = 0
    cache.kv[at][0] = codes[0]
    cache.kv_sc[at] = math.log(30000.0) * math.sqrt(D) / 1.0
    q = q.to(torch.bfloat16)
    out, lse = run_window(csa, cache, q, np.array([[n - 1]], np.int32), 1 << 30, 0)
    check(out, lse, reference(q, np.array([[n - 1]], np.int32), [(cache, True)], None, 0))


@pytest.mark.parametrize("n,Q", [(30001, 1), (20000, 5)])
def test_weight_behind_a_first_token(csa, n, Q):
    """The same with scales as a normalised latent has them: the first token's weight comes from the query's direction."""
    cache = Cache(3, [n], 64)
    for j in range(n):
        at = cache.row(0, j)
        cache.kv[at][0] = 0
        cache.kv_sc[at] = 0.01
    at = cache.row(0, 0)
    cache.kv[at] = 0
    cache.kv[at][0] = 0x7E   # 448
    cache.kv_sc[at] = 0.0163
    q = torch.zeros((1, Q, H, D))
    q[..., 0] = math.log(n) * math.sqrt(D) / (448 * 0.0163)
    q_pos = np.arange(n - Q, n, dtype=np.int32)[None]
    q = q.to(torch.bfloat16)
    out, lse = run_window(csa, cache, q, q_pos, 1 << 30, 0)
    check(out, lse, reference(q, q_pos, [(cache, True)], None, 0))


# ---- shared prefix -----------------------------------------------------------------------------

def run_prefix(csa, prefix, own, q, q_pos, **kw):
    r = csa.csa2_prefix_attn(q.cuda(), prefix.gpu(), own.gpu(), torch.from_numpy(np.asarray(q_pos, np.int32)).cuda(),
                             lse=True, **kw)
    csa.csa2_flag_status()
    return r


@pytest.mark.parametrize("B,Q,n_prefix,own,page", [
    (1, 1, 1, [1], 64), (2, 1, 300, [1, 40], 16), (3, 1, 129, [5, 0, 130], 64), (4, 1, 1000, [1, 2, 3, 4], 8),
    (5, 2, 513, [2, 300, 9, 64, 65], 64), (7, 3, 250, [3, 3, 3, 3, 3, 3, 140], 32), (33, 1, 640, list(range(1, 34)), 64),
    (2, 9, 77, [9, 200], 24), (1, 4, 2000, [4], 128), (6, 1, 4001, [17] * 6, 64)])
def test_prefix(csa, B, Q, n_prefix, own, page):
    prefix, mine = Cache(B, [n_prefix], page), Cache(B + 1, own, page, pos0=n_prefix)
    q = queries(B, B, Q)
    q_pos = np.array([[n_prefix + n - Q + i for i in range(Q)] for n in own], np.int32)
    out, lse = run_prefix(csa, prefix, mine, q, q_pos)
    check(out, lse, reference(q, q_pos, [(prefix, False), (mine, True)]))


def test_prefix_masks(csa):
    """Queries inside the prefix (causal in it), behind it, none; an absent prefix page; a prefix shorter than its table."""
    prefix, mine = Cache(1, [200], 16, max_pages=20), Cache(2, [30, 7, 0, 90, 64], 16, pos0=200)
    prefix.table[0, 4] = -1
    q_pos = np.array([[10, 199], [-1, 206], [205, 0], [220, 289], [-7, -1]], np.int32)
    q = queries(1, 5, 2)
    clean = run_prefix(csa, prefix, mine, q, q_pos)
    ref = reference(q, q_pos, [(prefix, False), (mine, True)])
    check(*clean, ref)
    prefix.poison_dead({prefix.row(0, j) for i in q_pos.flatten() for j in visible(prefix, 0, int(i))})
    mine.poison_dead({mine.row(b, j) for b in range(5) for i in q_pos[b] for j in visible(mine, b, int(i))})
    dirty = run_prefix(csa, prefix, mine, q, q_pos)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


def test_prefix_equals_each_sequence_alone(csa):
    """The same tokens as one table per sequence: the shared form and the window form agree within both bounds."""
    prefix = Cache(3, [333], 37 // 37 * 16)
    mine = Cache(4, [20, 51, 1], 16, pos0=333)
    q_pos = np.array([[333 + n - 1] for n in (20, 51, 1)], np.int32)
    q = queries(6, 3, 1)
    ref = reference(q, q_pos, [(prefix, False), (mine, True)])
    check(*run_prefix(csa, prefix, mine, q, q_pos), ref)
    whole = Cache(5, [353, 384, 334], 16)
    for b, n in enumerate((20, 51, 1)):
        for j in range(333 + n):
            c, r = (prefix, 0) if j < 333 else (mine, b)
            whole.kv[whole.row(b, j)], whole.kv_sc[whole.row(b, j)] = c.kv[c.row(r, j)], c.kv_sc[c.row(r, j)]
    check(*run_window(csa, whole, q, q_pos, 1 << 30, 0), ref)


@pytest.mark.parametrize("B,Q,window,sink,page", [(400, 1, 50, 3, 16), (310, 2, 20, 0, 32), (3, 250, 24, 2, 64), (160, 3, 5, 1, 8)])
def test_more_items_than_the_gpu_holds(csa, B, Q, window, sink, page):
    """CTAs walk over several items each, some of them without a query or a token."""
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(0, 2 * Q + 60, B)]
    lens[B // 3] = 0
    cache = Cache(B + Q, lens, page)
    q, q_pos = queries(B, B, Q), tail_positions(lens, Q)
    out, lse = run_window(csa, cache, q, q_pos, window, sink)
    check(out, lse, reference(q, q_pos, [(cache, True)], window, sink))


@pytest.mark.parametrize("Q", [1, 3, 2, 20])
def test_window_table_that_starts_later(csa, Q):
    """pos0 > 0: the table's first slot is a later token; sinks count by position."""
    lens = [300, 41]
    cache = Cache(17, lens, 16, pos0=1000)
    q, q_pos = queries(8, 2, Q), tail_positions(lens, Q) + 1000
    for window, sink in ((70, 0), (70, 1013), (16, 5)):
        out, lse = run_window(csa, cache, q, q_pos, window, sink)
        check(out, lse, reference(q, q_pos, [(cache, True)], window, sink))


@pytest.mark.parametrize("Q", [1, 4])
def test_positions_up_to_the_last(csa, Q):
    """Tables that end just below 2^31: every position is a position, none a mark for "no token"."""
    for pos0 in (2 ** 31 - 129 - 128, 2 ** 31 - 256 - 16, 2 ** 31 - 129):
        cache = Cache(19, [128], 16, pos0=pos0)
        cache.table[0, 5] = -1
        q, q_pos = queries(10, 1, Q), tail_positions([128], Q) + pos0
        for window, sink in ((70, 0), (100, pos0 + 3), (1 << 30, 5)):
            out, lse = run_window(csa, cache, q, q_pos, window, sink)
            check(out, lse, reference(q, q_pos, [(cache, True)], window, sink))


@pytest.mark.parametrize("page_prefix,page_own", [(64, 16), (8, 128), (256, 64), (24, 40)])
def test_prefix_pages_of_another_size(csa, page_prefix, page_own):
    prefix, mine = Cache(51, [777], page_prefix), Cache(52, [130, 1, 64, 9, 300], page_own, pos0=777)
    q, q_pos = queries(7, 5, 1), np.array([[777 + n - 1] for n in (130, 1, 64, 9, 300)], np.int32)
    check(*run_prefix(csa, prefix, mine, q, q_pos), reference(q, q_pos, [(prefix, False), (mine, True)]))


def test_prefix_without_own_tokens_or_prefix(csa):
    """An empty prefix, sequences of no token, and both."""
    q_pos = np.array([[5], [0], [9], [3]], np.int32)
    q = queries(12, 4, 1)
    for n, own in ((0, [6, 1, 10, 0]), (7, [0, 0, 3, 0]), (0, [0, 0, 0, 0])):
        prefix, mine = Cache(61, [n], 16), Cache(62, own, 16, pos0=n)
        check(*run_prefix(csa, prefix, mine, q, q_pos), reference(q, q_pos, [(prefix, False), (mine, True)]))


def test_a_table_wider_than_memory(csa):
    """A table that could name 2^31 - 64 tokens: the sizes stay within 32 bits (the pages it names are few)."""
    width = (1 << 31) // 4096 - 1
    small = Cache(63, [4096 + 50], 4096, n_pages=3)
    kv, sc = torch.from_numpy(small.kv).cuda(), torch.from_numpy(small.kv_sc).cuda()
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    last = width * 4096   # positions last - 4096 - 50 ..: the table's end
    table[0, width - 2:] = torch.from_numpy(small.table[0]).cuda()
    pages = csa.Pages.of(kv, sc, table, torch.full((1,), last, dtype=torch.int32, device="cuda"))
    shifted = Cache(63, [4096 + 50], 4096, n_pages=3, pos0=last - 8192)
    shifted.n_tokens[0] = 8192
    q, q_pos = queries(14, 1, 2), np.array([[last - 1, last - 4000]], np.int32)
    out, lse = run_window(csa, pages, q, q_pos, 300, 0)
    check(out, lse, reference(q, q_pos, [(shifted, True)], 300, 0))


@pytest.mark.parametrize("Q", [1, 4])
def test_zero_queries_do_not_hide_masked_nan(csa, Q):
    """Heads of zeros beside NaN slots: zero times NaN must not reach the output."""
    lens = [200]
    cache = Cache(64, lens, 16)
    q, q_pos = queries(15, 1, Q), tail_positions(lens, Q)
    q[:, :, :5] = 0
    cache.poison_dead({cache.row(0, j) for i in q_pos[0] for j in visible(cache, 0, int(i), 30, 2)})
    check(*run_window(csa, cache, q, q_pos, 30, 2), reference(q, q_pos, [(cache, True)], 30, 2))


@pytest.mark.parametrize("Q,n", [(1, 200), (1, 3000), (4, 200), (9, 700)])
def test_a_query_of_nan_or_infinity_keeps_to_itself(csa, Q, n):
    """NaN and infinite heads give NaN; every other head's result is bit-identical to the clean call's."""
    cache = Cache(65, [n], 64)
    q, q_pos = queries(16, 1, Q), tail_positions([n], Q)
    clean = run_window(csa, cache, q, q_pos, 1 << 30, 0)
    bad = q.clone()
    bad[0, 0, 3, 17], bad[0, Q - 1, 9, 500] = float("nan"), float("inf")
    out, lse = run_window(csa, cache, bad, q_pos, 1 << 30, 0)
    hit = torch.zeros((1, Q, H), dtype=torch.bool)
    hit[0, 0, 3] = hit[0, Q - 1, 9] = True
    hit = hit.cuda()
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ps", [16, 64])
def test_keys_that_a_nan_query_does_not_see(csa, ps, value):
    """A first query whose every head holds NaN or infinity leaves the keys behind it, which it does not see, to the
    queries of its tile that do."""
    cache = Cache(66, [300], ps)
    q, q_pos = queries(17, 1, 8), np.array([[100, 299, 298, 101, 40, 41, 42, 299]], np.int32)
    clean = run_window(csa, cache, q, q_pos, 1 << 30, 0)
    bad = q.clone()
    bad[0, 0, :, 7] = value
    bad[0, 4, 0, 511] = value
    out, lse = run_window(csa, cache, bad, q_pos, 1 << 30, 0)
    assert out[0, 0].isnan().all() and out[0, 4, 0].isnan().all() and lse[0, 0].isnan().all()
    keep = torch.ones((1, 8, H), dtype=torch.bool)
    keep[0, 0], keep[0, 4, 0] = False, False
    keep = keep.cuda()
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


# ---- single queries with long lists: two warpgroups take a query's tiles in turn --------------

def long_lists(seed, B, n, page, **kw):
    """Sequences around the tiles' borders, a third of the others up to n tokens, the rest short."""
    rng = np.random.default_rng(seed)
    lens = [int(v) for v in np.where(np.arange(B) % 3 == 0, rng.integers(0, n, B), rng.integers(0, 300, B))]
    lens[:11] = [n, 0, 1, 127, 128, 129, 255, 256, 257, 384, 385]
    return lens, Cache(seed, lens, page, **kw)


@pytest.mark.parametrize("B,n,window,sink,page", [
    (60, 2300, 1 << 30, 0, 16), (160, 2200, 2100, 5, 64), (100, 700, 1 << 30, 0, 8), (148, 640, 600, 70, 24), (320, 2049, 2048, 1, 32)])
def test_long_lists(csa, B, n, window, sink, page):
    lens, cache = long_lists(B, B, n, page)
    q, q_pos = queries(B, B, 1), tail_positions(lens, 1)
    out, lse = run_window(csa, cache, q, q_pos, window, sink)
    check(out, lse, reference(q, q_pos, [(cache, True)], window, sink))


def test_long_lists_masked_nan_and_bad_queries(csa):
    lens, cache = long_lists(3, 60, 2300, 16)
    q, q_pos = queries(6, 60, 1), tail_positions(lens, 1)
    clean = run_window(csa, cache, q, q_pos, 2200, 9)
    cache.poison_dead({cache.row(b, j) for b in range(60) for i in q_pos[b] for j in visible(cache, b, int(i), 2200, 9)})
    bad = q.clone()
    bad[0, 0, 0, 3], bad[20, 0, 15, 400] = float("nan"), float("inf")
    out, lse = run_window(csa, cache, bad, q_pos, 2200, 9)
    keep = torch.ones((60, 1, H), dtype=torch.bool)
    keep[0, 0, 0] = keep[20, 0, 15] = False
    keep = keep.cuda()
    assert out[~keep].isnan().all() and lse[~keep].isnan().all()
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


def test_long_lists_extreme_keys_and_queries(csa):
    lens = [2000] * 2 + [3] * 58
    cache = Cache(22, lens, 64)
    order = [cache.row(0, j) for j in range(2000)]
    for j in (0, 5, 1999):
        cache.kv[order[j]], cache.kv_sc[order[j]] = 0, 0.0
    for j in range(100, 200):
        cache.kv_sc[order[j]] *= 1e-20
    for j in list(range(300, 310)) + [700, 1500, 1900]:
        cache.kv_sc[order[j]] *= 30.0
    q, q_pos = queries(5, 60, 1), tail_positions(lens, 1)
    q[0, :, 3] = 0
    q[0, :, 4] *= 2.0 ** 100
    q[0, :, 5] *= 2.0 ** -100
    q[0, 0, 6] = torch.from_numpy(E4M3[cache.kv[order[1000]]]).to(torch.bfloat16) * 0.05   # looks straight at token 1000
    q[1, 0, 6] = torch.from_numpy(E4M3[cache.kv[cache.row(1, 130)]]).to(torch.bfloat16) * 0.05
    q[0, :, 7, 100] = 300.0
    out, lse = run_window(csa, cache, q, q_pos, 1 << 30, 0)
    check(out, lse, reference(q, q_pos, [(cache, True)], None, 0))


@pytest.mark.parametrize("n", [9000, 60000])
def test_many_splits(csa, n):
    """Splits by the hundred: a row's join is shared by several CTAs."""
    lens = [n, n // 3]
    cache = Cache(n, lens, 64)
    q, q_pos = queries(7, 2, 1), tail_positions(lens, 1)
    out, lse = run_window(csa, cache, q, q_pos, 1 << 30, 0)
    check(out, lse, reference(q, q_pos, [(cache, True)], None, 0))
    prefix, own = Cache(n + 1, [n], 64), Cache(n + 2, [1, 70, 0, 5], 64, pos0=n)
    q, q_pos = queries(8, 4, 1), np.array([[n], [n + 69], [n - 1], [n + 4]], np.int32)
    out, lse = run_prefix(csa, prefix, own, q, q_pos)
    check(out, lse, reference(q, q_pos, [(prefix, False), (own, True)]))


# ---- as they are used --------------------------------------------------------------------------

def test_decode_run(csa):
    """A prompt appended and attended chunk by chunk, then decode steps: every attention reads what the appends wrote."""
    B, page, window, sink = 3, 16, 40, 3
    g = torch.Generator().manual_seed(0)
    pages = csa.Pages(B, 20, n_pages=61, page_size=page)
    pages.table.copy_(torch.randperm(61, generator=g)[:60].view(3, 20).to(torch.int32))
    f = inv_freq_table()
    seen, done = [[] for _ in range(B)], np.zeros(B, np.int64)
    for step, counts in enumerate([[70, 33, 5], [20, 64, 1]] + [[1, 1, 1]] * 3):
        rows, Q = sum(counts), max(counts)
        x = torch.randn((rows, D), generator=g).to(torch.bfloat16).cuda()
        seq = torch.cat([torch.full((c,), b) for b, c in enumerate(counts)]).to(torch.int32).cuda()
        pos = torch.cat([torch.arange(done[b], done[b] + c) for b, c in enumerate(counts)]).to(torch.int32).cuda()
        csa.csa2_pages_append(x, pages, seq, pos, inv_freq=f)
        done += counts
        pages.n_tokens.copy_(torch.from_numpy(done.astype(np.int32)))
        q_pos = np.full((B, Q), -1, np.int32)
        for b, c in enumerate(counts):
            q_pos[b, :c] = np.arange(done[b] - c, done[b])
        q = queries(step, B, Q)
        out, lse = run_window(csa, pages, q, q_pos, window, sink)
        now = Cache(0, [1] * B, page)
        now.kv, now.kv_sc = pages.kv.cpu().numpy(), pages.kv_sc.cpu().numpy()
        now.table, now.n_tokens = pages.table.cpu().numpy(), pages.n_tokens.cpu().numpy()
        check(out, lse, reference(q, q_pos, [(now, True)], window, sink))


def test_prefix_run(csa):
    """A prompt appended once, then four answers drawn from it: shared prefix pages and own pages in one pool."""
    g = torch.Generator().manual_seed(8)
    page, n = 64, 150
    pool = csa.Pages(1, 3, n_pages=12, page_size=page)
    pool.table.copy_(torch.tensor([[7, 2, 9]], dtype=torch.int32))
    f = inv_freq_table()
    x = torch.randn((n, D), generator=g).to(torch.bfloat16).cuda()
    csa.csa2_pages_append(x, pool, torch.zeros(n, dtype=torch.int32).cuda(), torch.arange(n, dtype=torch.int32).cuda(), inv_freq=f)
    pool.n_tokens.fill_(n)
    own = csa.Pages.of(pool.kv, pool.kv_sc, torch.tensor([[0, -1], [1, -1], [3, 11], [5, -1]], dtype=torch.int32).cuda(),
                       torch.zeros(4, dtype=torch.int32).cuda(), pos0=n)
    for step in range(3):
        x = torch.randn((4, D), generator=g).to(torch.bfloat16).cuda()
        csa.csa2_pages_append(x, own, torch.arange(4, dtype=torch.int32).cuda(),
                              torch.full((4,), n + step, dtype=torch.int32).cuda(), inv_freq=f)
        own.n_tokens.fill_(step + 1)
        q, q_pos = queries(step, 4, 1), np.full((4, 1), n + step, np.int32)
        out, lse = csa.csa2_prefix_attn(q.cuda(), pool, own, torch.from_numpy(q_pos).cuda(), lse=True)
        csa.csa2_flag_status()
        caches = []
        for p, per_row in ((pool, False), (own, True)):
            c = Cache(0, [1] * p.B, page, pos0=p.pos0)
            c.kv, c.kv_sc = p.kv.cpu().numpy(), p.kv_sc.cpu().numpy()
            c.table, c.n_tokens = p.table.cpu().numpy(), p.n_tokens.cpu().numpy()
            caches.append((c, per_row))
        check(out, lse, reference(q, q_pos, caches))


def test_captured_calls(csa):
    """A decode step (append, window attention, prefix attention) captured twice, replayed at the same time on two streams
    with new tokens in place: each replay gives what the eager calls give, bit for bit."""
    B, page = 4, 16
    graphs = []
    for k in range(2):
        cache = Cache(30 + k, [400] * B, page, max_pages=26)
        prefix = Cache(40 + k, [2000], page)
        s = dict(pages=cache.gpu(), prefix=prefix.gpu(), q=queries(k, B, 1).cuda(), x=queries(50 + k, B, 1)[:, 0, 0].cuda(),
                 seq=torch.arange(B, dtype=torch.int32).cuda(), pos=torch.full((B,), 400, dtype=torch.int32).cuda(),
                 f=inv_freq_table())
        s["own"] = csa.Pages.of(s["pages"].kv, s["pages"].kv_sc, s["pages"].table, s["pages"].n_tokens, pos0=0)

        def step(s=s):
            csa.csa2_pages_append(s["x"], s["pages"], s["seq"], s["pos"], inv_freq=s["f"])
            s["pages"].n_tokens.copy_(s["pos"] + 1)
            qp = s["pos"].view(B, 1)
            return (*csa.csa2_window_attn(s["q"], s["pages"], qp, window=300, n_sink=2, lse=True),
                    *csa.csa2_prefix_attn(s["q"], s["prefix"], s["own"], qp, lse=True))
        step()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            held = step()
        graphs.append((gr, held, s, step))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for t in range(401, 405):
        for gr, held, s, step in graphs:
            s["pos"].fill_(t)
            s["x"].copy_(torch.randn(B, D))
        torch.cuda.synchronize()
        for (gr, held, s, step), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                for _ in range(3):
                    gr.replay()
        torch.cuda.synchronize()
        for gr, held, s, step in graphs:
            got = [h.clone() for h in held]
            want = step()
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)
    csa.csa2_flag_status()


def test_two_streams_at_once(csa):
    caches = [Cache(60 + k, [3000, 100], 64) for k in range(2)]
    pages, qs = [c.gpu() for c in caches], [queries(k, 2, 1).cuda() for k in range(2)]
    qp = torch.tensor([[2999], [99]], dtype=torch.int32).cuda()
    want = [csa.csa2_window_attn(q, p, qp, window=1 << 30, lse=True) for p, q in zip(pages, qs)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(20):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(csa.csa2_window_attn(qs[k], pages[k], qp, window=1 << 30, lse=True))
    torch.cuda.synchronize()
    for k in range(2):
        for out, lse in got[k]:
            assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])


def test_pool_beyond_32_bit_offsets(csa):
    """Pages at the end of a pool of more than 2^32 bytes, written by the append and read by both attentions."""
    page, n_pages = 64, 132000   # 4.3 GB of rows
    small = Cache(70, [150, 90], page)
    pages = csa.Pages(2, 3, n_pages=n_pages, page_size=page)
    far = torch.tensor([[n_pages - 1, n_pages - 3, n_pages - 2], [n_pages - 5, 3, -1]], dtype=torch.int32)
    pages.table.copy_(far)
    for b in range(2):
        for j in range(3):
            if small.table[b, j] >= 0 and far[b, j] >= 0:
                pages.kv[far[b, j]] = torch.from_numpy(small.kv[small.table[b, j]]).cuda()
                pages.kv_sc[far[b, j]] = torch.from_numpy(small.kv_sc[small.table[b, j]]).cuda()
    pages.n_tokens.copy_(torch.tensor([150, 90], dtype=torch.int32))
    q, q_pos = queries(1, 2, 1), np.array([[149], [89]], np.int32)
    check(*run_window(csa, pages, q, q_pos, 128, 4), reference(q, q_pos, [(small, True)], 128, 4))
    x = torch.randn((1, D)).to(torch.bfloat16)
    csa.csa2_pages_append(x.cuda(), pages, torch.zeros(1, dtype=torch.int32).cuda(), torch.full((1,), 150, dtype=torch.int32).cuda())
    y, scale = append_reference(x, np.array([150]), None, None, 1e-6, True)
    got = E4M3[pages.kv[n_pages - 2, 150 % page].cpu().numpy()]
    assert (np.abs(got - y[0] / scale[0]) <= 2.0 ** -4 * np.abs(y[0] / scale[0]) + 2.0 ** -10 + 448 * 2.0 ** -18).all()


def test_outputs_only_where_asked(csa):
    """out and lse given by the caller inside larger buffers: the rows around them stay as they were."""
    cache, Q = Cache(80, [90, 300], 64), 3
    q, q_pos = queries(2, 2, Q), tail_positions([90, 300], Q)
    big, bigl = torch.full((2 * Q + 2, H, D), 7.0, dtype=torch.bfloat16).cuda(), torch.full((2 * Q + 2, H), 7.0).cuda()
    run_window(csa, cache, q, q_pos, 128, 4, out=big[1:-1].view(2, Q, H, D))
    want = run_window(csa, cache, q, q_pos, 128, 4)
    csa.csa2_window_attn(q.cuda(), cache.gpu(), torch.from_numpy(q_pos).cuda(), n_sink=4, out=big[1:-1].view(2, Q, H, D),
                         lse=bigl[1:-1].view(2, Q, H))
    assert torch.equal(big[1:-1].view(2, Q, H, D), want[0]) and torch.equal(bigl[1:-1].view(2, Q, H), want[1])
    for t in (big, bigl):
        assert (t[0] == 7).all() and (t[-1] == 7).all()


def test_refusals_on_the_device(csa):
    cache = Cache(81, [90], 64)
    pages = cache.gpu()
    q, qp = queries(2, 1, 1).cuda(), torch.tensor([[89]], dtype=torch.int32).cuda()
    with pytest.raises(ValueError):
        csa.csa2_window_attn(q.cpu(), pages, qp)
    with pytest.raises(ValueError):
        csa.csa2_window_attn(q.half(), pages, qp)
    with pytest.raises(ValueError):
        csa.csa2_window_attn(q, pages, qp.long())
    with pytest.raises(ValueError):
        csa.csa2_window_attn(q[:, :, :8], pages, qp)
    with pytest.raises(ValueError):
        csa.csa2_window_attn(q, pages, torch.tensor([[89], [1]], dtype=torch.int32).cuda())
    with pytest.raises(csa.CSA2Error):
        csa.csa2_window_attn(q, pages, qp, window=0)
    with pytest.raises(csa.CSA2Error):
        csa.csa2_prefix_attn(q.expand(2, 1, H, D).contiguous(), Cache(1, [4, 4]).gpu(), Cache(1, [4, 4]).gpu(), qp.expand(2, 1).contiguous())
    with pytest.raises(ValueError):
        csa.csa2_pages_append(q[0, 0].t(), pages, qp[0], qp[0])
    with pytest.raises(csa.CSA2Error):
        csa.csa2_pages_append(torch.zeros(4, 516, dtype=torch.bfloat16).cuda()[:, :D], pages,
                              torch.zeros(4, dtype=torch.int32).cuda(), torch.zeros(4, dtype=torch.int32).cuda())


def test_timeout_is_reported(csa):
    """A producer that issues no copies (the library's test hook): the waits run out after 2 s, the call ends, the flag is
    set and read, and the next call on the same context is right again."""
    cache = Cache(90, [300, 90], 64)
    q, q_pos = queries(3, 2, 1), tail_positions([300, 90], 1)
    prefix = Cache(91, [700], 64)
    own = Cache(92, [5, 9], 64, pos0=700)
    pq_pos = np.array([[704], [708]], np.int32)
    csa.csa2_flag_status()
    for call in (lambda: csa.csa2_window_attn(q.cuda(), cache.gpu(), torch.from_numpy(q_pos).cuda()),
                 lambda: csa.csa2_prefix_attn(q.cuda(), prefix.gpu(), own.gpu(), torch.from_numpy(pq_pos).cuda())):
        csa.lib().csa2_test_starve_copies(1)
        try:
            call()
            with pytest.raises(csa.CSA2Error, match="TIMEOUT"):
                csa.csa2_flag_status(clear=True)
        finally:
            csa.lib().csa2_test_starve_copies(0)
        csa.csa2_flag_status()
    check(*run_window(csa, cache, q, q_pos, 128, 4), reference(q, q_pos, [(cache, True)], 128, 4))
    check(*run_prefix(csa, prefix, own, q, pq_pos), reference(q, pq_pos, [(prefix, False), (own, True)]))


def test_timeout_of_long_lists(csa):
    """The same where two warpgroups share a query."""
    lens, cache = long_lists(5, 60, 2300, 16)
    q, q_pos = queries(6, 60, 1), tail_positions(lens, 1)
    csa.csa2_flag_status()
    csa.lib().csa2_test_starve_copies(1)
    try:
        csa.csa2_window_attn(q.cuda(), cache.gpu(), torch.from_numpy(q_pos).cuda(), window=2200)
        with pytest.raises(csa.CSA2Error, match="TIMEOUT"):
            csa.csa2_flag_status(clear=True)
    finally:
        csa.lib().csa2_test_starve_copies(0)
    csa.csa2_flag_status()
    check(*run_window(csa, cache, q, q_pos, 2200, 4), reference(q, q_pos, [(cache, True)], 2200, 4))


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
@pytest.mark.parametrize("rope", [False, True])
def test_append_zero_rows(csa, eps, rope):
    """A zero row is stored as zeros of scale 0, without an epsilon too, and reads as a token of logit 0."""
    rows = 37
    x = torch.randn((rows, D), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    x[::4] = 0
    cache = Cache(82, [rows], 8)
    cache.kv_sc[:] = -7.0
    pages = cache.gpu()
    w, f = (torch.arange(D) / D + 0.5).cuda(), inv_freq_table() if rope else None
    pos = torch.arange(rows, dtype=torch.int32).cuda()
    csa.csa2_pages_append(x.cuda(), pages, torch.zeros_like(pos), pos, inv_freq=f, norm_w=w, eps=eps)
    kv, sc = pages.kv.cpu().numpy(), pages.kv_sc.cpu().numpy()
    live = np.arange(rows) % 4 != 0
    y, scale = append_reference(x[live], np.arange(rows)[live], f, w, eps, True)
    for r in range(0, rows, 4):
        assert not E4M3[kv[cache.row(0, r)]].any() and sc[cache.row(0, r)] == 0
    for r, yr, s in zip(np.flatnonzero(live), y, scale):
        at = cache.row(0, int(r))
        assert abs(sc[at] - s) <= 2.0 ** -18 * s
        assert (np.abs(E4M3[kv[at]] - yr / s) <= 2.0 ** -4 * np.abs(yr / s) + 2.0 ** -10 + 448 * 2.0 ** -18).all()
    now = Cache(0, [rows], 8)
    now.kv, now.kv_sc, now.table = kv, sc, cache.table
    q, q_pos = queries(4, 1, 1), np.array([[rows - 1]], np.int32)
    check(*run_window(csa, pages, q, q_pos, 1 << 30, 0), reference(q, q_pos, [(now, True)], 1 << 30, 0))
