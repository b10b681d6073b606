"""The paged attentions where much work is at hand, so that four queries share a CTA: the tests of small calls once
more, with their sequences repeated until that is the case."""
import numpy as np
import pytest
import torch

import test_gpu_pages as base
from test_gpu_pages import csa   # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

small_window, small_prefix = base.run_window, base.run_prefix


def repeated(cache, k):
    import sparse_attention_fp4_quant_b200 as csa
    kv, sc, table, n = (torch.from_numpy(a.copy()) for a in (cache.kv, cache.kv_sc, cache.table, cache.n_tokens))
    return csa.Pages.of(kv.cuda(), sc.cuda(), table.repeat(k, 1).cuda(), n.repeat(k).cuda(), pos0=cache.pos0)


def first_of(result, B):
    """The first copy's results, whose bits every other copy must have."""
    for t in result:
        copies = t.view(-1, B, *t.shape[1:])
        assert torch.equal(copies.nan_to_num(7.0), copies[:1].expand_as(copies).nan_to_num(7.0))
    return tuple(t[:B] for t in result)


@pytest.fixture(autouse=True)
def many(monkeypatch):
    def window(csa, cache, q, q_pos, window, sink, start=None, **kw):
        B, Q = q_pos.shape
        k = 300 // (B * Q) + 1
        r = small_window(csa, repeated(cache, k), q.repeat(k, 1, 1, 1), np.tile(q_pos, (k, 1)), window, sink,
                         None if start is None else start * k, **kw)
        return first_of(r, B)

    def prefix(csa, prefix, own, q, q_pos, **kw):
        B, Q = q_pos.shape
        k = 300 // (B * Q) + 1
        r = small_prefix(csa, prefix, Many(own, k), q.repeat(k, 1, 1, 1), np.tile(q_pos, (k, 1)), **kw)
        return tuple(t[-B:] for t in r)   # blocks of four reach over copies, whose keys are then split otherwise

    class Many:
        def __init__(self, cache, k):
            self.gpu = lambda: repeated(cache, k)

    monkeypatch.setattr(base, "run_window", window)
    monkeypatch.setattr(base, "run_prefix", prefix)


@pytest.mark.parametrize("lens,Q,window,sink,page", [
    ([700, 3], 2, 64, 1, 32), ([90, 400], 3, 33, 0, 8), ([513], 4, 128, 130, 128), ([260, 7, 31], 5, 16, 3, 24),
    ([150], 37, 20, 2, 64), ([97], 97, 2147483647, 0, 16), ([3001, 2999], 2, 1 << 30, 0, 40), ([640], 9, 1, 1, 64),
    ([2100], 7, 2000, 700, 16), ([33, 128, 129, 256], 4, 128, 0, 64)])
def test_window(csa, lens, Q, window, sink, page):
    base.test_window(csa, lens, Q, window, sink, page)


@pytest.mark.parametrize("Q", [2, 4, 11])
def test_window_positions_in_any_order(csa, Q):
    base.test_window_positions_in_any_order(csa, Q)


@pytest.mark.parametrize("Q,page", [(128, 64), (30, 16)])
def test_window_replay(csa, Q, page):
    base.test_window_replay(csa, Q, page)


@pytest.mark.parametrize("Q,window,sink,page", [(2, 100, 3, 64), (3, 40, 0, 16), (6, 130, 17, 8), (40, 77, 1, 64)])
def test_window_never_reads_a_masked_value(csa, Q, window, sink, page):
    base.test_window_never_reads_a_masked_value(csa, Q, window, sink, page)


@pytest.mark.parametrize("Q", [4, 8])
def test_extreme_keys_and_queries(csa, Q):
    base.test_extreme_keys_and_queries(csa, Q)


@pytest.mark.parametrize("Q", [2, 3, 20])
def test_window_table_that_starts_later(csa, Q):
    base.test_window_table_that_starts_later(csa, Q)


@pytest.mark.parametrize("Q,n", [(4, 200), (9, 700)])
def test_a_query_of_nan_or_infinity_keeps_to_itself(csa, Q, n):
    base.test_a_query_of_nan_or_infinity_keeps_to_itself(csa, Q, n)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("ps", [16, 64])
def test_keys_that_a_nan_query_does_not_see(csa, ps, value):
    base.test_keys_that_a_nan_query_does_not_see(csa, ps, value)


def test_zero_queries_do_not_hide_masked_nan(csa):
    base.test_zero_queries_do_not_hide_masked_nan(csa, 4)


def test_positions_up_to_the_last(csa):
    base.test_positions_up_to_the_last(csa, 4)


@pytest.mark.parametrize("B,Q,n_prefix,own", [(1, 1, 700, [5]), (3, 1, 130, [0, 129, 61]), (5, 2, 513, [2, 300, 7, 128, 40]), (2, 7, 64, [7, 200])])
@pytest.mark.parametrize("page", [8, 64])
def test_prefix(csa, B, Q, n_prefix, own, page):
    base.test_prefix(csa, B, Q, n_prefix, own, page)


def test_prefix_masks(csa):
    base.test_prefix_masks(csa)


@pytest.mark.parametrize("page_prefix,page_own", [(64, 16), (8, 128), (24, 40)])
def test_prefix_pages_of_another_size(csa, page_prefix, page_own):
    base.test_prefix_pages_of_another_size(csa, page_prefix, page_own)


def test_prefix_without_own_tokens_or_prefix(csa):
    base.test_prefix_without_own_tokens_or_prefix(csa)


def test_timeout_of_many(csa):
    """The starved copies of the timeout tests, where four queries share a CTA and CTAs walk over items."""
    B, Q = 200, 4
    cache = base.Cache(5, [60] * B, 16)
    q, q_pos = base.queries(6, B, Q), base.tail_positions([60] * B, Q)
    csa.csa2_flag_status()
    csa.lib().csa2_test_starve_copies(1)
    try:
        csa.csa2_window_attn(q.cuda(), cache.gpu(), torch.from_numpy(q_pos).cuda(), window=50)
        with pytest.raises(csa.CSA2Error, match="TIMEOUT"):
            csa.csa2_flag_status(clear=True)
    finally:
        csa.lib().csa2_test_starve_copies(0)
    csa.csa2_flag_status()
    base.check(*small_window(csa, cache, q, q_pos, 50, 4), base.reference(q, q_pos, [(cache, True)], 50, 4))
