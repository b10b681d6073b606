"""The paged cache's calls as programs with several host threads make them."""
import threading

import pytest
import torch

from pages_common import Cache, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def csa():
    import sparse_attention_fp4_quant_b200 as csa
    csa.lib()
    return csa


@pytest.mark.parametrize("op", ["append", "window", "prefix"])
def test_first_call_of_a_thread(csa, op):
    """A thread that has not used the device before: its first call is one of these."""
    cache, prefix, own = Cache(90, [300], 64), Cache(91, [700], 64), Cache(92, [9], 64, pos0=700)
    pages, prefix, own = cache.gpu(), prefix.gpu(), own.gpu()
    q, qp = queries(3, 1, 1).cuda(), torch.tensor([[299]], dtype=torch.int32).cuda()
    x, at = queries(4, 1, 1)[0, 0, :1].cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    flat, qp_prefix = qp[0], qp + 409

    def call():
        if op == "append":
            csa.csa2_pages_append(x, pages, at, flat)
            return pages.kv, pages.kv_sc
        if op == "window":
            return csa.csa2_window_attn(q, pages, qp, n_sink=4, lse=True)
        return csa.csa2_prefix_attn(q, prefix, own, qp_prefix, lse=True)
    want = [t.clone() for t in call()]
    if op == "append":
        pages.kv[:], pages.kv_sc[:] = torch.from_numpy(cache.kv).cuda(), torch.from_numpy(cache.kv_sc).cuda()
    torch.cuda.synchronize()
    got = []

    t = threading.Thread(target=lambda: got.append(call()))
    t.start()
    t.join()
    torch.cuda.synchronize()
    csa.csa2_flag_status()
    assert len(got) == 1 and all(torch.equal(a, b) for a, b in zip(got[0], want))


def test_two_threads_on_one_stream(csa):
    """Calls that split their keys, and so join partial results of a workspace, made by two threads on the default stream."""
    n, page = 6000, 64
    caches = [Cache(100 + k, [n, n // 2], page) for k in range(2)]
    pages, qs = [c.gpu() for c in caches], [queries(k, 2, 1).cuda() for k in range(2)]
    qp = torch.tensor([[n - 1], [n // 2 - 1]], dtype=torch.int32).cuda()
    assert csa.csa2_workspace_bytes(csa.OP_WINDOW_ATTN, 2, 1, pages[0].cap, 0) > 256   # split

    def call(k):
        return csa.csa2_window_attn(qs[k], pages[k], qp, window=1 << 30, lse=True)
    want = [call(k) for k in range(2)]
    torch.cuda.synchronize()
    got, start = [[], []], threading.Barrier(2)

    def work(k):
        start.wait()
        for _ in range(300):
            got[k].append(call(k))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    csa.csa2_flag_status()
    for k in range(2):
        assert len(got[k]) == 300
        for out, lse in got[k]:
            assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])
