"""The paged cache's calls as programs make them: from several host threads, between other calls, at the largest sizes."""
import threading

import numpy as np
import pytest
import torch

from pages_common import Cache, check, queries, reference

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


def test_between_index_calls(csa):
    """Index searches of several shapes and paged attentions in turn on one stream: both take tensor memory, and each starts
    while the one before it ends."""
    B, cap = 4, 4096
    g = torch.Generator().manual_seed(5)
    kv = csa.KV(B, cap)
    kv.ik.copy_(torch.randint(0, 256, kv.ik.shape, generator=g, dtype=torch.uint8))
    kv.ik_sc.fill_(0x38)
    kv.n_entries.fill_(cap)
    cache = Cache(3, [1000, 300, 64, 7] * 4, 64)
    pages = cache.gpu()
    index = []
    for Q in (1, 2, 64):
        q = torch.randint(0, 256, (B, Q, 128), generator=g, dtype=torch.uint8).cuda()
        sc, w = torch.full((B, Q, 16), 0x38, dtype=torch.uint8).cuda(), torch.rand((B, Q, 4), generator=g).cuda()
        index.append((q, sc, w, torch.full((B, Q), cap - 1, dtype=torch.int32).cuda()))
    paged = [(queries(Q, 16, Q).cuda(), torch.randint(0, 1000, (16, Q), generator=g, dtype=torch.int32).cuda())
             for Q in (1, 40)]

    def call(k):
        if k % 2:
            q, qp = paged[(k // 2) % 2]
            return csa.csa2_window_attn(q, pages, qp, window=(100, 1 << 30)[(k // 4) % 2], n_sink=4, lse=True)
        q, sc, w, qp = index[(k // 2) % 3]
        return (csa.csa2_index_topk(q, sc, w, kv, qp, 512),)
    want = []
    for k in range(24):   # one at a time
        want.append(call(k))
        torch.cuda.synchronize()
    for _ in range(5):
        got = [call(k) for k in range(24)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    csa.csa2_flag_status()


def test_largest_calls(csa):
    """65,535 queries: one chunk of a prompt, and a batch of single queries whose keys are split (4.3 GB of workspace)."""
    n = 65535
    cache = Cache(4, [n], 128)
    pages, q = cache.gpu(), torch.randn((1, n, 16, 512), generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    qp = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)
    out, lse = csa.csa2_window_attn(q, pages, qp, window=20, n_sink=2, lse=True)
    for lo, hi in ((0, 32768), (32768, n)):   # in parts: the same blocks of four queries
        o, l = csa.csa2_window_attn(q[:, lo:hi], pages, qp[:, lo:hi].contiguous(), window=20, n_sink=2, lse=True)
        assert torch.equal(o, out[:, lo:hi]) and torch.equal(l, lse[:, lo:hi])
    with pytest.raises(csa.CSA2Error):
        csa.csa2_window_attn(torch.cat([q, q[:, :1]], 1), pages, torch.zeros((1, n + 1), dtype=torch.int32, device="cuda"))
    lens, few = [2100, 1, 1999, 130, 0, 2048, 700, 129], 8
    small = Cache(5, lens, 64)
    some, pos = queries(6, few, 1), np.array([[m - 1] for m in lens], np.int32)
    copies = -(-n // few)
    wide = csa.Pages.of(torch.from_numpy(small.kv).cuda(), torch.from_numpy(small.kv_sc).cuda(),
                        torch.from_numpy(small.table).repeat(copies, 1)[:n].contiguous().cuda(),
                        torch.from_numpy(small.n_tokens).repeat(copies)[:n].contiguous().cuda())
    out, lse = csa.csa2_window_attn(some.cuda().repeat(copies, 1, 1, 1)[:n].contiguous(), wide,
                                    torch.from_numpy(pos).repeat(copies, 1)[:n].contiguous().cuda(), window=1 << 30, lse=True)
    check(out[:few], lse[:few], reference(some, pos, [(small, True)]))
    for t in (out, lse):
        full = t[:n // few * few].view(n // few, few, *t.shape[1:])
        assert torch.equal(full, full[:1].expand_as(full)) and torch.equal(t[n // few * few:], t[:n % few])
    csa.csa2_flag_status()


def test_append_of_many_rows(csa):
    """More rows than the grid takes at once many times over, in one call and in parts."""
    n = 400003
    x = torch.randn((n, 512), generator=torch.Generator("cuda").manual_seed(2), device="cuda").bfloat16()
    pos, seq = torch.randperm(n, generator=torch.Generator("cuda").manual_seed(3), device="cuda").int(), torch.zeros(n, dtype=torch.int32, device="cuda")
    whole, parts = (csa.Pages(1, -(-n // 128), page_size=128) for _ in range(2))
    for p in (whole, parts):
        p.table.copy_(torch.randperm(p.n_pages, generator=torch.Generator().manual_seed(4))[None].int())
    csa.csa2_pages_append(x, whole, seq, pos)
    for lo in range(0, n, 99991):
        csa.csa2_pages_append(x[lo:lo + 99991], parts, seq[lo:lo + 99991], pos[lo:lo + 99991])
    assert torch.equal(whole.kv, parts.kv) and torch.equal(whole.kv_sc, parts.kv_sc)
    assert int((whole.kv_sc > 0).sum()) == n
