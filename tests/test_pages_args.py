"""The paged cache's entry points refuse invalid arguments on the host, before anything runs (no GPU needed)."""
import ctypes

import pytest

P = ctypes.c_void_p
FAKE = P(0x1000)


@pytest.fixture(scope="module")
def csa():
    from sparse_attention_fp4_quant_b200 import build
    import sparse_attention_fp4_quant_b200 as csa
    build.build()
    return csa


def pages(csa, **kw):
    a = dict(kv=0x1000, kv_sc=0x1000, table=0x1000, n_tokens=0x1000, n_pages=8, page_size=64, B=2, max_pages=4, pos0=0)
    a.update(kw)
    return csa.csa2_pages(**a)


BAD_PAGES = [dict(kv=None), dict(kv_sc=None), dict(table=None), dict(n_tokens=None), dict(kv=0x1008), dict(kv_sc=0x1008), dict(page_size=0),
             dict(page_size=12), dict(page_size=8192), dict(B=0), dict(max_pages=0), dict(n_pages=0), dict(pos0=-1),
             dict(n_pages=1 << 26, page_size=64), dict(max_pages=1 << 25, page_size=64),
             dict(pos0=(1 << 31) - 10)]


@pytest.mark.parametrize("bad", BAD_PAGES)
def test_bad_pages(csa, bad):
    L, pg = csa.lib(), pages(csa, **bad)
    ref = ctypes.byref(pg)
    assert L.csa2_pages_append(FAKE, 512, 4, FAKE, FAKE, None, None, 1e-6, 1, ref, None) == 1
    assert L.csa2_window_attn(FAKE, ref, FAKE, 1, 128, 0, None, 0.04, FAKE, None, FAKE, 1 << 30, None, None) == 1
    good = pages(csa, B=1)
    assert L.csa2_prefix_attn(FAKE, ctypes.byref(good), ref, FAKE, 1, 0.04, FAKE, None, FAKE, 1 << 30, None, None) == 1
    assert L.csa2_prefix_attn(FAKE, ref, ctypes.byref(good), FAKE, 1, 0.04, FAKE, None, FAKE, 1 << 30, None, None) == 1


def test_append_arguments(csa):
    L, pg = csa.lib(), pages(csa)
    ref = ctypes.byref(pg)

    def call(x=FAKE, stride=512, rows=4, seq=FAKE, pos=FAKE, norm=None, eps=1e-6, p=ref):
        return L.csa2_pages_append(x, stride, rows, seq, pos, None, norm, eps, 1, p, None)
    assert call(rows=0) == 0 and call(x=None, seq=None, pos=None, rows=0) == 0
    assert call(rows=-1) == 1
    assert call(x=None) == 1 and call(seq=None) == 1 and call(pos=None) == 1 and call(p=None) == 1
    assert call(x=P(0x1002)) == 1
    assert call(stride=504) == 1 and call(stride=516) == 1
    assert call(norm=P(0x1004)) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1


def test_attention_arguments(csa):
    L, pg, px = csa.lib(), pages(csa), pages(csa, B=1)
    ref, rpx = ctypes.byref(pg), ctypes.byref(px)

    def window(q=FAKE, p=ref, q_pos=FAKE, Q=1, w=128, ns=0, scale=0.04, out=FAKE, ws=FAKE, n=1 << 30):
        return L.csa2_window_attn(q, p, q_pos, Q, w, ns, None, scale, out, None, ws, n, None, None)

    def prefix(q=FAKE, a=rpx, b=ref, q_pos=FAKE, Q=1, scale=0.04, out=FAKE, ws=FAKE, n=1 << 30):
        return L.csa2_prefix_attn(q, a, b, q_pos, Q, scale, out, None, ws, n, None, None)
    for call in (window, prefix):
        assert call(q=None) == 1 and call(q_pos=None) == 1 and call(out=None) == 1 and call(ws=None) == 1
        assert call(q=P(0x1008)) == 1 and call(out=P(0x1008)) == 1 and call(ws=P(0x1008)) == 1
        assert call(Q=0) == 1 and call(Q=40000) == 1
        assert call(scale=0.0) == 1 and call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
        assert call(n=0) == 3
    assert window(w=0) == 1 and window(ns=-1) == 1 and window(p=None) == 1
    assert prefix(a=ref) == 1 and prefix(a=None) == 1 and prefix(b=None) == 1   # a prefix has one table row
    assert L.csa2_flag_status(None, 0, None) == 1


def test_workspace_sizes(csa):
    L = csa.lib()
    for op in (csa.OP_WINDOW_ATTN, csa.OP_PREFIX_ATTN):
        assert L.csa2_workspace_bytes(op, 0, 1, 100, 0, 0) == 0
        for B, Q, cap in ((1, 1, 1), (32, 1, 131072), (1, 4096, 65536), (65535, 1, 1 << 31)):
            assert L.csa2_workspace_bytes(op, B, Q, cap, 0, 0) >= 256
    # a long context is split over the GPU's SMs, no further: the workspace does not grow with it
    a = L.csa2_workspace_bytes(csa.OP_PREFIX_ATTN, 4, 1, 1 << 20, 0, 0)
    assert a == L.csa2_workspace_bytes(csa.OP_PREFIX_ATTN, 4, 1, 1 << 30, 0, 0) < 1 << 27


def test_binding_refuses(csa):
    import torch
    t = dict(kv=torch.zeros(4, 64, 512, dtype=torch.uint8), kv_sc=torch.zeros(4, 64),
             table=torch.zeros(2, 2, dtype=torch.int32), n_tokens=torch.zeros(2, dtype=torch.int32))
    for bad in (dict(kv=torch.zeros(4, 64, 256, dtype=torch.uint8)), dict(kv=torch.zeros(4, 60, 512, dtype=torch.uint8)),
                dict(kv_sc=torch.zeros(4, 32)), dict(kv_sc=torch.zeros(4, 64, dtype=torch.float64)),
                dict(table=torch.zeros(4, dtype=torch.int32)), dict(n_tokens=torch.zeros(3, dtype=torch.int32)),
                dict(table=torch.zeros(2, 4, dtype=torch.int32)[:, ::2])):
        with pytest.raises(ValueError):
            csa.Pages.of(*{**t, **bad}.values())
    with pytest.raises(ValueError):
        csa.Pages.of(*t.values(), pos0=-1)
    csa.Pages.of(*t.values())


@pytest.mark.parametrize("window,n_sink", [(2 ** 32 + 5, 0), (2 ** 31, 0), (128, 2 ** 32), (-2 ** 32 + 5, 4)])
def test_window_beyond_32_bits_is_refused(csa, window, n_sink):
    """Not cut down to some other window."""
    with pytest.raises(ValueError, match="32-bit"):
        csa.csa2_window_attn(None, None, None, window=window, n_sink=n_sink)


def test_workspace_of_sizes_that_no_call_takes(csa):
    """Block counts beyond 32 bits end in a size of zero, tables beyond any in the largest one's."""
    L = csa.lib()
    for op in (csa.OP_WINDOW_ATTN, csa.OP_PREFIX_ATTN):
        for B, Q in ((1 << 18, 1 << 16), (65536, 65536), (2 ** 31 - 1, 2 ** 31 - 1), (1, 65536), (65536, 1), (256, 256)):
            assert L.csa2_workspace_bytes(op, B, Q, 1000, 0, 0) == 0
        for B, Q in ((1, 1), (4, 1), (1, 65535), (65535, 1), (21, 2)):
            assert L.csa2_workspace_bytes(op, B, Q, -5, 0, 0) == L.csa2_workspace_bytes(op, B, Q, 0, 0, 0) >= 256
            top = L.csa2_workspace_bytes(op, B, Q, 1 << 32, 0, 0)
            assert L.csa2_workspace_bytes(op, B, Q, 2 ** 63 - 1, 0, 0) == top >= 256


def test_workspace_of_calls_of_any_shape(csa):
    """The bound that the header gives for a buffer that serves every shape; sizes are not monotone in any argument."""
    L, larger = csa.lib(), 0
    for op in (csa.OP_WINDOW_ATTN, csa.OP_PREFIX_ATTN):
        for B in (*range(1, 40), 61, 74, 75, 148, 149, 296, 297, 512, 4096, 65535):
            for Q in (*range(1, 12), 16, 128, 1017, 4096, 65535):
                if B * Q > 65535:
                    continue
                sizes = [L.csa2_workspace_bytes(op, B, Q, n, 0, 0) for n in (1, 132, 384, 385, 600, 2048, 5000, 131072, 1 << 32)]
                assert 256 <= min(sizes) and max(sizes) <= 256 + max(19474432, 65792 * B * Q)
                larger = max(larger, *sizes)
    assert larger == 256 + 65792 * 65535
    assert L.csa2_workspace_bytes(csa.OP_WINDOW_ATTN, 1, 4096, 1028, 0, 0) == 256
    assert L.csa2_workspace_bytes(csa.OP_WINDOW_ATTN, 1, 1, 1028, 0, 0) > 256
