"""The Python binding of the paged cache, on the host alone: a stand-in for the library looks at what it is handed."""
import threading
import time
import weakref

import pytest
import torch

import sparse_attention_fp4_quant_b200 as csa


class Rows(torch.Tensor):
    """Queries that note each tensor made from them."""

    made = []

    def new_empty_strided(self, *args, **kw):
        t = super().new_empty_strided(*args, **kw)
        Rows.made.append((t.dtype, t.data_ptr(), weakref.ref(t)))
        return t


class Library:
    """Notes whether the workspace that it is handed (its argument number `at`) is held by anyone."""

    def __init__(self):
        self.held = []

    def csa2_workspace_bytes(self, *args):
        return 1 << 16

    def _look(self, address):
        self.held.append([ref() is not None for dtype, ptr, ref in Rows.made if dtype == torch.uint8 and ptr == address])
        return 0

    def csa2_window_attn(self, *args):
        return self._look(args[10])

    def csa2_prefix_attn(self, *args):
        return self._look(args[8])


@pytest.fixture
def host(monkeypatch):
    """The binding with tensors of the host and no device."""
    library = Library()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(csa, "lib", lambda: library)
    monkeypatch.setattr(csa, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(csa, "_flag", lambda dev: 0x1000)
    monkeypatch.setattr(csa, "_ws_bytes", {})
    monkeypatch.setattr(Rows, "made", [])
    return library


@pytest.mark.parametrize("lse", [False, True])
@pytest.mark.parametrize("call", ["window", "prefix"])
def test_workspace_is_held_during_the_call(host, call, lse):
    """The call makes several launches without the interpreter's lock: another thread's allocations must not get the
    workspace before all of them are on the stream."""
    pages, prefix = csa.Pages(2, 40, device="cpu"), csa.Pages(1, 40, device="cpu")
    q = torch.zeros((2, 1, csa.H, csa.D), dtype=torch.bfloat16).as_subclass(Rows)
    q_pos = torch.zeros((2, 1), dtype=torch.int32)
    if call == "window":
        csa.csa2_window_attn(q, pages, q_pos, window=2000, lse=lse)
    else:
        csa.csa2_prefix_attn(q, prefix, pages, q_pos, lse=lse)
    assert host.held == [[True]]
    assert [ref() for dtype, ptr, ref in Rows.made if dtype == torch.uint8] == [None]   # and by nobody after it


def test_one_flag_for_all_threads(monkeypatch):
    """Threads whose first calls come together share one flag, which stays: the kernels keep its address."""
    made = []

    def zeros(*args, **kw):
        made.append(torch.ones(64, dtype=torch.int32))
        time.sleep(0.05)   # the other threads come past meanwhile
        return made[-1]

    class Stream:
        def synchronize(self):
            pass
    monkeypatch.setattr(csa, "_flags", {})
    monkeypatch.setattr(torch, "zeros", zeros)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    got, start = [], threading.Barrier(4)

    def work():
        start.wait()
        got.append(csa._flag(0))
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(made) == 1 and got == [made[0].data_ptr()] * 4 and csa._flag(0) == got[0]
