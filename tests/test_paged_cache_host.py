"""device.PagedCache and PagedCache4 on the host: which calls each makes."""
import ctypes

import pytest
import torch

from speculative_tree_verify_gb300 import abi, build
from speculative_tree_verify_gb300.device import PagedCache, PagedCache4
from speculative_tree_verify_gb300.synth import Dims


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return abi.load()


@pytest.mark.parametrize("kind,prefix,attend", [(PagedCache, "tv_pages_", "tv_attend_paged_"), (PagedCache4, "tv_pages4_", "tv_attend_paged4_")])
def test_the_calls_of_a_kind(kind, prefix, attend, monkeypatch):
    """Their names are the class's: no call puts one together."""
    for name in ("extend", "fork", "release", "compact", "write", "read"):
        assert getattr(kind, "_" + name) == prefix + name
    assert (kind._ws_size, kind._attend_ws_size) == (prefix + "workspace_size", attend + "workspace_size")
    c = kind.alloc(Dims(hidden=64, n_q_heads=4, n_kv_heads=2, head_dim=64, vocab=64), 1, 4, 16, 2, 3, device="cpu")
    assert type(c.pool) is kind._pool and c.ws.numel() == getattr(abi, kind._ws_size)(c.pool, c.seqs)
    got = []
    for name in ("extend", "fork", "release", "compact", "write", "read"):
        for x in ("tv_pages_", "tv_pages4_"):
            monkeypatch.setattr(abi, x + name, lambda *a, name=x + name: got.append(name) or 0)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    rows, caches = torch.zeros(3, 8 * 64, dtype=torch.bfloat16), torch.zeros(2, 5, 64, dtype=torch.bfloat16)
    c.extend(i32(0), i32(3)), c.fork(i32(0), i32(1)), c.release(i32(0), i32(0)), c.compact(i32(0, 0, 0, 0), i32(0))
    c.write(0, i32(0), i32(0), i32(0, 3), rows), c.read_into(0, i32(0), i32(0), i32(0, 3), 3, caches, caches)
    c.write_from(0, i32(0), i32(0), i32(0, 3), 3, caches, caches)
    assert got == [prefix + x for x in ("extend", "fork", "release", "compact", "write", "read", "write")]


@pytest.mark.parametrize("name", ["tv_attend_prompt_window", "tv_attend_paged_window", "tv_attend_paged4"])
def test_windows_that_no_int_holds(name, monkeypatch):
    """A window of 2^32 + 5 hides no more than one of 2^31 - 1, and sinks of as many are all rows."""
    got = []

    class Lib:
        def __getattr__(self, _):
            return lambda *a: got.append([ctypes.c_int(x).value for x in a if type(x) is int]) or 0

    monkeypatch.setattr(abi, "load", Lib)
    F = 0x10000
    pool, seqs = (abi.TvPool4 if "4" in name else abi.TvPool)(), abi.TvSeqs()
    for window, sinks, want in (((1 << 32) + 5, 1 << 32, [abi.NO_WINDOW, abi.NO_WINDOW]), (7, 3, [7, 3]), (-(1 << 33), -1, [-(1 << 31), -1])):
        if name == "tv_attend_prompt_window":
            abi.tv_attend_prompt_window(4, 2, 64, window, sinks, F, F, F, 512, 512, F, 2, 9, F, F)
            assert got.pop()[3:5] == want
        else:
            getattr(abi, name)(pool, 0, seqs, F, 3, 4, window, sinks, F, 512, F, F, 512, F, F, 1 << 30, F)
            assert got.pop()[4:6] == want


def test_contexts_that_no_int_holds():
    for ctx in ((1 << 32) + 8192, 1 << 31, -1):
        with pytest.raises(ValueError, match="ARG"):
            abi.tv_rope_init(64, scaling=abi.TV_ROPE_BLEND, factor=2.0, original_ctx=ctx)
