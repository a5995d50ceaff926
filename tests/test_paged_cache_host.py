"""device.PagedCache and PagedCache4 on the host: which calls each makes."""
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
def test_the_calls_of_a_kind(kind, prefix, attend):
    """They are the class's: a call looks nothing up by its name."""
    for name in ("extend", "fork", "release", "compact", "write", "read"):
        assert getattr(kind, "_" + name) is getattr(abi, prefix + name)
    assert kind._ws_size is getattr(abi, prefix + "workspace_size") and kind._attend_ws_size is getattr(abi, attend + "workspace_size")
    c = kind.alloc(Dims(hidden=64, n_q_heads=4, n_kv_heads=2, head_dim=64, vocab=64), 1, 4, 16, 2, 3, device="cpu")
    assert type(c.pool) is kind._pool and c.ws.numel() == kind._ws_size(c.pool, c.seqs)
