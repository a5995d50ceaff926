"""The windowed attentions where keys that every row sees lie between hidden ones, with
test_gpu_window_attn.py's cases and tolerances."""
import numpy as np
import pytest
import torch

from oracle import bf16_to_f64, longctx
from test_gpu_paged_attn import bits, close, host
from test_gpu_window_attn import WindowPrompt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [np.inf, -np.inf])
@pytest.mark.parametrize("sinks", [0, 130])
@pytest.mark.parametrize("q_heads,kv_heads,dim,window", [(4, 1, 64, 100), (10, 2, 128, 110), (16, 1, 64, 125), (1, 1, 128, 200), (2, 1, 64, 90)])
def test_infinities_between_hidden_keys(gpu, q_heads, kv_heads, dim, window, sinks, value):
    """Infinities of V in keys that every row of a pair of tiles sees, in windows of 128 whose ends hide keys, with
    weights that round to zero: rows that see one hold the infinity or NaN in its dimension, the same bits every run,
    and nothing else is changed."""
    L, where = 620, [(j, i % dim) for i, j in enumerate(range(100, 600, 23))]

    def edit(p):
        p.q[..., 0], p.k[..., 0] = bits(np.array([8.0]))[0], 0
        for j, d in where:
            p.v[j, 0, d] = bits(np.array([value]))[0]
            p.k[j, :, 0] = bits(np.array([-15 * np.sqrt(dim)]))[0]
    p = WindowPrompt([L], window, sinks, q_heads, kv_heads, dim, seed=9, edit=edit)
    got = p.result().reshape(L, q_heads, dim)
    hit = np.zeros((L, dim), bool)
    for t in range(L):
        see = set(longctx.seen(t, window, sinks))
        for j, d in where:
            hit[t, d] |= j in see
    special = np.zeros(got.shape, bool)
    special[:, :q_heads // kv_heads] = hit[:, None, :]
    assert (np.isnan(got[special]) | (got[special] == value)).all()
    v = bf16_to_f64(p.v)
    v[~np.isfinite(v)] = 0.0
    o, off = longctx.attend_prompt(bf16_to_f64(p.q), bf16_to_f64(p.k), v, p.starts, window, sinks)
    close(np.where(special, 0, got), np.where(special, 0, o), off)
    first = host(p.out).copy()
    for _ in range(20):
        p.out.fill_(77)
        assert p.run() == 0
        torch.cuda.synchronize()
        assert (host(p.out) == first).all()
