"""The windowed attentions where keys that every row sees lie between hidden ones, with
test_gpu_window_attn.py's cases and tolerances."""
import numpy as np
import pytest
import torch

from oracle import bf16_to_f64, longctx
from test_gpu_paged_attn import bits, close, host
from test_gpu_paged4_attn import Case4
from test_gpu_window_attn import WindowCase, WindowPrompt, check_tokens

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


def forget_hidden(c):
    """Entries of pages that hold nothing but hidden tokens name no page."""
    ps, gone = c.k.shape[3] if isinstance(c, WindowCase) else c.ps, 0
    for i, x in enumerate(c.lens):
        see = set(longctx.seen(x - 1, c.window, c.sinks)) if x else set()
        for j in range(-(-x // ps)):
            if not see & set(range(j * ps, (j + 1) * ps)):
                c.pages[c.ids[i], j] = 1 << 30 if j % 2 else -7
                gone += 1
    assert gone


@pytest.mark.parametrize("new", [True, False])
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("window,sinks", [(20, 0), (70, 4), (33, 17), (130, 65)])
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_hidden_pages_beside_visible_ones(gpu, ps, window, sinks, four, new):
    """Entries between sinks and window may name anything, those in one tile of 64 tokens with a visible page among them."""
    lens, heads = [700, 3, 129, 1283, 410, 64], (8, 2, 128) if ps < 64 else (12, 1, 64)
    if four:
        c = Case4(lens, *heads, ps, window, sinks, seed=ps, new=new)
        forget_hidden(c)
        c.check()
    else:
        c = WindowCase(window, sinks, lens, *heads, ps, seed=ps, new=new, lost=False)
        forget_hidden(c)
        check_tokens(c)
