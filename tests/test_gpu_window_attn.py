"""tv_attend_prompt_window and tv_attend_paged_window against oracle/longctx.py
(fp64): the tolerances of the calls without a window, which
test_gpu_paged_attn.py derives (they hold for any set of keys)."""
import numpy as np
import pytest
import torch

from oracle import bf16_to_f64, longctx
from oracle.paged import attend
from speculative_tree_verify_gb300 import abi
from test_gpu_paged_attn import NAN, Case, bits, close, dev, host, i32
from test_gpu_prompt_attn import Prompt

pytestmark = pytest.mark.gpu

ALL = abi.NO_WINDOW


class WindowPrompt(Prompt):
    def __init__(self, lens, window, sinks, *args, **kw):
        self.window, self.sinks = window, sinks
        super().__init__(lens, *args, **kw)

    def run(self, stream=None, starts=None):
        Hq, Hkv, D = self.dims
        return abi.tv_attend_prompt_window(Hq, Hkv, D, self.window, self.sinks, self.x, self.x[:, Hq * D:], self.x[:, (Hq + Hkv) * D:],
                                           self.width, self.width, self.gstarts if starts is None else starts, len(self.lens),
                                           self.rows, self.out, self.status, stream)

    def want(self):
        return longctx.attend_prompt(bf16_to_f64(self.q), bf16_to_f64(self.k), bf16_to_f64(self.v), self.starts, self.window, self.sinks)

    def check(self):
        got = self.result()
        o, off = self.want()
        used = slice(self.starts[0], self.starts[-1])
        close(got, o[used], off[used])


HEADS = [(4, 2, 64), (5, 1, 128), (2, 2, 128), (1, 1, 64), (24, 1, 128), (128, 1, 64)]


@pytest.mark.parametrize("q_heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 0), (64, 4), (128, 0), (200, 33), (300, 130), (ALL, 0), (ALL, ALL), (5, ALL)])
def test_one_sequence(gpu, q_heads, kv_heads, dim, window, sinks):
    WindowPrompt([421], window, sinks, q_heads, kv_heads, dim, seed=421).check()


@pytest.mark.parametrize("length", [1, 2, 127, 128, 129, 256, 257, 700])
@pytest.mark.parametrize("window,sinks", [(127, 0), (128, 1), (129, 15), (130, 16), (60, 17), (256, 129)])
def test_edges(gpu, length, window, sinks):
    """Windows and sinks that end at, before and behind a tile's, a step's and the window's own border."""
    WindowPrompt([length], window, sinks, 8, 2, 64, seed=length).check()
    WindowPrompt([length], window, sinks, 2, 1, 128, seed=length + 1).check()


@pytest.mark.parametrize("q_heads,kv_heads,dim", HEADS[:5])
@pytest.mark.parametrize("window,sinks", [(40, 4), (250, 40)])
def test_packed_with_nan_around(gpu, q_heads, kv_heads, dim, window, sinks):
    WindowPrompt([3, 0, 127, 128, 1, 255, 0, 60, 300, 513], window, sinks, q_heads, kv_heads, dim, seed=q_heads, before=5, behind=40, pad=8).check()


@pytest.mark.parametrize("q_heads,kv_heads,dim,window,sinks", [(10, 2, 128, 300, 4), (4, 4, 64, 128, 0), (10, 2, 64, 513, 130), (48, 2, 64, 77, 8)])
def test_more_places_than_blocks(gpu, q_heads, kv_heads, dim, window, sinks):
    tokens = 128 // (q_heads // kv_heads)
    lens = [1500, tokens, 900, 3 * tokens, 1, 700, 2 * tokens + 1, 1111, 130, 5 * tokens - 1, 600, 257, 1, 800]
    WindowPrompt(lens if dim == 128 or q_heads > 4 else lens * 3, window, sinks, q_heads, kv_heads, dim, seed=dim + q_heads).check()


@pytest.mark.parametrize("dim", [64, 128])
def test_a_window_of_everything_is_no_window(gpu, dim):
    """The same rows, and the same but for the order of sums as the call without a window."""
    a, b = Prompt([700, 33], 4, 2, dim, seed=6), WindowPrompt([700, 33], ALL, 0, 4, 2, dim, seed=6)
    assert np.abs(a.result() - b.result()).max() <= 2.0 ** -7 * np.abs(a.result()).max()


def test_large_scores_and_loud_sinks(gpu):
    """Scores that move the offsets; sinks that outweigh the window, which the last keys looked at are."""
    WindowPrompt([700, 130], 100, 4, 4, 2, 64, seed=3, scale=30.0).check()

    def edit(p):
        p.k[p.starts[0]:p.starts[0] + 3] = bits(np.full((3, *p.k.shape[1:]), 3.0))
        p.q[:] = bits(np.abs(bf16_to_f64(p.q)))
    WindowPrompt([900], 64, 3, 8, 2, 128, seed=4, edit=edit).check()


def test_quiet_first_keys(gpu):
    """Rows whose window scores 200 powers of two below what is hidden from them."""
    def edit(p):
        p.q[:], p.k[:] = bits(np.ones(p.q.shape)), bits(np.zeros(p.k.shape))
        p.k[:, :, 0] = bits(np.repeat(np.linspace(1500, -1500, p.rows)[:, None], p.k.shape[1], 1))
    WindowPrompt([800], 90, 0, 4, 2, 64, seed=5, edit=edit).check()


@pytest.mark.parametrize("value,to", [(np.inf, np.inf), (-np.inf, -np.inf), (np.nan, np.nan)])
@pytest.mark.parametrize("q_heads,kv_heads,dim,window,sinks", [(4, 2, 64, 50, 3), (5, 1, 128, 200, 20), (1, 1, 64, 100, 0), (2, 1, 128, 30, 130)])
def test_what_is_hidden_does_not_reach_a_row(gpu, q_heads, kv_heads, dim, window, sinks, value, to):
    """V that is not finite is the result of the rows that see it, in its dimension, and of no other."""
    L, where = 460, [(0, 1), (2, 5), (19, 7), (25, 3), (131, dim - 1), (260, 0), (261, 0), (400, 9), (459, 2)]

    def edit(p):
        for j, d in where:
            p.v[j, 0, d] = bits(np.array([value]))[0] if not np.isnan(value) else NAN
    p = WindowPrompt([L], window, sinks, q_heads, kv_heads, dim, seed=9, edit=edit)
    got = p.result().reshape(L, q_heads, dim)
    v = bf16_to_f64(p.v)
    hit = np.zeros((L, dim), bool)
    for t in range(L):
        see = set(longctx.seen(t, window, sinks))
        for j, d in where:
            hit[t, d] |= j in see
    v[~np.isfinite(v)] = 0.0
    o, off = longctx.attend_prompt(bf16_to_f64(p.q), bf16_to_f64(p.k), v, p.starts, window, sinks)
    group = q_heads // kv_heads
    special = np.zeros(got.shape, bool)
    special[:, :group] = hit[:, None, :]
    assert np.array_equal(got[special], np.full(special.sum(), to), equal_nan=True)
    # the others' tolerance may count what the special ones' V would have been: they hold none of it
    close(np.where(special, 0, got), np.where(special, 0, o), off)


def test_hidden_keys_may_be_anything(gpu):
    """NaN and infinities in K and V between the sinks and every row's window: rows behind them are as without."""
    def run(poison):
        def edit(p):
            if poison:
                p.k[4:300], p.v[4:300] = NAN, 0x7F80
        p = WindowPrompt([600], 100, 4, 8, 2, 128, seed=10, edit=edit)
        return p.result()[400:]
    a, b = run(True), run(False)
    assert np.isfinite(a).all() and (a == b).all()


def test_prompt_refusals_and_streams(gpu):
    p = WindowPrompt([300, 40], 64, 4, 4, 2, 64, seed=12)
    assert p.run(starts=i32([0, 400, 340])) == 0
    torch.cuda.synchronize()
    assert abi.STATUS[int(p.status.item())] == "TV_E_SEQ" and (host(p.out) == 77).all()
    p.status.zero_()
    q = WindowPrompt([301, 41], 80, 0, 4, 2, 64, seed=13)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    assert p.run(streams[0]) == 0 and q.run(streams[1]) == 0
    torch.cuda.synchronize()
    p.check(), q.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert p.run(torch.cuda.current_stream()) == 0
    p.out.fill_(77)
    g.replay()
    torch.cuda.synchronize()
    first = host(p.out).copy()
    p.check()
    assert (host(p.out) == first).all()


# ---- single tokens ------------------------------------------------------------------
class WindowCase(Case):
    """As Case; what the new token does not see is NaN or, whole pages of it, no page at all."""

    def __init__(self, window, sinks, *args, lost=True, **kw):
        self.window, self.sinks = window, sinks
        super().__init__(*args, **kw)
        ps = self.k.shape[3]
        for i, x in enumerate(self.lens):
            see = set(longctx.seen(x - 1, window, sinks)) if x else set()
            for j in range(-(-x // ps)):
                p = self.pages[self.ids[i], j]
                hidden = [t for t in range(j * ps, min(x, (j + 1) * ps)) if t not in see]
                for t in hidden:
                    self.k[self.layer, p, :, t % ps], self.v[self.layer, p, :, t % ps] = NAN, 0x7F80
                # sinks and window are loaded in tiles of 64: pages that share none with either
                if lost and hidden and all(abs(t // 64 - s // 64) > 0 for s in (min(see), *see) for t in (j * ps, j * ps + ps - 1)):
                    self.pages[self.ids[i], j] = 1 << 30


def run_tokens(c, heads=None, stream=None):
    """The case through tv_attend_paged_window: (out, k, v) bits."""
    q_heads, kv_heads, dim = c.dims
    k, v, qkv = dev(c.k), dev(c.v), dev(c.qkv)
    lens = np.zeros(len(c.pages), np.int32)
    for i, x in enumerate(c.lens):
        lens[c.ids[i]] = x
    refs, pages, glens, ids, status = i32(np.ones(c.k.shape[1])), i32(c.pages), i32(lens), i32(c.ids), i32([0])
    pool = abi.TvPool(k.data_ptr(), v.data_ptr(), refs.data_ptr(), *c.k.shape)
    seqs = abi.TvSeqs(pages.data_ptr(), glens.data_ptr(), *c.pages.shape)
    n = len(c.lens)
    size = abi.tv_attend_paged_workspace_size(pool, q_heads, n)
    ws, out = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.full((n, q_heads, dim), 77, dtype=torch.int16, device="cuda")
    kn, vn = (qkv[:, (q_heads + i * kv_heads) * dim:] for i in (0, 1)) if c.new else (None, None)
    assert abi.tv_attend_paged_window(pool, c.layer, seqs, ids, n, q_heads, c.window, c.sinks, qkv, c.width, kn, vn, c.width, out, ws, size,
                                      status, stream) == 0
    torch.cuda.synchronize()
    assert int(status.item()) == 0, abi.STATUS.get(int(status.item()))
    return host(out), host(k), host(v)


def check_tokens(c):
    out, k, v = run_tokens(c)
    q = bf16_to_f64(c.q)
    for i, x in enumerate(c.lens):
        see = longctx.seen(x - 1, c.window, c.sinks) if x else []
        o, off = attend(q[i], bf16_to_f64(c.kv[i][0][see]), bf16_to_f64(c.kv[i][1][see]), True)
        close(bf16_to_f64(out[i]), o, off, f"sequence {i} of {x} tokens")
        if x and c.new:   # the new rows are stored
            ps = c.k.shape[3]
            p = c.pages[c.ids[i], (x - 1) // ps]
            assert (k[c.layer, p, :, (x - 1) % ps] == c.kv[i][0][-1]).all() and (v[c.layer, p, :, (x - 1) % ps] == c.kv[i][1][-1]).all()


WINDOWS = [(1, 0), (1, 1), (16, 0), (63, 4), (64, 64), (65, 16), (200, 5), (1000, 130), (ALL, 0), (7, ALL)]


@pytest.mark.parametrize("new", [True, False])
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("q_heads,kv_heads,dim,ps", [(4, 2, 64, 16), (10, 2, 128, 32), (24, 1, 128, 64), (3, 1, 64, 128)])
def test_tokens(gpu, q_heads, kv_heads, dim, ps, window, sinks, new):
    check_tokens(WindowCase(window, sinks, [1, 0, 2, 64, 65, 130, 700, 1283, 3], q_heads, kv_heads, dim, ps, layers=2, layer=1, seed=window % 97, new=new))


@pytest.mark.parametrize("window,sinks", [(300, 4), (2000, 0)])
@pytest.mark.parametrize("lens", [[9001], [20011, 1, 5000], [700] * 40, [5, 900, 64] * 60])
def test_long_and_many(gpu, lens, window, sinks):
    check_tokens(WindowCase(window, sinks, lens, 8, 2, 128, 16, seed=len(lens)))


@pytest.mark.parametrize("q_heads,kv_heads,dim", [(24, 1, 64), (40, 2, 128), (16, 16, 64)])
def test_many_short_runs(gpu, q_heads, kv_heads, dim):
    """More runs a block than places for their queries."""
    rng = np.random.default_rng(3)
    check_tokens(WindowCase(70, 2, rng.integers(0, 200, 900).tolist(), q_heads, kv_heads, dim, 16, seed=4, lost=False))


@pytest.mark.parametrize("value", [np.inf, -np.inf])
def test_an_infinity_that_is_seen(gpu, value):
    """In V of a sink, of the window's first token and of the last one."""
    c = WindowCase(100, 4, [500, 3], 4, 2, 64, 16, seed=8)
    bit = bits(np.array([value]))[0]
    for t, d in ((0, 3), (3, 7), (400, 20), (499, 33)):
        c.kv[0][1][t, 1, d] = bit
        p = c.pages[c.ids[0], t // 16]
        c.v[0, p, 1, t % 16, d] = bit
    c.qkv[0, (4 + 2 + 1) * 64 + 33] = bit
    out, _, _ = run_tokens(c)
    got = bf16_to_f64(out[0])
    assert (got[2:, [3, 7, 20, 33]] == value).all()
    rest = [d for d in range(64) if d not in (3, 7, 20, 33)]
    assert np.isfinite(got[:2]).all() and np.isfinite(got[2:, rest]).all()


def test_the_same_bits_twice(gpu):
    c = WindowCase(300, 4, [3000, 17, 900], 40, 8, 128, 16, seed=9)
    a, b = run_tokens(c), run_tokens(c)
    assert all((x == y).all() for x, y in zip(a, b))


@pytest.mark.parametrize("four", [False, True])
def test_the_longest_length(gpu, four):
    """2^31 - 16 tokens, of which a window and the sinks are seen; the entries of all pages between name none."""
    ps, D, n_pages, window, sinks = 16, 64, 2 ** 27 - 1, 100, 20
    rng = np.random.default_rng(14)
    k, v = (bits(rng.standard_normal((12, ps, D))) for _ in range(2))
    q = bits(rng.standard_normal((1, 4, D)))
    table = torch.full((1, n_pages), 1 << 30, dtype=torch.int32, device="cuda")
    L = n_pages * ps
    # sinks and window are looked up in tiles of 64 tokens: pages 0 .. 3, and the last 8 (the window lies in 7 of them)
    table[0, :4] = i32([0, 1, 2, 3])
    table[0, -8:] = i32([4, 5, 6, 7, 8, 9, 10, 11])
    refs, lens, ids, st = i32(np.ones(12)), i32([L]), i32([0]), i32([0])
    out, gq = torch.zeros(1, 4, D, dtype=torch.int16, device="cuda"), dev(q)
    seqs = abi.TvSeqs(table.data_ptr(), lens.data_ptr(), 1, n_pages)
    if four:
        raw = [np.zeros((1, 12, 1, 1, 9 * D), np.uint8) for _ in range(2)]
        rows, held = longctx.Pages4(*raw, ps, D), []
        for name, x in zip("kv", (k, v)):
            codes, scales = longctx.quantise(x)
            held.append(longctx.stands_for(codes, scales))
            for p in range(12):
                for t in range(ps):
                    rows.put(name, 0, p, t, codes[p, t][None], scales[p, t][None])
        gk, gv = (torch.from_numpy(x).cuda() for x in raw)
        pool = abi.TvPool4(gk.data_ptr(), gv.data_ptr(), refs.data_ptr(), 1, 12, 1, ps, D)
        size, call = abi.tv_attend_paged4_workspace_size(pool, 4, 1), abi.tv_attend_paged4
    else:
        held, gk, gv = [bf16_to_f64(k), bf16_to_f64(v)], dev(k), dev(v)
        pool = abi.TvPool(gk.data_ptr(), gv.data_ptr(), refs.data_ptr(), 1, 12, 1, ps, D)
        size, call = abi.tv_attend_paged_workspace_size(pool, 4, 1), abi.tv_attend_paged_window
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert call(pool, 0, seqs, ids, 1, 4, window, sinks, gq, 4 * D, None, None, 0, out, ws, size, st) == 0
    assert int(st.item()) == 0
    kk, vv = (np.concatenate([x.reshape(-1, 1, D)[:sinks], x.reshape(-1, 1, D)[-window:]]) for x in held)
    o, off = attend(bf16_to_f64(q[0]), kk, vv, True)
    # 4 bits: 2^-11 of sum w |v| more, which is at most |o| and the spread together
    close(bf16_to_f64(host(out))[0], o, off + (2.0 ** -3 * (np.abs(o) + off) if four else 0))
