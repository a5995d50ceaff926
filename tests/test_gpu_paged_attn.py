"""tv_attend_paged against oracle/paged.py (fp64).

Tolerance, per element: with weights w and result o, P rounded to bf16 moves
every weight by at most 2^-8 of itself, in the sum and the products alike, so
the result by at most 2^-8 A, A = sum_j w_j |v_j - o|.  fp32 scores (128
products, each within 2^-24 of sum |q||k|, below 100 here) and the SFU's
exponential move a weight by less than 1e-3 of itself.  The result is rounded
to bf16 once, 2^-8 of its size (and of the error's).  fp32 sums of at most
32768 terms, joined pairwise over warps and CTAs: below 2^-10 A + 2^-16 |o|."""
import numpy as np
import pytest
import torch

from oracle import bf16_to_f64
from oracle.paged import attend
from speculative_tree_verify_gb300 import abi

pytestmark = pytest.mark.gpu

NAN = 0x7FC0


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def bits(x):
    """fp32 values rounded to bf16, as bit patterns."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x).view(np.int16)).cuda()


def host(t):
    return t.cpu().numpy().view(np.uint16)


def close(got, o, off, what=""):
    err = np.abs(got - o)
    tol = 2.0 ** -8 * np.abs(o) * (1 + 2.0 ** -7) + (2.0 ** -8 + 1e-3 + 2.0 ** -10) * (1 + 2.0 ** -7) * off + 1e-30
    assert np.isfinite(got).all(), what
    assert (err <= tol).all(), f"{what}: worst {np.max(err / tol):.3f} of the tolerance"


class Case:
    """A pool whose every slot outside the sequences is NaN; sequences of random pages."""

    def __init__(self, lens, q_heads, kv_heads, dim, ps, layers=1, layer=0, seed=0, new=True, scale=1.0, unlisted=2, pad=0):
        rng = np.random.default_rng(seed)
        self.lens, self.dims, self.layer, self.new = lens, (q_heads, kv_heads, dim), layer, new
        n = len(lens)
        need = [-(-x // ps) for x in lens]
        n_pages = sum(need) + 3
        self.k = np.full((layers, n_pages, kv_heads, ps, dim), NAN, np.uint16)
        self.v = self.k.copy()
        places, at = rng.permutation(n_pages), 0
        rows = rng.permutation(n + unlisted)
        self.ids = rows[:n].tolist()
        self.pages = np.full((n + unlisted, max(1, max(need))), -3, np.int32)
        all_lens = np.zeros(n + unlisted, np.int32)
        self.kv = []
        for i, x in enumerate(lens):
            self.pages[self.ids[i], :need[i]] = places[at:at + need[i]]
            at += need[i]
            all_lens[self.ids[i]] = x
            kv = [bits(rng.standard_normal((x, kv_heads, dim))) for _ in range(2)]
            self.kv.append(kv)
            for t in range(x - (1 if new else 0)):   # the last token's slot waits for the new rows
                p = self.pages[self.ids[i], t // ps]
                self.k[layer, p, :, t % ps], self.v[layer, p, :, t % ps] = kv[0][t], kv[1][t]
        self.width = (q_heads + 2 * kv_heads) * dim + pad
        self.qkv = np.full((n, self.width), NAN, np.uint16)
        self.q = bits(rng.standard_normal((n, q_heads, dim)) * scale)
        self.qkv[:, :q_heads * dim] = self.q.reshape(n, -1)
        for i, x in enumerate(lens):
            if x:
                self.qkv[i, q_heads * dim:(q_heads + kv_heads) * dim] = self.kv[i][0][-1].reshape(-1)
                self.qkv[i, (q_heads + kv_heads) * dim:(q_heads + 2 * kv_heads) * dim] = self.kv[i][1][-1].reshape(-1)
        self.gk, self.gv, self.gq = dev(self.k), dev(self.v), dev(self.qkv)
        self.refs, self.gpages, self.glens = torch.ones(n_pages, dtype=torch.int32, device="cuda"), i32(self.pages), i32(all_lens)
        self.pool = abi.TvPool(self.gk.data_ptr(), self.gv.data_ptr(), self.refs.data_ptr(), layers, n_pages, kv_heads, ps, dim)
        self.seqs = abi.TvSeqs(self.gpages.data_ptr(), self.glens.data_ptr(), n + unlisted, self.pages.shape[1])
        self.gids, self.status = i32(self.ids), i32([0])
        self.out = torch.full((n + 1, q_heads, dim), 77, dtype=torch.int16, device="cuda")
        self.wsb = abi.tv_attend_paged_workspace_size(self.pool, q_heads, n)
        self.ws = torch.full((self.wsb,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN to whoever reads what it did not write

    def run(self, stream=None, ids=None, n=None):
        Hq, Hkv, D = self.dims
        k, v = (self.gq[:, Hq * D:], self.gq[:, (Hq + Hkv) * D:]) if self.new else (None, None)
        return abi.tv_attend_paged(self.pool, self.layer, self.seqs, self.gids if ids is None else ids, n or len(self.lens), Hq, self.gq,
                                   self.width, k, v, self.width, self.out, self.ws, self.wsb, self.status, stream)

    def check(self):
        assert self.run() == 0
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0, abi.STATUS.get(int(self.status.item()))
        got = bf16_to_f64(host(self.out))
        for i, x in enumerate(self.lens):
            o, off = attend(bf16_to_f64(self.q[i]), bf16_to_f64(self.kv[i][0]), bf16_to_f64(self.kv[i][1]), True)
            close(got[i], o, off, f"sequence {i} of length {x}")
        assert (host(self.out)[-1] == 77).all()          # the row behind the last sequence
        k, v, ps = self.k.copy(), self.v.copy(), self.pool.page_size
        for i, x in enumerate(self.lens):
            if x and self.new:
                p, s = self.pages[self.ids[i], (x - 1) // ps], (x - 1) % ps
                k[self.layer, p, :, s], v[self.layer, p, :, s] = self.kv[i][0][-1], self.kv[i][1][-1]
        assert np.array_equal(host(self.gk), k) and np.array_equal(host(self.gv), v)   # the new rows, and nothing else


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 0, 255]


@pytest.mark.parametrize("new", [True, False])
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(4, 2, 64), (40, 8, 128), (8, 8, 128), (24, 1, 128), (33, 1, 64), (16, 1, 64)])
def test_lengths_and_heads(gpu, q_heads, kv_heads, dim, new):
    Case(EDGES, q_heads, kv_heads, dim, 16, layers=2, layer=1, seed=q_heads, new=new, pad=8).check()


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
def test_page_sizes(gpu, ps, dim):
    Case(EDGES + [3 * ps - 1, 3 * ps, 3 * ps + 1], 8, 2, dim, ps, seed=ps).check()


@pytest.mark.parametrize("lens", [[1], [7], [64 * 9], [20011], [1, 9001, 3, 1], [700] * 40, [5] * 33 + [900], [3, 0, 70] * 230, [1, 2] * 1024],
                         ids=lambda x: f"{len(x)} of {x[0]}")
def test_long_short_and_many(gpu, lens):
    Case(lens, 8, 2, 128, 32, seed=len(lens)).check()


@pytest.mark.parametrize("dim,ps", [(128, 64), (64, 16)])
def test_many_tiles_a_cta(gpu, dim, ps):
    """Some thirty tiles a CTA: the ring of stages goes round often.  Every run gives the same bits."""
    c = Case([40001, 5], 16, 8, dim, ps, new=False)
    c.check()
    first = host(c.out).copy()
    for _ in range(200):
        assert c.run() == 0
    assert np.array_equal(host(c.out), first) and int(c.status.item()) == 0


def test_large_scores_move_the_offsets(gpu):
    """Scores of some hundreds, rising along the sequence: every offset moves, small weights vanish."""
    c = Case([333, 1000], 8, 2, 64, 16, new=False, scale=30.0)
    c.check()


def test_equal_values_pass_through(gpu):
    """All V rows equal: the result is that row exactly, whatever the weights."""
    c = Case([501], 4, 2, 64, 16, new=False)
    row = bits(np.random.default_rng(3).standard_normal((2, 64)))
    for t in range(501):
        c.v[0, c.pages[c.ids[0], t // 16], :, t % 16] = row
    c.gv.copy_(dev(c.v))
    assert c.run() == 0
    got = host(c.out)[0]
    a, b = bf16_to_f64(got), bf16_to_f64(np.repeat(row, 2, axis=0))
    assert (np.abs(a - b) <= 2.0 ** -8 * np.abs(b)).all()   # one rounding of a sum that is right to 2^-16


def test_a_nan_stays_in_its_column(gpu):
    c = Case([100, 100], 4, 2, 64, 16, new=False)
    c.v[0, c.pages[c.ids[0], 2], 1, 5, 9] = NAN       # token 37, KV head 1, dimension 9
    c.gv.copy_(dev(c.v))
    assert c.run() == 0
    bad = np.isnan(bf16_to_f64(host(c.out)[:2]))
    want = np.zeros_like(bad)
    want[0, 2:, 9] = True
    assert np.array_equal(bad, want)


def test_rows_past_two_to_the_31(gpu):
    """The last pages of a pool of more than 2^31 values."""
    n_pages, ps, D = 2 ** 31 // (16 * 64) + 5000, 16, 64
    k, v = (torch.zeros(n_pages, ps, D, dtype=torch.int16, device="cuda") for _ in range(2))
    rng = np.random.default_rng(1)
    pages = [n_pages - 1, n_pages - 4000, 3]
    kk, vv = (bits(rng.standard_normal((40, 1, D))) for _ in range(2))
    for x, src in ((k, kk), (v, vv)):
        for t in range(39):
            x[pages[t // ps], t % ps] = dev(src[t, 0])
    q = bits(rng.standard_normal((1, 2, D)))
    refs, table, lens = torch.ones(n_pages, dtype=torch.int32, device="cuda"), i32([pages]), i32([40])
    pool, seqs = abi.TvPool(k.data_ptr(), v.data_ptr(), refs.data_ptr(), 1, n_pages, 1, ps, D), abi.TvSeqs(table.data_ptr(), lens.data_ptr(), 1, 3)
    out, st = torch.zeros(1, 2, D, dtype=torch.int16, device="cuda"), i32([0])
    wsb = abi.tv_attend_paged_workspace_size(pool, 2, 1)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    qkv = dev(np.concatenate([q.reshape(-1), kk[-1].reshape(-1), vv[-1].reshape(-1)]))
    assert abi.tv_attend_paged(pool, 0, seqs, i32([0]), 1, 2, qkv, 128, qkv[128:], qkv[192:], 64, out, ws, wsb, st) == 0
    assert int(st.item()) == 0
    o, off = attend(bf16_to_f64(q[0]), bf16_to_f64(kk), bf16_to_f64(vv), True)
    close(bf16_to_f64(host(out))[0], o, off)
    assert np.array_equal(host(k[3, 7]), kk[39, 0]) and np.array_equal(host(v[3, 7]), vv[39, 0])


def test_the_longest_length(gpu):
    """2^31 - 16 tokens: a table row that names one page over and over, but for its last place.

    A CTA adds up 2^24 / 148 tiles or fewer, two products each, and a sum that drops what lies below its
    last place loses at most 2^-23 of itself a product: 2^18 2^-23 = 2^-5 of sum w |v|, and half of that
    of the denominator.  The other page's 16 tokens weigh less than 2^-20 (scores differ by less than 4)."""
    ps, D, n_pages = 16, 64, 2 ** 27 - 1
    rng = np.random.default_rng(2)
    k, v = (bits(rng.standard_normal((2, ps, D)) / 8) for _ in range(2))
    q = bits(rng.standard_normal((1, 4, D)) / 2)
    table = torch.zeros(1, n_pages, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    gk, gv, refs, lens = dev(k), dev(v), i32([1, 1]), i32([n_pages * ps])
    pool, seqs = abi.TvPool(gk.data_ptr(), gv.data_ptr(), refs.data_ptr(), 1, 2, 1, ps, D), abi.TvSeqs(table.data_ptr(), lens.data_ptr(), 1, n_pages)
    out, st, gq = torch.zeros(1, 4, D, dtype=torch.int16, device="cuda"), i32([0]), dev(q)
    wsb = abi.tv_attend_paged_workspace_size(pool, 4, 1)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    assert abi.tv_attend_paged(pool, 0, seqs, i32([0]), 1, 4, gq, 4 * D, None, None, 0, out, ws, wsb, st) == 0
    assert int(st.item()) == 0
    qf, kf, vf = bf16_to_f64(q[0]), bf16_to_f64(k[0]), bf16_to_f64(v[0])
    w = np.exp(qf @ kf.T / np.sqrt(D))
    w /= w.sum(1, keepdims=True)
    o, size = w @ vf, w @ np.abs(vf)
    assert (np.abs(bf16_to_f64(host(out))[0] - o) <= (2.0 ** -5 + 2.0 ** -6 + 3 * 2.0 ** -8 + 2.0 ** -19) * size).all()


def test_refusals(gpu):
    E = abi.CODES
    for ids in ([0, 99, 1], [0, -1, 1], [1, 0, 1], list(range(38)) + [40], list(range(38)) + [99999], [3] + list(range(38))):
        c = Case([20, 30, 40] if len(ids) == 3 else [20] * 39, 4, 2, 64, 16, unlisted=1)
        if ids[-1] == 40:
            c.glens[40 - 1] = 1000                           # (longer than its table row)
            ids = ids[:-1] + [39]
        assert c.run(ids=i32(ids)) == 0
        assert int(c.status.item()) == E["TV_E_SEQ"]
        assert (host(c.out) == 77).all() and np.array_equal(host(c.gk), c.k) and np.array_equal(host(c.gv), c.v)
    c = Case([20, 30, 40], 4, 2, 64, 16)
    c.glens[c.ids[1]] = 49                                   # longer than its table row
    assert c.run() == 0 and int(c.status.item()) == E["TV_E_SEQ"]
    for wrong in (-1, 1 << 30):
        c = Case([20, 300, 40], 4, 2, 64, 16)
        c.gpages[c.ids[1], 5] = wrong
        assert c.run() == 0 and int(c.status.item()) == E["TV_E_PAGE"]
    c = Case([20, 30, 40], 4, 2, 64, 16)
    c.status.fill_(E["TV_E_TOKEN"])
    assert c.run() == 0 and int(c.status.item()) == E["TV_E_TOKEN"] and (host(c.out) == 77).all()


def test_listed_twice_without_new_rows(gpu):
    c = Case([20, 300, 40], 4, 2, 64, 16, new=False)
    c.gq[1] = c.gq[0]
    assert c.run(ids=i32([c.ids[0], c.ids[0], c.ids[2]])) == 0 and int(c.status.item()) == 0
    assert np.array_equal(host(c.out)[0], host(c.out)[1])


def test_two_calls_at_once(gpu):
    """On two streams, each with its own pool, workspace and status."""
    cs = [Case([3000 + 500 * i, 70, 1], 8, 2, 128, 16, seed=30 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(cs, streams):
            assert c.run(s) == 0
    torch.cuda.synchronize()
    got = [c.out.clone() for c in cs]
    for c, g in zip(cs, got):
        c.check()
        assert torch.equal(c.out, g)


def test_graphs_share_a_workspace_and_lengths_grow(gpu):
    """Two captured calls on one workspace; replayed as the lengths change, each gives what a plain call gives, twice."""
    a, b = Case([900, 77, 5], 8, 2, 128, 16, seed=1, new=False), Case([64, 2000, 1], 8, 2, 128, 16, seed=2, new=False)
    b.ws = a.ws
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            assert c.run(torch.cuda.current_stream()) == 0
        graphs.append(g)
    for lens in ([900, 77, 5], [899, 16, 5], [64, 0, 1]):
        for c, full in ((a, [900, 77, 5]), (b, [64, 2000, 1])):
            for i in range(3):
                c.lens[i] = min(lens[i], full[i])
                c.glens[c.ids[i]] = c.lens[i]
        for _ in range(2):
            a.out.fill_(77)
            b.out.fill_(77)
            graphs[0].replay()
            graphs[1].replay()
            torch.cuda.synchronize()
            got = [host(a.out).copy(), host(b.out).copy()]
            for c, x in zip((a, b), got):
                short = [[kv[0][:c.lens[i]], kv[1][:c.lens[i]]] for i, kv in enumerate(c.kv)]
                assert int(c.status.item()) == 0
                for i in range(3):
                    o, off = attend(bf16_to_f64(c.q[i]), bf16_to_f64(short[i][0]), bf16_to_f64(short[i][1]), True)
                    close(bf16_to_f64(x[i]), o, off)
                c.out.fill_(77)
                assert c.run() == 0
                assert np.array_equal(host(c.out), x)     # the same bits


@pytest.mark.parametrize("q_heads,kv_heads,dim", [(10, 2, 128), (16, 2, 64), (12, 1, 64), (16, 1, 128), (24, 1, 64)])
@pytest.mark.parametrize("n", [600, 2048])
def test_many_sequences_of_one_tile(gpu, q_heads, kv_heads, dim, n):
    """Groups of 5 to 24 heads, whose queries have 6 to 2 places, and runs that the two halves of a block take in turn;
    lists whose rows and lengths lie in shared memory and longer ones.  The same bits every time."""
    lens = np.random.default_rng(n + q_heads).integers(1, 65, n).tolist()
    c = Case(lens, q_heads, kv_heads, dim, 16, seed=n)
    c.check()
    first = host(c.out).copy()
    for _ in range(100):
        assert c.run() == 0
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0, abi.STATUS.get(int(c.status.item()))
    assert np.array_equal(host(c.out), first)


def _set_value(c, i, t, g, d, value):
    """V of token t of listed sequence i; the last one comes with the new rows where there are any."""
    Hq, Hkv, D = c.dims
    word = int(np.array(value, np.uint16).view(np.int16))
    if c.new and t == c.lens[i] - 1:
        c.gq[i, (Hq + Hkv + g) * D + d] = word
    else:
        c.gv[c.layer, c.pages[c.ids[i], t // c.pool.page_size], g, t % c.pool.page_size, d] = word


@pytest.mark.parametrize("new", [True, False])
@pytest.mark.parametrize("scale", [1.0, 30.0])
@pytest.mark.parametrize("q_heads,kv_heads,dim,ps,lens", [(4, 2, 64, 16, [1, 40, 64, 65, 700]), (10, 2, 128, 32, [9001, 3]), (24, 1, 128, 64, [30, 5000]),
                                                          (16, 8, 128, 16, [50] * 300 + [1000]), (33, 1, 64, 16, [60] * 200)])
def test_infinities_that_are_seen(gpu, q_heads, kv_heads, dim, ps, lens, scale, new):
    """An infinity in a token's V is the result in its dimension, whatever the token weighs; with the other infinity or
    a NaN beside it, NaN.  Every other element keeps its bits, and a query that is NaN stays so."""
    case = lambda: Case(lens, q_heads, kv_heads, dim, ps, layers=2, layer=1, seed=17, new=new, scale=scale)
    c, G = case(), q_heads // kv_heads
    assert c.run() == 0
    want = bf16_to_f64(host(c.out))[:len(lens)]
    assert np.isfinite(want).all()
    c = case()
    inf, ninf, nan = 0x7F80, 0xFF80, NAN
    for i in range(0, len(lens), max(1, len(lens) // 7)):
        n, g = lens[i], i % kv_heads
        heads = slice(g * G, (g + 1) * G)
        for d, marks, value in ((3, [(n - 1, inf)], np.inf), (9, [(0, ninf)], -np.inf), (16, [(n // 2, inf), (n - 1, inf)], np.inf),
                                (31, [(n // 3, nan)], np.nan), (dim - 1, [(0, inf), (n - 1, ninf)], np.nan), (40, [(0, nan), (n - 1, inf)], np.nan)):
            if n == 1 and len({m for _, m in marks}) > 1:
                continue
            for t, m in marks:
                _set_value(c, i, t, g, d, m)
            want[i, heads, d] = value
    c.gq[0, (q_heads - 1) * dim] = int(np.array(NAN, np.uint16).view(np.int16))
    want[0, q_heads - 1] = np.nan
    assert c.run() == 0
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    assert np.array_equal(bf16_to_f64(host(c.out))[:len(lens)], want, equal_nan=True)
