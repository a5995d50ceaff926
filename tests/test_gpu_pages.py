"""The paged cache on the GPU against oracle/paged.py: tables, counts and
lengths equal, every value of the pool equal bit for bit (rows are only moved,
so there is no tolerance)."""
import numpy as np
import pytest
import torch

from oracle.paged import Cache, Refused
from speculative_tree_verify_gb300 import abi

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


class Both:
    """The same cache on the GPU and in the oracle."""

    def __init__(self, layers=2, n_pages=40, heads=2, ps=16, dim=64, max_seqs=9, max_pages=12, seed=0):
        rng = np.random.default_rng(seed)
        k, v = (rng.integers(0, 1 << 16, (layers, n_pages, heads, ps, dim)).astype(np.uint16) for _ in range(2))
        self.o = Cache(k, v, np.zeros(n_pages, np.int32), np.full((max_seqs, max_pages), -7, np.int32), np.zeros(max_seqs, np.int32))
        self.k, self.v = (torch.from_numpy(x.view(np.int16).copy()).cuda() for x in (k, v))
        self.refs, self.pages, self.lens = i32(self.o.refs), i32(self.o.pages), i32(self.o.lens)
        self.pool = abi.TvPool(self.k.data_ptr(), self.v.data_ptr(), self.refs.data_ptr(), layers, n_pages, heads, ps, dim)
        self.seqs = abi.TvSeqs(self.pages.data_ptr(), self.lens.data_ptr(), max_seqs, max_pages)
        self.status = i32([0])
        self.wsb = abi.tv_pages_workspace_size(self.pool, self.seqs)
        self.ws = torch.zeros(self.wsb, dtype=torch.uint8, device="cuda")
        self.remap, self.used = i32(np.full(n_pages, -5)), i32([-5])

    def call(self, rc, oracle, *args):
        """One call on both sides; a refusal has to carry the oracle's code and change nothing."""
        assert rc == abi.TV_OK, abi.STATUS.get(rc, rc)
        want, got = 0, int(self.status.item())
        try:
            r = oracle(*args)
        except Refused as e:
            want, r = abi.CODES[str(e)], None
        assert got == want, (abi.STATUS.get(got), abi.STATUS.get(want), args)
        self.status.zero_()
        self.same()
        return r

    def same(self):
        for name in ("refs", "pages", "lens"):
            assert np.array_equal(getattr(self, name).cpu().numpy(), getattr(self.o, name)), name
        for name in ("k", "v"):
            assert np.array_equal(getattr(self, name).cpu().numpy().view(np.uint16), getattr(self.o, name)), name

    def extend(self, ids, add):
        return self.call(abi.tv_pages_extend(self.pool, self.seqs, i32(ids), i32(add), len(ids), self.ws, self.wsb, self.status), self.o.extend, ids, add)

    def fork(self, src, dst):
        return self.call(abi.tv_pages_fork(self.pool, self.seqs, i32(src), i32(dst), len(src), self.status), self.o.fork, src, dst)

    def release(self, ids, keep):
        return self.call(abi.tv_pages_release(self.pool, self.seqs, i32(ids), i32(keep), len(ids), self.status), self.o.release, ids, keep)

    def compact(self):
        r = self.call(abi.tv_pages_compact(self.pool, self.seqs, self.remap, self.used, self.ws, self.wsb, self.status), self.o.compact)
        if r is not None:
            assert np.array_equal(self.remap.cpu().numpy(), r[0]) and int(self.used.item()) == r[1]


@pytest.mark.parametrize("ps,dim,heads,layers", [(16, 64, 2, 2), (32, 128, 1, 3), (64, 64, 3, 1), (128, 128, 2, 1)])
def test_fork_extend_release_by_hand(gpu, ps, dim, heads, layers):
    b = Both(layers, 20, heads, ps, dim)
    b.extend([2, 0], [ps + 1, ps])
    b.fork([2, 2], [1, 3])
    b.extend([1, 2, 3, 0], [1, 2, 3, 0])             # three holders of the partly filled page: the last keeps it
    b.fork([1], [4])
    b.extend([4], [1])                               # one of two holders: it copies
    b.extend([5], [0])
    b.release([1, 3, 2], [0, ps, ps + 3])            # to nothing, to a page's edge, to its own length
    b.extend([3], [1])                               # from a page's edge: no copy
    b.compact()
    b.compact()                                      # nothing left to move


def test_refusals_change_nothing(gpu):
    b = Both(n_pages=10, max_seqs=5, max_pages=4)
    b.extend([0, 1], [20, 33])                       # five pages
    b.fork([1], [2])
    for ids, add in (([0, 0], [1, 1]), ([5], [1]), ([-1], [1]), ([0, 1], [1, -1]), ([0], [45]), ([0, 2], [40, 16]),
                     ([1, 2, 0], [31, 31, 40]), ([2, 1, 3], [1, 1, 64])):
        b.extend(ids, add)
    for src, dst in (([0], [0]), ([0, 1], [3, 3]), ([0], [1]), ([0], [5]), ([-1], [3]), ([3], [4]), ([3, 0], [4, 3])):
        b.fork(src, dst)
    b.release([4], [0])
    for ids, keep in (([0], [21]), ([0, 0], [1, 1]), ([0, 1], [2, -1]), ([7], [0])):
        b.release(ids, keep)
    # a table row that names a page outside the pool, and one that nobody holds
    for wrong, code in ((10, "TV_E_PAGE"), (-1, "TV_E_PAGE"), (9, "TV_E_PAGE")):
        keep = int(b.o.pages[1, 2])
        b.o.pages[1, 2] = wrong
        b.pages.copy_(i32(b.o.pages))
        b.release([0, 1], [0, 0])
        b.fork([1], [3])
        b.extend([1], [1])
        b.compact()
        b.o.pages[1, 2] = keep
        b.pages.copy_(i32(b.o.pages))
    b.o.lens[0] = 65                                 # longer than its row
    b.lens.copy_(i32(b.o.lens))
    b.release([0], [0])
    b.compact()


def test_status_stops_every_call(gpu):
    b = Both()
    b.extend([0, 1], [20, 33])
    b.status.fill_(abi.CODES["TV_E_TOKEN"])
    k, v = (torch.zeros(4, 2, 64, dtype=torch.int16, device="cuda") for _ in range(2))
    assert abi.tv_pages_extend(b.pool, b.seqs, i32([0]), i32([40]), 1, b.ws, b.wsb, b.status) == 0
    assert abi.tv_pages_fork(b.pool, b.seqs, i32([0]), i32([2]), 1, b.status) == 0
    assert abi.tv_pages_release(b.pool, b.seqs, i32([0]), i32([0]), 1, b.status) == 0
    assert abi.tv_pages_compact(b.pool, b.seqs, b.remap, b.used, b.ws, b.wsb, b.status) == 0
    assert abi.tv_pages_write(b.pool, 0, b.seqs, i32([0]), i32([0]), i32([0, 4]), 1, 4, k, v, 128, 64, b.status) == 0
    assert abi.tv_pages_read(b.pool, 0, b.seqs, i32([0]), i32([0]), i32([0, 4]), 1, 4, k, v, 128, 64, b.status) == 0
    assert int(b.status.item()) == abi.CODES["TV_E_TOKEN"]
    b.same()
    assert int(b.used.item()) == -5 and not k.any()


@pytest.mark.parametrize("seed,n_pages,max_seqs,max_pages,ps", [(1, 61, 9, 12, 16), (2, 200, 40, 6, 32), (3, 1500, 70, 90, 16)])
def test_churn(gpu, seed, n_pages, max_seqs, max_pages, ps):
    """Random lists of every call, refusals among them."""
    b = Both(1, n_pages, 1, ps, 64, max_seqs, max_pages, seed)
    rng = np.random.default_rng(seed)
    for step in range(60):
        live = [s for s in range(max_seqs) if b.o.lens[s] > 0]
        idle = [s for s in range(max_seqs) if b.o.lens[s] == 0]
        what = rng.integers(0, 8)
        if what < 4:
            ids = rng.permutation(max_seqs)[: rng.integers(1, max_seqs + 1)]
            b.extend(ids.tolist(), rng.integers(0, 2 * ps if what else 6 * ps, len(ids)).tolist())
        elif what == 4 and live and idle:
            dst = rng.permutation(idle)[: rng.integers(1, len(idle) + 1)]
            b.fork([int(rng.choice(live)) for _ in dst], dst.tolist())
        elif what in (5, 6) and live:
            ids = rng.permutation(live)[: rng.integers(1, len(live) + 1)]
            b.release(ids.tolist(), [int(rng.integers(0, b.o.lens[s] + 1)) if rng.random() < .7 else 0 for s in ids])
        elif what == 7:
            b.compact()
        held = np.zeros(n_pages, np.int64)
        for s in range(max_seqs):
            for j in range(-(-int(b.o.lens[s]) // ps)):
                held[b.o.pages[s, j]] += 1
        assert np.array_equal(held, b.o.refs)


def test_the_longest_lists(gpu):
    """4096 sequences in one call, of 65536 table rows."""
    b = Both(1, 9000, 1, 16, 64, 65536, 2, 4)
    ids = np.random.default_rng(4).permutation(65536)[:4096].tolist()
    b.extend(ids, [1 + i % 17 for i in range(4096)])
    b.fork(ids[:100], np.setdiff1d(np.arange(65536), ids)[:100].tolist())
    b.extend(ids[:200], [1] * 200)
    b.release(ids, [i % 2 for i in range(4096)])
    b.compact()


@pytest.mark.parametrize("ps,dim,heads", [(16, 64, 1), (32, 128, 8), (128, 128, 3)])
def test_rows(gpu, ps, dim, heads):
    b = Both(2, 60, heads, ps, dim, 6, 9, 5)
    lens = [1, 3 * ps, 0, 2 * ps + 5, ps - 1]
    b.extend([0, 1, 2, 3, 4], lens)
    b.compact()
    rng = np.random.default_rng(6)
    # a projection's rows: q heads in front, two rows before and three behind the listed ones
    ids, pos, counts = [3, 1, 2, 4, 0], [4, 0, 0, ps - 2, 0], [ps + 9, 3 * ps, 0, 1, 1]
    starts = np.concatenate([[2], 2 + np.cumsum(counts)])
    rows = int(starts[-1]) + 3
    width = (3 + 2 * heads) * dim
    x = rng.integers(0, 1 << 16, (rows, width)).astype(np.uint16)
    xg = torch.from_numpy(x.view(np.int16)).cuda()
    kg, vg = xg[:, 3 * dim:], xg[:, (3 + heads) * dim:]
    rc = abi.tv_pages_write(b.pool, 1, b.seqs, i32(ids), i32(pos), i32(starts), 5, rows, kg, vg, width, dim, b.status)
    assert rc == 0 and int(b.status.item()) == 0
    k, v = (x[:, o:o + heads * dim].reshape(rows, heads, dim) for o in (3 * dim, (3 + heads) * dim))
    for i, s in enumerate(ids):
        b.o.write(1, s, pos[i], k[starts[i]:starts[i + 1]], v[starts[i]:starts[i + 1]])
    b.same()
    # back again into other rows, the rest of them left alone; a sequence may be read twice
    back = torch.full((rows, width), 77, dtype=torch.int16, device="cuda")
    rc = abi.tv_pages_read(b.pool, 1, b.seqs, i32(ids[:4] + [3]), i32(pos), i32(starts), 5, rows, back[:, 3 * dim:], back[:, (3 + heads) * dim:],
                           width, dim, b.status)
    assert rc == 0 and int(b.status.item()) == 0
    want = np.full((rows, width), 77, np.uint16)
    for i, s in enumerate(ids[:4] + [3]):
        a, e = starts[i], starts[i + 1]
        kk, vv = b.o.rows(1, s, pos[i], e - a)
        want[a:e, 3 * dim:(3 + heads) * dim], want[a:e, (3 + heads) * dim:] = kk.reshape(e - a, heads * dim), vv.reshape(e - a, heads * dim)
    assert np.array_equal(back.cpu().numpy().view(np.uint16), want)
    # one sequence as a contiguous cache [heads][capacity][dim], from slot 2 on
    cap = 3 * ps + 7
    ck, cv = (torch.full((heads, cap, dim), 5, dtype=torch.int16, device="cuda") for _ in range(2))
    rc = abi.tv_pages_read(b.pool, 0, b.seqs, i32([1]), i32([0]), i32([0, 3 * ps]), 1, 3 * ps, ck[:, 2:], cv[:, 2:], dim, cap * dim, b.status)
    assert rc == 0 and int(b.status.item()) == 0
    for got, want in zip((ck, cv), b.o.rows(0, 1, 0, 3 * ps)):
        got = got.cpu().numpy().view(np.uint16)
        assert np.array_equal(got[:, 2:2 + 3 * ps], want.transpose(1, 0, 2)) and (got[:, :2] == 5).all() and (got[:, 2 + 3 * ps:] == 5).all()


def test_rows_refusals(gpu):
    b = Both(n_pages=10, max_seqs=4, max_pages=4)
    b.extend([0, 1], [20, 33])
    k, v = (torch.zeros(64, 2, 64, dtype=torch.int16, device="cuda") for _ in range(2))
    E = abi.CODES
    for ids, pos, starts, code in (([0, 4], [0, 0], [0, 1, 2], "TV_E_SEQ"), ([0, -1], [0, 0], [0, 1, 2], "TV_E_SEQ"),
                                   ([0, 1], [0, -1], [0, 1, 2], "TV_E_SEQ"), ([0, 1], [0, 0], [0, 5, 4], "TV_E_SEQ"),
                                   ([0, 1], [0, 0], [0, 5, 65], "TV_E_SEQ"), ([0, 1], [0, 0], [-1, 5, 6], "TV_E_SEQ"),
                                   ([0, 1], [0, 30], [0, 5, 9], "TV_E_CAPACITY"), ([0, 2], [0, 0], [0, 5, 6], "TV_E_CAPACITY")):
        for fn in (abi.tv_pages_write, abi.tv_pages_read):
            assert fn(b.pool, 0, b.seqs, i32(ids), i32(pos), i32(starts), 2, 64, k, v, 128, 64, b.status) == 0
            assert int(b.status.item()) == E[code], (fn, ids, pos, starts)
            b.status.zero_()
    assert abi.tv_pages_write(b.pool, 0, b.seqs, i32([0, 0]), i32([0, 9]), i32([0, 1, 2]), 2, 64, k, v, 128, 64, b.status) == 0
    assert int(b.status.item()) == E["TV_E_SEQ"]
    b.same()
    assert not k.any() and not v.any()
    # a page outside the pool: that row is left out, the others are written
    b.status.zero_()
    b.o.pages[0, 1] = 10
    b.pages.copy_(i32(b.o.pages))
    assert abi.tv_pages_write(b.pool, 0, b.seqs, i32([0]), i32([14]), i32([0, 4]), 1, 64, k, v, 128, 64, b.status) == 0
    assert int(b.status.item()) == E["TV_E_PAGE"]
    for x in (b.o.k, b.o.v):
        x[0, b.o.pages[0, 0], :, 14:16] = 0
    b.same()


@pytest.mark.parametrize("which", [0, 1, 2])
def test_many_rows_around_a_bad_page(gpu, which):
    """Rows for several waves of blocks; a bad entry in the first page, a middle one or the last leaves out its own rows
    and no other, every time, and the next call does nothing."""
    ps, heads, dim, lens = 16, 1, 64, [9000, 12000, 20000]
    b = Both(1, sum(-(-x // ps) for x in lens) + 3, heads, ps, dim, 4, 1300, 21)
    b.extend([2, 0, 1], lens)
    ids, rows = [2, 0, 1], sum(lens)
    starts = np.concatenate([[0], np.cumsum(lens)])
    s, j = ((2, 0), (0, 400), (1, 1249))[which]
    b.o.pages[s, j] = b.o.refs.shape[0] if which else -1
    b.pages.copy_(i32(b.o.pages))
    left = starts[ids.index(s)] + ps * j
    E = abi.CODES
    rng = np.random.default_rng(which)
    for _ in range(10):
        x = rng.integers(0, 1 << 16, (2, rows, heads, dim)).astype(np.uint16)
        k, v = (torch.from_numpy(y.view(np.int16)).cuda() for y in x)
        assert abi.tv_pages_write(b.pool, 0, b.seqs, i32(ids), i32([0] * 3), i32(starts), 3, rows, k, v, dim, dim, b.status) == 0
        assert int(b.status.item()) == E["TV_E_PAGE"]
        for i, q in enumerate(ids):
            for m in range(-(-lens[i] // ps)):
                p, a, e = b.o.pages[q, m], starts[i] + ps * m, min(starts[i] + ps * (m + 1), starts[i + 1])
                if (q, m) != (s, j):
                    b.o.k[0, p, :, :e - a], b.o.v[0, p, :, :e - a] = x[0, a:e].transpose(1, 0, 2), x[1, a:e].transpose(1, 0, 2)
        b.same()
        got = [torch.full((rows, heads, dim), 77, dtype=torch.int16, device="cuda") for _ in range(2)]
        read = lambda: abi.tv_pages_read(b.pool, 0, b.seqs, i32(ids), i32([0] * 3), i32(starts), 3, rows, *got, dim, dim, b.status)
        assert read() == 0 and all((g == 77).all() for g in got)          # stopped by the status
        b.status.zero_()
        assert read() == 0 and int(b.status.item()) == E["TV_E_PAGE"]
        b.status.zero_()
        for g, y in zip(got, x):
            want = y.copy()
            want[left:left + min(ps, starts[ids.index(s) + 1] - left)] = 77
            assert np.array_equal(g.cpu().numpy().view(np.uint16), want)


def test_a_page_of_2_to_the_32_bytes(gpu):
    """131,073 heads of 128 tokens: what a copy-on-write and a compaction move has more bytes than 32 bits hold."""
    heads, ps, dim = 2 ** 17 + 1, 128, 128
    k, v = (torch.zeros(1, 3, heads, ps, dim, dtype=torch.int16, device="cuda") for _ in range(2))
    for x in (k, v):
        x[0, 0].view(-1, 1 << 14)[:, 0] = torch.arange(heads * ps * dim >> 14, device="cuda").to(torch.int16)
        x[0, 0, -1] = 7
    refs, table, lens, status = i32([1, 0, 0]), i32([[0], [-1]]), i32([5, 0]), i32([0])
    pool, seqs = abi.TvPool(k.data_ptr(), v.data_ptr(), refs.data_ptr(), 1, 3, heads, ps, dim), abi.TvSeqs(table.data_ptr(), lens.data_ptr(), 2, 1)
    wsb = abi.tv_pages_workspace_size(pool, seqs)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    assert abi.tv_pages_fork(pool, seqs, i32([0]), i32([1]), 1, status) == 0
    assert abi.tv_pages_extend(pool, seqs, i32([1]), i32([1]), 1, ws, wsb, status) == 0
    assert int(status.item()) == 0 and table.tolist() == [[0], [1]]
    assert torch.equal(k[0, 1], k[0, 0]) and torch.equal(v[0, 1], v[0, 0])
    assert abi.tv_pages_release(pool, seqs, i32([0]), i32([0]), 1, status) == 0
    k[0, 0], v[0, 0] = 0, 0
    assert abi.tv_pages_compact(pool, seqs, i32([0] * 3), i32([0]), ws, wsb, status) == 0
    assert int(status.item()) == 0 and table.tolist() == [[0], [0]]
    assert torch.equal(k[0, 1], k[0, 0]) and torch.equal(v[0, 1], v[0, 0])


def test_captured_and_replayed_on_other_lists(gpu):
    """One graph of release, fork, extend and compact, replayed with other lists in the same tensors, on a side stream."""
    b = Both(2, 80, 2, 16, 64, 9, 12, 8)
    b.extend([0], [50])
    kids, par, add, none = i32([1, 2, 3]), i32([0, 0, 0]), i32([0, 0, 0]), i32([0, 0, 0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        st = torch.cuda.current_stream()
        assert abi.tv_pages_release(b.pool, b.seqs, kids, none, 3, b.status, st) == 0
        assert abi.tv_pages_fork(b.pool, b.seqs, par, kids, 3, b.status, st) == 0
        assert abi.tv_pages_extend(b.pool, b.seqs, kids, add, 3, b.ws, b.wsb, b.status, st) == 0
        assert abi.tv_pages_compact(b.pool, b.seqs, b.remap, b.used, b.ws, b.wsb, b.status, st) == 0
    b.same()   # capturing runs nothing
    for k, a in (([1, 2, 3], [1, 2, 40]), ([4, 2, 8], [16, 0, 3]), ([3, 1, 5], [5, 6, 7])):
        kids.copy_(i32(k))
        add.copy_(i32(a))
        g.replay()
        torch.cuda.synchronize()
        assert int(b.status.item()) == 0
        b.o.release(k, [0] * 3)
        b.o.fork([0] * 3, k)
        b.o.extend(k, a)
        b.o.compact()
        b.same()


@pytest.mark.parametrize("n,max_pages", [(1, 33), (17, 32), (16, 1025), (35, 700), (20, 4000), (2, 8192), (33, 3000), (1, 8200)])
def test_lists_of_every_width(gpu, n, max_pages):
    """From one block's work to many blocks'; the first, a middle and the last sequence can refuse."""
    rows, long = 2 * n + 3, max_pages * 16 - 3
    b = Both(1, 2 * max_pages + 3 * n + 8, 1, 16, 64, rows, max_pages, n)
    rng = np.random.default_rng(n)
    order = rng.permutation(rows).tolist()
    parents, kids, more = order[:2], order[2:2 + n], order[2 + n:2 + 2 * n]
    b.extend(parents, [long, long // 2])
    b.fork([parents[i * i % 3 % 2] for i in range(n)], kids)           # runs of one source, and changes
    b.extend(kids, [i % 3 for i in range(n)])                          # some last pages are their own now
    b.fork(kids, more)
    j = (long + 15) // 16 - 1
    for row in {kids[0], kids[n // 2], kids[-1]}:                      # one bad entry: nothing changes
        at = min(j, -(-int(b.o.lens[row]) // 16) - 1)
        for wrong in (-1, b.o.refs.shape[0], int(np.flatnonzero(b.o.refs == 0)[0])):
            keep, b.o.pages[row, at] = int(b.o.pages[row, at]), wrong
            b.pages.copy_(i32(b.o.pages))
            b.release(kids, [0] * n)
            b.fork([row], [order[-1]])
            b.o.pages[row, at] = keep
            b.pages.copy_(i32(b.o.pages))
    if n > 1:
        b.release(kids[:-1] + [kids[0]], [0] * n)
        b.fork([parents[0]] * n, [order[-1]] * n)
        b.release(kids, [0] * (n - 1) + [int(b.o.lens[kids[-1]]) + 1])
        b.release(kids[:-1] + [rows], [0] * n)
    b.release(kids, [int(rng.integers(0, int(b.o.lens[s]) + 1)) if i % 4 else 0 for i, s in enumerate(kids)])
    b.release(more + parents, [i % 2 for i in range(n)] + [0, 0])
    b.release(kids, [0] * n)
    b.release(more, [0] * n)
    assert not b.o.refs.any() and not b.refs.any()
