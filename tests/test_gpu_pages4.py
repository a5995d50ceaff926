"""The page calls over a pool in 4 bits against oracle/longctx.py and
oracle/paged.py: codes, scales and tables are equal, byte by byte."""
import numpy as np
import pytest
import torch

from oracle import bf16_to_f64, longctx, paged
from speculative_tree_verify_gb300 import abi
from speculative_tree_verify_gb300.device import PagedCache, PagedCache4
from speculative_tree_verify_gb300.synth import Dims
from test_gpu_paged_attn import NAN, bits, dev, host, i32

pytestmark = pytest.mark.gpu


def make(heads, dim, layers=1, n_pages=40, ps=16, max_seqs=8, max_pages=12, seed=0):
    """A cache whose every byte is random."""
    d = Dims(hidden=64, n_q_heads=heads, n_kv_heads=heads, head_dim=dim, vocab=64)
    c = PagedCache4.alloc(d, layers, n_pages, ps, max_seqs, max_pages)
    rng = np.random.default_rng(seed)
    for x in (c.k, c.v):
        x.copy_(torch.from_numpy(rng.integers(0, 256, tuple(x.shape), dtype=np.uint8)))
    return c


def twin(c):
    """The oracle's view: (rows, tables) over the same bytes."""
    k, v = c.k.cpu().numpy().copy(), c.v.cpu().numpy().copy()
    rows = longctx.Pages4(k, v, c.pool.page_size, c.dims.head_dim)
    # a page's bytes as "rows" of the page size, so that the table's rules and copies are the bf16 pool's
    shape = (*k.shape[:3], c.pool.page_size, -1)
    tables = paged.Cache(k.reshape(shape), v.reshape(shape), c.refs.cpu().numpy().copy(), c.pages.cpu().numpy().copy(), c.lens.cpu().numpy().copy())
    return rows, tables


def same(c, rows, tables):
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0, abi.STATUS.get(int(c.status.item()))
    assert (c.refs.cpu().numpy() == tables.refs).all() and (c.lens.cpu().numpy() == tables.lens).all()
    for s, n in enumerate(tables.lens):
        held = -(-int(n) // c.pool.page_size)
        assert (c.pages.cpu().numpy()[s, :held] == tables.pages[s, :held]).all()
    assert (c.k.cpu().numpy() == rows.pools["k"]).all() and (c.v.cpu().numpy() == rows.pools["v"]).all()


def values(rng, shape, kind):
    x = rng.standard_normal(shape)
    if kind == "wide":   # exponents from the smallest to the largest, zeros among them
        x = x * 2.0 ** rng.integers(-140, 120, (*shape[:-1], 1)) * (rng.random(shape) < 0.9)
    if kind == "halves":  # scales that are powers of two: quotients that end in a half
        x = rng.integers(-14, 15, shape) / 2.0
        x[..., ::32] = 7.0
    if kind == "bad":
        x[rng.random(shape) < 0.01] = np.inf
        x[rng.random(shape) < 0.01] = np.nan
    with np.errstate(all="ignore"):
        return bits(x.astype(np.float32))


@pytest.mark.parametrize("kind", ["normal", "wide", "halves", "bad"])
@pytest.mark.parametrize("ps,dim,heads,layers", [(16, 128, 8, 1), (32, 64, 3, 2), (64, 128, 1, 1), (128, 64, 9, 1)])
def test_write_and_read(gpu, ps, dim, heads, layers, kind):
    """Ranges that begin and end anywhere, odd rows, empty ones; rows around them and other layers stay as they were."""
    c = make(heads, dim, layers, ps=ps, seed=ps)
    lens = [5, 100 % (ps * 12), 1, 33, 2 * ps, 0, 47]
    ids, layer = [3, 0, 6, 1, 5, 2, 4], layers - 1
    assert c.extend(i32(ids), i32(lens)) == 0
    torch.cuda.synchronize()
    rows, tables = twin(c)
    rng = np.random.default_rng(dim)
    pos = [rng.integers(0, n + 1) for n in lens]
    take = [int(rng.integers(0, n - p + 1)) if n else 0 for n, p in zip(lens, pos)]
    take[1], pos[1] = lens[1] - 3, 3
    starts = np.concatenate([[2], 2 + np.cumsum(take)])
    total = int(starts[-1]) + 3
    qkv = values(rng, (total, 3 * heads * dim + 8), kind)
    g = dev(qkv)
    assert c.write(layer, i32(ids), i32(pos), i32(starts), g) == 0
    k, v = (qkv[:, i * heads * dim:(i + 1) * heads * dim].reshape(total, heads, dim) for i in (1, 2))
    for i, s in enumerate(ids):
        for r in range(take[i]):
            page, slot = tables.slot(s, pos[i] + r)
            for name, x in (("k", k), ("v", v)):
                rows.put(name, layer, page, slot, *longctx.quantise(x[starts[i] + r]))
    same(c, rows, tables)
    # and back, into rows of another shape
    back = torch.full((total, 2, heads, dim), 77, dtype=torch.int16, device="cuda")
    assert abi.tv_pages4_read(c.pool, layer, c.seqs, i32(ids), i32(pos), i32(starts), len(ids), total, back, back[:, 1], 2 * heads * dim, dim,
                              c.status) == 0
    torch.cuda.synchronize()
    got = host(back)
    for which, x in ((0, k), (1, v)):
        want = longctx.stands_for(*longctx.quantise(x))
        a, b = got[starts[0]:starts[-1], which], longctx.bf16(want)[starts[0]:starts[-1]]
        assert ((a == b) | (np.isnan(bf16_to_f64(a)) & np.isnan(want[starts[0]:starts[-1]])) | ((a & 0x7FFF == 0) & (b & 0x7FFF == 0))).all()
    assert (got[:starts[0]] == 77).all() and (got[starts[-1]:] == 77).all()
    same(c, rows, tables)


def test_every_quotient(gpu):
    """Every value of a bf16 octave beside scales of every mantissa: codes at and next to every border."""
    mant = np.arange(128, 256)
    x = np.zeros((128, 4, 32))
    for i, m in enumerate(mant):
        x[i, :, 0] = m / 16.0   # the group's largest
        x[i, :, 1:] = np.resize(np.concatenate([mant / 128.0 * f for f in (0.5, 1, 2, 4)]), 4 * 31 * 4)[i % 4 * 124:][:124].reshape(4, 31) * (m / 256)
    x[..., 1::2] *= -1
    c = make(1, 128, n_pages=20, max_pages=10, seed=3)
    rows = bits(x.reshape(128, 128).astype(np.float32))
    qkv = np.concatenate([rows, rows, rows[:, ::-1]], 1)
    assert c.extend(i32([0]), i32([128])) == 0
    assert c.write(0, i32([0]), i32([0]), i32([0, 128]), dev(qkv)) == 0
    torch.cuda.synchronize()
    o, tables = twin(c)
    for t in range(128):
        page, slot = tables.slot(0, t)
        for name, y in (("k", rows[t]), ("v", rows[t, ::-1])):
            codes, scales = longctx.quantise(y[None])
            a, b = o.get(name, 0, page, slot)
            assert (a == codes).all() and (b == scales).all(), (t, name)


@pytest.mark.parametrize("seed,ps,dim,heads,layers", [(1, 16, 64, 1, 2), (2, 32, 128, 2, 1), (3, 128, 64, 1, 3)])
def test_churn(gpu, seed, ps, dim, heads, layers):
    """Fork, extend with copy-on-write, release and compact: the bf16 pool's rules, and the bytes moved whole."""
    rng = np.random.default_rng(seed)
    c = make(heads, dim, layers, n_pages=50, ps=ps, max_seqs=7, max_pages=9, seed=seed)
    rows, tables = twin(c)
    tables.k, tables.v = (x.reshape(*x.shape[:3], ps, -1) for x in (rows.pools["k"], rows.pools["v"]))   # views of the same bytes
    remap, used = i32(np.zeros(50)), i32([0])
    for _ in range(40):
        live = [s for s in range(7) if tables.lens[s] > 0]
        empty = [s for s in range(7) if tables.lens[s] == 0]
        op = rng.integers(0, 4)
        try:
            if op == 0:
                ids = rng.permutation(7)[:rng.integers(1, 5)].tolist()
                add = rng.integers(0, 2 * ps, len(ids)).tolist()
                tables.extend(ids, add)
                assert c.extend(i32(ids), i32(add)) == 0
            elif op == 1 and live and empty:
                n = int(rng.integers(1, len(empty) + 1))
                src = [int(rng.choice(live)) for _ in range(n)]
                tables.fork(src, empty[:n])
                assert c.fork(i32(src), i32(empty[:n])) == 0
            elif op == 2 and live:
                ids = rng.permutation(live)[:rng.integers(1, 4)].tolist()
                keep = [int(rng.integers(0, tables.lens[s] + 1)) for s in ids]
                tables.release(ids, keep)
                assert c.release(i32(ids), i32(keep)) == 0
            elif op == 3:
                want, n = tables.compact()
                assert c.compact(remap, used) == 0
                torch.cuda.synchronize()
                assert (remap.cpu().numpy() == want).all() and int(used.item()) == n
        except paged.Refused as e:
            if op == 0:
                assert c.extend(i32(ids), i32(add)) == 0
                torch.cuda.synchronize()
                assert abi.STATUS[int(c.status.item())] == str(e)
                c.status.zero_()
            continue
        same(c, rows, tables)


@pytest.mark.parametrize("n", [2, 600])
def test_refusals(gpu, n):
    """A bad list changes nothing; a bad page leaves out its own rows alone."""
    c = make(2, 64, n_pages=1300, max_seqs=620, max_pages=2, seed=n)
    ids, lens = list(range(n)), [20] * n
    assert c.extend(i32(ids), i32(lens)) == 0
    torch.cuda.synchronize()
    rows, tables = twin(c)
    x = dev(bits(np.random.default_rng(0).standard_normal((20 * n, 3 * 128))))
    starts = list(range(0, 20 * n + 1, 20))

    def refused(code, ids=ids, pos=None, starts=starts):
        assert c.write(0, i32(ids), i32([0] * n if pos is None else pos), i32(starts), x) == 0
        torch.cuda.synchronize()
        assert abi.STATUS[int(c.status.item())] == code
        c.status.zero_()
        same(c, rows, tables)

    refused("TV_E_SEQ", ids=[0] * n)
    refused("TV_E_SEQ", ids=ids[:-1] + [620])
    refused("TV_E_SEQ", starts=starts[:-1] + [20 * n + 1])
    refused("TV_E_SEQ", starts=[5] + starts[1:-2] + [0] + starts[-1:])
    refused("TV_E_SEQ", pos=[-1] + [0] * (n - 1))
    refused("TV_E_CAPACITY", pos=[1] + [0] * (n - 1))
    c.pages[n // 2, 1] = 1300
    assert c.write(0, i32(ids), i32([0] * n), i32(starts), x) == 0
    torch.cuda.synchronize()
    assert abi.STATUS[int(c.status.item())] == "TV_E_PAGE"
    c.status.zero_()
    c.pages[n // 2, 1] = int(tables.pages[n // 2, 1])
    X = host(x)
    for i in ids:
        for r in range(20):
            if i == n // 2 and r >= 16:
                continue
            page, slot = tables.slot(i, r)
            for name, at in (("k", 128), ("v", 256)):
                rows.put(name, 0, page, slot, *longctx.quantise(X[20 * i + r, at:at + 128].reshape(2, 64)))
    same(c, rows, tables)
    # the class refuses what a kernel would take for something else
    with pytest.raises(ValueError):
        c.write(0, i32(ids), i32([0] * n), i32(starts), x[:, ::2])
    with pytest.raises(ValueError):
        c.extend(i32(ids), i32(lens)[:1].expand(n + 1))


def test_from_a_contiguous_cache(gpu):
    """Rows of a tv_kv cache in, and back into one (a paged sequence verified, what was committed written back)."""
    heads, dim, cap = 3, 128, 80
    c = make(heads, dim, n_pages=12, max_pages=6, ps=32, seed=4)
    rng = np.random.default_rng(5)
    k, v = (bits(rng.standard_normal((heads, cap, dim))) for _ in range(2))
    assert c.extend(i32([2]), i32([70])) == 0
    assert c.write_from(0, i32([2]), i32([0]), i32([0, 70]), 70, dev(k), dev(v)) == 0
    gk, gv = (torch.full((heads, cap, dim), 77, dtype=torch.int16, device="cuda") for _ in range(2))
    assert c.read_into(0, i32([2]), i32([0]), i32([0, 70]), 70, gk, gv) == 0
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    for x, got in ((k, host(gk)), (v, host(gv))):
        want = longctx.bf16(longctx.stands_for(*longctx.quantise(x)))
        same_zero = (got[:, :70] & 0x7FFF == 0) & (want[:, :70] & 0x7FFF == 0)
        assert ((got[:, :70] == want[:, :70]) | same_zero).all() and (got[:, 70:] == 77).all()
        # what came back is written again as it is
    assert c.write_from(0, i32([2]), i32([0]), i32([0, 70]), 70, gk, gv) == 0
    hk = torch.zeros_like(gk)
    assert c.read_into(0, i32([2]), i32([0]), i32([0, 70]), 70, hk, torch.zeros_like(gv)) == 0
    torch.cuda.synchronize()
    a, b = bf16_to_f64(host(hk)[:, :70]), bf16_to_f64(host(gk)[:, :70])
    # 7 s rounded to bf16 and divided by 7 is s to 2^-8 of it, half a step of bf16: codes stay, values move by two roundings
    assert (np.abs(a - b) <= 2.0 ** -7 * np.abs(b)).all()


def test_pools_beside_each_other(gpu):
    """A bf16 and a 4-bit pool of the same dims on two streams."""
    d = Dims(hidden=64, n_q_heads=2, n_kv_heads=2, head_dim=64, vocab=64)
    a, b = PagedCache.alloc(d, 1, 40, 16, 4, 10), make(2, 64)
    x = dev(bits(np.random.default_rng(1).standard_normal((100, 3 * 128))))
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for c, s in ((a, st[0]), (b, st[1])):
        assert c.extend(i32([1]), i32([100]), s) == 0
        assert c.write(0, i32([1]), i32([0]), i32([0, 100]), x, s) == 0
        k, v = (torch.zeros(2, 100, 64, dtype=torch.int16, device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        assert c.read_into(0, i32([1]), i32([0]), i32([0, 100]), 100, k, v, s) == 0
        outs.append(k)
    torch.cuda.synchronize()
    assert int(a.status.item()) == int(b.status.item()) == 0
    exact, held = (bf16_to_f64(host(o)) for o in outs)
    # half of a step: the scale is the largest / 7 to 2^-8 of itself, the value rounded once more
    top = np.abs(exact).reshape(2, 100, 2, 32).max(-1, keepdims=True).repeat(32, -1).reshape(exact.shape)
    assert (np.abs(exact - held) <= top / 7 * (0.5 + 2.0 ** -5)).all()
