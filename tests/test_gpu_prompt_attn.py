"""tv_attend_prompt against oracle/paged.py (fp64), and a whole serving run:
prompts, pages, tokens, forks, and a tree verify of a paged sequence.

Tolerance: as test_gpu_paged_attn.py derives it (P rounded to bf16: 2^-8 of the
weights' spread around the result; fp32 scores; one rounding of the result)."""
import numpy as np
import pytest
import torch

from oracle import bf16_to_f64
from oracle.paged import attend, attend_prompt
from speculative_tree_verify_gb300 import abi
from test_gpu_paged_attn import NAN, bits, close, dev, host, i32

pytestmark = pytest.mark.gpu


class Prompt:
    """Packed sequences in rows of a QKV projection; what lies before, behind and beside them is NaN."""

    def __init__(self, lens, q_heads, kv_heads, dim, seed=0, before=0, behind=0, pad=0, scale=1.0, edit=None):
        rng = np.random.default_rng(seed)
        self.dims, self.lens = (q_heads, kv_heads, dim), lens
        self.starts = (before + np.concatenate([[0], np.cumsum(lens)])).tolist()
        rows, used = self.starts[-1] + behind, slice(before, self.starts[-1])
        self.rows, self.width = max(rows, 1), (q_heads + 2 * kv_heads) * dim + pad
        total = sum(lens)
        full = lambda h: np.full((self.rows, h, dim), NAN, np.uint16)
        self.q, self.k, self.v = full(q_heads), full(kv_heads), full(kv_heads)
        self.q[used] = bits(rng.standard_normal((total, q_heads, dim)) * scale)
        self.k[used] = bits(rng.standard_normal((total, kv_heads, dim)))
        self.v[used] = bits(rng.standard_normal((total, kv_heads, dim)))
        if edit:
            edit(self)
        x = np.full((self.rows, self.width), NAN, np.uint16)
        for part, at in ((self.q, 0), (self.k, q_heads * dim), (self.v, (q_heads + kv_heads) * dim)):
            x[:, at:at + part.shape[1] * dim] = part.reshape(self.rows, -1)
        self.x = dev(x)
        self.out = torch.full((self.rows, q_heads, dim), 77, dtype=torch.int16, device="cuda")
        self.gstarts, self.status = i32(self.starts), i32([0])

    def run(self, stream=None, starts=None):
        Hq, Hkv, D = self.dims
        return abi.tv_attend_prompt(Hq, Hkv, D, self.x, self.x[:, Hq * D:], self.x[:, (Hq + Hkv) * D:], self.width, self.width,
                                    self.gstarts if starts is None else starts, len(self.lens), self.rows, self.out, self.status, stream)

    def result(self):
        assert self.run() == 0
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0, abi.STATUS.get(int(self.status.item()))
        out = host(self.out)
        assert (out[:self.starts[0]] == 77).all() and (out[self.starts[-1]:] == 77).all()   # rows of no sequence
        return bf16_to_f64(out)[self.starts[0]:self.starts[-1]]

    def check(self):
        got = self.result()
        o, off = attend_prompt(bf16_to_f64(self.q), bf16_to_f64(self.k), bf16_to_f64(self.v), self.starts, True)
        used = slice(self.starts[0], self.starts[-1])
        close(got, o[used], off[used])


HEADS = [(4, 2, 64), (40, 8, 128), (8, 2, 128), (2, 2, 128), (1, 1, 64), (24, 1, 128), (33, 1, 64), (128, 1, 64)]


@pytest.mark.parametrize("q_heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("length", [1, 2, 64, 129])
def test_one_sequence(gpu, q_heads, kv_heads, dim, length):
    Prompt([length], q_heads, kv_heads, dim, seed=length).check()


@pytest.mark.parametrize("q_heads,kv_heads,dim", HEADS[:6])
def test_packed_with_nan_around(gpu, q_heads, kv_heads, dim):
    """Odd lengths, empty sequences, rows before and behind, a padded row stride, NaN wherever no sequence is."""
    Prompt([3, 0, 127, 128, 1, 255, 0, 60, 300], q_heads, kv_heads, dim, seed=q_heads, before=5, behind=40, pad=8).check()


@pytest.mark.parametrize("q_heads,kv_heads,dim,length", [(5, 1, 128, 1500), (1, 1, 128, 1281), (2, 1, 64, 1024), (8, 1, 64, 777)])
def test_long(gpu, q_heads, kv_heads, dim, length):
    """Many windows a tile; one query head to a tile of 128 tokens and more."""
    Prompt([length, 257], q_heads, kv_heads, dim, seed=length).check()


@pytest.mark.parametrize("q_heads,kv_heads,dim", [(10, 2, 64), (10, 2, 128), (4, 4, 64), (48, 2, 64)])
def test_more_places_than_blocks(gpu, q_heads, kv_heads, dim):
    """Blocks that take over several places each, of one window to many, of one tile of queries and of two."""
    tokens = 128 // (q_heads // kv_heads)
    lens = [1500, tokens, 900, 3 * tokens, 1, 700, 2 * tokens + 1, 1111, 130, 5 * tokens - 1, 600, 257, 1, 800]
    Prompt(lens if dim == 128 or q_heads > 4 else lens * 3, q_heads, kv_heads, dim, seed=dim + q_heads).check()


def test_many_short(gpu):
    rng = np.random.default_rng(1)
    Prompt(rng.integers(0, 9, 700).tolist(), 4, 2, 64, seed=2).check()


def test_no_sequence_at_all(gpu):
    p = Prompt([0, 0], 4, 2, 64, before=2, behind=3)
    assert len(p.result()) == 0


def test_large_scores_move_the_offsets(gpu):
    Prompt([700, 130], 4, 2, 64, seed=3, scale=30.0).check()


def test_rising_scores_rescale_every_window(gpu):
    """Keys that grow towards the front, where the windows go: every window moves every offset."""
    def edit(p):
        p.q[:], p.k[:] = bits(np.ones(p.q.shape)), bits(np.zeros(p.k.shape))
        p.k[:, :, 0] = bits(np.repeat(np.linspace(400, 0, p.rows)[:, None], p.k.shape[1], 1))
    Prompt([1100], 4, 2, 128, seed=4, edit=edit).check()


@pytest.mark.parametrize("up", [1.0, 2.0 ** 7, -2.0 ** 7])
def test_scores_at_the_end_of_their_precision(gpu, up):
    """Scores of 2^20 and 2^27 (powers of two), known to half of 2^-4 and of 2^3.

    The products are integers below 2^24 times `up`, so the scores are exact.  The second window's are chosen so
    that an offset taken from the first one's, 20 beyond it, seems to be right for them (they round to at most 2
    above it) while 64 exponentials add up to more than the 256 that an offset may have."""
    f = np.float32
    scale = f(1.4426950408889634 / 8)
    for first in range(4_000_000, 4_002_000):
        x = (first + np.arange(-300, 400)) * up
        m = f(f(f(first * up) * scale) + f(20))
        over = x * float(scale) - float(m)
        found = np.flatnonzero((x.astype(f) * scale <= f(m + f(2))) & (over > 2.012) & (over < 60))
        if found.size:
            break
    assert found.size
    second = int(found[0]) - 300 + first

    def rows(dot):
        whole, rest = divmod(dot, 256)
        return np.array([whole // 63 + (i < whole % 63) for i in range(63)] + [rest], np.float64)

    def edit(p):
        p.q[:], p.k[:] = bits(np.full(p.q.shape, 256.0 * up)), bits(np.broadcast_to(rows(first), p.k.shape))
        p.q[:, :, 63] = bits(np.array([up]))[0]
        p.k[256:384] = bits(rows(second))
    Prompt([700], 1, 1, 64, seed=11, edit=edit).check()


@pytest.mark.parametrize("q_heads,kv_heads,dim", [(5, 1, 128), (3, 1, 64), (1, 1, 128)])
def test_very_low_scores(gpu, q_heads, kv_heads, dim):
    """Scores of minus some hundreds everywhere: an offset that is not the row's own would leave nothing of it."""
    def edit(p):
        p.q[:, :, 0], p.k[:] = bits(np.full(p.q.shape[:2], 64.0)), bits(np.zeros(p.k.shape))
        p.k[:, :, 0] = bits(np.random.default_rng(9).uniform(-64, -60, p.k.shape[:2]))
    Prompt([300, 131, 128, 9], q_heads, kv_heads, dim, seed=8, edit=edit).check()


@pytest.mark.parametrize("value", [0x7FC0, 0x7F80, 0xFF80])
@pytest.mark.parametrize("q_heads,kv_heads,dim,lens", [(4, 2, 64, [300, 90]), (2, 2, 128, [513, 3]), (40, 8, 128, [70, 200])])
def test_what_a_row_may_not_see_does_not_reach_it(gpu, value, q_heads, kv_heads, dim, lens):
    """NaN and infinities in V (and NaN in K) of one token: the rows before it and the other sequences are as without it;
    the rows from it on have the value in that dimension (NaN in K: NaN everywhere)."""
    for at in (0, 1, lens[0] // 2, lens[0] - 1, lens[0]):
        plain = Prompt(lens, q_heads, kv_heads, dim, seed=5).result()

        def edit(p):
            p.v[at, kv_heads - 1, 7] = value
        got = Prompt(lens, q_heads, kv_heads, dim, seed=5, edit=edit).result()
        seen = np.zeros(got.shape, bool)
        G = q_heads // kv_heads
        seen[at:(lens[0] if at < lens[0] else sum(lens)), (kv_heads - 1) * G:, 7] = True
        assert np.array_equal(got[~seen], plain[~seen])
        want = bf16_to_f64(np.array([value], np.uint16))[0]
        assert np.array_equal(got[seen], np.full(seen.sum(), want), equal_nan=True)
    both = Prompt(lens, q_heads, kv_heads, dim, seed=5, edit=lambda p: p.v.__setitem__((slice(10, 13, 2), 0, 3), [0x7F80, 0xFF80])).result()
    assert np.isposinf(both[10:12, 0, 3]).all() and np.isnan(both[12:lens[0], 0, 3]).all() and np.isfinite(both[:10]).all()
    k = Prompt(lens, q_heads, kv_heads, dim, seed=5, edit=lambda p: p.k.__setitem__((20, 0, 3), NAN)).result()
    assert np.isfinite(k[:20]).all() and np.isnan(k[20:lens[0], :q_heads // kv_heads]).all() and np.isfinite(k[lens[0]:]).all()


@pytest.mark.parametrize("q_heads,kv_heads,dim", [(4, 2, 64), (5, 1, 128), (1, 1, 128)])
@pytest.mark.parametrize("early,late", [(0x7FC0, 0x7F80), (0x7FC0, 0xFF80), (0xFF80, 0x7F80), (0x7F80, 0xFF80), (0x7F80, 0x7F80), (0xFF80, 0xFF80)])
def test_values_that_are_not_finite_add_up(gpu, early, late, q_heads, kv_heads, dim):
    """An early token's value comes through the products, that of a row's own tile pair beside them: both together are
    what their sum is, wherever the tile pairs begin."""
    n = 700
    plain = Prompt([n], q_heads, kv_heads, dim, seed=13).result()
    a, b = bf16_to_f64(np.array([early, late], np.uint16))
    with np.errstate(invalid="ignore"):
        both = a + b
    for first, second in ((10, 200), (3, 520), (130, 699), (255, 257), (0, 1)):
        def edit(p):
            p.v[first, 0, 3], p.v[second, 0, 3] = early, late
        got = Prompt([n], q_heads, kv_heads, dim, seed=13, edit=edit).result()
        want = plain.copy()
        G = q_heads // kv_heads
        want[first:, :G, 3], want[second:, :G, 3] = a, both
        assert np.array_equal(got, want, equal_nan=True), (first, second)


@pytest.mark.parametrize("value", [0x7FC0, 0x7F80, 0xFF80])
@pytest.mark.parametrize("what", ["q", "k"])
def test_a_row_that_is_nan_stays_nan_beside_them(gpu, what, value):
    """NaN in a row's query, or in a key that rows see, next to a V that is not finite in a token of the same tile pair."""
    def edit(p):
        p.v[200, 0, 3] = value
        if what == "q":
            p.q[210, 1, 5] = NAN
        else:
            p.k[190, 0, 5] = NAN
    got = Prompt([300], 4, 2, 64, seed=14, edit=edit).result()
    want = bf16_to_f64(np.array([value], np.uint16))[0]
    nan = np.zeros(got.shape, bool)
    if what == "q":
        nan[210, 1] = True
        hit = nan.copy()
        hit[200:, :2, 3] = True
        assert np.array_equal(got[hit & ~nan], np.full((hit & ~nan).sum(), want), equal_nan=True)
        assert np.isfinite(got[~hit]).all()
    else:
        nan[190:, :2] = True
        assert np.isfinite(got[~nan]).all()
    assert np.isnan(got[nan]).all()


def test_separate_tensors_with_strides_of_their_own(gpu):
    p = Prompt([150, 70], 6, 2, 64, seed=12)
    o, off = attend_prompt(bf16_to_f64(p.q), bf16_to_f64(p.k), bf16_to_f64(p.v), p.starts, True)
    q, k, v = dev(p.q), dev(np.pad(p.k.reshape(220, -1), ((0, 0), (0, 24)), constant_values=NAN)), None
    v = dev(np.pad(p.v.reshape(220, -1), ((0, 0), (0, 24)), constant_values=NAN))
    assert abi.tv_attend_prompt(6, 2, 64, q, k, v, 384, 152, p.gstarts, 2, 220, p.out, p.status) == 0
    assert int(p.status.item()) == 0
    close(bf16_to_f64(host(p.out)), o, off)


def test_two_calls_at_once(gpu):
    """On two streams, each on its own tensors and status."""
    ps = [Prompt([900 + 300 * i, 5], 8, 2, 128, seed=20 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip(ps, streams):
            assert p.run(s) == 0
    torch.cuda.synchronize()
    got = [p.out.clone() for p in ps]
    for p, g in zip(ps, got):
        assert int(p.status.item()) == 0
        p.check()
        assert torch.equal(p.out, g)


def test_refusals(gpu):
    for starts in ([5, 4, 6], [-1, 4, 6], [0, 4, 101], [0, 101, 100]):
        p = Prompt([40, 60], 4, 2, 64)
        assert p.run(starts=i32(starts)) == 0
        assert int(p.status.item()) == abi.CODES["TV_E_SEQ"] and (host(p.out) == 77).all()
    p = Prompt([40, 60], 4, 2, 64)
    p.status.fill_(abi.CODES["TV_E_TOKEN"])
    assert p.run() == 0
    assert int(p.status.item()) == abi.CODES["TV_E_TOKEN"] and (host(p.out) == 77).all()


def test_captured_and_replayed_with_other_starts(gpu):
    """The same bits from a plain call, from a replay and on a side stream; the starts are read when it runs."""
    p = Prompt([300, 211], 8, 2, 128, seed=6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        assert p.run(torch.cuda.current_stream()) == 0
    for starts in ([0, 300, 511], [100, 100, 511], [0, 1, 2]):
        p.starts = starts
        p.gstarts.copy_(i32(starts))
        p.out.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        a = host(p.out).copy()
        p.out.fill_(77)
        p.check()
        assert np.array_equal(a, host(p.out))


def test_the_same_bits_every_time(gpu):
    p = Prompt([2000, 1], 10, 2, 128, seed=7)
    assert p.run() == 0
    first = p.out.clone()
    for _ in range(100):
        assert p.run() == 0
        assert torch.equal(p.out, first)


def test_a_serving_run(gpu):
    """Two prompts through attention into pages, tokens decoded, a sequence forked, drafts given back, the pool
    compacted, and the paged sequence verified as a contiguous cache and its committed rows written back; every result
    against the oracle on the rows that were put in."""
    import oracle
    from speculative_tree_verify_gb300 import device as dv
    from speculative_tree_verify_gb300 import synth
    d, ps, layers = synth.TINY, 16, 2
    Hq, Hkv, D = d.n_q_heads, d.n_kv_heads, d.head_dim
    rng = np.random.default_rng(11)
    c = dv.PagedCache.alloc(d, layers, 24, ps, 5, 6)
    c.k.fill_(float("nan"))
    c.v.fill_(float("nan"))
    rows_of = {0: [], 2: [], 3: []}              # what the oracle keeps: (k, v) of every token

    def ok(rc, what):
        dv.check(rc, what)
        assert int(c.status.item()) == 0, (what, abi.STATUS.get(int(c.status.item())))

    def rows(n):
        x = bits(rng.standard_normal((n, (Hq + 2 * Hkv) * D)))
        parts = x[:, :Hq * D].reshape(n, Hq, D), x[:, Hq * D:(Hq + Hkv) * D].reshape(n, Hkv, D), x[:, (Hq + Hkv) * D:].reshape(n, Hkv, D)
        return dev(x).view(torch.bfloat16), parts

    def kv(s):
        return (bf16_to_f64(np.array([r[i] for r in rows_of[s]])) for i in (0, 1))

    # prompts of 37 and 16 tokens in one pass
    lens = [37, 16]
    starts, ids = i32([0, 37, 53]), i32([2, 0])
    x, (q, k, v) = rows(53)
    out = torch.zeros(53, Hq, D, device="cuda", dtype=torch.bfloat16)
    ok(c.attend_prompt(x, starts, out), "attend_prompt")
    o, off = attend_prompt(bf16_to_f64(q), bf16_to_f64(k), bf16_to_f64(v), [0, 37, 53], True)
    close(bf16_to_f64(host(out.view(torch.int16))), o, off, "prompts")
    ok(c.extend(ids, i32(lens)), "extend")
    for layer in range(layers):
        ok(c.write(layer, ids, i32([0, 0]), starts, x), "write")
    rows_of[2] = [(k[t], v[t]) for t in range(37)]
    rows_of[0] = [(k[t], v[t]) for t in range(37, 53)]

    def decode(seqs):
        x, (q, k, v) = rows(len(seqs))
        ids, out = i32(seqs), torch.zeros(len(seqs), Hq, D, device="cuda", dtype=torch.bfloat16)
        ok(c.extend(ids, i32([1] * len(seqs))), "extend")
        for layer in range(layers):
            ok(c.attend(layer, ids, x, out), "attend")
        for i, s in enumerate(seqs):
            rows_of[s] = rows_of[s] + [(k[i], v[i])]
            o, off = attend(bf16_to_f64(q[i]), *kv(s), True)
            close(bf16_to_f64(host(out.view(torch.int16))[i]), o, off, f"token of sequence {s}")

    for _ in range(3):
        decode([0, 2])
    ok(c.fork(i32([2]), i32([3])), "fork")
    rows_of[3] = list(rows_of[2])
    for _ in range(9):                            # the two part ways: over a page's end
        decode([3, 0, 2])
    ok(c.release(i32([3, 0]), i32([41, 0])), "release")
    rows_of[3], rows_of[0] = rows_of[3][:41], []
    remap, used = i32([0] * 24), i32([0])
    ok(c.compact(remap, used), "compact")
    held = c.refs.cpu().numpy()
    assert (held[:int(used.item())] > 0).all() and not held[int(used.item()):].any()
    decode([2, 3])
    # sequence 3 as a contiguous cache under a tree verify, and its committed path back into pages
    n, tree = len(rows_of[3]), synth.tree_spine_random(8, 4, d.vocab, 3)
    model = synth.gen_model(d, 1, random_gains=True)
    cache = synth.gen_cache(d, n, n + 16, 5)
    gk, gv = (dev(getattr(cache, w)).view(torch.bfloat16) for w in "kv")
    gk[:, :n] = 0
    gv[:, :n] = 0
    ok(c.read_into(1, i32([3]), i32([0]), i32([0, n]), n, gk, gv), "read")
    for t, (a, b) in enumerate(rows_of[3]):
        cache.k[:, t], cache.v[:, t] = a, b
    assert np.array_equal(host(gk.view(torch.int16)), cache.k) and np.array_equal(host(gv.view(torch.int16)), cache.v)
    req = dv.DeviceRequest(gk, gv, n, torch.from_numpy(tree.parent.copy()).cuda(), torch.from_numpy(tree.token.copy()).cuda())
    b = dv.RoundBuffers.alloc(d, tree.n, 1, n)
    dv.run_round(dv.DeviceModel.from_host(model), [req], b)
    torch.cuda.synchronize()
    assert int(b.status.item()) == 0
    orc = oracle.verify_tree(model, cache, tree)
    lg, ol = b.logits.cpu().numpy().astype(np.float64), orc["logits"].astype(np.float64)
    assert (np.abs(lg - ol).max(1) <= 2e-2 * np.sqrt((ol * ol).mean(1))).all()
    more = int(b.new_ctx.item()) - n
    assert more == int(b.accept_len.item()) + 1
    ok(c.extend(i32([3]), i32([more])), "extend")
    ok(c.write_from(1, i32([3]), i32([n]), i32([0, more]), more, gk[:, n:], gv[:, n:]), "write_from")
    back = torch.zeros_like(gk), torch.zeros_like(gv)
    ok(c.read_into(1, i32([3]), i32([0]), i32([0, n + more]), n + more, *back), "read")
    for a, w in zip(back, (gk, gv)):
        assert torch.equal(a[:, :n + more].view(torch.int16), w[:, :n + more].view(torch.int16))
