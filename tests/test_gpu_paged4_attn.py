"""tv_attend_paged4 against fp64 attention over what the cache stands for.

Tolerance, per element, with weights w, result o and A = sum w |v - o|, B = sum
w |v|: a weight times a scale is rounded to fp16 for the product with V, 2^-11 of
itself, while the sum of the weights is not: 2^-11 B.  Below fp16's normal values
(2^-14, the largest weight times the largest scale being 2^7 or more) half a step
is 2^-25, 2^-32 of the largest, of at most 15 tokens' codes each: 2^-28 B' with
B' = tokens * the largest |v|.  Scores as test_gpu_paged_attn.py has them (1e-3 of
a weight: the first sums here are at most 16 times a product's size): 1e-3 A.
fp32 sums and joins: 2^-10 A + 2^-16 |o|, and the offset of the codes, at most
16/7 of the largest value a token, rounds in them with 2^-22 B'' (B'' = sum w
times the largest |v| of the group, at most the largest).  One rounding of the
result to bf16, 2^-8."""
import numpy as np
import pytest
import torch

from oracle import bf16_to_f64, longctx
from speculative_tree_verify_gb300 import abi
from speculative_tree_verify_gb300.device import PagedCache, PagedCache4, rotate
from speculative_tree_verify_gb300.synth import Dims
from test_gpu_paged_attn import NAN, bits, dev, host, i32

pytestmark = pytest.mark.gpu

ALL = abi.NO_WINDOW


def spreads(q, k, v):
    """(o, A, B, largest |v|) of one token: q [heads][D], k and v [tokens][kv_heads][D]."""
    heads, D = q.shape
    o, A, B = (np.zeros((heads, D)) for _ in range(3))
    for h in range(heads if len(k) else 0):
        g = h * k.shape[1] // heads
        a = k[:, g] @ q[h] / np.sqrt(D)
        w = np.exp(a - a.max())
        w /= w.sum()
        o[h] = w @ v[:, g]
        A[h], B[h] = w @ np.abs(v[:, g] - o[h]), w @ np.abs(v[:, g])
    return o, A, B, np.abs(v).max() if len(k) else 0.0


def close4(got, q, k, v, what="", but=None):
    """but: elements that are not compared."""
    o, A, B, top = spreads(q, k, v)
    if but is not None:
        got = np.where(but, o, got)
    err = np.abs(got - o)
    tol = (2.0 ** -11 * B + (1e-3 + 2.0 ** -10) * A + 2.0 ** -16 * np.abs(o) + (2.0 ** -28 * len(k) + 2.0 ** -22) * top) * (1 + 2.0 ** -7) \
        + 2.0 ** -8 * np.abs(o) * (1 + 2.0 ** -7) + 1e-30
    assert np.isfinite(got).all(), what
    assert (err <= tol).all(), f"{what}: worst {np.max(err / tol):.3f} of the tolerance"


class Case4:
    """Sequences in random pages of a pool whose other bytes are random, scales that are NaN among them."""

    def __init__(self, lens, q_heads, kv_heads, dim, ps, window=ALL, sinks=0, layers=1, layer=0, seed=0, new=True, scale=1.0, vscale=1.0,
                 unlisted=2, pad=0, edit=None):
        rng = np.random.default_rng(seed)
        self.lens, self.dims, self.layer, self.new, self.window, self.sinks = lens, (q_heads, kv_heads, dim), layer, new, window, sinks
        n = len(lens)
        need = [-(-x // ps) for x in lens]
        n_pages = sum(need) + 3
        shape = (layers, n_pages, kv_heads, ps // 16, 9 * dim)
        self.k, self.v = (rng.integers(0, 256, shape, dtype=np.uint8) for _ in range(2))
        self.rows, self.ps = longctx.Pages4(self.k, self.v, ps, dim), ps
        places, at = rng.permutation(n_pages), 0
        self.ids = rng.permutation(n + unlisted)[:n].tolist()
        self.pages = np.full((n + unlisted, max(1, max(need))), -3, np.int32)
        self.all_lens = np.zeros(n + unlisted, np.int32)
        self.kv = []   # bf16 rows, before the rounding
        for i, x in enumerate(lens):
            self.pages[self.ids[i], :need[i]] = places[at:at + need[i]]
            at += need[i]
            self.all_lens[self.ids[i]] = x
            self.kv.append([bits(rng.standard_normal((x, kv_heads, dim))), bits(rng.standard_normal((x, kv_heads, dim)) * vscale)])
        self.q = bits(rng.standard_normal((n, q_heads, dim)) * scale)
        if edit:
            edit(self)
        self.held = []
        for i, x in enumerate(lens):
            pair = []
            see = set(longctx.seen(x - 1, window, sinks)) if x else ()
            for name, y in zip("kv", self.kv[i]):
                codes, scales = longctx.quantise(y)
                pair.append((codes, scales))
                for t in range(x - (1 if new else 0)):
                    p = self.pages[self.ids[i], t // ps]
                    # what is not seen stands for NaN
                    self.rows.put(name, layer, p, t % ps, codes[t], scales[t] if t in see else np.full_like(scales[t], 0x7FC0))
            self.held.append(pair)
        self.width = (q_heads + 2 * kv_heads) * dim + pad
        self.qkv = np.full((n, self.width), NAN, np.uint16)
        self.qkv[:, :q_heads * dim] = self.q.reshape(n, -1)
        for i, x in enumerate(lens):
            if x:
                for j in (0, 1):
                    a = (q_heads + j * kv_heads) * dim
                    self.qkv[i, a:a + kv_heads * dim] = self.kv[i][j][-1].reshape(-1)

    def upload(self):
        n, (Hq, Hkv, D) = len(self.lens), self.dims
        self.gk, self.gv = torch.from_numpy(self.k).cuda(), torch.from_numpy(self.v).cuda()
        self.refs, self.gpages, self.glens, self.gids = i32(np.ones(self.k.shape[1])), i32(self.pages), i32(self.all_lens), i32(self.ids)
        self.status, self.gqkv = i32([0]), dev(self.qkv)
        self.pool = abi.TvPool4(self.gk.data_ptr(), self.gv.data_ptr(), self.refs.data_ptr(), self.k.shape[0], self.k.shape[1], Hkv, self.ps, D)
        self.seqs = abi.TvSeqs(self.gpages.data_ptr(), self.glens.data_ptr(), *self.pages.shape)
        self.size = abi.tv_attend_paged4_workspace_size(self.pool, Hq, n)
        self.ws = torch.empty(self.size, dtype=torch.uint8, device="cuda")
        self.out = torch.full((n, Hq, D), 77, dtype=torch.int16, device="cuda")

    def call(self, stream=None, ids=None):
        n, (Hq, Hkv, D) = len(self.lens), self.dims
        kn, vn = (self.gqkv[:, (Hq + i * Hkv) * D:] for i in (0, 1)) if self.new else (None, None)
        return abi.tv_attend_paged4(self.pool, self.layer, self.seqs, self.gids if ids is None else ids, n, Hq, self.window, self.sinks, self.gqkv,
                                    self.width, kn, vn, self.width, self.out, self.ws, self.size, self.status, stream)

    def run(self):
        self.upload()
        assert self.call() == 0
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0, abi.STATUS.get(int(self.status.item()))
        return bf16_to_f64(host(self.out))

    def rows_of(self, i):
        see = longctx.seen(self.lens[i] - 1, self.window, self.sinks) if self.lens[i] else []
        return tuple(longctx.stands_for(c[see], s[see]) for c, s in self.held[i])

    def check(self):
        got, q = self.run(), bf16_to_f64(self.q)
        for i, x in enumerate(self.lens):
            close4(got[i], q[i], *self.rows_of(i), f"sequence {i} of {x} tokens")
        self.stored()

    def stored(self):
        """The new rows' codes are in their slots, and nothing else has changed."""
        if self.new:
            for i, x in enumerate(self.lens):
                if x:
                    p = self.pages[self.ids[i], (x - 1) // self.ps]
                    for name, (codes, scales) in zip("kv", self.held[i]):
                        self.rows.put(name, self.layer, p, (x - 1) % self.ps, codes[-1], scales[-1])
        assert (self.gk.cpu().numpy() == self.k).all() and (self.gv.cpu().numpy() == self.v).all()


@pytest.mark.parametrize("new", [True, False])
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(4, 2, 64), (40, 8, 128), (8, 8, 128), (8, 1, 64), (9, 1, 128), (24, 1, 128), (33, 1, 64), (16, 1, 64)])
def test_lengths_and_heads(gpu, q_heads, kv_heads, dim, new):
    Case4([1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 0, 300, 1000], q_heads, kv_heads, dim, 16, layers=2, layer=1, seed=q_heads, new=new, pad=8).check()


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(ALL, 0), (1, 0), (1, 1), (16, 0), (63, 4), (64, 64), (200, 5), (1000, 130), (7, ALL)])
def test_pages_and_windows(gpu, ps, dim, window, sinks):
    Case4([700, 3, 129, 1283, 64], 4, 2, dim, ps, window, sinks, seed=ps).check()


@pytest.mark.parametrize("lens", [[1], [64 * 9], [20011], [1, 9001, 3, 1], [700] * 40, [5] * 33 + [900], [3, 0, 70] * 230, [1, 2] * 1024],
                         ids=lambda x: f"{len(x)}x{max(x)}")
def test_long_short_and_many(gpu, lens):
    Case4(lens, 4, 2, 64, 16, seed=len(lens)).check()


@pytest.mark.parametrize("dim,ps", [(128, 64), (64, 16)])
@pytest.mark.parametrize("q_heads", [3, 12])
def test_many_tiles_a_cta(gpu, dim, ps, q_heads):
    Case4([33000, 7000, 1, 500], q_heads, 1, dim, ps, seed=dim).check()


@pytest.mark.parametrize("q_heads,kv_heads,dim", [(10, 2, 128), (16, 2, 64), (12, 1, 64), (24, 1, 64), (40, 1, 128)])
@pytest.mark.parametrize("n", [600, 2048])
def test_many_sequences_of_one_tile(gpu, q_heads, kv_heads, dim, n):
    """More runs a block than places for their queries, whatever those are."""
    rng = np.random.default_rng(n)
    Case4(rng.integers(1, 65, n).tolist(), q_heads, kv_heads, dim, 16, seed=n + dim).check()


@pytest.mark.parametrize("scale", [30.0, 1e-30, 2.0 ** 90])
def test_queries_of_any_size(gpu, scale):
    """Offsets that move; queries whose scores are all but equal; those of an exponent no score can hold are spread over
    keys as small."""
    def edit(c):
        if scale > 1e20:
            for pair in c.kv:
                pair[0][:] = bits((bf16_to_f64(pair[0]) / scale).astype(np.float32))
    Case4([700, 130, 3000], 8, 2, 128, 32, seed=3, scale=scale, edit=edit).check()


@pytest.mark.parametrize("scale,kscale", [(2.0 ** -112, 2.0 ** 111), (2.0 ** -115, 2.0 ** 114), (2.0 ** -118, 2.0 ** 117), (2.0 ** -125, 2.0 ** 123)])
def test_the_smallest_queries(gpu, scale, kscale):
    """Down to values that are not normal, beside keys that make scores of them."""
    def edit(c):
        for pair in c.kv:
            pair[0] = bits(bf16_to_f64(pair[0]) * kscale)
    for heads in ((8, 2, 128), (12, 1, 64)):
        Case4([1, 70, 700], *heads, 32, scale=scale, seed=41, edit=edit).check()


@pytest.mark.parametrize("vscale", [2.0 ** -60, 1e-4, 1e4, 2.0 ** 90])
def test_values_of_any_size(gpu, vscale):
    Case4([700, 65], 8, 2, 128, 32, seed=4, vscale=vscale).check()


def test_scales_that_grow_and_shrink(gpu):
    """Values of every size in one sequence: the weights' range follows the largest so far."""
    def edit(c):
        for pair in c.kv:
            x = bf16_to_f64(pair[1])
            n = len(x)
            pair[1][:] = bits((x * 2.0 ** np.linspace(-40, 30, n)[:, None, None]).astype(np.float32))
    Case4([2000, 300], 5, 1, 128, 64, seed=5, edit=edit).check()


def test_one_loud_token(gpu):
    """A value 2^20 times the others', which weighs next to nothing, does not cost the others their digits."""
    def edit(c):
        c.kv[0][1][100] = bits(bf16_to_f64(c.kv[0][1][100]) * 2.0 ** 20)
        c.kv[0][0][100] = bits(-8 * np.sign(bf16_to_f64(c.q[0]).reshape(2, 4, 128).mean(1)))
    c = Case4([900], 8, 2, 128, 16, seed=6, edit=edit)
    got, q = c.run(), bf16_to_f64(c.q)
    close4(got[0], q[0], *c.rows_of(0))


def test_equal_values_pass_through(gpu):
    """V that is the same in every token comes out as it stands, whatever the weights are, to the roundings of them."""
    def edit(c):
        for pair in c.kv:
            pair[1][:] = pair[1][:1]
    c = Case4([1000, 40], 8, 2, 64, 16, seed=7, edit=edit)
    got = c.run()
    for i in range(2):
        v = c.rows_of(i)[1][0].repeat(4, 0)
        assert (np.abs(got[i] - v) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16) * (1 + 2.0 ** -7) * np.abs(v) + 2.0 ** -22 * np.abs(v).max()).all()


def test_groups_that_are_not_finite(gpu):
    """A K group of NaN makes its heads' rows NaN; a V group its 32 dimensions, whatever it weighs; nothing else."""
    def edit(c):
        c.kv[0][0][50, 0, 3] = 0x7F80
        c.kv[1][1][20, 1, 70] = NAN
        c.kv[2][1][-1, 0, 5] = 0xFF80   # the new token's own
    c = Case4([200, 90, 33], 8, 2, 128, 16, seed=8, edit=edit)
    got, q = c.run(), bf16_to_f64(c.q)
    assert np.isnan(got[0, :4]).all() and np.isfinite(got[0, 4:]).all()
    bad = np.zeros((8, 128), bool)
    bad[4:, 64:96] = True
    assert np.isnan(got[1][bad]).all() and np.isfinite(got[1][~bad]).all()
    bad = np.zeros((8, 128), bool)
    bad[:4, :32] = True
    assert np.isnan(got[2][bad]).all() and np.isfinite(got[2][~bad]).all()
    for i in (1, 2):
        k, v = c.rows_of(i)
        close4(got[i], q[i], k, np.where(np.isnan(v), 0, v), but=np.isnan(got[i]))


def test_refusals(gpu):
    c = Case4([100, 40, 70], 4, 2, 64, 16, seed=9)
    c.upload()

    def refused(code, ids):
        assert c.call(ids=i32(ids)) == 0
        torch.cuda.synchronize()
        assert abi.STATUS[int(c.status.item())] == code
        c.status.zero_()
        assert (host(c.out) == 77).all() and (c.gk.cpu().numpy() == c.k).all()

    refused("TV_E_SEQ", [c.ids[0], c.ids[1], c.ids[0]])
    refused("TV_E_SEQ", [c.ids[0], c.ids[1], len(c.pages)])
    refused("TV_E_SEQ", [-1, c.ids[1], c.ids[2]])
    c.glens[c.ids[2]] = c.pages.shape[1] * 16 + 1
    refused("TV_E_SEQ", c.ids)
    c.glens[c.ids[2]] = 70
    c.status.fill_(-5)
    assert c.call() == 0
    torch.cuda.synchronize()
    assert int(c.status.item()) == -5 and (host(c.out) == 77).all()
    c.status.zero_()
    c.gpages[c.ids[0], 2] = c.k.shape[1]
    assert c.call() == 0
    torch.cuda.synchronize()
    assert abi.STATUS[int(c.status.item())] == "TV_E_PAGE"


def test_listed_twice_without_new_rows(gpu):
    c = Case4([100, 40], 4, 2, 64, 16, seed=10, new=False)
    c.upload()
    assert c.call(ids=i32([c.ids[0], c.ids[0]])) == 0
    torch.cuda.synchronize()
    got = host(c.out)
    assert int(c.status.item()) == 0
    close4(bf16_to_f64(got[0]), bf16_to_f64(c.q[0]), *c.rows_of(0))
    close4(bf16_to_f64(got[1]), bf16_to_f64(c.q[1]), *c.rows_of(0))


def test_two_calls_at_once_and_the_same_bits(gpu):
    a, b = Case4([3000, 5, 900], 40, 8, 128, 16, seed=11), Case4([70, 8000], 12, 1, 64, 32, seed=12)
    first = [c.run() for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for c in (a, b):
            c.out.fill_(77)
        torch.cuda.synchronize()
        for c, s in zip((a, b), streams):
            assert c.call(s) == 0
        torch.cuda.synchronize()
        for c, f in zip((a, b), first):
            assert np.array_equal(bf16_to_f64(host(c.out)), f)


def test_graphs_share_a_workspace(gpu):
    """Two captured calls on one workspace, replayed in turn as the sequence grows."""
    d = Dims(hidden=64, n_q_heads=10, n_kv_heads=2, head_dim=128, vocab=64)
    c = PagedCache4.alloc(d, 2, 60, 16, 3, 20)
    rng = np.random.default_rng(13)
    ids, one = i32([2]), i32([1])
    rows = bits(rng.standard_normal((2, 300, (10 + 4) * 128)))
    assert c.extend(ids, i32([255])) == 0
    for layer in (0, 1):
        assert c.write(layer, ids, i32([0]), i32([0, 255]), dev(rows[layer, :255])) == 0
    qkv = [torch.zeros(1, 14 * 128, dtype=torch.int16, device="cuda") for _ in (0, 1)]
    out = [torch.zeros(1, 10, 128, dtype=torch.int16, device="cuda") for _ in (0, 1)]
    graphs = []
    for layer in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s = torch.cuda.current_stream()
            if layer == 0:
                assert c.extend(ids, one, s) == 0
            assert c.attend(layer, ids, qkv[layer], out[layer], s, window=200, sinks=3) == 0
        graphs.append(g)
    for t in range(255, 300):
        for layer in (0, 1):
            qkv[layer].copy_(dev(rows[layer, t:t + 1]))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0 and int(c.lens[2]) == t + 1
        if t in (255, 256, 270, 299):
            for layer in (0, 1):
                x = rows[layer, :t + 1]
                see = longctx.seen(t, 200, 3)
                k, v = (longctx.stands_for(*longctx.quantise(x[see, (10 + 2 * i) * 128:(12 + 2 * i) * 128].reshape(-1, 2, 128))) for i in (0, 1))
                close4(bf16_to_f64(host(out[layer])[0]), bf16_to_f64(x[-1, :1280].reshape(10, 128)), k, v, f"layer {layer} at {t}")


@pytest.mark.parametrize("kind", [PagedCache, PagedCache4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_serving_run(gpu, kind, interleaved):
    """Projections' rows to answers: positions, windowed prompts, pages, a fork, and tokens that each see the window and
    the sinks of their own sequence; against fp64 over the rows as each step held them."""
    Hq, Hkv, D, window, sinks = 8, 2, 64, 90, 4
    d = Dims(hidden=64, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=D, vocab=64)
    c = kind.alloc(d, 1, 80, 16, 5, 20)
    rng = np.random.default_rng(20 + interleaved)
    rope = abi.tv_rope_init(32, interleaved, 1e4, abi.TV_ROPE_BLEND, 4.0, 64, 1.0, 4.0, 1.1)
    lens = [150, 37]
    starts, ids = [0, 150, 187], i32([3, 1])
    raw = bits(rng.standard_normal((187, (Hq + 2 * Hkv) * D)))
    x, pos = dev(raw), i32(list(range(150)) + list(range(37)))
    assert rotate(rope, x, pos, Hq + Hkv, D, c.status) == 0
    out = torch.zeros(187, Hq, D, dtype=torch.int16, device="cuda")
    assert c.attend_prompt(x, i32(starts), out, window=window, sinks=sinks) == 0
    assert c.extend(ids, i32(lens)) == 0
    assert c.write(0, ids, i32([0, 0]), i32(starts), x) == 0
    assert c.fork(i32([3]), i32([0])) == 0
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    turned = host(x)
    part = lambda y, a, h: y[:, a * D:(a + h) * D].reshape(-1, h, D)
    q, k, v = (bf16_to_f64(part(turned, a, h)) for a, h in ((0, Hq), (Hq, Hkv), (Hq + Hkv, Hkv)))
    # P of the prompt is bf16: test_gpu_paged_attn.py's tolerance
    from test_gpu_paged_attn import close
    o, off = longctx.attend_prompt(q, k, v, starts, window, sinks)
    close(bf16_to_f64(host(out)), o, off)
    held = (lambda y: bf16_to_f64(y)) if kind is PagedCache else (lambda y: longctx.stands_for(*longctx.quantise(y)))
    kb, vb = part(turned, Hq, Hkv), part(turned, Hq + Hkv, Hkv)
    history = {3: [kb[:150], vb[:150]], 1: [kb[150:], vb[150:]]}
    history[0] = [y.copy() for y in history[3]]
    order = [0, 1, 3]
    for step in range(20):
        raw = bits(rng.standard_normal((3, (Hq + 2 * Hkv) * D)))
        x = dev(raw)
        assert rotate(rope, x, i32([len(history[s][0]) for s in order]), Hq + Hkv, D, c.status) == 0
        assert c.extend(i32(order), i32([1] * 3)) == 0
        out = torch.zeros(3, Hq, D, dtype=torch.int16, device="cuda")
        assert c.attend(0, i32(order), x, out, window=window, sinks=sinks) == 0
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        turned, got = host(x), bf16_to_f64(host(out))
        for i, s in enumerate(order):
            for j, a in ((0, Hq), (1, Hq + Hkv)):
                history[s][j] = np.concatenate([history[s][j], part(turned[i:i + 1], a, Hkv)])
            see = longctx.seen(len(history[s][0]) - 1, window, sinks)
            close4(got[i], bf16_to_f64(part(turned[i:i + 1], 0, Hq))[0], held(history[s][0])[see], held(history[s][1])[see], f"step {step}, sequence {s}")


def test_the_longest_length(gpu):
    """2^31 - 16 tokens: a table row that names one page over and over, but for its last place (its 16 tokens weigh less
    than 2^-20).  A warp adds up 2^25 / (6 * 148) tiles of two products or fewer; sums that drop what lies below their last
    place lose at most 2^-23 of themselves a product: 2^17 2^-23 = 2^-6 of sum w |v|, and half of that of the denominator."""
    ps, D, n_pages = 16, 64, 2 ** 27 - 1
    rng = np.random.default_rng(21)
    raw = [np.zeros((1, 2, 1, 1, 9 * D), np.uint8) for _ in range(2)]
    rows, held = longctx.Pages4(*raw, ps, D), []
    for name in "kv":
        codes, scales = longctx.quantise(bits(rng.standard_normal((2, ps, D)) / 8))
        held.append(longctx.stands_for(codes, scales)[0])
        for p in range(2):
            for t in range(ps):
                rows.put(name, 0, p, t, codes[p, t][None], scales[p, t][None])
    q = bits(rng.standard_normal((1, 4, D)) / 2)
    table = torch.zeros(1, n_pages, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    gk, gv, refs, lens = *(torch.from_numpy(x).cuda() for x in raw), i32([1, 1]), i32([n_pages * ps])
    pool, seqs = abi.TvPool4(gk.data_ptr(), gv.data_ptr(), refs.data_ptr(), 1, 2, 1, ps, D), abi.TvSeqs(table.data_ptr(), lens.data_ptr(), 1, n_pages)
    out, st, gq = torch.zeros(1, 4, D, dtype=torch.int16, device="cuda"), i32([0]), dev(q)
    size = abi.tv_attend_paged4_workspace_size(pool, 4, 1)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert abi.tv_attend_paged4(pool, 0, seqs, i32([0]), 1, 4, ALL, 0, gq, 4 * D, None, None, 0, out, ws, size, st) == 0
    assert int(st.item()) == 0
    qf, (kf, vf) = bf16_to_f64(q[0]), held
    w = np.exp(qf @ kf.T / np.sqrt(D))
    w /= w.sum(1, keepdims=True)
    o, mag = w @ vf, w @ np.abs(vf)
    assert (np.abs(bf16_to_f64(host(out))[0] - o) <= (2.0 ** -6 + 2.0 ** -7 + 3 * 2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -22).all()


def test_pages_past_two_to_the_32_bytes(gpu):
    """The last pages of a pool whose K alone is more than 2^32 bytes: written, read, and attended to."""
    ps, D = 16, 64
    n_pages = 2 ** 32 // (9 * D) + 5000
    k, v = (torch.zeros(1, n_pages, 1, 1, 9 * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    rng = np.random.default_rng(22)
    pages = [n_pages - 1, n_pages - 4000, 3]
    kk, vv = (bits(rng.standard_normal((40, 1, D))) for _ in range(2))
    q = bits(rng.standard_normal((1, 2, D)))
    refs, table, lens, ids, st = torch.ones(n_pages, dtype=torch.int32, device="cuda"), i32([pages]), i32([40]), i32([0]), i32([0])
    pool, seqs = abi.TvPool4(k.data_ptr(), v.data_ptr(), refs.data_ptr(), 1, n_pages, 1, ps, D), abi.TvSeqs(table.data_ptr(), lens.data_ptr(), 1, 3)
    assert abi.tv_pages4_write(pool, 0, seqs, ids, i32([0]), i32([0, 39]), 1, 39, dev(kk), dev(vv), D, D, st) == 0
    out = torch.zeros(1, 2, D, dtype=torch.int16, device="cuda")
    size = abi.tv_attend_paged4_workspace_size(pool, 2, 1)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    qkv = dev(np.concatenate([q.reshape(-1), kk[-1].reshape(-1), vv[-1].reshape(-1)]))
    assert abi.tv_attend_paged4(pool, 0, seqs, ids, 1, 2, ALL, 0, qkv, 128, qkv[128:], qkv[192:], 64, out, ws, size, st) == 0
    back = [torch.zeros(40, D, dtype=torch.int16, device="cuda") for _ in range(2)]
    assert abi.tv_pages4_read(pool, 0, seqs, ids, i32([0]), i32([0, 40]), 1, 40, *back, D, D, st) == 0
    assert int(st.item()) == 0
    held = [longctx.stands_for(*longctx.quantise(x)) for x in (kk, vv)]
    for x, b in zip(held, back):
        assert (bf16_to_f64(host(b)) == bf16_to_f64(longctx.bf16(x[:, 0]))).all()
    close4(bf16_to_f64(host(out))[0], bf16_to_f64(q[0]), *held)


def test_many_tokens_without_values(gpu):
    """Weights whose V is zero are summed as all others are, however many they are: 2^18 tokens of one
    sequence a CTA, V zero (a scale of zero) but in the last 128 tokens, whose values are 7; scores 0 in the first
    384 tokens, which is where each warp has its offset from, and 5.375 in all others.
    Tolerance: a weight times a scale is fp16 (2^-11), scores 1e-3, sums of 2^18 / 96 fp32 terms a thread
    2^-12 (each step 2^-24 of the sum), joins 2^-16, the result's rounding 2^-8."""
    D, ps, tokens, n = 64, 128, 1 << 18, torch.cuda.get_device_properties(0).multi_processor_count
    k = torch.full((1, tokens // ps, 1, ps // 16, 9 * D), 0x99, dtype=torch.uint8, device="cuda")   # codes: 1
    v = torch.full_like(k, 0xFF)                                                                    # 7
    ks, vs = (x[..., 8 * D:].view(torch.int16) for x in (k, v))
    ks.fill_(0x3F2C)     # 0.671875
    ks[:, :384 // ps] = 0
    vs.zero_()
    vs[:, -1] = 0x3F80   # 1
    refs, status = i32(np.full(tokens // ps, n)), i32([0])
    pages, lens, ids = i32(np.tile(np.arange(tokens // ps), (n, 1))), i32(np.full(n, tokens)), i32(np.arange(n))
    pool = abi.TvPool4(k.data_ptr(), v.data_ptr(), refs.data_ptr(), 1, tokens // ps, 1, ps, D)
    seqs = abi.TvSeqs(pages.data_ptr(), lens.data_ptr(), n, tokens // ps)
    size = abi.tv_attend_paged4_workspace_size(pool, 2, n)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    q = torch.ones((n, 2, D), dtype=torch.bfloat16, device="cuda").view(torch.int16)
    out = torch.empty_like(q)
    assert abi.tv_attend_paged4(pool, 0, seqs, ids, n, 2, ALL, 0, q, 2 * D, None, None, 0, out, ws, size, status) == 0
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    w = np.exp(D * 0.671875 / 8)
    o = 7 * 128 * w / (384 + (tokens - 384) * w)
    err = np.abs(bf16_to_f64(host(out)) - o)
    assert (err <= o * ((2.0 ** -11 + 2e-3 + 2.0 ** -12 + 2.0 ** -16) * (1 + 2.0 ** -7) + 2.0 ** -8 * (1 + 2.0 ** -7))).all(), err.max() / o


def test_captured_first(gpu):
    """A process whose first call of each kind is made while capturing."""
    import subprocess
    import sys
    code = """
import torch
from speculative_tree_verify_gb300 import abi
from speculative_tree_verify_gb300.device import PagedCache, PagedCache4, rotate
from speculative_tree_verify_gb300.synth import Dims
d = Dims(hidden=64, n_q_heads=4, n_kv_heads=2, head_dim=128, vocab=64)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
x, out = torch.randn(40, 8 * 128, device="cuda").bfloat16(), torch.zeros(40, 4, 128, device="cuda", dtype=torch.bfloat16)
caches = [kind.alloc(d, 1, 9, 16, 2, 6) for kind in (PagedCache, PagedCache4)]
lists = i32([0]), i32([40]), i32([0, 40]), i32(list(range(40)))
rope = abi.tv_rope_init(128)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    s = torch.cuda.current_stream()
    for c in caches:
        assert rotate(rope, x, lists[3], 6, 128, c.status, stream=s) == 0
        assert c.attend_prompt(x, lists[2], out, s, window=9, sinks=2) == 0
        assert c.extend(lists[0], lists[1], s) == 0
        assert c.write(0, lists[0], lists[0], lists[2], x, s) == 0
        assert c.attend(0, lists[0], x, out, s, window=9, sinks=2) == 0
        assert c.release(lists[0], lists[0], s) == 0
g.replay()
g.replay()
torch.cuda.synchronize()
assert [int(c.status.item()) for c in caches] == [0, 0]
assert torch.isfinite(out.float()).all()
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]
