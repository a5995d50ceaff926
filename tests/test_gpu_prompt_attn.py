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
