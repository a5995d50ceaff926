"""tv_rope_rows against oracle/longctx.py (fp64).

Tolerance, per element, u and w the pair: the angle as a fraction of a turn is a
64-bit product of the position and a frequency that a double holds to 2^-53 of
itself: positions below 2^31 and frequencies up to one radian, 2^-24.6 of a turn
at most (the oracle's the same once more), rounded to fp32 at half a turn at most
(2^-25); sincospif within 2 units in the last place; gain and products rounded to
fp32 (3 of 2^-24).  Together below 2^-19 (|u| + |w|) gain.  The result is
rounded to bf16 once: 2^-8 of it, and of the error."""
import numpy as np
import pytest
import torch

from oracle import bf16_to_f64, longctx
from speculative_tree_verify_gb300 import abi
from speculative_tree_verify_gb300.device import rotate
from test_gpu_paged_attn import NAN, bits, dev, host, i32

pytestmark = pytest.mark.gpu


def check(got, x, pos, rope, heads, dim):
    """Bits of rows got, x [rows][heads * dim]."""
    freq, inter, gain = list(rope.freq)[:rope.rot_dim // 2], bool(rope.interleaved), rope.gain
    X = bf16_to_f64(x).reshape(-1, heads, dim)
    want = longctx.rotate(X, pos, freq, inter, gain)
    rot = rope.rot_dim
    pairs = np.abs(X[..., :rot]).reshape(*X.shape[:2], -1, 2).sum(-1).repeat(2, -1) if inter else \
        np.tile(np.abs(X[..., :rot // 2]) + np.abs(X[..., rot // 2:rot]), 2)
    got = got.reshape(-1, heads, dim)
    assert (got[..., rot:] == x.reshape(-1, heads, dim)[..., rot:]).all()   # what does not turn stays as it is
    err = np.abs(bf16_to_f64(got)[..., :rot] - want[..., :rot])
    tol = 2.0 ** -8 * np.abs(want[..., :rot]) + 2.0 ** -19 * (1 + 2.0 ** -8) * pairs * abs(gain) + 2.0 ** -134
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3f} of the tolerance"


class Rows:
    def __init__(self, rows, heads, dim, pos=None, seed=0, pad=0, extra=1):
        """`extra` heads (V) and a padding behind those that turn: NaN, to be left alone."""
        rng = np.random.default_rng(seed)
        self.rows, self.heads, self.dim = rows, heads, dim
        self.x = np.full((rows, (heads + extra) * dim + pad), NAN, np.uint16)
        self.x[:, :heads * dim] = bits(rng.standard_normal((rows, heads * dim)) * 3)
        self.pos = rng.integers(0, 1 << 20, rows).tolist() if pos is None else pos
        self.gx, self.gpos, self.status = dev(self.x), i32(self.pos), i32([0])

    def run(self, rope, in_place=True, stream=None):
        out = self.gx if in_place else torch.full_like(self.gx, 77)
        assert rotate(rope, self.gx, self.gpos, self.heads, self.dim, self.status, out, stream) == 0
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        got, used = host(out), self.heads * self.dim
        assert (got[:, used:] == (NAN if in_place else 77)).all()
        check(np.ascontiguousarray(got[:, :used]), self.x[:, :used].copy(), self.pos, rope, self.heads, self.dim)
        if not in_place:
            assert (host(self.gx) == self.x).all()


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,dim,rot", [(48, 128, 128), (6, 64, 64), (1, 128, 64), (10, 64, 48), (5, 128, 16), (3, 64, 16), (48, 128, 112)])
def test_layouts(gpu, heads, dim, rot, interleaved, in_place):
    Rows(7, heads, dim, seed=rot, pad=8).run(abi.tv_rope_init(rot, interleaved), in_place)


@pytest.mark.parametrize("rows", [1, 2, 151, 1217, 2500, 5001, 10007])
def test_rows_a_block(gpu, rows):
    """One row a block to eight, the last block ragged."""
    Rows(rows, 3, 64, seed=rows).run(abi.tv_rope_init(32))


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(gpu, interleaved):
    pos = [0, 1, 2 ** 31 - 1, -(2 ** 31), -1, 1 << 24, (1 << 24) + 1, 123456789, 10 ** 6, 2 ** 30 + 12345]
    Rows(len(pos), 4, 128, pos, seed=5).run(abi.tv_rope_init(128, interleaved, 1e6))


@pytest.mark.parametrize("scaling", [abi.TV_ROPE_LINEAR, abi.TV_ROPE_BASE, abi.TV_ROPE_BLEND])
def test_scaled(gpu, scaling):
    Rows(9, 4, 128, seed=scaling).run(abi.tv_rope_init(128, False, 1e4, scaling, 8.0, 8192, 1.0, 4.0, 1.2079441541679836))


def test_own_frequencies(gpu):
    """Zero, negative ones and such of more than a turn a position."""
    rope = abi.tv_rope_init(16, False, gain=-0.5)
    for i, f in enumerate([0.0, -0.25, -1.0, 7.5, -100.25, 2 * np.pi, 1e-300, -1e-9]):
        rope.freq[i] = f
    Rows(12, 2, 64, list(range(-5, 7)), seed=7).run(rope)


def test_values_at_the_ends(gpu):
    """Infinities and NaN stay in their pair; a position of zero leaves every value as it is."""
    rope, r = abi.tv_rope_init(64), Rows(4, 2, 64, [0, 3, 5, 9], seed=8)
    r.x[1, 5], r.x[2, 64 + 40] = 0x7F80, NAN
    r.gx = dev(r.x)
    assert rotate(rope, r.gx, r.gpos, 2, 64, r.status) == 0
    got = host(r.gx)
    assert (got[0, :128] == r.x[0, :128]).all()
    bad = ~np.isfinite(bf16_to_f64(got[:, :128]))
    assert set(zip(*np.nonzero(bad))) == {(1, 5), (1, 37), (2, 64 + 8), (2, 64 + 40)}


def test_refused_and_stopped(gpu):
    rope, r = abi.tv_rope_init(64), Rows(4, 2, 64, seed=9)
    for bad in (lambda: rotate(rope, r.gx[:, ::2], r.gpos, 1, 64, r.status), lambda: rotate(rope, r.gx, r.gpos[:3], 2, 64, r.status),
                lambda: rotate(rope, r.gx, r.gpos.long(), 2, 64, r.status), lambda: rotate(rope, r.gx.float(), r.gpos, 2, 64, r.status),
                lambda: rotate(rope, r.gx, r.gpos, 4, 64, r.status), lambda: rotate(rope, r.gx, r.gpos, 2, 64, r.status, r.gx[:3]),
                lambda: rotate(rope, r.gx.cpu(), r.gpos, 2, 64, r.status)):
        with pytest.raises(ValueError):
            bad()
    assert rotate(abi.tv_rope_init(128), r.gx, r.gpos, 1, 64, r.status) == abi.CODES["TV_E_UNSUPPORTED"]
    r.status.fill_(-16)
    assert rotate(rope, r.gx, r.gpos, 2, 64, r.status) == 0
    assert (host(r.gx) == r.x).all() and int(r.status.item()) == -16


def test_streams_and_graphs(gpu):
    """Two streams at once, and a graph replayed on other positions."""
    rope, a, b = abi.tv_rope_init(128), Rows(300, 8, 128, seed=10), Rows(300, 8, 128, seed=11)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    a.run(rope, False, streams[0])
    b.run(rope, True, streams[1])
    g, out, r = torch.cuda.CUDAGraph(), torch.zeros_like(a.gx), Rows(300, 8, 128, seed=12)
    with torch.cuda.graph(g):
        assert rotate(rope, r.gx, r.gpos, 8, 128, r.status, out, torch.cuda.current_stream()) == 0
    for step in (1, 77):
        pos = [(i * step + 5) % 9999 for i in range(300)]
        r.gpos.copy_(i32(pos))
        g.replay()
        torch.cuda.synchronize()
        check(np.ascontiguousarray(host(out)[:, :1024]), r.x[:, :1024].copy(), pos, rope, 8, 128)
