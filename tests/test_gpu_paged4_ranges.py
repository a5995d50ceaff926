"""tv_attend_paged4 over the whole of its stated range, with test_gpu_paged4_attn.py's
cases and tolerance."""
import numpy as np
import pytest
import torch

from oracle import bf16_to_f64
from test_gpu_paged4_attn import Case4, bits, close4, spreads

pytestmark = pytest.mark.gpu

# 8 (or 16) heads a KV head: six (or four) pairs of warps take a head block's tiles in turn, and a block of the grid has
# whole head blocks of 15 tiles, so that what comes late in a sequence comes late in every warp
LATE = [(8, 8, 64, 40), (8, 8, 128, 40), (32, 2, 64, 80)]


@pytest.mark.parametrize("early,late", [(0.0, 2.0 ** 46), (0.0, 2.0 ** 60), (0.0, 2.0 ** 90), (2.0 ** -30, 2.0 ** 97)])
@pytest.mark.parametrize("q_heads,kv_heads,dim,n", LATE)
def test_values_that_come_late(gpu, q_heads, kv_heads, dim, n, early, late):
    """Nothing (or next to it) in V of every warp's first tiles, then values of any size: the weights of the first tokens
    count, whatever the scales grow by."""
    def edit(c):
        for pair in c.kv:
            x = bf16_to_f64(pair[1])
            pair[1] = bits(x * np.where(np.arange(len(x)) < 400, early, late)[:, None, None])
    c = Case4([900] * n, q_heads, kv_heads, dim, 64, seed=30, edit=edit)
    got, q = c.run(), bf16_to_f64(c.q)
    for i in range(n):
        close4(got[i], q[i], *c.rows_of(i), f"sequence {i}")


@pytest.mark.parametrize("q_heads,kv_heads,dim", [(8, 2, 128), (8, 2, 64), (12, 1, 64), (24, 1, 128)])
def test_small_queries_beside_large_ones(gpu, q_heads, kv_heads, dim):
    """Whole numbers up to 3 beside 2^18, which meets zeros of K alone: the scores are what the small ones make of them,
    and exact (products and their sums are whole numbers below 2^24 of a scale)."""
    def edit(c):
        q = np.random.default_rng(37).integers(-3, 4, c.q.shape).astype(np.float64)
        q[..., 4::32], q[..., 6::32] = 2.0 ** 18, -2.0 ** 18
        c.q[:] = bits(q)
        for pair in c.kv:
            k = bf16_to_f64(pair[0])
            k[..., 4::32] = k[..., 6::32] = 0
            pair[0] = bits(k)
    Case4([700, 33], q_heads, kv_heads, dim, 32, seed=38, edit=edit).check()


@pytest.mark.parametrize("less", [9, 12, 14, 16])
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(8, 2, 128), (8, 2, 64), (12, 1, 64), (24, 1, 128)])
def test_light_tokens_beside_heavy_ones(gpu, q_heads, kv_heads, dim, less):
    """15 of 16 tokens weigh 2^-less of the 16th, whose V is zero in the odd dimensions: there the others' V is the
    result."""
    def edit(c):
        q = np.zeros(c.q.shape)
        q[..., 0] = 8
        c.q[:] = bits(q)
        for pair in c.kv:
            k, v = np.zeros(pair[0].shape), np.zeros(pair[0].shape)
            light = np.arange(len(k)) % 16 != 5
            k[light, :, 0] = -(less * np.log(2) - 0.1) * np.sqrt(dim) / 8
            v[~light, :, 0::2], v[light, :, 1::2] = 7, 1
            v[..., 30::32] = 7   # a scale of one
            pair[0], pair[1] = bits(k), bits(v)
    Case4([700, 40], q_heads, kv_heads, dim, 32, seed=39, edit=edit).check()


@pytest.mark.parametrize("step", [2.0 ** -3, 2.0 ** 3, 2.0 ** 10])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("q_heads,kv_heads,dim,n", LATE)
def test_scores_of_any_size(gpu, q_heads, kv_heads, dim, n, first, step):
    """Scores up to 2^27, exact in fp32: tokens of equal scores weigh the same wherever they are, and whichever warp and
    block has them.

    q is 8^i step in dimensions 0 .. 6 and K of these the digits of a whole number below 8^7, so that products and sums
    are whole numbers below 2^24 times step.  V is 1 in a warp's first tiles and -1 behind them (or, where the scores rise
    from next to nothing after 400 tokens, in the tile that they rise in and behind it): weights that depend on
    the place do not cancel.  Tolerance: close4's, whose 1e-3 of a weight is for rounding scores of some hundreds; here
    what is left of a score less an offset is exact, or at most 2^-24 of some hundreds."""
    L, rise, turn = 900, 0 if first else 400, 400 if first else 784

    def edit(c):
        rng = np.random.default_rng(31)
        q = np.zeros(c.q.shape)
        q[..., :7] = 8.0 ** np.arange(7) * step
        c.q[:] = bits(q)
        for i, pair in enumerate(c.kv):
            k = np.zeros((L, kv_heads, dim))
            top = 2 ** 20 - 1234 * (i + 1) + rng.integers(-3, 1, (L, kv_heads)) * (1 if step > 1 else 8)
            top[:rise] = rng.integers(0, 9, (rise, kv_heads))
            k[..., :7] = top[..., None] // 8 ** np.arange(7) % 8
            k[..., 7::32] = 7   # a scale of one
            pair[0] = bits(k)
            pair[1] = bits(np.broadcast_to(np.where(np.arange(L) < turn, 1.0, -1.0)[:, None, None], k.shape))
    c = Case4([L] * n, q_heads, kv_heads, dim, 64, seed=32, edit=edit)
    got, q = c.run(), bf16_to_f64(c.q)
    for i in range(n):
        close4(got[i], q[i], *c.rows_of(i), f"sequence {i}")


def close_loud(got, q, k, v, scale, quiet, what=""):
    """Where values of very different size meet.  scale: the largest of V's scales that are seen, quiet: the dimensions
    compared.  With weights w, their largest m, o and A as in close4, B = sum w |v|, C = sum w times the largest |v| of the
    token's 32: a weight times a scale is fp16, 2^-11 of itself (B) or half of 2^-24, 2^-31 of m times `scale`, of codes up to
    7; a run's few fp32 products lose 2^-23 of C each; scores, sums and the result's rounding as in close4."""
    heads, tokens = len(q), len(k)
    o, A, B, _ = spreads(q, k, v)
    for h in range(heads):
        g = h * k.shape[1] // heads
        a = k[:, g] @ q[h] / np.sqrt(q.shape[1])
        w = np.exp(a - a.max())
        w /= w.sum()
        C = (w @ np.abs(v[:, g]).reshape(tokens, -1, 32).max(-1)).repeat(32)
        tol = (2.0 ** -11 * B[h] + (1e-3 + 2.0 ** -10) * A[h] + 2.0 ** -16 * np.abs(o[h]) + 2.0 ** -20 * C
               + 7 * 2.0 ** -31 * tokens * w.max() * scale) * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(o[h]) * (1 + 2.0 ** -7)
        err = np.abs(got[h] - o[h])
        assert (tol[quiet] < 0.5 * np.abs(o[h][quiet])).all(), "the bound says something"
        assert (err[quiet] <= tol[quiet]).all(), f"{what}: head {h}, worst {np.max(err[quiet] / tol[quiet]):.3f} of the tolerance"


HEADS = [(8, 2, 128), (8, 2, 64), (12, 1, 64)]


@pytest.mark.parametrize("up", [10, 16, 20, 24])
@pytest.mark.parametrize("q_heads,kv_heads,dim", HEADS)
def test_a_loud_token_that_weighs_nothing(gpu, q_heads, kv_heads, dim, up):
    """One token's V is 2^up times the others', its weight below 2^-90."""
    at = [7, 450]

    def edit(c):
        rng = np.random.default_rng(33)
        q = bf16_to_f64(c.q)
        q[..., 0] = 8
        c.q[:] = bits(q)
        for i, pair in enumerate(c.kv):
            k, v = bf16_to_f64(pair[0]), rng.uniform(0.5, 1, pair[1].shape)
            k[..., 0], k[at[i]], v[at[i]] = 0, 0, v[at[i]] * 2.0 ** up
            k[at[i], :, 0] = -12 * np.sqrt(dim)
            pair[0], pair[1] = bits(k), bits(v)
    c = Case4([60, 900], q_heads, kv_heads, dim, 16, seed=34, edit=edit)
    got, q = c.run(), bf16_to_f64(c.q)
    for i in range(2):
        k, v = c.rows_of(i)
        close_loud(got[i], q[i], k, v, bf16_to_f64(c.held[i][1][1]).max(), slice(None), f"sequence {i}")


@pytest.mark.parametrize("up", [10, 16, 20, 24])
@pytest.mark.parametrize("q_heads,kv_heads,dim", HEADS)
def test_a_loud_group(gpu, q_heads, kv_heads, dim, up):
    """Every token's V is 2^up times as large in its last 32 dimensions as in the others."""
    def edit(c):
        rng = np.random.default_rng(35)
        for pair in c.kv:
            v = rng.uniform(0.5, 1, pair[1].shape)
            v[..., -32:] *= 2.0 ** up
            pair[1] = bits(v)
    c = Case4([60, 900], q_heads, kv_heads, dim, 16, seed=36, edit=edit)
    got, q = c.run(), bf16_to_f64(c.q)
    for i in range(2):
        k, v = c.rows_of(i)
        for part in (slice(0, -32), slice(-32, None)):
            close_loud(got[i], q[i], k, v, bf16_to_f64(c.held[i][1][1]).max(), part, f"sequence {i}")


@pytest.mark.parametrize("early", [0, 400])
@pytest.mark.parametrize("q_heads,kv_heads,dim,n", LATE)
def test_the_largest_scores_keep_their_digits(gpu, q_heads, kv_heads, dim, n, early):
    """One token in 16 has a score near 2^27, all others (after `early` tokens next to nothing) 2^7 less or lower still:
    its V is the result, to a weight's 2^-11 and the result's rounding, however the offsets were rounded."""
    def edit(c):
        rng = np.random.default_rng(40)
        q = np.zeros(c.q.shape)
        q[..., :7] = 8.0 ** np.arange(7) * 2.0 ** 10
        c.q[:] = bits(q)
        for pair in c.kv:
            k = np.zeros(pair[0].shape)
            top = rng.integers(2 ** 19, 2 ** 20, (1, kv_heads)) - (np.arange(len(k)) % 16 != 5)[:, None]
            top[:early] = rng.integers(0, 9, (early, kv_heads))
            k[..., :7] = top[..., None] // 8 ** np.arange(7) % 8
            k[..., 7::32] = 7   # a scale of one
            pair[0] = bits(k)
            pair[1] = bits(np.broadcast_to(rng.uniform(0.5, 1, (1, kv_heads, dim)), k.shape))
    c = Case4([900] * n, q_heads, kv_heads, dim, 64, seed=41, edit=edit)
    got = c.run()
    for i in range(n):
        v = c.rows_of(i)[1][-1].repeat(q_heads // kv_heads, 0)
        assert (np.abs(got[i] - v) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16) * (1 + 2.0 ** -7) * np.abs(v) + 2.0 ** -22 * np.abs(v).max()).all(), i


@pytest.mark.parametrize("q_heads,kv_heads,dim", [(8, 2, 128), (12, 1, 64)])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_a_query_that_is_not_finite(gpu, q_heads, kv_heads, dim, value):
    """Its head is NaN (all of K counts towards it), and no other one is touched."""
    def edit(c):
        c.q[:, 3, 5] = bits(np.array([value]))[0] if np.isinf(value) else 0x7FC0
    c = Case4([900, 40], q_heads, kv_heads, dim, 16, seed=42, edit=edit)
    got, q = c.run(), bf16_to_f64(c.q)
    assert np.isnan(got[:, 3]).all()
    for i in range(2):
        bad = np.zeros(got[i].shape, bool)
        bad[3] = True
        with np.errstate(invalid="ignore"):
            close4(got[i], np.where(np.isfinite(q[i]), q[i], 0), *c.rows_of(i), but=bad)
