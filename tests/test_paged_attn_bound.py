"""The single-token attention held to what it states: P as two bf16 parts, fp32 sums, one rounding of the output.

The bound, per element, with weights w, result o, A = sum_j w_j |v_j - o| and B = sum_j w_j |v_j|:

- a score is a sum of D products; each addition is off by at most 2^-23 of the size of what has been added (whether it
  rounds or cuts off), so it is within (D + 8) 2^-23 S of exact, S = max_j sum_i |q_i k_ji| / sqrt(D), the 8 being the
  scale's and the product's roundings and the subtraction's of an offset (below 2 S + 8 powers of two away: 8 (S + 4)
  2^-23 covers it); 2^x is within 2^-22 of itself.  A weight moves by that much of itself in the sums above and below
  alike, the result so by at most e A, e = (D + 8) 2^-23 S + 32 2^-23 + 2^-22 (the 32 also covers the few further 2^x
  that bring warps and blocks to one offset);
- P enters the product as its nearest bf16 and the nearest bf16 to the rest: within 2^-8 2^-8 of itself, of P above
  only, so 2^-16 B;
- sums over n tokens: an element passes through at most n / 16 + 64 additions (tiles of one warp, 16 tokens each,
  products of a tile, warps, blocks), above and below: 2 (n / 16 + 64) 2^-23 B;
- the output is rounded once: 2^-8 of its size, the error's included.

P as one bf16 part would be off by up to 2^-8 of every weight on its own, which shows where o is small beside A."""
import numpy as np
import pytest
import torch

from oracle import bf16_to_f64
from test_gpu_paged_attn import Case, bits, host


def reference(q, k, v, round_p=lambda p: p, drop=None):
    """One KV head: q [G][D], k and v [n][D] -> result and its bound.  round_p: how P enters the product."""
    D, n = q.shape[1], len(k)
    s = q @ k.T / np.sqrt(D)
    size = (np.abs(q) @ np.abs(k).T / np.sqrt(D)).max(1, keepdims=True)
    p = np.exp(s - s.max(1, keepdims=True))
    if drop is not None:
        p[:, drop] = 0
    w = p / p.sum(1, keepdims=True)
    o = (round_p(p) @ v) / p.sum(1, keepdims=True)
    away = (w[:, :, None] * np.abs(v[None] - o[:, None])).sum(1)
    total = w @ np.abs(v)
    e = (D + 8) * 2.0 ** -23 * size + 32 * 2.0 ** -23 + 2.0 ** -22
    inner = e * away + (2.0 ** -16 + 2 * (n / 16 + 64) * 2.0 ** -23) * total
    return o, 2.0 ** -8 * (np.abs(o) + inner) + inner


def rounded(x):
    return bf16_to_f64(bits(x))


def two_parts(p):
    hi = rounded(p)
    return hi + rounded(p - hi)


LENS = [1, 2, 5, 17, 40, 64, 65, 100, 300, 1000, 3000]


@pytest.mark.parametrize("dim", [64, 128])
def test_the_bound_tells_one_part_from_two(dim):
    """On the CPU: two parts stay within it; one part, a part of the wrong scale and a lost token do not."""
    rng = np.random.default_rng(dim)
    worst = dict(two=0.0, one=0.0, scaled=0.0, lost=0.0)
    for n in LENS[2:]:
        q, k, v = (rounded(rng.standard_normal((rows, dim))) for rows in (5, n, n))
        o, tol = reference(q, k, v)
        half = lambda p: rounded(p) + rounded(p - rounded(p)) / 2
        for name, got in (("two", reference(q, k, v, two_parts)[0]), ("one", reference(q, k, v, rounded)[0]),
                          ("scaled", reference(q, k, v, half)[0]), ("lost", reference(q, k, v, drop=n // 2)[0])):
            worst[name] = max(worst[name], (np.abs(rounded(got) - o) / tol).max())
    assert worst["two"] <= 1 < min(worst["one"], worst["scaled"], worst["lost"]), worst


@pytest.mark.gpu
@pytest.mark.parametrize("new", [True, False])
@pytest.mark.parametrize("q_heads,kv_heads,dim,ps", [(4, 2, 64, 16), (10, 2, 128, 32), (8, 8, 128, 16), (24, 1, 128, 64), (33, 1, 64, 16)])
def test_two_parts_of_p(gpu, q_heads, kv_heads, dim, ps, new):
    c = Case(LENS, q_heads, kv_heads, dim, ps, seed=q_heads, new=new)
    assert c.run() == 0
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    got, G = bf16_to_f64(host(c.out)), q_heads // kv_heads
    for i, n in enumerate(LENS):
        k, v = (bf16_to_f64(x) for x in c.kv[i])
        for g in range(kv_heads):
            h = slice(g * G, (g + 1) * G)
            o, tol = reference(bf16_to_f64(c.q[i, h]), k[:, g], v[:, g])
            err = np.abs(got[i, h] - o)
            assert (err <= tol).all(), f"sequence of {n}: worst {np.max(err / tol):.3f} of the bound"
