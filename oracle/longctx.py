"""Plain references of the long-context operators, in fp64: rotary positions,
attention through a window with sinks, and the cache in 4 bits.

The pages of the method name none of them; the rules are those include/tv.h
states at tv_rope_rows, tv_attend_prompt_window and tv_pool4.  bf16 values are
uint16 bit patterns.
"""
from __future__ import annotations

import math

import numpy as np

from . import bf16_to_f64
from .paged import attend


def bf16(x):
    """fp64 rounded to the nearest bf16 (ties to even), as bits.  NaN stays one."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
    ulp = np.maximum(e - 8, -133)                       # 8 bits of significand, subnormals below 2^-126
    y = np.ldexp(np.rint(np.ldexp(m, e - ulp)), ulp)
    y = np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, y), y)
    y = np.where(np.isfinite(x), y, x).astype(np.float32)
    return (y.view(np.uint32) >> 16).astype(np.uint16) | np.where(np.isnan(y), 0x40, 0).astype(np.uint16)


# ---- rotary positions ----------------------------------------------------------
def frequencies(rot_dim, theta, scaling="plain", factor=1.0, original_ctx=1, low_turns=1.0, high_turns=32.0):
    got = []
    if scaling == "base":
        theta *= factor ** (rot_dim / (rot_dim - 2))
    for i in range(rot_dim // 2):
        f = theta ** (-2 * i / rot_dim)
        if scaling == "linear":
            f /= factor
        if scaling == "blend":
            turns = original_ctx * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low_turns) / (high_turns - low_turns)))
            f = keep * f + (1 - keep) * f / factor
        got.append(f)
    return got


def rotate(x, pos, freq, interleaved, gain=1.0):
    """x [rows][heads][D] fp64; the angle's turns are taken exactly (integers of 2^-80 of one)."""
    y = x.copy()
    half = len(freq)
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        turn = int(f / (2 * math.pi) * 2.0 ** 80)
        frac = np.array([(int(p) * turn % 2 ** 80) / 2.0 ** 80 for p in pos])
        c, s = np.cos(2 * np.pi * frac)[:, None] * gain, np.sin(2 * np.pi * frac)[:, None] * gain
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


# ---- a window and sinks ----------------------------------------------------------
def seen(t, window, sinks):
    """The rows that row t sees, ascending."""
    return [j for j in range(t + 1) if j > t - window or j < sinks]


def attend_prompt(q, k, v, starts, window, sinks):
    """(out, spread) as oracle.paged.attend_prompt."""
    out, off = np.full(q.shape, np.nan), np.zeros(q.shape)
    for a, b in zip(starts[:-1], starts[1:]):
        for t in range(a, b):
            j = [a + x for x in seen(t - a, window, sinks)]
            out[t], off[t] = attend(q[t], k[j], v[j], True)
    return out, off


# ---- 4 bits ----------------------------------------------------------------------
def quantise(x):
    """bits [..., D] -> (codes [..., D], scales' bits [..., D / 32])."""
    g = bf16_to_f64(x).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    fine = np.isfinite(g).all(-1)
    g = np.where(fine[..., None], g, 0.0)
    scales = bf16(np.abs(g).max(-1) / 7)
    s = bf16_to_f64(scales)
    held = s >= 2.0 ** -126
    n = np.floor(np.abs(g) / np.where(held, s, 1.0)[..., None] + 0.5) * np.sign(g)   # halves away from zero
    codes = np.where(held[..., None], 8 + n, 8).astype(np.uint8)
    return codes.reshape(x.shape), np.where(fine, np.where(held, scales, 0), 0x7FC0).astype(np.uint16)


def stands_for(codes, scales):
    """fp64"""
    n = codes.astype(np.float64).reshape(*scales.shape, 32) - 8
    return (n * bf16_to_f64(scales)[..., None]).reshape(codes.shape)


def place(kind, t, d, D):
    """The byte of dimension d of token t in a block; the even dimensions are its low four bits."""
    G, g = D // 32, d // 32
    if kind == "k":
        return t * (D // 2) + (d % 32 // 8 * G + g) * 4 + d % 8 // 2
    return ((t // 8 * 32 + d % 32 // 4 * 4 + t % 8 // 2) * G + g) * 4 + t % 2 * 2 + d % 4 // 2


def scale_place(t, g, D):
    return 8 * D + ((t // 8 * 4 + t % 8 // 2) * (D // 32) + g) * 4 + t % 2 * 2


class Pages4:
    """The rows of a pool in 4 bits: k, v uint8 [layers][pages][heads][page_size / 16][9 D]."""

    def __init__(self, k, v, page_size, dim):
        self.pools, self.ps, self.dim = {"k": k, "v": v}, page_size, dim

    def _at(self, kind, slot):
        t, D = slot % 16, self.dim
        scales = [scale_place(t, g, D) + i for g in range(D // 32) for i in (0, 1)]
        return slot // 16, [place(kind, t, d, D) for d in range(0, D, 2)], scales

    def put(self, kind, layer, page, slot, codes, scales):
        """A token of every head: codes [heads][D], scales [heads][D / 32]."""
        block, at, sat = self._at(kind, slot)
        b = self.pools[kind][layer, page, :, block]
        b[:, at] = codes[:, 0::2] | codes[:, 1::2] << 4
        b[:, sat] = np.ascontiguousarray(scales, dtype="<u2").view(np.uint8)

    def get(self, kind, layer, page, slot):
        block, at, sat = self._at(kind, slot)
        b = self.pools[kind][layer, page, :, block]
        codes = np.stack([b[:, at] & 15, b[:, at] >> 4], -1).reshape(len(b), -1)
        return codes, np.ascontiguousarray(b[:, sat]).view("<u2")
