"""Host side of the long-context operators: argument checks (nothing is launched
when one fails), the rotary tables, the oracle's own rules by hand, and the ring
of loads that several warps keep, as a protocol on the CPU."""
import math
import re
from collections import deque
from pathlib import Path

import numpy as np
import pytest

from oracle import bf16_to_f64, longctx
from speculative_tree_verify_gb300 import abi, build

FAKE = 0x10000   # 16-byte aligned, never dereferenced on these paths
E = abi.CODES
CSRC = Path(__file__).parents[1] / "speculative_tree_verify_gb300" / "csrc"


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return abi.load()


def _pool(kind=abi.TvPool4, **over):
    a = dict(k=FAKE, v=FAKE, refs=FAKE, n_layers=2, n_pages=64, n_kv_heads=2, page_size=16, head_dim=64)
    a.update(over)
    return kind(*a.values())


def _seqs(**over):
    a = dict(pages=FAKE, lens=FAKE, max_seqs=8, max_pages=10)
    a.update(over)
    return abi.TvSeqs(*a.values())


CALLS = {
    "extend": lambda pool, seqs, n=3, ids=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE: abi.tv_pages4_extend(pool, seqs, ids, FAKE, n, ws, wsb, st),
    "fork": lambda pool, seqs, n=3, ids=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE: abi.tv_pages4_fork(pool, seqs, ids, FAKE, n, st),
    "release": lambda pool, seqs, n=3, ids=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE: abi.tv_pages4_release(pool, seqs, ids, FAKE, n, st),
    "compact": lambda pool, seqs, n=3, ids=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE: abi.tv_pages4_compact(pool, seqs, ids, FAKE, ws, wsb, st),
    "write": lambda pool, seqs, n=3, ids=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE: abi.tv_pages4_write(pool, 0, seqs, ids, FAKE, FAKE, n, 9, FAKE, FAKE, 128, 64, st),
    "read": lambda pool, seqs, n=3, ids=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE: abi.tv_pages4_read(pool, 0, seqs, ids, FAKE, FAKE, n, 9, FAKE, FAKE, 128, 64, st),
}


@pytest.mark.parametrize("name", CALLS)
def test_pages4_host_checks(name):
    call = CALLS[name]
    for over in (dict(k=None), dict(v=None), dict(refs=None), dict(k=FAKE + 8), dict(refs=FAKE + 4), dict(n_layers=0),
                 dict(n_pages=0), dict(n_kv_heads=0)):
        assert call(_pool(**over), _seqs()) == E["TV_E_ARG"], over
    for over in (dict(page_size=8), dict(page_size=24), dict(page_size=256), dict(head_dim=96), dict(head_dim=32),
                 dict(n_pages=1 << 30, n_layers=4), dict(n_pages=1 << 26)):
        assert call(_pool(**over), _seqs()) == E["TV_E_UNSUPPORTED"], over
    assert call(_pool(), _seqs(lens=None)) == E["TV_E_ARG"]
    assert call(_pool(), _seqs(max_seqs=65537)) == E["TV_E_UNSUPPORTED"]
    assert call(_pool(), _seqs(), ids=None) == E["TV_E_ARG"]
    assert call(_pool(), _seqs(), st=None) == E["TV_E_ARG"]
    if name != "compact":
        assert call(_pool(), _seqs(), n=0) == E["TV_E_ARG"]
        assert call(_pool(), _seqs(), n=4097) == E["TV_E_UNSUPPORTED"]
    if name in ("extend", "compact"):
        need = abi.tv_pages4_workspace_size(_pool(), _seqs())
        assert need > 0 and need % 256 == 0
        assert call(_pool(), _seqs(), wsb=need - 1) == E["TV_E_WORKSPACE"]


def _paged(kind, **over):
    a = dict(layer=0, n=3, heads=4, window=100, sinks=4, q=FAKE, qs=512, k=FAKE, v=FAKE, kvs=512, out=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE)
    a.update(over)
    call = abi.tv_attend_paged4 if kind is abi.TvPool4 else abi.tv_attend_paged_window
    return call(a.get("pool") or _pool(kind), a["layer"], a.get("seqs") or _seqs(), FAKE, a["n"], a["heads"], a["window"], a["sinks"],
                a["q"], a["qs"], a["k"], a["v"], a["kvs"], a["out"], a["ws"], a["wsb"], a["st"])


@pytest.mark.parametrize("kind", [abi.TvPool, abi.TvPool4])
def test_token_host_checks(kind):
    for over in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(layer=2), dict(layer=-1), dict(n=0), dict(heads=0), dict(q=None),
                 dict(q=FAKE + 8), dict(qs=252), dict(qs=250 + 8), dict(k=None), dict(v=None), dict(kvs=120), dict(kvs=132), dict(out=None),
                 dict(out=FAKE + 4), dict(st=None)):
        assert _paged(kind, **over) == E["TV_E_ARG"], over
    for over in (dict(heads=5), dict(heads=65538), dict(n=2049), dict(seqs=_seqs(max_pages=1 << 27), n=2048)):
        assert _paged(kind, **over) == E["TV_E_UNSUPPORTED"], over
    size = abi.tv_attend_paged4_workspace_size if kind is abi.TvPool4 else abi.tv_attend_paged_workspace_size
    need = size(_pool(kind), 4, 3)
    for over in (dict(wsb=need - 1), dict(ws=None), dict(ws=FAKE + 8)):
        assert _paged(kind, **over) == E["TV_E_WORKSPACE"], over
    with pytest.raises(ValueError, match="UNSUPPORTED"):
        size(_pool(kind), 5, 3)


def test_prompt_host_checks():
    def call(heads=(4, 2, 64), window=100, sinks=4, q=FAKE, qs=512, kvs=512, n=2, rows=9, out=FAKE, st=FAKE):
        return abi.tv_attend_prompt_window(*heads, window, sinks, q, FAKE, FAKE, qs, kvs, FAKE, n, rows, out, st)

    for over in (dict(window=0), dict(window=-5), dict(sinks=-1), dict(q=None), dict(q=FAKE + 2), dict(qs=248), dict(kvs=60), dict(n=0),
                 dict(rows=0), dict(out=FAKE + 16), dict(st=None), dict(heads=(0, 2, 64))):
        assert call(**over) == E["TV_E_ARG"], over
    for over in (dict(heads=(4, 2, 96)), dict(heads=(5, 2, 64)), dict(heads=(258, 2, 64)), dict(n=4097)):
        assert call(**over) == E["TV_E_UNSUPPORTED"], over


def test_rope_host_checks():
    r = abi.tv_rope_init(64)

    def call(rope=r, x=FAKE, xs=512, out=FAKE, outs=512, heads=4, dim=128, pos=FAKE, rows=3, st=FAKE):
        return abi.tv_rope_rows(rope, x, xs, out, outs, heads, dim, pos, rows, st)

    for over in (dict(x=None), dict(x=FAKE + 8), dict(out=None), dict(out=FAKE + 2), dict(xs=511), dict(xs=504), dict(outs=640), dict(pos=None),
                 dict(heads=0), dict(rows=0), dict(st=None)):
        assert call(**over) == E["TV_E_ARG"], over
    for over in (dict(dim=96), dict(dim=256, xs=4096, outs=4096), dict(heads=65537, xs=1 << 24, outs=1 << 24)):
        assert call(**over) == E["TV_E_UNSUPPORTED"], over
    assert call(rope=abi.tv_rope_init(128), dim=64) == E["TV_E_UNSUPPORTED"]
    for field, value in (("rot_dim", 24), ("rot_dim", 0), ("rot_dim", 144), ("interleaved", 2), ("gain", math.inf)):
        bad = abi.tv_rope_init(64)
        setattr(bad, field, value)
        assert call(rope=bad) == E["TV_E_ARG"], field
    bad = abi.tv_rope_init(64)
    bad.freq[31] = math.nan
    assert call(rope=bad) == E["TV_E_ARG"]


def test_a_gain_no_float_holds():
    rope = abi.tv_rope_init(64, gain=3e38)
    for gain in (1e39, -1e300):
        with pytest.raises(ValueError, match="ARG"):
            abi.tv_rope_init(64, gain=gain)
        rope.gain = gain
        assert abi.tv_rope_rows(rope, FAKE, 512, FAKE, 512, 4, 128, FAKE, 3, FAKE) == E["TV_E_ARG"]


def test_rope_tables():
    for args, kw in (((64, False, 10000.0), {}), ((128, True, 5e5), dict(scaling="linear", factor=4.0)), ((48, False, 1e4), dict(scaling="base", factor=8.0)),
                     ((128, False, 1e6), dict(scaling="blend", factor=8.0, original_ctx=8192, low_turns=1.0, high_turns=4.0)),
                     ((16, True, 1e4), dict(scaling="blend", factor=2.0, original_ctx=100, low_turns=0.0, high_turns=0.5))):
        names = dict(plain=abi.TV_ROPE_PLAIN, linear=abi.TV_ROPE_LINEAR, base=abi.TV_ROPE_BASE, blend=abi.TV_ROPE_BLEND)
        got = abi.tv_rope_init(*args, names[kw.get("scaling", "plain")], **{k: v for k, v in kw.items() if k != "scaling"}, gain=1.25)
        want = longctx.frequencies(args[0], args[2], **kw)
        assert (got.rot_dim, got.interleaved, got.gain) == (args[0], int(args[1]), 1.25)
        assert np.allclose(got.freq[:len(want)], want, rtol=2.0 ** -45, atol=0)   # a few roundings of pow's last place, 64 of them at most
        assert not any(got.freq[len(want):])
    # the slowest pair as LINEAR, the fastest as it was
    base, lin, plain = (abi.tv_rope_init(128, False, 1e4, k, 8.0).freq for k in (abi.TV_ROPE_BASE, abi.TV_ROPE_LINEAR, abi.TV_ROPE_PLAIN))
    assert math.isclose(base[63], lin[63], rel_tol=1e-12) and base[0] == plain[0] == 1.0
    for bad in (dict(rot_dim=8), dict(rot_dim=130), dict(rot_dim=20), dict(theta=0.0), dict(theta=math.nan), dict(scaling=4), dict(scaling=-1),
                dict(scaling=abi.TV_ROPE_LINEAR, factor=0.0), dict(scaling=abi.TV_ROPE_BASE, factor=math.inf), dict(gain=math.nan),
                dict(scaling=abi.TV_ROPE_BLEND, factor=2.0, original_ctx=0), dict(scaling=abi.TV_ROPE_BLEND, factor=2.0, low_turns=4.0, high_turns=4.0),
                dict(scaling=abi.TV_ROPE_BLEND, factor=2.0, low_turns=-1.0), dict(theta=1e-300, scaling=abi.TV_ROPE_BASE, factor=1e300),
                dict(scaling=abi.TV_ROPE_LINEAR, factor=1e-320)):
        with pytest.raises(ValueError, match="ARG"):
            abi.tv_rope_init(**{"rot_dim": 64, **bad})


def test_oracle_by_hand():
    assert longctx.seen(5, 2, 0) == [4, 5] and longctx.seen(5, 2, 1) == [0, 4, 5] and longctx.seen(5, 1, 9) == [0, 1, 2, 3, 4, 5]
    assert longctx.seen(0, 1, 0) == [0] and longctx.seen(3, 100, 0) == [0, 1, 2, 3]
    # bf16: ties to even, subnormals, overflow
    for x, want in ((1.0, 0x3F80), (1 + 2.0 ** -8, 0x3F80), (1 + 3 * 2.0 ** -8, 0x3F82), (-2.0 ** -133, 0x8001), (2.0 ** -134, 0), (3.4e38, 0x7F80),
                    (math.inf, 0x7F80)):
        assert longctx.bf16(x) == want, x
    # codes: a scale of one, halves away from zero; a group of zeros; one that is not finite
    x = np.zeros((1, 96))
    x[0, :6] = 7, -7, 2.5, -2.5, 0.5, -0.4375
    x[0, 64] = np.inf
    codes, scales = longctx.quantise(longctx.bf16(x))
    assert codes[0, :7].tolist() == [15, 1, 11, 5, 9, 8, 8] and (codes[0, 32:] == 8).all()
    assert scales[0].tolist() == [0x3F80, 0, 0x7FC0]
    y = longctx.stands_for(codes, scales)
    assert y[0, :6].tolist() == [7, -7, 3, -3, 1, 0] and np.isnan(y[0, 64:]).all()
    # every value and every scale of a block has its own place
    for D in (64, 128):
        for kind in ("k", "v"):
            places = {longctx.place(kind, t, d, D) for t in range(16) for d in range(0, D, 2)}
            assert places == set(range(8 * D))
            assert all(longctx.place(kind, t, d, D) == longctx.place(kind, t, d + 1, D) for t in range(16) for d in range(0, D, 2))
        assert {longctx.scale_place(t, g, D) for t in range(16) for g in range(D // 32)} == set(range(8 * D, 9 * D, 2))
    # rotating there and back
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 64))
    f = longctx.frequencies(32, 1e4)
    for inter in (False, True):
        y = longctx.rotate(longctx.rotate(x, [5, 2 ** 31 - 1, -9], f, inter), [-5, 1 - 2 ** 31, 9], f, inter)
        assert np.abs(y - x).max() < 1e-9 and (y[..., 32:] == x[..., 32:]).all()
    assert np.allclose(longctx.rotate(x, [0, 0, 0], f, False, 2.0)[..., :32], 2 * x[..., :32])


# ---- several loading warps and one ring --------------------------------------------
def _constant(source, name):
    return int(re.search(rf"constexpr int {name} = (\d+);", (CSRC / source).read_text()).group(1))


def passes(completed, phase):
    """try_wait.parity of phase `phase` (counted from 0) after `completed` phases."""
    return (completed & 1) != (phase & 1)


def search(places, stages, loaders, teams, runs, query_of, tile_of):
    """What goes wrong, or None, in every order of events of runs of one tile.

    Run r's queries are issued by loader query_of(r), its tile (tile r) by tile_of(r), each loader in order of runs, once
    the place that they go to is given up; copies land in any order.  Team r mod `teams` takes the queries, the tile, and
    gives the queries' place up; the others wait for the queries and go on, which counts too."""
    items = [[(r, k) for r in range(runs) for k in "qt" if (query_of if k == "q" else tile_of)(r) == w] for w in range(loaders)]
    lists = [[(r, k) for r in range(runs) for k in (("q", "t", "f") if r % teams == g else ("s",))] for g in range(teams)]
    issue = {x: (w, i) for w in range(loaders) for i, x in enumerate(items[w])}
    step = {x: i + 1 for g in range(teams) for i, x in enumerate(lists[g]) if x[1] != "s"}
    skip = {(r, g): i + 1 for g in range(teams) for i, (r, k) in enumerate(lists[g]) if k == "s"}
    start = ((0,) * loaders, frozenset(), (0,) * teams)
    seen, todo = {start}, deque([start])
    while todo:
        load, flying, at = todo.popleft()

        def landed(r, k):
            w, i = issue[(r, k)]
            return load[w] > i and (r, k) not in flying

        def given_up(r, k):
            if k == "t":
                return at[r % teams] >= step[(r, "t")]
            return at[r % teams] >= step[(r, "f")] and all(at[g] >= skip[(r, g)] for g in range(teams) if g != r % teams)

        def phases(f, r, k, size):
            return sum(f(x, k) for x in range(r % size, runs, size))
        nexts = [(load, flying - {f}, at) for f in flying]
        for w in range(loaders):
            if load[w] == len(items[w]):
                continue
            r, k = items[w][load[w]]
            size = places if k == "q" else stages
            if r >= size:
                if not passes(phases(given_up, r, k, size), r // size - 1):
                    continue
                if not given_up(r - size, k):
                    return "loaded over"
            nexts.append((load[:w] + (load[w] + 1,) + load[w + 1:], flying | {(r, k)}, at))
        for g in range(teams):
            if at[g] == len(lists[g]):
                continue
            r, k = lists[g][at[g]]
            kind, size = ("t", stages) if k == "t" else ("q", places)
            if k != "f":
                if not passes(phases(landed, r, kind, size), r // size):
                    continue
                if not landed(r, kind):
                    return "read too early"
            nexts.append((load, flying, at[:g] + (at[g] + 1,) + at[g + 1:]))
        if not nexts and not (all(map(lambda w: load[w] == len(items[w]), range(loaders))) and all(at[g] == len(lists[g]) for g in range(teams))):
            return "dead end"
        for s in nexts:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return None


@pytest.mark.parametrize("places", [2, 3, 4])
def test_each_place_has_one_loading_warp(places):
    stages, loaders = _constant("tv_paged_attn.cu", "kStages"), _constant("tv_paged_attn.cu", "kLoadWarps")
    assert search(places, stages, loaders, 2, places + 4, lambda r: r % places % loaders, lambda r: r % stages % loaders) is None


@pytest.mark.parametrize("places", [2, 3])
def test_rings_of_the_4_bit_kernel(places):
    stages, loaders = _constant("tv_paged4_attn.cu", "kStages"), _constant("tv_paged4_attn.cu", "kLoadWarps")
    assert stages % loaders == 0
    # as many stages as loaders: the same protocol with fewer states
    assert search(places, loaders, loaders, 2, 7, lambda r: r % places % loaders, lambda r: r % loaders) is None


def test_places_that_change_hands_do_not_do():
    """What the rule is for: a warp that sees every other phase of a place takes one for the next."""
    assert search(2, 6, 4, 2, 8, lambda r: r % 4, lambda r: r % 4) == "loaded over"
