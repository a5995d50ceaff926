"""Host side of the paged cache: argument checks (nothing is launched when one
fails) and the oracle's own rules by hand on a small pool."""
import numpy as np
import pytest

from speculative_tree_verify_gb300 import abi, build

FAKE = 0x10000   # 16-byte aligned, never dereferenced on these paths


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return abi.load()


def _pool(**over):
    a = dict(k=FAKE, v=FAKE, refs=FAKE, n_layers=2, n_pages=64, n_kv_heads=2, page_size=16, head_dim=64)
    a.update(over)
    return abi.TvPool(*a.values())


def _seqs(**over):
    a = dict(pages=FAKE, lens=FAKE, max_seqs=8, max_pages=10)
    a.update(over)
    return abi.TvSeqs(*a.values())


CALLS = {
    "extend": lambda pool, seqs, n=3, ids=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE: abi.tv_pages_extend(pool, seqs, ids, FAKE, n, ws, wsb, st),
    "fork": lambda pool, seqs, n=3, ids=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE: abi.tv_pages_fork(pool, seqs, ids, FAKE, n, st),
    "release": lambda pool, seqs, n=3, ids=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE: abi.tv_pages_release(pool, seqs, ids, FAKE, n, st),
    "compact": lambda pool, seqs, n=3, ids=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE: abi.tv_pages_compact(pool, seqs, ids, FAKE, ws, wsb, st),
    "write": lambda pool, seqs, n=3, ids=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE: abi.tv_pages_write(pool, 0, seqs, ids, FAKE, FAKE, n, 9, FAKE, FAKE, 128, 64, st),
    "read": lambda pool, seqs, n=3, ids=FAKE, ws=FAKE, wsb=1 << 30, st=FAKE: abi.tv_pages_read(pool, 0, seqs, ids, FAKE, FAKE, n, 9, FAKE, FAKE, 128, 64, st),
}


@pytest.mark.parametrize("name", CALLS)
def test_pages_host_checks(name):
    call, E = CALLS[name], abi.CODES
    for over in (dict(k=None), dict(v=None), dict(refs=None), dict(k=FAKE + 2), dict(refs=FAKE + 4), dict(n_layers=0),
                 dict(n_pages=0), dict(n_kv_heads=0)):
        assert call(_pool(**over), _seqs()) == E["TV_E_ARG"], over
    for over in (dict(page_size=8), dict(page_size=24), dict(page_size=256), dict(head_dim=96), dict(head_dim=0),
                 dict(n_pages=1 << 30, n_layers=4), dict(n_pages=1 << 26)):
        assert call(_pool(**over), _seqs()) == E["TV_E_UNSUPPORTED"], over
    for over in (dict(pages=None), dict(lens=None), dict(max_seqs=0), dict(max_pages=0)):
        assert call(_pool(), _seqs(**over)) == E["TV_E_ARG"], over
    for over in (dict(max_seqs=65537), dict(max_pages=1 << 28)):
        assert call(_pool(), _seqs(**over)) == E["TV_E_UNSUPPORTED"], over
    assert call(_pool(), _seqs(), ids=None) == E["TV_E_ARG"]
    assert call(_pool(), _seqs(), st=None) == E["TV_E_ARG"]
    if name != "compact":
        assert call(_pool(), _seqs(), n=0) == E["TV_E_ARG"]
        assert call(_pool(), _seqs(), n=4097) == E["TV_E_UNSUPPORTED"]
    if name in ("extend", "compact"):
        need = abi.tv_pages_workspace_size(_pool(), _seqs())
        assert need > 0 and need % 256 == 0
        assert call(_pool(), _seqs(), wsb=need - 1) == E["TV_E_WORKSPACE"]
        assert call(_pool(), _seqs(), ws=None) == E["TV_E_WORKSPACE"]
        assert call(_pool(), _seqs(), ws=FAKE + 8) == E["TV_E_WORKSPACE"]


@pytest.mark.parametrize("fn", [abi.tv_pages_write, abi.tv_pages_read])
def test_rows_host_checks(fn):
    E = abi.CODES

    def call(layer=1, rows=9, k=FAKE, v=FAKE, rs=128, hs=64):
        return fn(_pool(), layer, _seqs(), FAKE, FAKE, FAKE, 3, rows, k, v, rs, hs, FAKE)

    for over in (dict(layer=-1), dict(layer=2), dict(rows=-1), dict(k=None), dict(v=None), dict(k=FAKE + 2), dict(v=FAKE + 8),
                 dict(rs=129), dict(hs=68)):
        assert call(**over) == E["TV_E_ARG"], over


def test_attend_paged_host_checks():
    E = abi.CODES
    need = abi.tv_attend_paged_workspace_size(_pool(), 8, 3)
    assert need > 0 and need % 256 == 0
    with pytest.raises(ValueError, match="UNSUPPORTED"):
        abi.tv_attend_paged_workspace_size(_pool(), 7, 3)
    with pytest.raises(ValueError, match="ARG"):
        abi.tv_attend_paged_workspace_size(_pool(), 0, 3)

    def call(pool=None, layer=0, seqs=None, ids=FAKE, n=3, hq=8, q=FAKE, qs=512, k=FAKE, v=FAKE, kvs=128, out=FAKE, ws=FAKE, wsb=need, st=FAKE):
        return abi.tv_attend_paged(pool or _pool(), layer, seqs or _seqs(), ids, n, hq, q, qs, k, v, kvs, out, ws, wsb, st)

    for over in (dict(ids=None), dict(q=None), dict(out=None), dict(st=None), dict(k=None), dict(v=None), dict(layer=2), dict(layer=-1),
                 dict(n=0), dict(hq=0), dict(q=FAKE + 2), dict(out=FAKE + 8), dict(k=FAKE + 2), dict(v=FAKE + 2), dict(qs=516), dict(qs=504),
                 dict(kvs=132), dict(kvs=120), dict(pool=_pool(k=None)), dict(seqs=_seqs(lens=None))):
        assert call(**over) == E["TV_E_ARG"], over
    for over in (dict(n=4097), dict(n=2049), dict(hq=9), dict(pool=_pool(head_dim=96)), dict(pool=_pool(page_size=20))):
        assert call(**over) == E["TV_E_UNSUPPORTED"], over
    for over in (dict(wsb=need - 1), dict(ws=None), dict(ws=FAKE + 8)):
        assert call(**over) == E["TV_E_WORKSPACE"], over


def test_attend_prompt_host_checks():
    E = abi.CODES

    def call(hq=8, hkv=2, d=64, q=FAKE, k=FAKE, v=FAKE, qs=512, kvs=128, starts=FAKE, n=3, rows=9, out=FAKE, st=FAKE):
        return abi.tv_attend_prompt(hq, hkv, d, q, k, v, qs, kvs, starts, n, rows, out, st)

    for over in (dict(hq=0), dict(hkv=0), dict(q=None), dict(k=None), dict(v=None), dict(starts=None), dict(out=None), dict(st=None),
                 dict(n=0), dict(rows=0), dict(q=FAKE + 2), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(out=FAKE + 4), dict(out=FAKE + 16), dict(qs=516), dict(qs=504),
                 dict(kvs=132), dict(kvs=120)):
        assert call(**over) == E["TV_E_ARG"], over
    for over in (dict(n=4097), dict(d=96), dict(hq=9), dict(hq=258, hkv=2, qs=258 * 64), dict(rows=2 ** 31 - 1, hq=256, hkv=8, kvs=512, qs=256 * 64)):
        assert call(**over) == E["TV_E_UNSUPPORTED"], over


def test_what_is_an_address():
    """None and ints go as they are, without an exception on the way; tensors by their address."""
    import sys

    import torch
    x, raised = torch.zeros(4), []

    def trace(frame, event, arg):
        if event == "exception":
            raised.append(arg)
        return trace
    sys.settrace(trace)
    try:
        got = [abi._p(a) for a in (None, 0, FAKE, x, x[1:])]
    finally:
        sys.settrace(None)
    assert got == [None, 0, FAKE, x.data_ptr(), x.data_ptr() + 4] and not raised


@pytest.mark.parametrize("what", [b"x" * 64, "x", 1.5, np.zeros(4, np.int32), [1]])
def test_what_is_no_address(what):
    with pytest.raises(AttributeError):
        CALLS["fork"](_pool(), _seqs(), ids=what)


def _paged_cache():
    import torch

    from speculative_tree_verify_gb300 import device, synth
    c = device.PagedCache.alloc(synth.TINY, 2, 24, 16, 5, 6, device="cpu")
    d = c.dims
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    width = (d.n_q_heads + 2 * d.n_kv_heads) * d.head_dim
    bf16 = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)
    return c, i32, bf16, width, (d.n_q_heads, d.n_kv_heads, d.head_dim)


def _reached(monkeypatch):
    """The C calls replaced by a note that they were reached: what is accepted is not launched here."""
    calls = []
    for name in abi.SYMBOLS:
        if name.startswith(("tv_pages", "tv_attend")) and not name.endswith("size"):
            monkeypatch.setattr(abi, name, lambda *a, _n=name, **k: calls.append(_n) or 0)
    return calls


def test_paged_cache_takes_what_fits(monkeypatch):
    c, i32, bf16, width, (Hq, Hkv, D) = _paged_cache()
    calls, ids = _reached(monkeypatch), i32(0, 1)
    qkv, k = bf16(9, width + 8)[:, :width], bf16(Hkv, 32, D)
    c.extend(ids, i32(3, 4))
    c.fork(ids, i32(2, 3))
    c.release(ids, i32(0, 0))
    c.compact(i32(*[0] * 24), i32(0))
    c.write(0, ids, i32(0, 0), i32(0, 4, 9), qkv)
    c.read_into(0, ids, i32(0, 0), i32(0, 4, 9), 9, k, k.clone())
    c.write_from(0, ids, i32(0, 0), i32(0, 4, 9), 9, k[:, 5:], k.clone()[:, 5:])
    c.attend_prompt(qkv, i32(0, 4, 9), bf16(9, Hq, D))
    c.attend(0, ids, qkv, bf16(2, Hq, D))
    assert len(calls) == 9


def test_paged_cache_refuses(monkeypatch):
    """Lists of other lengths, types or strides, tensors of another device or layout, too few rows: nothing is called."""
    import torch
    c, i32, bf16, width, (Hq, Hkv, D) = _paged_cache()
    calls, ids, one = _reached(monkeypatch), i32(0, 1), i32(0)
    qkv, out, k = bf16(9, width), bf16(9, Hq, D), bf16(Hkv, 32, D)
    long, strided, far = torch.tensor([0, 1]), i32(0, 7, 1, 7)[::2], ids.to("meta")
    starts = i32(0, 4, 9)
    for bad in (one, long, strided, far, ids.float()):
        for call in (c.extend, c.fork, c.release):
            with pytest.raises(ValueError):
                call(ids, bad)
        for call in (lambda: c.write(0, ids, bad, starts, qkv), lambda: c.read_into(0, ids, bad, starts, 9, k, k),
                     lambda: c.write_from(0, ids, bad, starts, 9, k, k), lambda: c.write(0, ids, ids, bad, qkv),
                     lambda: c.read_into(0, ids, ids, bad, 9, k, k), lambda: c.write_from(0, ids, ids, bad, 9, k, k),
                     lambda: c.compact(bad, one)):
            with pytest.raises(ValueError):
                call()
    for bad in (long, strided, far):
        for call in (lambda: c.extend(bad, ids), lambda: c.attend(0, bad, qkv, out), lambda: c.attend_prompt(qkv, bad, out)):
            with pytest.raises(ValueError):
                call()
    for bad in (bf16(9, width - 1), bf16(9, width).float(), bf16(9, width).to("meta"), bf16(width, 9).T, bf16(9 * width)):
        for call in (lambda: c.write(0, ids, ids, starts, bad), lambda: c.attend(0, ids, bad, out), lambda: c.attend_prompt(bad, starts, out)):
            with pytest.raises(ValueError):
                call()
    for call in (lambda: c.attend(0, ids, qkv[:1], out), lambda: c.attend(0, ids, qkv, out[:1]), lambda: c.attend_prompt(qkv, starts, out[:8]),
                 lambda: c.attend_prompt(qkv, starts, bf16(Hq, 9, D).transpose(0, 1)), lambda: c.compact(i32(*[0] * 24), ids)):
        with pytest.raises(ValueError):
            call()
    for a, b, rows in ((k, bf16(Hkv, 33, D), 9), (k, bf16(Hkv, 33, D)[:, :32], 9), (k, k, 33), (k, k, -1), (bf16(32, Hkv, D), bf16(32, Hkv, D), 2),
                       (k.float(), k, 9), (k, k.to("meta"), 9), (k[..., :1], k[..., :1], 9), (bf16(Hkv, D, 32).transpose(1, 2),) * 2 + (9,)):
        for call in (c.read_into, c.write_from):
            with pytest.raises(ValueError):
                call(0, ids, ids, starts, rows, a, b)
    assert not calls


def test_workspace_refuses_bad_shapes():
    with pytest.raises(ValueError, match="UNSUPPORTED"):
        abi.tv_pages_workspace_size(_pool(page_size=17), _seqs())
    with pytest.raises(ValueError, match="ARG"):
        abi.tv_pages_workspace_size(_pool(), _seqs(max_pages=0))


# ---- the oracle by hand, and with planted mistakes ------------------------------
def _cache(P, n_pages=6, max_seqs=4, max_pages=3):
    k = np.arange(2 * n_pages * 16 * 4, dtype=np.uint16).reshape(2, n_pages, 1, 16, 4)
    return P.Cache(k.copy(), k + 7, np.zeros(n_pages, np.int32), np.full((max_seqs, max_pages), -9, np.int32), np.zeros(max_seqs, np.int32))


def _pin_pages(P):
    c = _cache(P)
    c.extend([2, 0], [17, 16])
    assert c.pages[2].tolist() == [0, 1, -9] and c.pages[0].tolist() == [2, -9, -9]
    assert c.refs.tolist() == [1, 1, 1, 0, 0, 0] and c.lens.tolist() == [16, 0, 17, 0]
    c.fork([2, 2], [1, 3])
    assert c.refs.tolist() == [3, 3, 1, 0, 0, 0] and c.lens.tolist() == [16, 17, 17, 17]
    old = c.k[:, 1].copy(), c.v[:, 1].copy()
    c.extend([1, 2, 3, 0], [1, 2, 3, 0])   # three holders of page 1: the last in the list keeps it
    assert c.pages[1].tolist() == [0, 3, -9] and c.pages[2].tolist() == [0, 4, -9] and c.pages[3].tolist() == [0, 1, -9]
    assert c.refs.tolist() == [3, 1, 1, 1, 1, 0]
    for p in (3, 4):
        assert (c.k[:, p] == old[0]).all() and (c.v[:, p] == old[1]).all()
    with pytest.raises(P.Refused, match="CAPACITY"):
        c.extend([0, 3], [16, 14])
    assert c.lens.tolist() == [16, 18, 19, 20] and c.refs.tolist() == [3, 1, 1, 1, 1, 0]
    c.release([1, 3], [0, 16])
    assert c.refs.tolist() == [2, 0, 1, 0, 1, 0] and c.lens.tolist() == [16, 0, 19, 16]
    last = c.k[:, 4].copy()
    remap, used = c.compact()
    assert used == 3 and remap.tolist() == [0, -1, 2, -1, 1, -1] and c.refs.tolist() == [2, 1, 1, 0, 0, 0]
    assert c.pages[2].tolist() == [0, 1, -9] and (c.k[:, 1] == last).all()
    c.write(1, 2, 14, np.full((4, 1, 4), 500, np.uint16), np.full((4, 1, 4), 600, np.uint16))
    assert (c.k[1, 0, 0, 14:] == 500).all() and (c.v[1, 1, 0, :2] == 600).all() and not (c.k[0] == 500).any()
    k, v = c.rows(1, 2, 13, 3)
    assert (k[1:] == 500).all() and (v[1:] == 600).all() and (k[0] != 500).all()
    for bad in (([0, 0], [1, 1]), ([4], [1]), ([0], [-1])):
        with pytest.raises(P.Refused, match="SEQ"):
            c.extend(*bad)
    for bad in (([0], [0]), ([0], [2]), ([0, 0], [1, 1])):
        with pytest.raises(P.Refused, match="SEQ"):
            c.fork(*bad)
    with pytest.raises(P.Refused, match="SEQ"):
        c.release([0], [17])
    c.pages[0, 0] = 5
    with pytest.raises(P.Refused, match="PAGE"):
        c.release([0], [0])


def _pin_attention(P):
    rng = np.random.default_rng(0)
    v = rng.standard_normal((5, 2, 8))
    q = np.zeros((4, 8))
    out = P.attend(q, rng.standard_normal((5, 2, 8)), v)   # no preference: the mean
    assert np.allclose(out, np.repeat(v.mean(0), 2, axis=0))
    k = np.zeros((5, 2, 8))
    k[3] = 1000.0
    assert np.allclose(P.attend(np.ones((4, 8)), k, v), np.repeat(v[3], 2, axis=0))   # one key takes all
    k[3], k[1] = 0.0, np.sqrt(8.0) * np.log(3.0) / 8.0                                   # one key three times as heavy
    assert np.allclose(P.attend(np.ones((4, 8)), k, v), np.repeat((v.sum(0) + 2 * v[1]) / 7, 2, axis=0))
    k[1, 1], k[4, 1] = 0.0, 1000.0                                                       # each KV head its own keys
    assert np.allclose(P.attend(np.ones((4, 8)), k, v), [(v[:, 0].sum(0) + 2 * v[1, 0]) / 7] * 2 + [v[4, 1]] * 2)
    assert (P.attend(q, k[:0], v[:0]) == 0).all()
    o = P.attend_prompt(np.zeros((7, 4, 8)), np.zeros((7, 2, 8)), np.concatenate([v, v[:2]]), [1, 4, 4, 6])
    assert np.isnan(o[0]).all() and np.isnan(o[6]).all()
    assert np.allclose(o[1], np.repeat(v[1], 2, axis=0)) and np.allclose(o[3], np.repeat(v[1:4].mean(0), 2, axis=0))
    assert np.allclose(o[4], np.repeat(v[4], 2, axis=0))
    # the spread around the result: of two equally heavy values half their distance
    assert np.allclose(P.attend(q, k[:2] * 0, v[:2], True)[1], np.repeat(np.abs(v[0] - v[1]) / 2, 2, axis=0))


def test_oracle_pins():
    import oracle.paged
    _pin_pages(oracle.paged)
    _pin_attention(oracle.paged)


MISTAKES = [("refs[self.pages[s, have - 1]] > 1", "refs[self.pages[s, have - 1]] > 0"), ("n % self.ps and refs", "refs"),
            ("            refs[self.pages[s, have - 1]] -= 1\n", ""), ("if refs[p] == 0]", "if refs[p] == 0][::-1]"),
            ("self.k[:, p], self.v[:, p] = self.k[:, old], self.v[:, old]", "self.k[:, p] = self.k[:, old]"),
            ("self.refs[self.pages[s, j]] += 1", "pass"), ("or self.lens[d] != 0 ", ""), ("range(self._held(m), self._held(int", "range(self._held(m) + 1, self._held(int"),
            ("if not 0 <= m <= n", "if not 0 <= m"), ("self.refs[b], self.refs[a] = self.refs[a], 0", "self.refs[b] = self.refs[a]"),
            ("self.pages[s, j] = remap[self.pages[s, j]]", "pass"), ("p, o = self.slot(s, pos + r)", "p, o = self.slot(s, pos)"),
            ("/ np.sqrt(dim)", ""), ("k[:, h // group] @", "k[:, h % k.shape[1]] @"), ("k[a:t + 1], v[a:t + 1], True", "k[a:t], v[a:t], True"),
            ("k[a:t + 1], v[a:t + 1], True", "k[:t + 1], v[:t + 1], True"), ("np.abs(v[:, h // group] - out[h])", "np.abs(v[:, h // group])")]


@pytest.mark.parametrize("old,new", MISTAKES, ids=range(len(MISTAKES)))
def test_planted_mistakes_fail_a_pin(old, new):
    import types

    import oracle.paged
    text = open(oracle.paged.__file__).read()
    assert old in text
    m = types.ModuleType("planted")
    exec(compile(text.replace(old, new), "planted", "exec"), m.__dict__)
    with pytest.raises((AssertionError, IndexError, ValueError, m.Refused, pytest.fail.Exception)):
        _pin_pages(m)
        _pin_attention(m)
