"""Operators of long contexts, as a serving program calls them, with their plain forms.

Five operators of one path, from a projection's rows to a token's attention: rotary positions of the
rows; attention of packed prompts through a sliding window with a few first tokens that stay visible
(sinks); the rows into a paged cache held in 4 bits, and back; attention of one new token a sequence
over that cache; and of one new token over the bf16 pages through a window.

A case holds plain values only; sequence lengths follow from its "mix" number, so that work() knows
them, and every tensor's contents follow from the seed.  A window of 0 is no window.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EVERYTHING = (1 << 31) - 1   # a window that hides nothing


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short prompt to the smallest layer, a window a fraction of it: latency is all
        dict(name="window prompt short", op="prompt", n=1, longest=300, ragged=False, mix=1, q_heads=4, kv_heads=2, head_dim=64, pad=0, window=64, sinks=4),
        # a batch of prompts of every length packed into one pass, some shorter than the window
        dict(name="window prompts packed", op="prompt", n=24, longest=1531, ragged=True, mix=3, q_heads=40, kv_heads=8, head_dim=128, pad=37, window=512, sinks=4),
        # a long document
        dict(name="window prompt 16k", op="prompt", n=1, longest=16384, ragged=False, mix=4, q_heads=40, kv_heads=8, head_dim=128, pad=0, window=1024, sinks=4),
        # one user far into a conversation, a layer that looks back 1k tokens: latency
        dict(name="window token 32k", op="token", n=1, longest=32768, ragged=False, mix=6, q_heads=40, kv_heads=8, head_dim=128, page=64, window=1024, sinks=4),
        # a serving batch of mixed contexts, odd lengths and an odd window
        dict(name="window tokens ragged", op="token", n=128, longest=8191, ragged=True, mix=7, q_heads=40, kv_heads=8, head_dim=128, page=16, window=2047, sinks=4),
        # one user decoding at 32k from 4 bits, its last row stored by an earlier call
        dict(name="4-bit token 32k", op="token4", n=1, longest=32768, ragged=False, mix=8, q_heads=40, kv_heads=8, head_dim=128, page=64, window=0, sinks=0, new=False),
        # a batch on a smaller layer through a window, the new rows stored in the same call
        dict(name="4-bit tokens ragged, window", op="token4", n=48, longest=8191, ragged=True, mix=9, q_heads=8, kv_heads=2, head_dim=128, page=16, window=1500, sinks=4, new=True),
        # the largest batch: 128 users at 8k
        dict(name="4-bit tokens 128 x 8k", op="token4", n=128, longest=8192, ragged=False, mix=10, q_heads=40, kv_heads=8, head_dim=128, page=32, window=0, sinks=0, new=True),
        # accepted drafts of a batch appended to its pages: few rows a sequence, none of them aligned
        dict(name="4-bit rows of drafts", op="rows4", n=64, longest=7, mix=11, layers=2, kv_heads=8, head_dim=128, page=16),
        # a batch of prompts into one layer's pages, and back
        dict(name="4-bit rows packed", op="rows4", n=24, longest=4093, mix=12, layers=1, kv_heads=8, head_dim=128, page=16),
        # the new tokens of a batch, each at its own far position, scaled for a long context
        dict(name="rotary tokens", op="rotary", rows=48, far=131072, mix=13, heads=48, head_dim=128, rot_dim=128, interleaved=False, scaling=2),
        # a long prompt, neighbouring pairs, half of the head
        dict(name="rotary 16k", op="rotary", rows=16384, far=16384, mix=14, heads=48, head_dim=128, rot_dim=64, interleaved=True, scaling=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    q, kv, d = rng.choice([(4, 2, 64), (8, 2, 128), (40, 8, 128), (32, 4, 64), (16, 16, 128), (24, 1, 128)])
    page = rng.choice([16, 32, 64, 128])
    window, sinks = _log(rng, 1, 8192), rng.choice([0, 1, 4, 4, 33, 130])
    op = rng.choice(["prompt", "prompt", "token", "token4", "token4", "rows4", "rotary"])
    if op == "prompt":  # at most 16384 tokens in all, and no more work than 40 heads of 128 at 16384 with a window of 1024
        n = _log(rng, 1, 64)
        longest = _log(rng, 1, 16384 // n)
        return dict(op=op, n=n, longest=longest, ragged=rng.random() < 0.7, mix=mix, q_heads=q, kv_heads=kv, head_dim=d, pad=rng.choice([0, 1, 50]),
                    window=max(1, min(window, 1024 * 16384 // (n * longest)) - sinks), sinks=sinks)
    if op == "token":
        n = _log(rng, 1, 256)
        longest = _log(rng, 1, min(65536, (1 << 20) * 8 // (n * max(kv, 1))))
        return dict(op=op, n=n, longest=longest, ragged=rng.random() < 0.7, mix=mix, q_heads=q, kv_heads=kv, head_dim=d, page=page,
                    window=max(1, min(window, 2048 * 128 * 8 // (n * kv))), sinks=sinks)
    if op == "token4":
        n = _log(rng, 1, 256)
        longest = _log(rng, 1, min(65536, (1 << 20) * 8 // (n * max(kv, 1))))
        if rng.random() < 0.5:
            window, sinks = 0, 0
        return dict(op=op, n=n, longest=longest, ragged=rng.random() < 0.7, mix=mix, q_heads=q, kv_heads=kv, head_dim=d, page=page,
                    window=window, sinks=sinks, new=rng.random() < 0.7)
    if op == "rows4":
        n = _log(rng, 1, 64)
        return dict(op=op, n=n, longest=_log(rng, 1, 65536 // n), mix=mix, layers=rng.randint(1, 4), kv_heads=min(kv, 8), head_dim=d, page=page)
    return dict(op=op, rows=_log(rng, 1, 16384), far=_log(rng, 16, 1 << 20), mix=mix, heads=rng.choice([q + kv, q, kv]), head_dim=d,
                rot_dim=rng.choice([16, 32, 48, 64, d]), interleaved=rng.random() < 0.5, scaling=rng.randrange(4))


def _lengths(c):
    """Sequence lengths: all the longest, or one the longest and the rest spread over the logarithm."""
    if not c.get("ragged", c["op"] == "rows4"):
        return [c["longest"]] * c["n"]
    r = random.Random(c["mix"])
    got = [c["longest"]] + [_log(r, 1, c["longest"]) for _ in range(c["n"] - 1)]
    r.shuffle(got)
    return got


def _before(c):
    """rows4: the tokens that a sequence holds already."""
    r = random.Random(c["mix"] + 2)
    return [r.randrange(0, 40) for _ in range(c["n"])]


def _sees(x, c):
    """How many of x tokens the last one sees."""
    return x if c["window"] == 0 else min(x, c["window"] + c["sinks"])


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ a cache in 4 bits
# 32 values of a token's head share a scale s = bf16(max |x| / 7); x is held as the code 8 + x / s, rounded to the
# nearest (halves away from zero).  16 tokens of a head are one block of bytes: 16 D / 2 of codes, then the scales.
def _places(D):
    """Byte offsets in a block of the values 2 i and 2 i + 1 (low and high four bits) of each token's K, of its V, and
    of its scales (in units of bf16)."""
    t, i = torch.arange(16, device=DEV)[:, None], torch.arange(D // 2, device=DEV)[None, :]
    d, G = 2 * i, D // 32
    k = t * (D // 2) + ((d % 32) // 8 * G + d // 32) * 4 + (d % 8) // 2
    pair, odd, half = t % 8 // 2, t % 2, t // 8
    v = half * 4 * D + (((d % 32) // 4 * 4 + pair) * G + d // 32) * 4 + odd * 2 + (d % 4) // 2
    g = torch.arange(G, device=DEV)[None, :]
    return k, v, 4 * D + ((half * 4 + pair) * G + g) * 2 + odd


def _codes(x):
    """fp32 [..., D] -> codes [..., D] in 0 .. 15 and scales bf16 [..., D / 32]."""
    g = x.unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    s = (top / 7.0).to(torch.bfloat16)
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    q = torch.floor(g.abs() / s.float()[..., None] + 0.5) * g.sign()
    return (torch.where(s[..., None] > 0, q, torch.zeros_like(q)) + 8.0).to(torch.uint8).flatten(-2), s


def _bytes(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _block_bytes(D):
    return 9 * D


def _values(blocks, at, scales_at):
    """[..., 9 D] bytes -> fp32 [..., 16, D]."""
    b = blocks[..., at]
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2).float() - 8.0
    s = blocks.view(torch.bfloat16)[..., scales_at].float()
    return (n.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(shape, g, scale=1.0):
    """bf16 normals, made in pieces: a pool's worth of fp32 is not needed at once."""
    out = torch.empty(shape, device=DEV, dtype=torch.bfloat16)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randn(part.shape, device=DEV, generator=g) * scale)
    return out


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pool4(layers, n_pages, c, g):
    """A pool of normals, in 4 bits; K with a few channels of large values, as the keys of a trained layer have."""
    Hkv, D = c["kv_heads"], c["head_dim"]
    shape = (layers, n_pages, Hkv, c["page"] // 16, _block_bytes(D))
    kb, vb, sb = _places(D)
    loud = torch.ones(D, device=DEV)
    loud[:: 37] = 6.0
    got = []
    for at, gain in ((kb, loud), (vb, torch.ones(D, device=DEV))):
        out = torch.empty(shape, device=DEV, dtype=torch.uint8)
        flat = out.view(-1, _block_bytes(D))
        for i in range(0, flat.shape[0], 1 << 16):
            part = flat[i:i + (1 << 16)]
            codes, s = _codes((torch.randn((part.shape[0], 16, D), device=DEV, generator=g) * gain).bfloat16().float())
            part[:, at] = _bytes(codes)
            part.view(torch.bfloat16)[:, sb] = s
        got.append(out)
    return dict(k=got[0], v=got[1])


def _starts(lens):
    s = [0]
    for x in lens:
        s.append(s[-1] + x)
    return s


def _rope(c):
    """Frequencies of the pairs and the factor on the result; scaling 1: all frequencies divided; 2: only those that
    turn seldom in the original context, blended between 1 and 4 turns; 3: a larger base."""
    r, theta, factor, first = c["rot_dim"], 10000.0, 8.0, 8192
    if c["scaling"] == 3:
        theta *= factor ** (r / (r - 2.0))
    f = [theta ** (-2.0 * i / r) for i in range(r // 2)]
    if c["scaling"] == 1:
        f = [x / factor for x in f]
    if c["scaling"] == 2:
        keep = [min(1.0, max(0.0, (first * x / (2.0 * math.pi) - 1.0) / 3.0)) for x in f]
        f = [x * k + x / factor * (1.0 - k) for x, k in zip(f, keep)]
    return f, (0.1 * math.log(factor) + 1.0 if c["scaling"] == 2 else 1.0)


def prepare(case, seed):
    c, g, op = case, _gen(seed), case["op"]
    s = dict(case=c, op=op, status=torch.zeros(1, dtype=torch.int32, device=DEV))
    D = c["head_dim"]
    if op == "rotary":
        r = random.Random(c["mix"])
        width = c["heads"] * D
        pos = list(range(c["rows"])) if c["rows"] == c["far"] else [r.randrange(c["far"]) for _ in range(c["rows"])]
        f, gain = _rope(c)
        s.update(x=_normal((c["rows"], width), g), pos=_ints(pos), out=torch.zeros(c["rows"], width, device=DEV, dtype=torch.bfloat16),
                 freq=torch.tensor(f, dtype=torch.float64, device=DEV), gain=gain)
        return s
    if op == "prompt":
        # the QKV projection's rows: the Q heads, the K heads, the V heads.  Queries of twice the usual size give
        # the peaked rows of a trained layer beside flat ones
        lens = _lengths(c)
        starts = _starts(lens)
        rows, Hq, Hkv = starts[-1] + c["pad"], c["q_heads"], c["kv_heads"]
        qkv = _normal((rows, (Hq + 2 * Hkv) * D), g)
        qkv[:, : Hq * D // 2] *= 2
        s.update(qkv=qkv, starts=_ints(starts), rows=rows, longest=max(lens), tokens=starts[-1],
                 out=torch.zeros(rows, Hq, D, device=DEV, dtype=torch.bfloat16))
        return s
    order, ps = random.Random(c["mix"] + 1), c["page"]
    if op == "rows4":
        lens, pos = _lengths(c), _before(c)
        need = [_ceil(x + p, ps) for x, p in zip(lens, pos)]
    else:
        lens = _lengths(c)
        need = [_ceil(x, ps) for x in lens]
    n_pages = sum(need) + 3
    places = list(range(n_pages))
    order.shuffle(places)
    max_pages = max(need) + 1
    table, at = [], 0
    for m in need:
        table.append(places[at:at + m] + [0] * (max_pages - m))
        at += m
    s.update(pages=_ints(table), refs=torch.ones(n_pages, dtype=torch.int32, device=DEV))
    if op == "rows4":
        starts = _starts(lens)
        width = 2 * c["kv_heads"] * D
        s.update(_pool4(c["layers"], n_pages, c, g), lens=_ints([x + p for x, p in zip(lens, pos)]), ids=_ints(range(c["n"])), pos=_ints(pos),
                 starts=_ints(starts), kv=_normal((starts[-1], width), g), back=torch.zeros(starts[-1], width, device=DEV, dtype=torch.bfloat16),
                 layer=c["layers"] - 1)
        return s
    Hq, Hkv = c["q_heads"], c["kv_heads"]
    qkv = _normal((c["n"], (Hq + 2 * Hkv) * D), g)
    qkv[:, : Hq * D // 2] *= 2
    ids = list(range(c["n"]))
    order.shuffle(ids)
    if op == "token":
        shape = (1, n_pages, Hkv, ps, D)
        s.update(k=_normal(shape, g), v=_normal(shape, g))
    else:
        s.update(_pool4(1, n_pages, c, g), back=torch.zeros(c["n"], 2 * Hkv * D, device=DEV, dtype=torch.bfloat16),
                 last=_ints([lens[i] - 1 for i in ids]), each=_ints(range(c["n"] + 1)))
    s.update(lens=_ints(lens), ids=_ints(ids), qkv=qkv, out=torch.zeros(c["n"], Hq, D, device=DEV, dtype=torch.bfloat16))
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return _calls(state) if own else _plain(state)


def _handles(s):
    """What a program makes once: the library's structs and the workspaces."""
    from speculative_tree_verify_gb300 import abi
    c, op = s["case"], s["op"]
    h = dict(abi=abi, ok=abi.TV_OK)
    D = c["head_dim"]
    if op == "rotary":
        kind = (abi.TV_ROPE_PLAIN, abi.TV_ROPE_LINEAR, abi.TV_ROPE_BLEND, abi.TV_ROPE_BASE)[c["scaling"]]
        h["rope"] = abi.tv_rope_init(c["rot_dim"], c["interleaved"], 10000.0, kind, 8.0, 8192, 1.0, 4.0, s["gain"])
    elif op == "prompt":
        Hq, Hkv = c["q_heads"], c["kv_heads"]
        h["qkv"] = s["qkv"], s["qkv"][:, Hq * D:], s["qkv"][:, (Hq + Hkv) * D:]
        h["heads"] = Hq, Hkv, D
    else:
        refs, Hkv = s["refs"], c["kv_heads"]
        pool = abi.TvPool if op == "token" else abi.TvPool4
        h["pool"] = pool(s["k"].data_ptr(), s["v"].data_ptr(), refs.data_ptr(), s["k"].shape[0], s["k"].shape[1], Hkv, c["page"], D)
        h["seqs"] = abi.TvSeqs(s["pages"].data_ptr(), s["lens"].data_ptr(), s["pages"].shape[0], s["pages"].shape[1])
        if op == "rows4":
            h["kv"] = s["kv"], s["kv"][:, Hkv * D:]
            h["back"] = s["back"], s["back"][:, Hkv * D:]
        else:
            Hq = c["q_heads"]
            h["qkv"] = s["qkv"], s["qkv"][:, Hq * D:], s["qkv"][:, (Hq + Hkv) * D:]
            size = abi.tv_attend_paged_workspace_size if op == "token" else abi.tv_attend_paged4_workspace_size
            h["bytes"] = size(h["pool"], Hq, c["n"])
            h["ws"] = torch.empty(h["bytes"], dtype=torch.uint8, device=DEV)
            if op == "token4":
                h["back"] = s["back"], s["back"][:, Hkv * D:]
    s["handles"] = h
    return h


def _calls(s):
    h = s.get("handles") or _handles(s)
    abi, c, op = h["abi"], s["case"], s["op"]
    stream = torch.cuda.current_stream()
    D = c["head_dim"]

    def call(rc):
        if rc != h["ok"]:
            raise RuntimeError(abi.tv_status_string(rc))

    if op == "rotary":
        call(abi.tv_rope_rows(h["rope"], s["x"], s["x"].shape[1], s["out"], s["out"].shape[1], c["heads"], D, s["pos"], c["rows"], s["status"], stream))
        return [s["out"]]
    window = c.get("window", 0) or EVERYTHING
    if op == "prompt":
        q, k, v = h["qkv"]
        call(abi.tv_attend_prompt_window(*h["heads"], window, c["sinks"], q, k, v, q.shape[1], q.shape[1], s["starts"], c["n"], s["rows"], s["out"],
                                         s["status"], stream))
        return [s["out"]]
    if op == "token":
        q, k, v = h["qkv"]
        call(abi.tv_attend_paged_window(h["pool"], 0, h["seqs"], s["ids"], c["n"], c["q_heads"], window, c["sinks"], q, q.shape[1], k, v, q.shape[1],
                                        s["out"], h["ws"], h["bytes"], s["status"], stream))
        return [s["out"], s["k"], s["v"]]
    if op == "token4":
        q, k, v = h["qkv"]
        call(abi.tv_attend_paged4(h["pool"], 0, h["seqs"], s["ids"], c["n"], c["q_heads"], window, c["sinks"], q, q.shape[1], k if c["new"] else None,
                                  v if c["new"] else None, q.shape[1], s["out"], h["ws"], h["bytes"], s["status"], stream))
        if not c["new"]:
            return [s["out"]]
        k, v = h["back"]   # what the call stored, as the values that it stands for
        call(abi.tv_pages4_read(h["pool"], 0, h["seqs"], s["ids"], s["last"], s["each"], c["n"], c["n"], k, v, k.shape[1], D, s["status"], stream))
        return [s["out"], s["back"]]
    k, v = h["kv"]
    call(abi.tv_pages4_write(h["pool"], s["layer"], h["seqs"], s["ids"], s["pos"], s["starts"], c["n"], k.shape[0], k, v, k.shape[1], D,
                             s["status"], stream))
    k, v = h["back"]
    call(abi.tv_pages4_read(h["pool"], s["layer"], h["seqs"], s["ids"], s["pos"], s["starts"], c["n"], k.shape[0], k, v, k.shape[1], D,
                            s["status"], stream))
    return [s["back"]]


# ------------------------------------------------------------------ plain forms
def _plain(s):
    if s["op"] == "rotary":
        return _plain_rotary(s)
    if s["op"] == "prompt":
        return _plain_prompt(s)
    if s["op"] == "rows4":
        return _plain_rows4(s)
    return _plain_token(s)


def _plain_rotary(s):
    """Pair i of a head's first rot_dim values turned by pos * freq[i], the angle in 64 bits."""
    c = s["case"]
    r = c["rot_dim"]
    x = s["x"].view(c["rows"], c["heads"], c["head_dim"]).float()
    a = s["pos"].double()[:, None] * s["freq"]
    cos, sin = (a.cos() * s["gain"]).float()[:, None], (a.sin() * s["gain"]).float()[:, None]
    u, w = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., : r // 2], x[..., r // 2:r])
    both = (u * cos - w * sin, u * sin + w * cos)
    turned = torch.stack(both, -1).flatten(-2) if c["interleaved"] else torch.cat(both, -1)
    s["out"].copy_(torch.cat([turned, x[..., r:]], -1).flatten(1))
    return [s["out"]]


def _plain_prompt(s):
    """softmax(Q K^T / sqrt(D)) V over each sequence's last `window` rows and its first `sinks`, the sequences padded
    to the longest."""
    c = s["case"]
    Hq, Hkv, D, n, L = c["q_heads"], c["kv_heads"], c["head_dim"], c["n"], s["longest"]
    G = Hq // Hkv
    first, last = s["starts"][:-1].long(), s["starts"][1:].long()
    t = torch.arange(L, device=DEV)
    here = t[None, :] < (last - first)[:, None]
    row = torch.where(here, first[:, None] + t[None, :], 0)
    hide = (t[None, :] > t[:, None]) | ((t[None, :] <= t[:, None] - c["window"]) & (t[None, :] >= c["sinks"]))
    out = torch.empty(n, L, Hq, D, device=DEV, dtype=torch.bfloat16)
    for h in range(Hkv):  # a KV head at a time: all heads' scores at once would not fit
        q = s["qkv"][:, h * G * D:(h + 1) * G * D][row].view(n, L, G, D).permute(0, 2, 1, 3).float()
        k = s["qkv"][:, (Hq + h) * D:(Hq + h + 1) * D][row].view(n, 1, L, D).float()
        v = s["qkv"][:, (Hq + Hkv + h) * D:(Hq + Hkv + h + 1) * D][row].view(n, 1, L, D).float()
        p = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).masked_fill_(hide, -math.inf)
        p = p.sub_(p.amax(-1, keepdim=True)).exp_()
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
        out[:, :, h * G:(h + 1) * G] = o.permute(0, 2, 1, 3)
    s["out"][row[here]] = out[here]
    return [s["out"]]


def _store4(s, layer, page, slot, k, v):
    """Rows of fp32 [rows, Hkv, D] into slots of pages."""
    D = s["case"]["head_dim"]
    kb, vb, sb = _places(D)
    block, t = (slot // 16)[:, None, None], slot % 16
    head = torch.arange(s["case"]["kv_heads"], device=DEV)[None, :, None]
    for pool, x, at in ((s["k"], k, kb), (s["v"], v, vb)):
        codes, sc = _codes(x)
        pool[layer][page[:, None, None], head, block, at[t][:, None]] = _bytes(codes)
        pool.view(torch.bfloat16)[layer][page[:, None, None], head, block, sb[t][:, None]] = sc


def _load4(s, layer, page, slot):
    """The values of slots of pages, fp32 [rows, Hkv, D]."""
    D = s["case"]["head_dim"]
    kb, vb, sb = _places(D)
    block, t = (slot // 16)[:, None, None], slot % 16
    head = torch.arange(s["case"]["kv_heads"], device=DEV)[None, :, None]
    got = []
    for pool, at in ((s["k"], kb), (s["v"], vb)):
        b = pool[layer][page[:, None, None], head, block, at[t][:, None]]
        sc = pool.view(torch.bfloat16)[layer][page[:, None, None], head, block, sb[t][:, None]].float()
        x = torch.stack([b & 15, b >> 4], -1).flatten(-2).float() - 8.0
        got.append((x.unflatten(-1, (-1, 32)) * sc[..., None]).flatten(-2))
    return got


def _plain_rows4(s):
    c = s["case"]
    ps, Hkv, D = c["page"], c["kv_heads"], c["head_dim"]
    first = s["starts"].long()
    r = torch.arange(s["kv"].shape[0], device=DEV)
    seq = torch.searchsorted(first[1:], r, right=True)
    at = s["pos"].long()[seq] + r - first[seq]
    page = s["pages"][s["ids"].long()[seq], at // ps].long()
    _store4(s, s["layer"], page, at % ps, s["kv"][:, : Hkv * D].view(-1, Hkv, D).float(), s["kv"][:, Hkv * D:].view(-1, Hkv, D).float())
    s["back"].copy_(torch.cat([x.flatten(1) for x in _load4(s, s["layer"], page, at % ps)], 1))
    return [s["back"]]


def _plain_token(s):
    """The new token's K and V into their slot, then softmax(q K^T / sqrt(D)) V over the slots that it sees."""
    c = s["case"]
    Hq, Hkv, D, n, ps = c["q_heads"], c["kv_heads"], c["head_dim"], c["n"], c["page"]
    ids, four = s["ids"].long(), s["op"] == "token4"
    lens, table = s["lens"][ids].long(), s["pages"][ids].long()
    q = s["qkv"][:, : Hq * D].view(n, Hkv, Hq // Hkv, D).float()
    at = lens - 1
    page = table.gather(1, (at // ps)[:, None])[:, 0]
    new_k, new_v = s["qkv"][:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D), s["qkv"][:, (Hq + Hkv) * D:].view(n, Hkv, D)
    if not four:
        s["k"][0, page, :, at % ps] = new_k
        s["v"][0, page, :, at % ps] = new_v
    elif c["new"]:
        _store4(s, 0, page, at % ps, new_k.float(), new_v.float())
        s["back"].copy_(torch.cat([x.flatten(1) for x in _load4(s, 0, page, at % ps)], 1))
    if c["window"] > 0:   # the tokens that are seen: the first ones, and those of the window
        most = min(c["longest"], c["window"] + c["sinks"])
        j = torch.arange(most, device=DEV)[None, :]
        tok = j + torch.where(j < c["sinks"], 0, (lens - (c["window"] + c["sinks"])).clamp(min=0)[:, None])
        seen = tok < lens[:, None]
        tok = torch.where(seen, tok, 0)
    else:
        tok = torch.arange(c["longest"], device=DEV)[None, :].expand(n, -1)
        seen = tok < lens[:, None]
        tok = torch.where(seen, tok, 0)
    pages = table.gather(1, tok // ps)

    def rows(which):   # [n, Hkv, tokens, D]
        if not four:
            return s[which][0][pages, :, tok % ps].transpose(1, 2).float()
        kb, vb, sb = _places(D)
        if c["window"] == 0:   # whole blocks
            x = _values(s[which][0][table[:, : _ceil(c["longest"], ps)]], kb if which == "k" else vb, sb)   # [n, pages, Hkv, blocks, 16, D]
            return x.permute(0, 2, 1, 3, 4, 5).reshape(n, Hkv, -1, D)[:, :, : c["longest"]]
        got = _load4(s, 0, pages.flatten(), (tok % ps).flatten())[0 if which == "k" else 1]
        return got.view(n, -1, Hkv, D).transpose(1, 2)

    k = rows("k")
    p = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    del k
    p = p.masked_fill(~seen[:, None, None, :], -math.inf)
    p = (p - p.amax(-1, keepdim=True)).exp()
    o = torch.matmul(p, rows("v")) / p.sum(-1, keepdim=True)
    s["out"].copy_(o.reshape(n, Hq, D))
    if four:
        return [s["out"], s["back"]] if c["new"] else [s["out"]]
    return [s["out"], s["k"], s["v"]]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, op, D = case, case["op"], case["head_dim"]
    if op == "rotary":
        turned = c["rows"] * c["heads"] * c["rot_dim"]
        return {"bytes": 4.0 * c["rows"] * c["heads"] * D + 4.0 * c["rows"], "flops": 3.0 * turned}
    row = c["kv_heads"] * D * 2   # bytes of one token's K (or V) in one layer, in bf16
    lens = _lengths(c)
    if op == "prompt":
        w, k = c["window"], c["sinks"]
        pairs = 0
        for x in lens:   # row t sees min(t + 1, w + min(k, the rows that the window has left behind))
            m = min(x, w + k)
            pairs += m * (m + 1) // 2 + (x - m) * (w + k)
        return {"bytes": sum(lens) * (2 * c["q_heads"] * D * 2 + 2 * row), "flops": 4.0 * pairs * c["q_heads"] * D}
    row4 = row * 9 // 32          # in 4 bits and a scale for every 32 of them
    if op == "rows4":
        return {"bytes": sum(lens) * (4.0 * row + 4.0 * row4), "flops": 0}
    seen = sum(_sees(x, c) for x in lens)
    heads = c["n"] * 2 * c["q_heads"] * D * 2
    if op == "token":
        return {"bytes": seen * 2.0 * row + heads + 2 * c["n"] * row, "flops": 4.0 * seen * c["q_heads"] * D}
    stored = c["n"] * (4 * row + 2 * row4) if c["new"] else 0   # the new rows read, stored, and returned
    return {"bytes": seen * 2.0 * row4 + heads + stored, "flops": 4.0 * seen * c["q_heads"] * D}


# ------------------------------------------------------------------ in 64 bits
def _decoded(blocks, D, v):
    """[..., 9 D] bytes as fp64 [..., 16, D], by the order in which a block holds its values."""
    lead, G = blocks.shape[:-1], D // 32
    b = blocks[..., : 8 * D]
    n = torch.stack([b & 15, b >> 4], -1).double() - 8
    if v:   # half of the tokens, 4 values of 32, token pair, 32 values, token of the pair, 2 bytes, 2 values
        n = n.reshape(*lead, 2, 8, 4, G, 2, 2, 2).movedim((-7, -5, -3, -4, -6, -2, -1), (-7, -6, -5, -4, -3, -2, -1))
    else:   # token, 8 values of 32, 32 values, 4 bytes, 2 values
        n = n.reshape(*lead, 16, 4, G, 4, 2).transpose(-4, -3)
    n = n.reshape(*lead, 16, G, 32)
    s = blocks[..., 8 * D:].contiguous().view(torch.bfloat16).double().reshape(*lead, 2, 4, G, 2).transpose(-2, -1)
    return (n * s.reshape(*lead, 16, G, 1)).reshape(*lead, 16, D)


def _held(x):
    """fp64 rows as a 4-bit cache gives them back."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    s = (g.abs().amax(-1, keepdim=True) / 7).float().bfloat16().double()
    n = torch.where(s > 0, torch.trunc(g / s + 0.5 * torch.sign(g)), 0.0)
    return (n * s).reshape(x.shape)


def exact(case, seed):
    c, D, op = case, case["head_dim"], case["op"]
    s = prepare(case, seed)
    if op == "rotary":
        r, x = c["rot_dim"], s["x"].double().view(c["rows"], c["heads"], D)
        for i, f in enumerate(_rope(c)[0]):
            z = torch.polar(torch.full_like(s["pos"], s["gain"], dtype=torch.float64), s["pos"].double() * f)[:, None]
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
            y = torch.complex(x[..., a].clone(), x[..., b].clone()) * z
            x[..., a], x[..., b] = y.real, y.imag
        return [x.reshape(c["rows"], -1)]
    if op == "rows4":
        return [_held(s["kv"].double())]
    Hq, Hkv, x = c["q_heads"], c["kv_heads"], s["qkv"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lens, w, sinks = _lengths(c), c["window"], c["sinks"]
    if op == "prompt":
        at = 0
        for L in lens:
            for h in range(Hq):
                g = h * Hkv // Hq
                k = x[at:at + L, (Hq + g) * D:(Hq + g + 1) * D]
                v = x[at:at + L, (Hq + Hkv + g) * D:(Hq + Hkv + g + 1) * D]
                for b in range(0, L, 2048):
                    e = min(L, b + 2048)
                    lo = max(0, b - w + 1)
                    j = torch.cat([torch.arange(min(sinks, lo), device=DEV), torch.arange(lo, e, device=DEV)])
                    t = torch.arange(b, e, device=DEV)[:, None]
                    a = x[at + b:at + e, h * D:(h + 1) * D] @ k[j].T / D ** 0.5
                    a = a.masked_fill((j > t) | ((t - j >= w) & (j >= sinks)), -math.inf)
                    out[at + b:at + e, h] = torch.softmax(a, -1) @ v[j]
            at += L
        return [out]
    ids, table, ps = s["ids"].tolist(), s["pages"].tolist(), c["page"]
    four = op == "token4"
    new = x[:, Hq * D:].view(c["n"], 2, Hkv, D)
    new = _held(new) if four else new
    for i, t in enumerate(ids):
        L = lens[t]
        p = torch.tensor(table[t][: _ceil(L, ps)], device=DEV)
        if four:
            k = _decoded(s["k"][0][p], D, False).transpose(0, 1).reshape(Hkv, -1, D)[:, :L].transpose(0, 1)
            v = _decoded(s["v"][0][p], D, True).transpose(0, 1).reshape(Hkv, -1, D)[:, :L].transpose(0, 1)
        else:
            k = s["k"][0][p].double().transpose(1, 2).reshape(-1, Hkv, D)[:L]
            v = s["v"][0][p].double().transpose(1, 2).reshape(-1, Hkv, D)[:L]
        if not four or c["new"]:
            k, v = k.clone(), v.clone()
            k[L - 1], v[L - 1] = new[i]
        if 0 < w < L - sinks:
            k, v = (torch.cat([y[:sinks], y[L - w:]]) for y in (k, v))
        q = x[i, : Hq * D].view(Hkv, Hq // Hkv, D)
        a = torch.softmax(torch.einsum("hgd,lhd->hgl", q, k) / D ** 0.5, -1)
        out[i] = torch.einsum("hgl,lhd->hgd", a, v).reshape(Hq, D)
    if four:
        return [out, new.reshape(c["n"], -1)] if c["new"] else [out]
    return [out, None, None]
