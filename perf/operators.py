"""The prompt and page-cache operators, as a serving program calls them, with their plain forms.

Three operators of one set: attention over packed prompts (what fills a cache), the pages of a
paged key-value cache (writing rows into them and reading them back, forking, extending with
copy-on-write, releasing, compacting), and attention of one new token over that cache.

A case holds plain values only; sequence lengths follow from its "mix" number, so that work() knows
them, and every tensor's contents follow from the seed.  Head counts are the layers' of this
repository: 4/2 heads of 64, 8/2 and 40/8 heads of 128.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short prompt to the smallest layer: latency is all
        dict(name="prompt short", op="prompt", n=1, longest=64, ragged=False, mix=1, q_heads=4, kv_heads=2, head_dim=64, pad=0),
        # one user's prompt of 1k tokens to the hidden-5120 layer
        dict(name="prompt 1k", op="prompt", n=1, longest=1024, ragged=False, mix=2, q_heads=40, kv_heads=8, head_dim=128, pad=0),
        # a batch of prompts of every length packed into one pass, padding rows behind them
        dict(name="prompt packed", op="prompt", n=24, longest=1531, ragged=True, mix=3, q_heads=40, kv_heads=8, head_dim=128, pad=37),
        # a long document
        dict(name="prompt 16k", op="prompt", n=1, longest=16384, ragged=False, mix=4, q_heads=40, kv_heads=8, head_dim=128, pad=0),
        # one user decoding at 1k: latency
        dict(name="token 1k", op="token", n=1, longest=1024, ragged=False, mix=5, q_heads=40, kv_heads=8, head_dim=128, page=16),
        # one user decoding at 32k
        dict(name="token 32k", op="token", n=1, longest=32768, ragged=False, mix=6, q_heads=40, kv_heads=8, head_dim=128, page=64),
        # a serving batch of mixed contexts on a smaller layer, odd lengths
        dict(name="token ragged", op="token", n=48, longest=8191, ragged=True, mix=7, q_heads=8, kv_heads=2, head_dim=128, page=16),
        # the largest batch: 128 users at 8k
        dict(name="token 128 x 8k", op="token", n=128, longest=8192, ragged=False, mix=8, q_heads=40, kv_heads=8, head_dim=128, page=32),
        # eight samples of a 1k prompt: fork, room for the next drafts, the rejected ones given back
        dict(name="fork 8 at 1k", op="fork", n=8, longest=1000, mix=9, layers=4, kv_heads=8, head_dim=128, page=16),
        # 32 samples of a 32k prompt
        dict(name="fork 32 at 32k", op="fork", n=32, longest=32759, mix=10, layers=4, kv_heads=8, head_dim=128, page=16),
        # a batch of prompts' keys and values into one layer's pages, and the longest read back as a contiguous cache
        dict(name="rows packed", op="rows", n=24, longest=4093, mix=11, layers=1, kv_heads=8, head_dim=128, page=16),
        # a pool that churn has left half empty, its used pages moved to the front
        dict(name="compact 8192 pages", op="compact", n=64, pages=8192, mix=12, layers=4, kv_heads=8, head_dim=128, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    q, kv, d = rng.choice([(4, 2, 64), (8, 2, 128), (40, 8, 128), (32, 4, 64), (16, 16, 128), (24, 1, 128)])
    page = rng.choice([16, 32, 64, 128])
    op = rng.choice(["prompt", "prompt", "token", "token", "fork", "rows", "compact"])
    if op == "prompt":  # at most 16384 tokens in all, and no more work than 40 heads of 128 at 16384
        n = _log(rng, 1, 64)
        longest = _log(rng, 1, 16384 // n)
        return dict(op=op, n=n, longest=longest, ragged=rng.random() < 0.7, mix=mix, q_heads=q, kv_heads=kv, head_dim=d, pad=rng.choice([0, 1, 50]))
    if op == "token":
        n = _log(rng, 1, 256)
        longest = _log(rng, 1, min(65536, (1 << 20) * 8 // (n * max(kv, 1))))
        return dict(op=op, n=n, longest=longest, ragged=rng.random() < 0.7, mix=mix, q_heads=q, kv_heads=kv, head_dim=d, page=page)
    layers = rng.randint(1, 4)
    if op == "fork":
        return dict(op=op, n=_log(rng, 1, 64), longest=_log(rng, 1, 32768), mix=mix, layers=layers, kv_heads=min(kv, 8), head_dim=d, page=page)
    if op == "rows":
        n = _log(rng, 1, 64)
        return dict(op=op, n=n, longest=_log(rng, 1, 65536 // n), mix=mix, layers=layers, kv_heads=min(kv, 8), head_dim=d, page=rng.choice([16, 32]))
    return dict(op=op, n=_log(rng, 4, 128), pages=_log(rng, 100, 8192 * 16 // page), mix=mix, layers=layers, kv_heads=min(kv, 8), head_dim=d, page=page)


def _lengths(c):
    """Sequence lengths: all the longest, or one the longest and the rest spread over the logarithm."""
    if not c.get("ragged", c["op"] == "rows"):
        return [c["longest"]] * c["n"]
    r = random.Random(c["mix"])
    got = [c["longest"]] + [_log(r, 1, c["longest"]) for _ in range(c["n"] - 1)]
    r.shuffle(got)
    return got


def _fork_plan(c):
    """Tokens each child grows by, and how many of them it keeps: 1 to 32 drafts, at least one kept."""
    r = random.Random(c["mix"])
    add = [r.randint(1, 32) for _ in range(c["n"])]
    return add, [r.randint(1, a) for a in add]


def _compact_plan(c):
    """The pages of each sequence in a pool left half used: random places, and the first quarter of every 8th
    sequence shared with the one before it (a fork)."""
    r = random.Random(c["mix"])
    places = list(range(c["pages"]))
    r.shuffle(places)
    left, per, rows = places[: c["pages"] // 2], c["pages"] // 2 // c["n"], []
    for i in range(c["n"]):
        take = r.randint(0, 2 * per) if i + 1 < c["n"] else per
        take = min(take, len(left))
        mine, left = left[:take], left[take:]
        if i % 8 == 7:
            mine = rows[i - 1][: len(rows[i - 1]) // 4] + mine
        rows.append(mine)
    lens = [max(0, len(m) * c["page"] - r.randrange(c["page"])) for m in rows]
    return rows, lens


def _ceil(a, b):
    return -(-a // b)


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


def _pool(c, n_pages, layers, g):
    shape = (layers, n_pages, c["kv_heads"], c["page"], c["head_dim"])
    return dict(k=_normal(shape, g), v=_normal(shape, g))


def _starts(lens):
    s = [0]
    for x in lens:
        s.append(s[-1] + x)
    return s


def prepare(case, seed):
    c, g, op = case, _gen(seed), case["op"]
    s = dict(case=c, op=op, status=torch.zeros(1, dtype=torch.int32, device=DEV))
    D = c["head_dim"]
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
    order = random.Random(c["mix"] + 1)
    if op == "token":
        lens = _lengths(c)
        need = [_ceil(x, c["page"]) for x in lens]
        n_pages = sum(need) + 3
        places = list(range(n_pages))
        order.shuffle(places)
        max_pages = max(need) + 1
        table, at = [], 0
        for m in need:
            table.append(places[at:at + m] + [0] * (max_pages - m))
            at += m
        Hq, Hkv = c["q_heads"], c["kv_heads"]
        qkv = _normal((c["n"], (Hq + 2 * Hkv) * D), g)
        qkv[:, : Hq * D // 2] *= 2
        ids = list(range(c["n"]))
        order.shuffle(ids)
        s.update(_pool(c, n_pages, 1, g), pages=_ints(table), lens=_ints(lens), refs=torch.ones(n_pages, dtype=torch.int32, device=DEV),
                 ids=_ints(ids), qkv=qkv, out=torch.zeros(c["n"], Hq, D, device=DEV, dtype=torch.bfloat16))
        return s
    ps = c["page"]
    if op == "fork":
        add, keep = _fork_plan(c)
        first = _ceil(c["longest"], ps)
        n_pages = first + sum(_ceil(c["longest"] % ps + a, ps) + 1 for a in add) + 8
        max_pages = _ceil(c["longest"] + 32, ps) + 1
        places = list(range(n_pages))
        order.shuffle(places)
        table = torch.full((c["n"] + 1, max_pages), -1, dtype=torch.int32, device=DEV)
        table[0, :first] = _ints(places[:first])
        refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        refs[table[0, :first].long()] = 1
        s.update(_pool(c, n_pages, c["layers"], g), pages=table, lens=_ints([c["longest"]] + [0] * c["n"]), refs=refs,
                 parent=_ints([0] * c["n"]), ids=_ints(range(1, c["n"] + 1)), add=_ints(add), none=_ints([0] * c["n"]),
                 keep=_ints([c["longest"] + k for k in keep]))
        return s
    if op == "rows":
        lens = _lengths(c)
        need = [_ceil(x, ps) for x in lens]
        n_pages = sum(need) + 3
        places = list(range(n_pages))
        order.shuffle(places)
        table, at = [], 0
        for m in need:
            table.append(places[at:at + m] + [-1] * (max(need) - m))
            at += m
        starts = _starts(lens)
        big = max(range(len(lens)), key=lambda i: lens[i])
        kv = _normal((starts[-1], 2 * c["kv_heads"] * D), g)
        shape = (c["kv_heads"], lens[big] + 32, D)  # a contiguous cache with room for a draft tree
        s.update(_pool(c, n_pages, c["layers"], g), pages=_ints(table), lens=_ints(lens), refs=torch.ones(n_pages, dtype=torch.int32, device=DEV),
                 ids=_ints(range(c["n"])), pos=_ints([0] * c["n"]), starts=_ints(starts), kv=kv, layer=c["layers"] - 1,
                 one=_ints([big]), one_pos=_ints([0]), one_starts=_ints([0, lens[big]]), cache_k=torch.zeros(shape, device=DEV, dtype=torch.bfloat16),
                 cache_v=torch.zeros(shape, device=DEV, dtype=torch.bfloat16), big=lens[big])
        return s
    rows, lens = _compact_plan(c)
    max_pages = max(1, max(len(r) for r in rows))
    refs = [0] * c["pages"]
    for r in rows:
        for p in r:
            refs[p] += 1
    pages0 = _ints([r + [-1] * (max_pages - len(r)) for r in rows])
    s.update(_pool(c, c["pages"], c["layers"], g), pages0=pages0, refs0=_ints(refs), lens=_ints(lens), pages=pages0.clone(), refs=_ints(refs),
             remap=torch.zeros(c["pages"], dtype=torch.int32, device=DEV), used=torch.zeros(1, dtype=torch.int32, device=DEV))
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return _calls(state) if own else _plain(state)


def _handles(s):
    """What a program makes once: the library's structs and the workspaces."""
    from speculative_tree_verify_gb300 import abi
    c, h = s["case"], dict(abi=abi, ok=abi.TV_OK)
    if s["op"] == "prompt":
        Hq, Hkv, D = c["q_heads"], c["kv_heads"], c["head_dim"]
        h["qkv"] = s["qkv"], s["qkv"][:, Hq * D:], s["qkv"][:, (Hq + Hkv) * D:]
        h["heads"] = Hq, Hkv, D
    else:
        k = s["k"]
        h["pool"] = abi.TvPool(k.data_ptr(), s["v"].data_ptr(), s["refs"].data_ptr(), k.shape[0], k.shape[1], k.shape[2], k.shape[3], k.shape[4])
        h["seqs"] = abi.TvSeqs(s["pages"].data_ptr(), s["lens"].data_ptr(), s["pages"].shape[0], s["pages"].shape[1])
        if s["op"] == "token":
            Hq, Hkv, D = c["q_heads"], c["kv_heads"], c["head_dim"]
            h["qkv"] = s["qkv"], s["qkv"][:, Hq * D:], s["qkv"][:, (Hq + Hkv) * D:]
            h["bytes"] = abi.tv_attend_paged_workspace_size(h["pool"], Hq, c["n"])
        else:
            h["bytes"] = abi.tv_pages_workspace_size(h["pool"], h["seqs"])
        if s["op"] == "rows":
            h["kv"] = s["kv"], s["kv"][:, c["kv_heads"] * c["head_dim"]:]
        h["ws"] = torch.empty(h["bytes"], dtype=torch.uint8, device=DEV)
    s["handles"] = h
    return h


def _calls(s):
    h = s.get("handles") or _handles(s)
    abi, c, op = h["abi"], s["case"], s["op"]
    stream = torch.cuda.current_stream()

    def call(rc):
        if rc != h["ok"]:
            raise RuntimeError(abi.tv_status_string(rc))

    if op == "prompt":
        q, k, v = h["qkv"]
        call(abi.tv_attend_prompt(*h["heads"], q, k, v, q.shape[1], q.shape[1], s["starts"], c["n"], s["rows"], s["out"], s["status"], stream))
        return [s["out"]]
    if op == "token":
        q, k, v = h["qkv"]
        call(abi.tv_attend_paged(h["pool"], 0, h["seqs"], s["ids"], c["n"], c["q_heads"], q, q.shape[1], k, v, q.shape[1], s["out"],
                                 h["ws"], h["bytes"], s["status"], stream))
        return [s["out"], s["k"], s["v"]]
    if op == "fork":
        call(abi.tv_pages_release(h["pool"], h["seqs"], s["ids"], s["none"], c["n"], s["status"], stream))
        call(abi.tv_pages_fork(h["pool"], h["seqs"], s["parent"], s["ids"], c["n"], s["status"], stream))
        call(abi.tv_pages_extend(h["pool"], h["seqs"], s["ids"], s["add"], c["n"], h["ws"], h["bytes"], s["status"], stream))
        call(abi.tv_pages_release(h["pool"], h["seqs"], s["ids"], s["keep"], c["n"], s["status"], stream))
        return [s["pages"], s["lens"], s["refs"], s["k"], s["v"]]
    if op == "rows":
        k, v = h["kv"]
        D, cap = c["head_dim"], s["cache_k"].shape[1]
        call(abi.tv_pages_write(h["pool"], s["layer"], h["seqs"], s["ids"], s["pos"], s["starts"], c["n"], k.shape[0], k, v, k.shape[1], D,
                                s["status"], stream))
        call(abi.tv_pages_read(h["pool"], s["layer"], h["seqs"], s["one"], s["one_pos"], s["one_starts"], 1, s["big"], s["cache_k"], s["cache_v"],
                               D, cap * D, s["status"], stream))
        return [s["k"], s["v"], s["cache_k"], s["cache_v"]]
    # the fragmented pool arrives: its tables and counts as they were before the last pass moved them
    s["pages"].copy_(s["pages0"])
    s["refs"].copy_(s["refs0"])
    call(abi.tv_pages_compact(h["pool"], h["seqs"], s["remap"], s["used"], h["ws"], h["bytes"], s["status"], stream))
    return [s["pages"], s["refs"], s["remap"], s["used"], s["k"], s["v"]]


# ------------------------------------------------------------------ plain forms
def _plain(s):
    op = s["op"]
    if op == "prompt":
        return _plain_prompt(s)
    if op == "token":
        return _plain_token(s)
    if op == "fork":
        _plain_release(s, s["none"])
        _plain_fork(s)
        _plain_extend(s)
        _plain_release(s, s["keep"])
        return [s["pages"], s["lens"], s["refs"], s["k"], s["v"]]
    if op == "rows":
        return _plain_rows(s)
    s["pages"].copy_(s["pages0"])
    s["refs"].copy_(s["refs0"])
    return _plain_compact(s)


def _plain_prompt(s):
    """softmax(Q K^T / sqrt(D)) V over each sequence's own earlier rows, the sequences padded to the longest."""
    c = s["case"]
    Hq, Hkv, D, n, L = c["q_heads"], c["kv_heads"], c["head_dim"], c["n"], s["longest"]
    G = Hq // Hkv
    first, last = s["starts"][:-1].long(), s["starts"][1:].long()
    t = torch.arange(L, device=DEV)
    here = t[None, :] < (last - first)[:, None]
    row = torch.where(here, first[:, None] + t[None, :], 0)
    hide = t[None, :] > t[:, None]
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


def _plain_token(s):
    """The new token's K and V into their slot, then softmax(q K^T / sqrt(D)) V over the sequence's slots."""
    c = s["case"]
    Hq, Hkv, D, n, ps = c["q_heads"], c["kv_heads"], c["head_dim"], c["n"], c["page"]
    ids = s["ids"].long()
    lens, table = s["lens"][ids].long(), s["pages"][ids].long()
    q = s["qkv"][:, : Hq * D].view(n, Hkv, Hq // Hkv, D).float()
    at = lens - 1
    page = table.gather(1, (at // ps)[:, None])[:, 0]
    s["k"][0, page, :, at % ps] = s["qkv"][:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D)
    s["v"][0, page, :, at % ps] = s["qkv"][:, (Hq + Hkv) * D:].view(n, Hkv, D)
    L = table.shape[1] * ps
    k = s["k"][0][table].permute(0, 2, 1, 3, 4).reshape(n, Hkv, L, D).float()
    p = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    del k
    p = p.masked_fill(torch.arange(L, device=DEV)[None, None, None, :] >= lens[:, None, None, None], -math.inf)
    p = (p - p.amax(-1, keepdim=True)).exp()
    v = s["v"][0][table].permute(0, 2, 1, 3, 4).reshape(n, Hkv, L, D).float()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    s["out"].copy_(o.reshape(n, Hq, D))
    return [s["out"], s["k"], s["v"]]


def _plain_release(s, keep):
    """Every page past the kept length loses a reference."""
    ps, ids = s["case"]["page"], s["ids"].long()
    lens, table = s["lens"][ids].long(), s["pages"][ids].long()
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    gone = (j >= ((keep.long() + ps - 1) // ps)[:, None]) & (j < ((lens + ps - 1) // ps)[:, None])
    s["refs"].index_add_(0, torch.where(gone, table, 0).view(-1), gone.to(torch.int32).view(-1), alpha=-1)
    s["lens"][ids] = keep


def _plain_fork(s):
    """The child's table is the parent's, each of its pages held once more."""
    ps, src, dst = s["case"]["page"], s["parent"].long(), s["ids"].long()
    lens, table = s["lens"][src], s["pages"][src]
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    held = j < ((lens + ps - 1) // ps)[:, None]
    s["refs"].index_add_(0, torch.where(held, table, 0).long().view(-1), held.to(torch.int32).view(-1))
    s["pages"][dst] = torch.where(held, table, s["pages"][dst])
    s["lens"][dst] = lens


def _plain_extend(s):
    """In list order: a shared page that new tokens would go into is copied to the lowest free page (the last holder
    keeps it), and new pages come from the lowest free ones."""
    ps, ids, n = s["case"]["page"], s["ids"].long(), s["case"]["n"]
    lens, table, refs, add = s["lens"][ids].long(), s["pages"][ids].long(), s["refs"], s["add"].long()
    have, want = (lens + ps - 1) // ps, (lens + add + ps - 1) // ps
    last = table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0].clamp(min=0)
    cand = (lens % ps != 0) & (add > 0) & (refs[last] > 1)
    order = torch.arange(n, device=DEV)
    held = torch.zeros(refs.shape[0], dtype=torch.int64, device=DEV).index_add_(0, last, cand.long())
    final = torch.full((refs.shape[0],), -1, dtype=torch.int64, device=DEV)
    final = final.scatter_reduce(0, last, torch.where(cand, order, -1), "amax")
    cow = cand & ~((held[last] == refs[last]) & (final[last] == order))
    need = want - have + cow.long()
    before = need.cumsum(0) - need
    free = torch.argsort((refs > 0).to(torch.int8), stable=True)
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    rank = torch.where(j >= have[:, None], before[:, None] + cow.long()[:, None] + j - have[:, None], before[:, None])
    new = ((j >= have[:, None]) & (j < want[:, None])) | ((j == have[:, None] - 1) & cow[:, None])
    got = free[rank.clamp(max=free.shape[0] - 1)]
    to = torch.where(cow, free[before.clamp(max=free.shape[0] - 1)], last)
    refs.index_add_(0, last, cow.to(torch.int32), alpha=-1)
    refs.index_add_(0, torch.where(new, got, 0).view(-1), new.to(torch.int32).view(-1))
    s["k"][:, to] = s["k"][:, last]
    s["v"][:, to] = s["v"][:, last]
    s["pages"][ids] = torch.where(new, got, table).to(torch.int32)
    s["lens"][ids] = (lens + add).to(torch.int32)


def _plain_rows(s):
    c = s["case"]
    ps, Hkv, D = c["page"], c["kv_heads"], c["head_dim"]
    first = s["starts"].long()
    r = torch.arange(s["kv"].shape[0], device=DEV)
    seq = torch.searchsorted(first[1:], r, right=True)
    at = s["pos"].long()[seq] + r - first[seq]
    page = s["pages"][s["ids"].long()[seq], at // ps].long()
    s["k"][s["layer"], page, :, at % ps] = s["kv"][:, : Hkv * D].view(-1, Hkv, D)
    s["v"][s["layer"], page, :, at % ps] = s["kv"][:, Hkv * D:].view(-1, Hkv, D)
    at = torch.arange(s["big"], device=DEV)
    page = s["pages"][s["one"].long(), at // ps].long()
    s["cache_k"][:, : s["big"]] = s["k"][s["layer"], page, :, at % ps].transpose(0, 1)
    s["cache_v"][:, : s["big"]] = s["v"][s["layer"], page, :, at % ps].transpose(0, 1)
    return [s["k"], s["v"], s["cache_k"], s["cache_v"]]


def _plain_compact(s):
    """The k-th used page at or past the number of used pages goes to the k-th free page below it."""
    ps, refs = s["case"]["page"], s["refs"]
    held = refs > 0
    i = torch.arange(refs.shape[0], device=DEV)
    used = held.sum()
    src, dst = (held & (i >= used)).nonzero()[:, 0], (~held & (i < used)).nonzero()[:, 0]
    remap = torch.where(held, i, -1)
    remap[src] = dst
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    j = torch.arange(s["pages"].shape[1], device=DEV)[None, :]
    live = j < ((s["lens"].long() + ps - 1) // ps)[:, None]
    s["pages"].copy_(torch.where(live, remap[s["pages"].long().clamp(min=0)], s["pages"].long()))
    refs[dst] = refs[src]
    refs[src] = 0
    s["remap"].copy_(remap)
    s["used"].copy_(used[None])
    return [s["pages"], refs, s["remap"], s["used"], s["k"], s["v"]]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, op, D = case, case["op"], case["head_dim"]
    row = c["kv_heads"] * D * 2  # bytes of one token's K (or V) in one layer
    if op == "prompt":
        lens = _lengths(c)
        pairs = sum(x * (x + 1) // 2 for x in lens)
        return {"bytes": sum(lens) * (2 * c["q_heads"] * D * 2 + 2 * row), "flops": 4.0 * pairs * c["q_heads"] * D}
    if op == "token":
        lens = _lengths(c)
        return {"bytes": sum(lens) * 2 * row + c["n"] * (2 * c["q_heads"] * D * 2 + 2 * row), "flops": 4.0 * sum(lens) * c["q_heads"] * D}
    ps = c["page"]
    if op == "fork":
        shared = _ceil(c["longest"], ps)
        copies = c["n"] if c["longest"] % ps else 0
        # tables: a child's entry is written by the fork and read by the release; the parent's are read once, the counts read and written
        return {"bytes": copies * c["layers"] * 4.0 * ps * row + 8.0 * c["n"] * shared + 12.0 * shared, "flops": 0}
    if op == "rows":
        lens = _lengths(c)
        return {"bytes": 4.0 * row * (sum(lens) + max(lens)), "flops": 0}
    rows, lens = _compact_plan(c)
    held = set(p for r in rows for p in r)
    moved = sum(p >= len(held) for p in held)
    return {"bytes": moved * c["layers"] * 4.0 * ps * row + 8.0 * sum(len(r) for r in rows) + 12.0 * c["pages"], "flops": 0}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if case["op"] not in ("prompt", "token"):
        return None  # whole numbers and moved values: nothing is computed
    s = prepare(case, seed)
    c, D = case, case["head_dim"]
    Hq, Hkv, x = c["q_heads"], c["kv_heads"], s["qkv"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lens = _lengths(c)
    if c["op"] == "prompt":
        at = 0
        for L in lens:
            for h in range(Hq):
                g = h * Hkv // Hq
                k = x[at:at + L, (Hq + g) * D:(Hq + g + 1) * D]
                v = x[at:at + L, (Hq + Hkv + g) * D:(Hq + Hkv + g + 1) * D]
                for b in range(0, L, 2048):
                    e = min(L, b + 2048)
                    a = x[at + b:at + e, h * D:(h + 1) * D] @ k[:e].T / D ** 0.5
                    a = torch.softmax(a + torch.full((e - b, e), -math.inf, dtype=torch.float64, device=DEV).triu_(b + 1), -1)
                    out[at + b:at + e, h] = a @ v[:e]
            at += L
        return [out]
    ids, table, ps = s["ids"].tolist(), s["pages"].tolist(), c["page"]
    for i, t in enumerate(ids):
        L = lens[t]
        p = torch.tensor(table[t][: _ceil(L, ps)], device=DEV)
        k = s["k"][0][p].double().transpose(1, 2).reshape(-1, Hkv, D)[:L]
        v = s["v"][0][p].double().transpose(1, 2).reshape(-1, Hkv, D)[:L]
        k[L - 1] = x[i, Hq * D:(Hq + Hkv) * D].view(Hkv, D)
        v[L - 1] = x[i, (Hq + Hkv) * D:].view(Hkv, D)
        q = x[i, : Hq * D].view(Hkv, Hq // Hkv, D)
        a = torch.softmax(torch.einsum("hgd,lhd->hgl", q, k) / D ** 0.5, -1)
        out[i] = torch.einsum("hgl,lhd->hgd", a, v).reshape(Hq, D)
    return [out, None, None]
