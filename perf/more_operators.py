"""What is measured of the operators that verify drafted tokens over the 8-bit cache.

A drafter proposes tokens behind each sequence's last one, as a tree: row 0 is
the last token itself, the parent of any other row comes before it.  One step
of the target model runs all rows over the cached prefix, and the drafts are
tested against its probabilities.  Four operators:

  mask    which rows every row sees (its ancestors and itself), and its position;
  attn    the rows attend to the cached keys and to the rows that they see;
  verify  the accepted path and the token behind it, from given random numbers;
  commit  the keys and values of the accepted rows are quantised into the pages.

``run`` computes them in elementary torch operations where ``own`` is false
and through the framework's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
HEADS = ((16, 8), (32, 8), (40, 8), (8, 4), (2, 2))
PAGES = (16, 32, 64, 128)


# ------------------------------------------------------------------- cases
def _case(name, op, n, rows, kids, length=0, Hq=16, Hkv=8, d=128, page=64, **more):
    """n sequences' trees of ``rows`` rows, at most ``kids`` children to a row (1: a chain)."""
    c = dict(name=name, op=op, n=n, rows=rows, kids=kids, len=length, Hq=Hq, Hkv=Hkv, d=d, page=page, ragged=n > 1,
             out="bf16", V=0, draft=False, type="f32")
    c.update(more)
    return c


def listed():
    return [
        # the masks of one step of 32 sequences with trees of 32
        _case("mask trees", "mask", 32, 32, 4, 8192),
        # drafted blocks, chains of 256 tokens behind 64 sequences
        _case("mask chains", "mask", 64, 256, 1, 8192),
        # one sequence that has just begun, a chain of 4 behind it: latency of the smallest step
        _case("attn chain tiny", "attn", 1, 4, 1, 256, 2, 2, 64, 16, out="f32"),
        # a chain of 4 drafted tokens behind the last one, for each of 32 sequences of up to 32768 tokens
        _case("attn chain batch", "attn", 32, 5, 1, 32768, 32, 8, 128, 64),
        # trees of 32 behind 16 sequences
        _case("attn tree 32", "attn", 16, 32, 4, 8192, 16, 8, 128, 32),
        # trees of 64 behind 8 long sequences, 5 query heads to a KV head
        _case("attn tree 64", "attn", 8, 64, 4, 32768, 40, 8, 128, 64),
        # a large tree behind one sequence of 131072 tokens
        _case("attn tree 256", "attn", 1, 256, 8, 131072, 16, 8, 128, 128),
        # one sequence's chain of 8, a small vocabulary: latency of the smallest test
        _case("verify chain tiny", "verify", 1, 8, 1, V=32000, draft=True),
        # drawn trees of 64 sequences, against the probabilities that they were drawn from
        _case("verify drawn trees", "verify", 64, 16, 3, V=131072, draft=True),
        # chosen trees (the likeliest tokens) of 16 sequences, an odd vocabulary, probabilities in bf16
        _case("verify chosen trees", "verify", 16, 64, 4, V=100003, type="bf16"),
        # the accepted rows of 32 sequences in flight: latency of the smallest write
        _case("commit batch", "commit", 32, 16, 3, 2048),
        # long accepted chains of 256 sequences
        _case("commit chains", "commit", 256, 128, 1, 4096, 32, 8, 128, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("mask", "attn", "attn", "attn", "verify", "verify", "commit"))
    Hq, Hkv = rng.choice(HEADS)
    d, page = rng.choice((64, 128)), rng.choice(PAGES)
    kids = rng.choice((1, 2, 3, 4, 8))
    more = dict(ragged=rng.random() < 0.8, out=rng.choice(("bf16", "f32")), type=rng.choice(("bf16", "f32")),
                draft=rng.random() < 0.6)
    if op == "mask":
        n, rows = _log(rng, 1, 64), _log(rng, 1, 256)
        c = _case("", op, n, rows, kids, _log(rng, 1, 8192), **more)
    elif op == "attn":
        n, rows, length = _log(rng, 1, 32), _log(rng, 1, 256), _log(rng, 16, 131072)
        length = max(1, min(length, (32 * 32768 * 1024) // (n * Hkv * d) // 2))
        rows = max(1, min(rows, (16 * 256 * 131072) // (n * Hq * (length + rows))))
        c = _case("", op, n, rows, kids, length, Hq, Hkv, d, page, **more)
    elif op == "verify":
        n, rows, V = _log(rng, 1, 64), _log(rng, 1, 64), _log(rng, 1000, 160000)
        rows = max(1, min(rows, (64 * 16 * 131072) // (n * V)))
        c = _case("", op, n, rows, kids, V=V, **more)
    else:
        n, rows, length = _log(rng, 1, 256), _log(rng, 1, 128), _log(rng, 1, 4096) - 1
        length = min(length, (256 * 4096 * 1024) // (n * Hkv * d))
        c = _case("", op, n, rows, kids, length, Hq, Hkv, d, page, **more)
    del c["name"]
    return c


def _lens(c):
    """Cached tokens of each sequence: the case's length, and with ``ragged`` shorter ones, the last sequence empty."""
    x = [c["len"]] * c["n"]
    if c["ragged"] and c["n"] > 1:
        x = [int(c["len"] * (1.0 if i == 0 else 0.25 + 0.75 * ((0.5 + 0.6180339887 * i) % 1.0))) for i in range(c["n"])]
        if c["n"] >= 4:
            x[-1] = 0
    return x


def _rows(c):
    """Rows of each sequence: the case's, and with ``ragged`` every third sequence's tree smaller; of 8 and more
    sequences the second has ended and has none."""
    x = [max(1, int(c["rows"] * ((0.3 + 0.7548776662 * i) % 1.0))) if c["ragged"] and i % 3 == 2 else c["rows"]
         for i in range(c["n"])]
    if c["ragged"] and c["n"] >= 8:
        x[1] = 0
    return x


def work(c):
    lens, rows = _lens(c), _rows(c)
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    T = sum(rows)
    words = -(-max(rows) // 32)
    if c["op"] == "mask":
        return {"bytes": T * (4 + 4 * words + 4) + 8 * c["n"], "flops": T * words}
    if c["op"] == "attn":
        pages = sum(-(-x // page) for x in lens)
        # own keys: half of them, as of a chain (a tree's rows see fewer)
        seen = sum(r * (x + (r + 1) / 2) for r, x in zip(rows, lens))
        o = 2 if c["out"] == "bf16" else 4
        live = sum(x for x, r in zip(lens, rows) if r)
        return {"bytes": live * Hkv * 2 * d + pages * Hkv * 8 + T * (Hq * (2 * d + o * d + 4) + 4 * Hkv * d + 4 * words),
                "flops": seen * Hq * 4 * d}
    if c["op"] == "verify":
        # the row that the token behind the path is drawn from
        n = sum(r > 0 for r in rows)
        e = (4 if c["type"] == "f32" else 2) * (2 if c["draft"] else 1)
        return {"bytes": n * c["V"] * e + T * 12, "flops": n * c["V"] * 2}
    # accepted rows: half of the deepest path on average
    took = sum(min(r, _depth(c)) + 1 for r in rows if r) / 2
    return {"bytes": took * Hkv * d * 6, "flops": took * Hkv * d * 4}


def _depth(c):
    """Rows on the longest path that a tree of the case is made with."""
    if c["kids"] == 1:
        return c["rows"]
    return max(2, 2 + int(math.log(max(c["rows"], 2)) / math.log(c["kids"]) * 1.5))


# ------------------------------------------------------------------ inputs
def _tree(rng, rows, kids, depth):
    """Parents of a random tree: every row hangs under an earlier one that has room, later ones more often."""
    par, deep, room = [-1], [1], [kids]
    for i in range(1, rows):
        free = [j for j in range(i) if room[j] and deep[j] < depth]
        j = free[int(len(free) * rng.random() ** 0.7)] if free else i - 1
        par.append(j)
        room[j] -= 1
        deep.append(deep[j] + 1)
        room.append(kids)
    return par, max(deep)


def prepare(c, seed):
    """The trees of a step, and what its operator reads."""
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    n, Hq, Hkv, d, page = c["n"], c["Hq"], c["Hkv"], c["d"], c["page"]
    lens, rows = _lens(c), _rows(c)
    T, R = sum(rows), max(rows)
    trees = [_tree(rng, r, c["kids"], _depth(c)) for r in rows if r]
    st = dict(case=dict(c), T=T, max_rows=R, words=-(-R // 32), scale=1.0 / math.sqrt(d),
              width=max(t[1] for t in trees))
    ints = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)
    st["parents"] = ints(np.concatenate([t[0] for t in trees]))
    if c["op"] == "mask":  # (positions count from the cached tokens)
        lens = [int(rng.integers(0, x + 1)) for x in lens]
    st["lens"] = ints(lens)
    st["row_offsets"] = ints(np.concatenate([[0], np.cumsum(rows)]))
    st["row_counts"] = torch.tensor(rows, dtype=torch.int64, device=DEV)
    st["row_seq"] = torch.tensor(np.repeat(np.arange(n), rows), dtype=torch.int64, device=DEV)
    st["row_pos"] = torch.arange(T, device=DEV) - st["row_offsets"].long()[st["row_seq"]]
    if c["op"] == "verify":
        return _prepare_verify(c, st, g, trees)
    room = c["rows"] if c["op"] == "commit" else 0
    max_pages = max(1, max(-(-(x + room) // page) for x in _lens(c)))
    n_pages = n * max_pages + 3
    st["table"] = torch.randperm(n_pages, generator=g, device=DEV)[: n * max_pages].to(torch.int32).reshape(n, max_pages)
    if c["op"] == "mask":
        Hkv, d = 1, 64  # (of the cache, the lengths alone count)
    for x in ("k", "v"):  # pages of unlike amplitude: codes use their upper range, the scale follows
        amp = torch.randint(-1, 2, (n_pages, Hkv), generator=g, device=DEV).float()
        codes = torch.randn((n_pages, Hkv, page, d), generator=g, device=DEV, dtype=torch.float32)
        st[x + "8"] = (codes * 96.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        st[x + "_scale"] = torch.exp2(amp - 7.0)
    rand = lambda H: torch.randn((T, H, d), generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    if c["op"] == "attn":
        st["Q"], st["K"], st["V"] = rand(Hq), rand(Hkv), rand(Hkv)
        st["visible"] = _plain_mask(st)[0]
    elif c["op"] == "commit":
        st["K"], st["V"] = rand(Hkv), rand(Hkv)
        # a path from row 0 down a chain of each tree's children, cut where the drafts stopped being accepted
        path, took = np.full((n, st["width"]), -1), np.zeros(n, np.int64)
        it = iter(trees)
        for s in range(n):
            if not rows[s]:
                continue
            par = np.asarray(next(it)[0])
            way = [0]
            while len(way) < st["width"] and (par == way[-1]).any():
                way.append(int(rng.choice(np.flatnonzero(par == way[-1]))))
            way = way[: int(rng.integers(1, len(way) + 1))]
            path[s, : len(way)], took[s] = way, len(way)
        st["path"], st["accepted"] = ints(path), ints(took)
        hit = [(s, j) for s in range(n) if took[s]
               for j in range(lens[s] // page, -(-(lens[s] + int(took[s])) // page))]
        st["hit_seq"] = torch.tensor([h[0] for h in hit], dtype=torch.int64, device=DEV)
        st["hit_page"] = torch.tensor([h[1] for h in hit], dtype=torch.int64, device=DEV)
        st["lens_out"] = torch.zeros(n, dtype=torch.int32, device=DEV)
    return st


def _prepare_verify(c, st, g, trees):
    """Probabilities of a target and of a drafter that is near it, and tokens drawn from the drafter or, without its
    probabilities, its likeliest ones."""
    T, V = st["T"], c["V"]
    dt = torch.float32 if c["type"] == "f32" else torch.bfloat16
    off = st["row_offsets"].long()[st["row_seq"]]
    parent = torch.where(st["parents"] >= 0, off + st["parents"], -1)
    order = np.concatenate([_ranks(t[0]) for t in trees])  # which child of its parent a row is
    st["kids"] = int(order.max()) + 1
    z = torch.randn((T, V), generator=g, device=DEV) * 3.0
    st["target"] = torch.softmax(z, 1).to(dt)
    z += torch.randn((T, V), generator=g, device=DEV) * 0.6
    q = torch.softmax(z, 1).to(dt)
    del z
    if c["draft"]:
        picks = torch.cat([torch.multinomial(part.float(), st["kids"], replacement=True, generator=g)
                           for part in q.split(256)])
        st["draft"] = q
    else:
        picks = torch.topk(q.float(), min(st["kids"], V), dim=1).indices
        st["draft"] = None
    rank = torch.tensor(order, dtype=torch.int64, device=DEV)
    tokens = picks[parent.clamp(min=0), rank.clamp(max=picks.shape[1] - 1)]
    st["tokens"] = torch.where(parent >= 0, tokens, 0).to(torch.int32)
    st["uniforms"] = torch.rand(T, generator=g, device=DEV)
    st["sample"] = torch.rand(c["n"], generator=g, device=DEV)
    return st


def _ranks(parents):
    seen, out = {}, []
    for p in parents:
        out.append(seen.get(p, 0))
        seen[p] = out[-1] + 1
    return np.asarray(out)


# ------------------------------------------------------------- plain forms
def _plain_mask(st):
    """Every row's ancestors and itself as bits, and its position behind the cached tokens."""
    n, R, T = st["case"]["n"], st["max_rows"], st["T"]
    seq, pos = st["row_seq"], st["row_pos"]
    sees = torch.zeros((T, st["words"] * 32), dtype=torch.int64, device=DEV)
    row = torch.arange(T, device=DEV)
    off = st["row_offsets"].long()[seq]
    at, depth = pos.clone(), torch.full((T,), -1, dtype=torch.int64, device=DEV)
    for _ in range(st["width"]):
        live = at >= 0
        sees[row, at.clamp(min=0)] |= live.long()
        depth += live
        at = torch.where(live, st["parents"].long()[(off + at).clamp(min=0)], -1)
    bit = torch.ones(32, dtype=torch.int64, device=DEV) << torch.arange(32, device=DEV)
    words = (sees.reshape(T, st["words"], 32) * bit).sum(2)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32), (st["lens"][seq] + depth).to(torch.int32)


def _pages(codes, scale, table):
    """[n, Hkv, tokens, d] fp32 values of the pages of a table."""
    t = table.long()
    x = codes.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * scale[t][..., None, None]
    n, P, H, page, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, H, P * page, d)


def _padded(x, st):
    """Packed rows [T, ...] as [n, max_rows, ...] (rows behind a sequence's last: others')."""
    at = st["row_offsets"][:-1, None].long() + torch.arange(st["max_rows"], device=DEV)
    return x[at.clamp_(max=st["T"] - 1)]


def _plain_attn(st):
    c = st["case"]
    n, Hq, Hkv, d, R = c["n"], c["Hq"], c["Hkv"], c["d"], st["max_rows"]
    rows = lambda x: _padded(x, st).float().transpose(1, 2)
    bit = torch.arange(st["words"] * 32, device=DEV)
    sees = ((st["visible"][:, bit // 32] >> (bit % 32)) & 1).bool()[:, :R]
    sees = _padded(sees, st) & (torch.arange(R, device=DEV) < st["row_counts"][:, None])[:, None, :]
    sees = sees.repeat(1, Hq // Hkv, 1)[:, None]  # rows of a KV head: by query head, then by row
    q = rows(st["Q"]).reshape(n, Hkv, -1, d) * st["scale"]
    s = q @ _pages(st["k8"], st["k_scale"], st["table"]).transpose(2, 3)
    cached = torch.arange(s.shape[3], device=DEV) < st["lens"][:, None]
    s.masked_fill_(~cached[:, None, None, :], -math.inf)
    mine = (q @ rows(st["K"]).transpose(2, 3)).masked_fill_(~sees, -math.inf)
    m = torch.maximum(s.amax(3, keepdim=True), mine.amax(3, keepdim=True))
    m = m.masked_fill(m == -math.inf, 0.0)
    p, own_p = s.sub_(m).exp_(), (mine - m).exp_()
    total = p.sum(3, keepdim=True) + own_p.sum(3, keepdim=True)
    o = p @ _pages(st["v8"], st["v_scale"], st["table"]) + own_p @ rows(st["V"])
    o = torch.where(total > 0, o / total, 0.0).reshape(n, Hq, R, d)
    lse = (m + total.log()).reshape(n, Hq, R)
    at = (st["row_seq"], slice(None), st["row_pos"])
    return o[at].to(torch.bfloat16 if c["out"] == "bf16" else torch.float32), lse[at].t().contiguous()


def _plain_verify(st):
    """All sequences a row at a time, in 64 bits: tests and the token behind the path stand next to borders."""
    c = st["case"]
    n, V, R, W = c["n"], c["V"], st["max_rows"], st["width"]
    have = torch.arange(R, device=DEV) < st["row_counts"][:, None]
    par = _padded(st["parents"], st).long().masked_fill(~have, -2)
    tok, u = _padded(st["tokens"], st).long(), _padded(st["uniforms"], st).double()
    off = st["row_offsets"][:-1].long().clamp(max=st["T"] - 1)
    seq = torch.arange(n, device=DEV)
    cur = torch.zeros(n, dtype=torch.int64, device=DEV)
    going = st["row_counts"] > 0
    path = torch.full((n, W), -1, dtype=torch.int64, device=DEV)
    path[:, 0] = torch.where(going, 0, -1)
    took = going.long()
    one = torch.ones(n, dtype=torch.float64, device=DEV)
    rest = torch.zeros((n, V), dtype=torch.float64, device=DEV)
    for step in range(W):
        p = st["target"][off + cur].double()
        q = st["draft"][off + cur].double() if c["draft"] else None
        r, z, w = p.clone(), one.clone(), torch.zeros_like(one)
        last, nxt = torch.full_like(cur, -1), torch.full_like(cur, -1)
        for _ in range(st["kids"] if step < W - 1 else 0):
            # the next child of cur behind the last one tested
            kid = (par == cur[:, None]) & (torch.arange(R, device=DEV) > last[:, None])
            j = torch.where(kid, torch.arange(R, device=DEV), R).amin(1)
            test = going & (j < R) & (nxt < 0)
            jj = j.clamp(max=R - 1)
            x = tok[seq, jj]
            left = r[seq, x]
            if c["draft"]:
                ok = test & (u[seq, jj] * q[seq, x] * z < left)
                lost = test & ~ok
                w = torch.where(lost, w + z, w)
                r = torch.where(lost[:, None], (p - w[:, None] * q).clamp_(min=0.0), r)
                z = torch.where(lost, r.sum(1), z)
            else:
                ok = test & (u[seq, jj] * z < left)
                lost = test & ~ok
                z = torch.where(lost, z - left, z)
                r[seq, x] = torch.where(lost, 0.0, left)
            nxt = torch.where(ok, jj, nxt)
            last = torch.where(test, jj, last)
        ends = going & (nxt < 0)
        rest = torch.where(ends[:, None], r, rest)
        going = going & (nxt >= 0)
        cur = torch.where(going, nxt, cur)
        if step < W - 1:
            path[:, step + 1] = torch.where(going, nxt, -1)
        took = took + going
    cdf = rest.cumsum(1)
    token = (cdf <= st["sample"].double()[:, None] * cdf[:, -1:]).sum(1)
    token = torch.where(st["row_counts"] > 0, token.clamp(max=V - 1), -1)
    return {"path": path.to(torch.int32), "accepted": took.to(torch.int32), "token": token.to(torch.int32)}


def _pow2_scale(amax):
    """The smallest power of two, at least 2^-64, that holds amax within e4m3's largest value, 448."""
    m, e = torch.frexp(amax)
    return torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875)).clamp(min=-64))


def _plain_commit(st):
    c = st["case"]
    seq, pg, page = st["hit_seq"], st["hit_page"], c["page"]
    pid = st["table"][seq, pg].long()
    rel = pg[:, None] * page + torch.arange(page, device=DEV) - st["lens"][seq, None]
    new, old = (rel >= 0) & (rel < st["accepted"][seq, None]), rel < 0
    row = st["path"][seq[:, None], rel.clamp(0, st["width"] - 1).long()].clamp(min=0)
    src = (st["row_offsets"][seq, None] + row).clamp_(0, st["T"] - 1).long()
    new, old = new[:, None, :, None], old[:, None, :, None]
    for x, name in ((st["K"], "k"), (st["V"], "v")):
        was = st[name + "8"].view(torch.uint8)[pid]
        s_was = st[name + "_scale"][pid][..., None, None]
        x = x[src].float().transpose(1, 2)
        s = _pow2_scale((x * new).abs().amax((2, 3), keepdim=True))
        s = torch.where(old.any(2, keepdim=True), torch.maximum(s, s_was), s)
        x = torch.where(new, x, was.view(torch.float8_e4m3fn).float() * s_was) / s
        code = torch.where(new | old, x.to(torch.float8_e4m3fn).view(torch.uint8), was)
        st[name + "8"].view(torch.uint8)[pid] = code
        st[name + "_scale"][pid] = s[..., 0, 0]
    st["lens_out"].copy_(st["lens"] + st["accepted"])
    return {x: st[x] for x in ("k8", "v8", "k_scale", "v_scale", "lens_out")}


PLAIN = {"mask": _plain_mask, "attn": _plain_attn, "verify": _plain_verify, "commit": _plain_commit}


# --------------------------------------------------- the framework's calls
def _handle(st):
    """The cache handle and the workspace that a program makes once and keeps."""
    import structured_mask_attention_gb300 as m
    c = st["case"]
    if c["op"] == "verify":
        st["ws"] = m.bdlm_verify_workspace(c["n"], st["max_rows"], c["V"], DEV)
    else:
        st["cache"] = m.BdlmCache(st["k8"], st["v8"], st["k_scale"], st["v_scale"], st["table"], st["lens"])
        st["ws"] = m.bdlm_cache_workspace(st["cache"], c["Hq"] if c["op"] == "attn" else 0, max(1, st["max_rows"]))
    st["m"] = m
    return m


def _own(st):
    m = st.get("m") or _handle(st)
    c, ws, off, R = st["case"], st["ws"], st["row_offsets"], st["max_rows"]
    if c["op"] == "mask":
        return m.bdlm_tree_mask(st["cache"], st["parents"], off, R, workspace=ws)
    if c["op"] == "attn":
        return m.bdlm_attn_tree(st["Q"], st["K"], st["V"], st["visible"], st["cache"], off, R, scale=st["scale"],
                                o_dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, workspace=ws)
    if c["op"] == "verify":
        path, accepted, token = m.bdlm_tree_verify(st["parents"], st["tokens"], st["target"], st["draft"],
                                                   st["uniforms"], st["sample"], off, R, max_path=st["width"],
                                                   workspace=ws)
        return {"path": path, "accepted": accepted, "token": token}
    m.bdlm_cache_commit(st["cache"], st["K"], st["V"], st["path"], st["accepted"], off, R, lens_out=st["lens_out"],
                        workspace=ws)
    return {x: st[x] for x in ("k8", "v8", "k_scale", "v_scale", "lens_out")}


def run(st):
    if own:
        return _own(st)
    return PLAIN[st["case"]["op"]](st)


# ------------------------------------------------------------------- exact
def _e4m3_table():
    """The 256 values of the e4m3 codes, from the format: sign, 4 exponent bits of bias 7, 3 mantissa bits."""
    v = []
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        x = f / 8.0 * 2.0 ** -6 if e == 0 else (1 + f / 8.0) * 2.0 ** (e - 7)
        v.append(math.nan if b & 127 == 127 else -x if b & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _nearest(x, scale):
    """x in units of scale, rounded to the nearest e4m3 value, ties to the even code, in 64 bits."""
    x = x / scale
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign(torch.round(a / step) * step, x)


def _scale64(amax):
    k = math.ceil(math.log2(amax / 448.0)) if amax > 0 else -64
    while 448.0 * 2.0 ** (k - 1) >= amax and k > -64:
        k -= 1
    return 2.0 ** max(k, -64)


def exact(c, seed):
    if c["op"] in ("mask", "verify"):  # whole numbers alone
        return None
    st = prepare(c, seed)
    lens, rows = _lens(c), _rows(c)
    off = np.concatenate([[0], np.cumsum(rows)]).tolist()
    val, page, Hkv, d = _e4m3_table(), c["page"], c["Hkv"], c["d"]
    table = st["table"].cpu().tolist()
    code = {x: st[x + "8"].view(torch.uint8) for x in ("k", "v")}
    scale = {x: st[x + "_scale"].double() for x in ("k", "v")}
    if c["op"] == "attn":
        T, Hq = st["T"], c["Hq"]
        g = Hq // Hkv
        o = torch.zeros((T, Hq, d), dtype=torch.float64, device=DEV)
        lse = torch.full((Hq, T), -math.inf, dtype=torch.float64, device=DEV)
        parents = st["parents"].cpu().tolist()
        for s in range(c["n"]):
            a, b = off[s], off[s + 1]
            if a == b:
                continue
            sees = np.zeros((b - a, b - a), bool)  # a row sees what its parent sees, and itself
            for i in range(b - a):
                if parents[a + i] >= 0:
                    sees[i] = sees[parents[a + i]]
                sees[i, i] = True
            hide = torch.cat([torch.zeros((b - a, lens[s]), dtype=torch.bool, device=DEV),
                              torch.from_numpy(~sees).to(DEV)], 1)
            ids = torch.tensor(table[s][: -(-lens[s] // page)], dtype=torch.int64, device=DEV)
            for h in range(Hkv):
                k, v = ((val[code[x][ids, h].long()] * scale[x][ids, h][:, None, None]).reshape(-1, d)[: lens[s]]
                        for x in ("k", "v"))
                k, v = torch.cat([k, st["K"][a:b, h].double()]), torch.cat([v, st["V"][a:b, h].double()])
                for x in range(h * g, (h + 1) * g):
                    z = (st["Q"][a:b, x].double() @ k.t() * st["scale"]).masked_fill(hide, -math.inf)
                    lse[x, a:b] = torch.logsumexp(z, 1)
                    o[a:b, x] = torch.softmax(z, 1) @ v
        return o, lse
    out = {x + "_scale": scale[x].clone() for x in ("k", "v")}
    num = {x: val[code[x].long()] for x in ("k", "v")}
    hit = list(zip(st["hit_seq"].tolist(), st["hit_page"].tolist()))
    path, took = st["path"].cpu().tolist(), st["accepted"].cpu().tolist()
    if len(hit) * Hkv > 8192:  # too many blocks for one at a time
        return None
    new = {"k": st["K"].double(), "v": st["V"].double()}
    for x in ("k", "v"):
        for s, j in hit:
            pid, first = table[s][j], max(lens[s], j * page)
            last = min(lens[s] + took[s], (j + 1) * page)
            part = new[x][[off[s] + r for r in path[s][first - lens[s]: last - lens[s]]]]
            big = part.abs().amax((0, 2)).tolist()
            for h in range(Hkv):
                sc, a = _scale64(big[h]), first - j * page
                if a > 0:
                    sc = max(sc, scale[x][pid, h].item())
                    num[x][pid, h, :a] = _nearest(num[x][pid, h, :a] * scale[x][pid, h], sc)
                num[x][pid, h, a: last - j * page] = _nearest(part[:, h], sc)
                out[x + "_scale"][pid, h] = sc
    return {"k8": num["k"], "v8": num["v"], **out, "lens_out": None}
