"""Workloads of the speculative and beam decode operators: attention for a tree of drafted tokens
over a compressed cache, and the pages of the exact tokens behind it (commit, fork, compact).

Every case has a plain form (elementary torch operations in 32 bits, rounded once at the end), the
call a program makes of the library, and an oracle in 64 bits.  Inputs are made from a seed: the
compressed layouts are drawn in the library's byte layout, with the anchor, coefficient and residual
statistics of long prompts, the pools with pages scattered as after long use.
"""
import functools
import math

import torch

own = False

D = 128          # head size of the codec
TILE = 128       # tokens of one word group of the residual bitmap
HEADER = 16      # leading int32 of a page state
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    tree = dict(op="tree", dtype="bf16", theta=0.05, page=64, batch=1, layouts=1)
    page = dict(dtype="bf16", layers=32, heads=8)
    return [
        # the smallest call: the fp32 reference shape with a handful of drafts, where latency counts
        dict(tree, name="tree fp32 n1024", tokens=1024, kv=1, q=4, theta=0.1, drafts=5, tail=37, page=16, dtype="fp32"),
        # ordinary decoding: one token of one sequence behind a 32k prompt
        dict(tree, name="tree 32k one token", tokens=32768, kv=8, q=32, drafts=1, tail=100),
        # a small drafted tree, the common size of speculative decoding
        dict(tree, name="tree 32k 16 drafts", tokens=32768, kv=8, q=32, drafts=16, tail=333),
        # the widest tree
        dict(tree, name="tree 32k 64 drafts", tokens=32768, kv=8, q=32, drafts=64, tail=1000),
        # a batch of sequences of unequal tails and unequal trees
        dict(tree, name="tree 32k batch 16", tokens=32768, kv=8, q=32, theta=0.1, drafts=8, tail=700, batch=16, layouts=16),
        # the longest prompt, eight query heads for each KV head
        dict(tree, name="tree 128k 24 drafts", tokens=131072, kv=8, q=64, drafts=24, tail=517),
        # one decoded token of one sequence, all layers
        dict(page, op="commit", name="commit one token", slots=1, drafts=1, tail=300, page=64),
        # verified paths of a batch
        dict(page, op="commit", name="commit 16 paths", slots=16, drafts=16, tail=301, page=64),
        # four beams of one prompt
        dict(page, op="fork", name="fork 4 beams", slots=4, beams=4, tail=203, page=64),
        # sixteen prompts of four beams
        dict(page, op="fork", name="fork 16x4 beams", slots=64, beams=4, tail=150, page=32),
        # a small pool of one layer group
        dict(page, op="compact", name="compact 24 pages", layers=4, pages=24, live=11, slots=4, page=16),
        # a pool that served many sequences, half of it free
        dict(page, op="compact", name="compact 160 pages", pages=160, live=83, slots=16, page=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "tree", "commit", "fork", "compact"))
    if op == "tree":
        kv, q = rng.choice(((1, 4), (2, 8), (2, 2), (3, 6), (8, 32), (8, 64), (4, 64)))
        dtype = "fp32" if rng.random() < 0.2 else "bf16"
        batch = _log(rng, 1, 16)
        c = dict(op=op, dtype=dtype, theta=round(rng.uniform(0.05, 0.4), 3), page=rng.choice((16, 32, 64, 128)),
                 batch=batch, layouts=rng.choice((1, batch)), kv=kv, q=q, drafts=_log(rng, 1, 64),
                 tail=_log(rng, 1, 1500), tokens=_log(rng, 40, 8192 if dtype == "fp32" else 131072))
        c["tokens"] = min(c["tokens"], (1 << 22) // (batch * kv))
        c["drafts"] = max(1, min(c["drafts"], (1 << 27) // (batch * c["tokens"] * q)))
        return c
    c = dict(op=op, dtype="bf16", layers=rng.choice((1, 2, 5, 16, 32)), heads=rng.choice((1, 2, 8)),
             page=rng.choice((16, 32, 64, 128)))
    room = 3 * 10**8 // (c["layers"] * c["heads"] * c["page"] * D * 2)      # pages of about 300 MB a side
    if op == "commit":
        c.update(slots=_log(rng, 1, 64), drafts=_log(rng, 1, 64), tail=_log(rng, 1, 900))
        while c["slots"] > 1 and c["slots"] * (2 + (c["tail"] + c["drafts"]) // c["page"]) > room:
            c["slots"] = (c["slots"] + 1) // 2
    elif op == "fork":
        beams = rng.choice((2, 3, 4, 8))
        c.update(beams=beams, slots=beams * _log(rng, 1, 16), tail=_log(rng, 1, 400))
        while c["slots"] > beams and c["slots"] * (2 + c["tail"] // c["page"]) > room:
            c["slots"] = max(beams, c["slots"] // beams // 2 * beams)
    else:
        c.update(pages=_log(rng, 8, max(9, min(400, room))), slots=_log(rng, 1, 32))
        c["live"] = max(1, int(c["pages"] * rng.uniform(0.2, 0.9)))
    return c


# ---------------------------------------------------------------- the codec's layout, by its published rules

def _layout(c):
    """Sections of one compressed layer: byte offsets, anchors k, residual records R."""
    n, h, e = c["tokens"], c["kv"], 4 if c["dtype"] == "fp32" else 2
    m = -(-n // 128)
    k = n if n - 32 <= m else 32 + m
    nt = -(-n // TILE)
    off, cur = {}, 0
    for name, size in (("ak", h * k * D * e), ("av", h * k * D * e), ("pos", 4 * h * k), ("tok", 8 * h * n),
                       ("bits", 32 * h * nt), ("prefix", 8 * h * (nt + 1))):
        off[name] = cur
        cur = (cur + size + 15) // 16 * 16
    budget = math.floor(c["theta"] * float(2 * h * n * D * e))
    r = min(2 * h * (n - k), max(0, (budget - cur) // 34))
    off["codes"], off["sigma"] = cur, cur + 32 * r
    return dict(off=off, k=k, r=r, nt=nt, total=cur + 34 * r, stride=(cur + 34 * r + 15) // 16 * 16)


@functools.cache
def _levels():
    """Outer and inner level of the four-level Lloyd-Max quantizer of N(0, 1), by Lloyd's iteration."""
    a, b = 0.4, 1.6
    density = lambda x: math.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)  # noqa: E731
    above = lambda x: 0.5 * math.erfc(x / math.sqrt(2))                  # noqa: E731
    for _ in range(2000):
        t = 0.5 * (a + b)
        a, b = (density(0.0) - density(t)) / (0.5 - above(t)), density(t) / above(t)
    return a, b


@functools.cache
def _signs(device):
    """The shared +-1 signs of the randomized rotation for seed 0 (SplitMix64 of 2^63 ^ j)."""
    out, m = [], (1 << 64) - 1
    for j in range(D):
        z = ((1 << 63) ^ j) + 0x9E3779B97F4A7C15 & m
        z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9 & m
        z = (z ^ (z >> 27)) * 0x94D049BB133111EB & m
        out.append(-1.0 if (z ^ (z >> 31)) & 1 else 1.0)
    return torch.tensor(out, dtype=torch.float64, device=device)


@functools.cache
def _rotation(device):
    """Rows of the orthonormal Hadamard matrix with the signs on its columns: r = z @ rotation."""
    i = torch.arange(D, device=device)
    x = i[:, None] & i[None, :]
    x = x ^ (x >> 4)
    x = x ^ (x >> 2)
    x = (x ^ (x >> 1)) & 1
    return ((1 - 2 * x).double() / math.sqrt(D)) * _signs(device)


def _bytes(t):
    return t.contiguous().view(torch.uint8).reshape(t.shape[0], -1)


def _make_layouts(c, g, dev):
    """`layouts` compressed layers, [layouts, stride] bytes."""
    lay, b, n, h, k, r = _layout(c), c["layouts"], c["tokens"], c["kv"], _layout(c)["k"], _layout(c)["r"]
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)           # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=g, device=dev)             # noqa: E731
    buf = torch.zeros(b, lay["stride"], dtype=torch.uint8, device=dev)
    size = torch.exp(0.5 * rand(2, b, h, k, 1))
    anchors = (rand(2, b, h, k, D) * size).to(_DT[c["dtype"]])           # unequal norms, as keys have
    pos = torch.argsort(uni(b, h, n), dim=-1)[..., :k].sort(dim=-1).values
    slot = torch.randint(0, k, (b, 2, h, n), generator=g, device=dev)
    gamma = (0.45 + 0.25 * rand(b, 2, h, n)).half()
    at = pos[:, None].expand(b, 2, h, k)
    slot.scatter_(3, at, torch.arange(k, device=dev).expand(b, 2, h, k))
    gamma.scatter_(3, at, torch.ones(b, 2, h, k, dtype=torch.float16, device=dev))
    tok = (slot | (gamma.view(torch.int16).long() & 0xFFFF) << 16)
    tok = torch.where(tok >= 1 << 31, tok - (1 << 32), tok).int()
    sel = torch.zeros(b, 2, h, lay["nt"] * TILE, dtype=torch.bool, device=dev)
    if r:
        key = uni(b, 2, h, n).scatter_(3, at, 2.0).reshape(b, -1)        # the anchors never carry a residual
        chosen = torch.zeros(b, 2 * h * n, dtype=torch.bool, device=dev)
        chosen.scatter_(1, key.argsort(dim=1)[:, :r], True)
        sel[..., :n] = chosen.reshape(b, 2, h, n)
    words = (sel.reshape(b, 2, h, lay["nt"], 4, 32).long() << torch.arange(32, device=dev)).sum(-1)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).int()
    count = sel.reshape(b, 2 * h, lay["nt"], TILE).sum(-1).reshape(b, -1).cumsum(1).reshape(b, 2 * h, lay["nt"])
    start = torch.cat([torch.zeros(b, 1, dtype=torch.long, device=dev), count[:, :-1, -1]], 1)
    prefix = torch.cat([start[..., None], count], 2).int()
    o = lay["off"]
    for name, t in (("ak", anchors[0]), ("av", anchors[1]), ("pos", pos.int()), ("tok", tok), ("bits", words), ("prefix", prefix)):
        t = _bytes(t)
        buf[:, o[name]:o[name] + t.shape[1]] = t
    if r:
        buf[:, o["codes"]:o["codes"] + 32 * r] = torch.randint(0, 256, (b, 32 * r), generator=g, device=dev, dtype=torch.uint8)
        buf[:, o["sigma"]:o["sigma"] + 2 * r] = _bytes((0.6 * torch.exp(0.4 * rand(b, r))).half())
    return buf


# ---------------------------------------------------------------- inputs

def _gen(case, seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1_000_003 + 17)
    return g


def _tails(c, slots):
    """Committed tail tokens of each slot: unequal, at least one."""
    return [max(1, c["tail"] - (29 * b) % (c["tail"] // 2 + 1)) for b in range(slots)]


def _counts(c, slots):
    """Drafted (or accepted) tokens of each slot: unequal beyond the first."""
    return [max(1, c["drafts"] - (3 * b) % (c["drafts"] // 2 + 1)) for b in range(slots)]


def _state(dev, n_pages, free, refs, lens, table):
    """The int32 page state: header (status, free pages), free list, references, lengths, page table."""
    head = torch.zeros(HEADER, dtype=torch.int32)
    head[1] = len(free)
    rest = torch.tensor(list(free) + [-1] * (n_pages - len(free)), dtype=torch.int32)
    return torch.cat([head, rest, torch.tensor(refs, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32),
                      torch.tensor(table, dtype=torch.int32).reshape(-1)]).to(dev)


def _scatter_pages(rng, n_pages, lens, page, most, groups=None):
    """Pages of each slot in scattered order; slots of one group share their full pages."""
    ids = torch.randperm(n_pages, generator=rng).tolist()
    refs, table = [0] * n_pages, []
    for b, n in enumerate(lens):
        first = (b // groups) * groups if groups else b
        row = []
        for j in range(-(-n // page)):
            if b != first and (j + 1) * page <= min(n, lens[first]):
                row.append(table[first][j])
            else:
                row.append(ids.pop())
            refs[row[-1]] += 1
        table.append(row + [-1] * (most - len(row)))
    return table, refs, ids


def _ancestors(rng, batch, drafts):
    """Bit j of word t: draft j is t itself or one of its ancestors, in a random tree for each sequence."""
    out = []
    for _ in range(batch):
        words = []
        for t in range(drafts):
            p = int(torch.randint(max(-1, t - 5), t, (1,), generator=rng)) if t else -1
            words.append((words[p] if p >= 0 else 0) | 1 << t)
        out.append([w - (1 << 64) if w >= 1 << 63 else w for w in words])
    return torch.tensor(out, dtype=torch.int64)


def prepare(case, seed):
    dev = torch.device("cuda")
    c, g = dict(case), _gen(case, seed, "cuda")
    rng = torch.Generator().manual_seed(seed + 5)
    dt = _DT[c["dtype"]]
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)           # noqa: E731
    s = dict(case=c)
    if c["op"] == "tree":
        b, t, h, q = c["batch"], c["drafts"], c["kv"], c["q"]
        lens = _tails(c, b)
        most = -(-c["tail"] // c["page"])
        n_pages = sum(-(-n // c["page"]) for n in lens) + 3
        table, refs, free = _scatter_pages(rng, n_pages, lens, c["page"], most)
        s["spec"] = dict(n_pages=n_pages, page_size=c["page"], n_slots=b, max_pages=most, n_layers=1, n_kv_heads=h, dtype=c["dtype"])
        s["state"] = _state(dev, n_pages, free, refs, lens, table)
        s["layouts"] = _make_layouts(c, g, dev)
        s["layout_of"] = torch.tensor([i % c["layouts"] for i in range(b)], dtype=torch.int32, device=dev)
        s["K"], s["V"] = (rand(n_pages, h, c["page"], D).to(dt) for _ in range(2))
        s["q"] = (2.0 * rand(b, t, q, D)).to(dt)
        s["K_new"], s["V_new"] = (rand(b, t, h, D).to(dt) for _ in range(2))
        s["mask"] = _ancestors(rng, b, t).to(dev)
        s["n_new"] = torch.tensor(_counts(c, b), dtype=torch.int32, device=dev)
        s["out"] = torch.zeros(b, t, q, D, dtype=dt, device=dev)
        return s
    n_layers, h, page, slots = c["layers"], c["heads"], c["page"], c["slots"]
    if c["op"] == "compact":
        n_pages, most = c["pages"], c["live"]
        cut = sorted(torch.randint(0, c["live"] + 1, (slots - 1,), generator=rng).tolist())
        sizes = [y - x for x, y in zip([0] + cut, cut + [c["live"]])]
        lens = [max(0, n * page - (7 * b) % page) if n else 0 for b, n in enumerate(sizes)]
        table, refs, free = _scatter_pages(rng, n_pages, lens, page, most)
    else:
        lens = _tails(c, slots)
        extra = c.get("drafts", 0)
        most = -(-(c["tail"] + extra) // page) + 1
        n_pages = sum(-(-(n + extra) // page) for n in lens) + slots + 2
        table, refs, free = _scatter_pages(rng, n_pages, lens, page, most, c.get("beams"))
    s["spec"] = dict(n_pages=n_pages, page_size=page, n_slots=slots, max_pages=most, n_layers=n_layers, n_kv_heads=h, dtype=c["dtype"])
    s["state"] = _state(dev, n_pages, free, refs, lens, table)
    s["state_out"] = s["state"].clone()
    s["K"], s["V"] = (torch.randn(n_layers, n_pages, h, page, D, generator=g, device=dev, dtype=dt) for _ in range(2))
    if c["op"] == "commit":
        t = c["drafts"]
        s["K_new"], s["V_new"] = (torch.randn(n_layers, slots, t, h, D, generator=g, device=dev, dtype=dt) for _ in range(2))
        s["n_accept"] = torch.tensor(_counts(c, slots), dtype=torch.int32, device=dev)
        # accepted nodes of the tree, in ascending order
        s["path"] = torch.stack([torch.randperm(t, generator=rng) for _ in range(slots)])
        for b, n in enumerate(_counts(c, slots)):
            s["path"][b, :n] = s["path"][b, :n].sort().values
        s["path"] = s["path"].int().to(dev)
    elif c["op"] == "fork":
        base = torch.arange(slots) // c["beams"] * c["beams"]
        parents = base + torch.randint(0, c["beams"], (slots,), generator=rng)
        parents[torch.rand(slots, generator=rng) < 0.06] = -1            # finished beams
        s["parents"] = parents.int().to(dev)
    return s


# ---------------------------------------------------------------- plain forms

def _view(s):
    """Parts of a page state."""
    x, st = s["spec"], s["state"]
    n, b = x["n_pages"], x["n_slots"]
    free, refs, lens = st[HEADER:HEADER + n].long(), st[HEADER + n:HEADER + 2 * n].long(), st[HEADER + 2 * n:HEADER + 2 * n + b].long()
    return st[1].long(), free, refs, lens, st[HEADER + 2 * n + b:].reshape(b, x["max_pages"]).long()


def _pack(n_free, free, refs, lens, table):
    n = torch.arange(free.numel(), device=free.device)
    head = torch.zeros(HEADER, dtype=torch.long, device=free.device)
    head[1] = n_free
    return torch.cat([head, torch.where(n < n_free, free, -1), refs, lens, table.reshape(-1)]).int()


def _rebuild(c, buf, side):
    """Dense keys (side 0) or values (side 1) of each layout, [layouts, H, N, D] in 32 bits."""
    lay, b, h, n = _layout(c), buf.shape[0], c["kv"], c["tokens"]
    o, k, r, dev = lay["off"], lay["k"], lay["r"], buf.device
    part = lambda at, size, dt: buf[:, at:at + size].contiguous().view(dt)                # noqa: E731
    e = 4 if c["dtype"] == "fp32" else 2
    anchors = part(o["av" if side else "ak"], h * k * D * e, _DT[c["dtype"]]).reshape(b, h, k, D).float()
    tok = part(o["tok"] + side * 4 * h * n, 4 * h * n, torch.int32).reshape(b, h, n)
    gamma = (tok >> 16).to(torch.int16).view(torch.float16).float()
    slot = (tok & 0xFFFF).long()
    x = torch.gather(anchors, 2, slot[..., None].expand(b, h, n, D)) * gamma[..., None]
    if r == 0:
        return x
    words = part(o["bits"], 32 * h * lay["nt"], torch.int32).reshape(b, 2 * h, lay["nt"] * 4)
    sel = ((words[..., None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1).reshape(b, 2 * h, -1)[..., :n]
    record = (sel.reshape(b, -1).cumsum(1) - 1).reshape(b, 2, h, n)[:, side].clamp(min=0)
    sel = sel.reshape(b, 2, h, n)[:, side].bool()
    codes = part(o["codes"], 32 * r, torch.uint8).reshape(b, r, 32, 1)
    codes = ((codes >> torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=dev)) & 3).reshape(b, r, D).int()
    inner, outer = _levels()
    level = torch.where((codes == 0) | (codes == 3), outer, inner) * (2 * (codes >> 1) - 1)
    level = level.float() * part(o["sigma"], 2 * r, torch.float16).float()[..., None]
    level = level @ _rotation(dev).float()
    res = torch.gather(level, 1, record.reshape(b, -1, 1).expand(b, h * n, D)).reshape(b, h, n, D)
    return x + torch.where(sel[..., None], res, 0.0)


def _tree_plain(s):
    c = s["case"]
    b, t, h, q = c["batch"], c["drafts"], c["kv"], c["q"]
    _, _, _, lens, table = _view(s)
    dev = table.device
    of = s["layout_of"].long()
    pages = table.clamp(min=0)
    tail = lambda pool, new: torch.cat([pool[pages].permute(0, 2, 1, 3, 4).reshape(b, h, -1, D), new.permute(0, 2, 1, 3)], 2).float()  # noqa: E731
    rows = s["q"].reshape(b, t, h, q // h, D).permute(0, 2, 1, 3, 4).reshape(b, h, -1, D).float()
    front = rows @ _rebuild(c, s["layouts"], 0)[of].transpose(2, 3) / math.sqrt(D)
    back = rows @ tail(s["K"], s["K_new"]).transpose(2, 3) / math.sqrt(D)
    m = back.shape[3] - t
    seen = torch.arange(m, device=dev) < lens[:, None]
    j = torch.arange(t, device=dev)
    tree = ((s["mask"][..., None] >> j) & 1).bool() & (j < s["n_new"][:, None])[:, None]
    seen = torch.cat([seen[:, None].expand(b, t, m), tree], 2)[:, None, :, None].expand(b, h, t, q // h, m + t).reshape(back.shape)
    back = torch.where(seen, back, -math.inf)
    top = torch.maximum(front.amax(3), back.amax(3))[..., None]
    front, back = torch.exp(front - top), torch.exp(back - top)
    o = front @ _rebuild(c, s["layouts"], 1)[of] + back @ tail(s["V"], s["V_new"])
    o = o / (front.sum(3) + back.sum(3))[..., None]
    o = o.reshape(b, h, t, q // h, D).permute(0, 2, 1, 3, 4).reshape(b, t, q, D).to(s["out"].dtype)
    return torch.where((j < s["n_new"][:, None])[..., None, None], o, s["out"])


def _commit_plain(s):
    page = s["spec"]["page_size"]
    n_free, free, refs, lens, table = _view(s)
    dev, t, n = free.device, s["path"].shape[1], s["n_accept"].long()
    after = lens + n
    had, has = (lens + page - 1) // page, (after + page - 1) // page
    first = (has - had).cumsum(0) - (has - had)
    col = torch.arange(table.shape[1], device=dev)
    fresh = (col >= had[:, None]) & (col < has[:, None])
    at = n_free - 1 - first[:, None] - (col - had[:, None])
    ids = free[at.clamp(0, free.numel() - 1)]
    table = torch.where(fresh, ids, table)
    refs[ids[fresh]] = 1
    i = torch.arange(t, device=dev)
    b, i = torch.where(i < n[:, None])
    pos = lens[b] + i
    p, r, src = table[b, pos // page], pos % page, s["path"].long()[b, i]
    s["K"][:, p, :, r] = s["K_new"][:, b, src].transpose(0, 1)
    s["V"][:, p, :, r] = s["V_new"][:, b, src].transpose(0, 1)
    return dict(K=s["K"], V=s["V"], state=_pack(n_free - (has - had).sum(), free, refs, after, table))


def _fork_plain(s):
    page, slots = s["spec"]["page_size"], s["spec"]["n_slots"]
    n_free, free, refs, lens, table = _view(s)
    dev, parent = free.device, s["parents"].long()
    col, n = torch.arange(table.shape[1], device=dev), torch.arange(free.numel(), device=dev)
    me = torch.arange(slots, device=dev)
    kept, par = parent >= 0, parent.clamp(min=0)
    length = torch.where(kept, lens[par], 0)
    full, part = length // page, length % page > 0
    keeper = torch.full((slots,), slots, device=dev).scatter_reduce(0, par, torch.where(kept, me, slots), "amin")
    copy = part & (keeper[par] != me)
    rows = table[par]
    mine = (col < full[:, None]) | ((col == full[:, None]) & (part & ~copy)[:, None])
    count = torch.zeros_like(refs).scatter_add(0, rows.clamp(min=0).reshape(-1), mine.reshape(-1).long())
    freed = (refs > 0) & (count == 0)
    free = free.scatter(0, n_free + freed.cumsum(0)[freed] - 1, n[freed])
    n_free = n_free + freed.sum()
    dst = free[(n_free - copy.cumsum(0)).clamp(min=0)]
    src = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    table = torch.where(mine, rows, torch.where((col == full[:, None]) & copy[:, None], dst[:, None], -1))
    count[dst[copy]] = 1
    a, z = src[copy], dst[copy]
    written = (torch.arange(page, device=dev) < (length % page)[copy][:, None])[None, :, None, :, None]
    s["K"][:, z] = torch.where(written, s["K"][:, a], s["K"][:, z])
    s["V"][:, z] = torch.where(written, s["V"][:, a], s["V"][:, z])
    return dict(K=s["K"], V=s["V"], state=_pack(n_free - copy.sum(), free, count, length, table))


def _compact_plain(s):
    _, free, refs, lens, table = _view(s)
    n = torch.arange(free.numel(), device=free.device)
    live = refs > 0
    n_live = live.sum()
    src, dst = n[live & (n >= n_live)], n[~live & (n < n_live)]
    to = n.scatter(0, src, dst)
    s["K"][:, dst] = s["K"][:, src]
    s["V"][:, dst] = s["V"][:, src]
    refs = torch.zeros_like(refs).scatter(0, to[live], refs[live])
    table = torch.where(table >= 0, to[table.clamp(min=0)], -1)
    return dict(K=s["K"], V=s["V"], state=_pack(n.numel() - n_live, n.numel() - 1 - n, refs, lens, table))


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from kv_cache_compression_anchorkv_b200 import api

    c = s["case"]
    if "handle" not in s:                                                # what a program keeps between calls
        spec = api.PageSpec(**s["spec"])
        if c["op"] == "tree":
            p = api.AnchorKVParams(n_tokens=c["tokens"], n_kv_heads=c["kv"], n_q_heads=c["q"], theta=c["theta"], dtype=c["dtype"])
            size = api.tree_workspace_bytes(p, c["batch"], c["drafts"], spec)
        else:
            p, size = None, api.pages_workspace_bytes(spec)
        s["handle"] = spec, p, torch.empty(size, dtype=torch.uint8, device="cuda")
    spec, p, ws = s["handle"]
    if c["op"] == "tree":
        return api.tree_attn(p, s["layouts"], s["q"], s["K_new"], s["V_new"], n_new=s["n_new"], mask=s["mask"], layout_of=s["layout_of"],
                             pages=spec, state=s["state"], K_pages=s["K"], V_pages=s["V"], out=s["out"], workspace=ws)
    to = dict(state_out=s["state_out"], workspace=ws)
    if c["op"] == "commit":
        st = api.pages_commit(spec, s["state"], s["K"], s["V"], s["K_new"], s["V_new"], s["n_accept"], path=s["path"], **to)
    elif c["op"] == "fork":
        st = api.pages_fork(spec, s["state"], s["K"], s["V"], s["parents"], **to)
    else:
        st = api.pages_compact(spec, s["state"], s["K"], s["V"], **to)
    return dict(K=s["K"], V=s["V"], state=st)


def run(state):
    if own:
        return _own(state)
    return {"tree": _tree_plain, "commit": _commit_plain, "fork": _fork_plain, "compact": _compact_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the work that cannot be left out

def work(case):
    c = case
    e = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "tree":
        lens, new = _tails(c, c["batch"]), _counts(c, c["batch"])
        rows = sum(new) * c["q"]
        tail = sum(lens) + sum(new)
        data = c["layouts"] * _layout(c)["total"] + 2 * tail * c["kv"] * D * e + 2 * rows * D * e
        return {"bytes": data, "flops": 4 * D * c["q"] * sum(m * (c["tokens"] + n) + m * (m + 1) // 2 for n, m in zip(lens, new))}
    row = 2 * c["layers"] * c["heads"] * D * e                           # keys and values of one token, all layers
    ints = 4 * (HEADER + 2)
    if c["op"] == "commit":
        return {"bytes": 2 * row * sum(_counts(c, c["slots"])) + ints * c["slots"], "flops": 0}
    if c["op"] == "fork":                                                # about a third of the slots keep their parent's page
        part = [n % c["page"] for n in _tails(c, c["slots"])]
        return {"bytes": 2 * row * sum(part) * 0.36 + ints * c["slots"], "flops": 0}
    moved = c["live"] * (1 - c["live"] / c["pages"])
    return {"bytes": 2 * row * c["page"] * moved + 8 * c["pages"], "flops": 0}


# ---------------------------------------------------------------- oracle, in 64 bits

def _exact_tree(s):
    import numpy as np

    c, lay = s["case"], _layout(s["case"])
    b, t, h, q, n = c["batch"], c["drafts"], c["kv"], c["q"], c["tokens"]
    if b * h * n * (64 + t * q // h) > 1 << 31:
        return None
    dev, o, k, r, e = s["q"].device, lay["off"], lay["k"], lay["r"], 4 if c["dtype"] == "fp32" else 2
    had = torch.ones(1, 1, dtype=torch.float64)
    while had.shape[0] < D:
        had = torch.cat([torch.cat([had, had], 1), torch.cat([had, -had], 1)], 0)
    had = had.to(dev) / math.sqrt(D)
    signs, (inner, outer) = _signs(dev), _levels()
    book = torch.tensor([-outer, -inner, inner, outer], dtype=torch.float64, device=dev)
    st = s["state"].cpu().numpy()
    x = s["spec"]
    lens = st[HEADER + 2 * x["n_pages"]:][:b]
    table = st[HEADER + 2 * x["n_pages"] + b:].reshape(b, -1)
    new, mask = s["n_new"].cpu().tolist(), s["mask"].cpu().tolist()
    out = torch.zeros(b, t, q, D, dtype=torch.float64, device=dev)
    for i in range(b):
        image = s["layouts"][int(s["layout_of"][i])]
        raw = image.cpu().numpy()
        prefix = raw[o["prefix"]:o["prefix"] + 8 * h * (lay["nt"] + 1)].view(np.int32).reshape(2, h, lay["nt"] + 1)
        ids = table[i][:-(-int(lens[i]) // c["page"])].tolist()
        seen = torch.tensor([[bool(mask[i][a] >> d & 1) for d in range(new[i])] for a in range(new[i])], device=dev)
        for j in range(h):
            dense = []
            for side, name in enumerate(("ak", "av")):
                a = image[o[name] + j * k * D * e:][:k * D * e].view(_DT[c["dtype"]]).reshape(k, D).double()
                word = image[o["tok"] + 4 * (side * h + j) * n:][:4 * n].view(torch.int32).long() & 0xFFFFFFFF
                g = np.asarray((word >> 16).cpu(), dtype=np.uint16).view(np.float16).astype(np.float64)
                x_hat = torch.tensor(g, device=dev)[:, None] * a[word & 0xFFFF]
                bits = raw[o["bits"] + 16 * (side * h + j) * lay["nt"]:][:16 * lay["nt"]]
                where = np.flatnonzero(np.unpackbits(bits, bitorder="little")[:n])
                if len(where):
                    r0 = int(prefix[side, j, 0])
                    code = image[o["codes"] + 32 * r0:][:32 * len(where)].reshape(-1, 32).long()
                    code = torch.stack([code >> 2 * u & 3 for u in range(4)], 2).reshape(-1, D)
                    sigma = torch.tensor(raw[o["sigma"] + 2 * r0:][:2 * len(where)].view(np.float16).astype(np.float64), device=dev)
                    x_hat[torch.tensor(where, device=dev)] += (book[code] * sigma[:, None]) @ had.T * signs
                pool, fresh = (s["V"], s["V_new"]) if side else (s["K"], s["K_new"])
                exact_tail = torch.cat([pool[p, j] for p in ids])[:int(lens[i])].double()
                dense.append(torch.cat([x_hat, exact_tail, fresh[i, :new[i], j].double()]))
            rows = s["q"][i, :new[i], j * (q // h):(j + 1) * (q // h)].double()
            z = torch.einsum("tgd,nd->tgn", rows, dense[0]) / math.sqrt(D)
            z[:, :, n + int(lens[i]):].masked_fill_(~seen[:, None], -math.inf)
            out[i, :new[i], j * (q // h):(j + 1) * (q // h)] = torch.softmax(z, 2) @ dense[1]
    return out


def _exact_pages(s):
    """The operations as a program of lists, one sequence after another."""
    c, x, page = s["case"], s["spec"], s["spec"]["page_size"]
    st = s["state"].cpu().tolist()
    n, slots, most = x["n_pages"], x["n_slots"], x["max_pages"]
    free = st[HEADER:HEADER + st[1]]
    refs, lens = st[HEADER + n:HEADER + 2 * n], st[HEADER + 2 * n:HEADER + 2 * n + slots]
    flat = st[HEADER + 2 * n + slots:]
    table = [flat[b * most:b * most + -(-lens[b] // page)] for b in range(slots)]
    pools = [s["K"], s["V"]]
    if c["op"] == "commit":
        path = s["path"].cpu().tolist()
        for b, m in enumerate(s["n_accept"].cpu().tolist()):
            for i in range(m):
                if lens[b] % page == 0:
                    table[b].append(free.pop())
                    refs[table[b][-1]] = 1
                for pool, fresh in zip(pools, (s["K_new"], s["V_new"])):
                    pool[:, table[b][-1], :, lens[b] % page] = fresh[:, b, path[b][i]]
                lens[b] += 1
    elif c["op"] == "fork":
        parents = s["parents"].cpu().tolist()
        old, old_lens, old_refs = table, lens, refs
        lens = [old_lens[p] if p >= 0 else 0 for p in parents]
        table, refs, copies, taken = [], [0] * n, [], set()
        for b, p in enumerate(parents):
            row = list(old[p]) if p >= 0 else []
            if lens[b] % page and p in taken:
                copies.append((b, row.pop()))
            taken.add(p)
            for u in row:
                refs[u] += 1
            table.append(row)
        free += [u for u in range(n) if old_refs[u] and not refs[u]]
        for b, src in copies:
            table[b].append(free.pop())
            refs[table[b][-1]] = 1
            for pool in pools:
                pool[:, table[b][-1], :, :lens[b] % page] = pool[:, src, :, :lens[b] % page].clone()
    else:
        n_live = sum(1 for u in refs if u)
        holes = [u for u in range(n_live) if not refs[u]]
        to = dict(zip([u for u in range(n_live, n) if refs[u]], holes))
        for src, dst in to.items():
            refs[dst], refs[src] = refs[src], 0
            for pool in pools:
                pool[:, dst] = pool[:, src]
        table = [[to.get(u, u) for u in row] for row in table]
        free = list(range(n - 1, n_live - 1, -1))
    table = [row + [-1] * (most - len(row)) for row in table]
    return dict(K=pools[0].double(), V=pools[1].double(), state=_state(s["state"].device, n, free, refs, lens, table))


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_tree(s) if case["op"] == "tree" else _exact_pages(s)
