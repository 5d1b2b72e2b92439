"""Operators of long-context serving on the paged KV cache, as measured workloads.

Five operators, each in a plain form (elementary torch operations) and as the
calls that a user makes of the library:

  tree     attention for a tree of drafted tokens over the cache
  sparse   decode over the pages that a score on the pages' key bounds selects
  append   a cache's growth: pages are reserved and new tokens written
  beam     one step of beam search on the cache: rows forked, old rows freed,
           room for the next token reserved (shared tail pages are copied)
  compact  live pages moved to the front of the pool, tables rewritten

``own`` False: run() computes the plain form.  ``own`` True: run() calls the
library.  Both take the state that prepare() makes.
"""
import math

import torch

own = False

PAGE = 64   # tokens of a page
DIM = 64    # head dimension
S, ALPHA, L_TRAIN, BETA = 8.0, 0.3, 2048, 1.0  # method constants


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # One conversation, a draft of eight tokens: the latency of a verification step.
        {"name": "tree one 8 nodes", "kind": "tree", "seqs": 1, "lo": 1501, "hi": 1501, "nodes": 8,
         "hq": 16, "hkv": 4},
        # A serving batch of mixed lengths with drafts of up to 26 tokens.
        {"name": "tree batch 26 nodes", "kind": "tree", "seqs": 32, "lo": 500, "hi": 8192,
         "nodes": 26, "hq": 16, "hkv": 4},
        # Long contexts verified with the widest tree: the most work.
        {"name": "tree long 64 nodes", "kind": "tree", "seqs": 8, "lo": 32768, "hi": 65536,
         "nodes": 64, "hq": 16, "hkv": 4},
        # One conversation over a 32K context that reads 32 of about 512 pages.
        {"name": "sparse one 32K", "kind": "sparse", "seqs": 1, "lo": 32700, "hi": 32700, "keep": 32,
         "hq": 16, "hkv": 4},
        # Short and odd lengths together, some below the number of kept pages; groups of eight.
        {"name": "sparse ragged keep 17", "kind": "sparse", "seqs": 5, "lo": 3, "hi": 20000,
         "keep": 17, "hq": 16, "hkv": 2},
        # The 64K-256K decode pool with an eighth or less of its pages read.
        {"name": "sparse long keep 256", "kind": "sparse", "seqs": 16, "lo": 65536, "hi": 262144,
         "keep": 256, "hq": 16, "hkv": 4},
        # Every decode step of a batch: one token for each sequence.
        {"name": "append step 64 seqs", "kind": "append", "seqs": 64, "lo": 100, "hi": 8000,
         "tokens": 1, "hkv": 4},
        # Prompts written into the cache after their prefill.
        {"name": "append prompts", "kind": "append", "seqs": 16, "lo": 0, "hi": 0, "tokens": 16384,
         "hkv": 4},
        # One prompt searched with four beams.
        {"name": "beam 1x4", "kind": "beam", "prompts": 1, "beams": 4, "lo": 300, "hi": 300,
         "hkv": 4},
        # A batch of long prompts with eight beams each.
        {"name": "beam 16x8", "kind": "beam", "prompts": 16, "beams": 8, "lo": 4000, "hi": 32768,
         "hkv": 4},
        # A small pool after a few sequences ended.
        {"name": "compact 512 pages", "kind": "compact", "pages": 512, "live": 0.6, "seqs": 9,
         "hkv": 2},
        # A 2 GB pool, half of it live, before it is shrunk.
        {"name": "compact 32768 pages", "kind": "compact", "pages": 32768, "live": 0.5, "seqs": 64,
         "hkv": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tree", "sparse", "append", "beam", "compact"])
    hkv = rng.choice([1, 2, 4, 8])
    if kind == "tree":
        seqs = _log(rng, 1, 32)
        hi = _log(rng, 1, min(65536, 400000 // seqs))
        group = rng.choice([1, 2, 4, 8])
        hkv = min(hkv, 4, 16 // group)
        return {"kind": kind, "seqs": seqs, "lo": rng.randint(0, hi), "hi": hi,
                "nodes": _log(rng, 1, 64), "hq": hkv * group, "hkv": hkv}
    if kind == "sparse":
        seqs = _log(rng, 1, 32)
        hi = _log(rng, 40, min(262144, 1800000 // seqs))
        hkv = min(hkv, 4)
        return {"kind": kind, "seqs": seqs, "lo": rng.randint(1, hi), "hi": hi,
                "keep": _log(rng, 1, 256), "hq": hkv * rng.choice([1, 2, 4, 8]), "hkv": hkv}
    if kind == "append":
        seqs, tokens = _log(rng, 1, 128), _log(rng, 1, 16384)
        while seqs * tokens * hkv > 16 * 16384 * 4:
            tokens = max(1, tokens // 2)
        hi = _log(rng, 1, 8000)
        return {"kind": kind, "seqs": seqs, "lo": rng.randint(0, hi), "hi": hi, "tokens": tokens,
                "hkv": hkv}
    if kind == "beam":
        hi = _log(rng, 1, 32768)
        return {"kind": kind, "prompts": _log(rng, 1, 16), "beams": rng.randint(2, 8),
                "lo": rng.randint(1, hi), "hi": hi, "hkv": min(hkv, 4)}
    pages = _log(rng, 64, 32768)
    return {"kind": kind, "pages": pages, "live": round(rng.uniform(0.05, 0.95), 3),
            "seqs": _log(rng, 1, min(64, pages // 8)), "hkv": min(hkv, 4)}


# ---------------------------------------------------------------- prepare ---

def _unit(x):
    return x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)


def _uniform(gen, lo, hi, n):
    """n whole numbers of [lo, hi], the last of them hi."""
    r = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    v = (lo + (r * (hi - lo + 1)).floor()).long().clamp(max=hi)
    v[-1] = hi
    return v


def _pool(gen, pages, hkv):
    """kv_pages [pages, 2, hkv, 64, 64] bf16: unit rows; the keys of a page lie
    about a direction of their own, as the keys of neighbouring tokens do."""
    kv = torch.empty((pages, 2, hkv, PAGE, DIM), device="cuda", dtype=torch.bfloat16)
    for p0 in range(0, pages, 4096):
        part = kv[p0:p0 + 4096]
        x = torch.randn(part.shape, generator=gen, device="cuda")
        x[:, 0] += torch.randn((x.shape[0], hkv, 1, DIM), generator=gen, device="cuda")
        part.copy_(_unit(x))
    return kv


def _table(gen, lens, max_pages, pages):
    """A page table over a random permutation of the pool; -1 past the end."""
    n = (lens + PAGE - 1) // PAGE
    first = torch.cumsum(n, 0) - n
    col = torch.arange(max_pages, device="cuda")
    perm = torch.randperm(pages, generator=gen, device="cuda")
    at = (first[:, None] + col).clamp(max=pages - 1)
    return torch.where(col < n[:, None], perm[at], -1).int().contiguous()


def _references(table, pages):
    used = table[table >= 0].long()
    return torch.bincount(used, minlength=pages).int()


def _bounds(kv):
    """Per page and head, the smallest and the largest key of each dimension."""
    return torch.stack((kv[:, 0].amin(2), kv[:, 0].amax(2)), 2).contiguous()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    st = {"case": dict(case)}
    kind, hkv = case["kind"], case["hkv"]
    if kind in ("tree", "sparse"):
        n, hq = case["seqs"], case["hq"]
        lens = _uniform(gen, case["lo"], case["hi"], n)
        max_pages = max(1, (case["hi"] + PAGE - 1) // PAGE)
        pages = max(1, int(((lens + PAGE - 1) // PAGE).sum()))
        st["kv"] = _pool(gen, pages, hkv)
        st["table"], st["lens"] = _table(gen, lens, max_pages, pages), lens.int()
        st["u"] = 0.02 * torch.randn((hq, DIM), generator=gen, device="cuda")
        rows = case.get("nodes", 1)
        q = _unit(torch.randn((n, rows, hq, DIM), generator=gen, device="cuda"))
        # Some cached keys match a query, as retrieved ones do.
        if int(lens.min()) > 0:
            at = (torch.rand((n, hkv), generator=gen, device="cuda") * lens[:, None]).long()
            at = at.clamp(max=lens[:, None] - 1)
            page = st["table"].long().gather(1, at // PAGE)
            near = q[:, 0].view(n, hkv, hq // hkv, DIM)[:, :, 0]
            noise = torch.randn(near.shape, generator=gen, device="cuda") * (0.1 / math.sqrt(DIM))
            st["kv"][page, 0, torch.arange(hkv, device="cuda"), at % PAGE] = _unit(
                near + noise).bfloat16()
        st["q"] = q.bfloat16().contiguous()
        if kind == "sparse":
            st["q"] = st["q"][:, 0].contiguous()
            st["bounds"] = _bounds(st["kv"])
            st["out"] = torch.empty_like(st["q"])
            return st
        kt = torch.randn((2, n, rows, hkv, DIM), generator=gen, device="cuda")
        st["k"], st["v"] = _unit(kt).bfloat16().contiguous().unbind(0)
        # Each node's parent is an earlier node or the cache's last token (-1).
        r = torch.rand((n, rows), generator=gen, device="cuda", dtype=torch.float64)
        parent = (r * (torch.arange(rows, device="cuda") + 1)).long() - 1
        seen = torch.zeros((n, rows, rows), dtype=torch.bool, device="cuda")
        for t in range(rows):
            up = seen.gather(1, parent[:, t].clamp(min=0)[:, None, None].expand(n, 1, rows))[:, 0]
            seen[:, t] = up & (parent[:, t] >= 0)[:, None]
            seen[:, t, t] = True
        bits = seen.long() << torch.arange(rows, device="cuda")
        st["mask"] = bits.sum(-1)  # distinct bits: the sum is their union
        st["nodes"] = _uniform(gen, max(1, rows // 2), rows, n).int()
        # Where a sequence drafted fewer nodes, its rows behind them stay as they are: zeros here.
        st["out"] = torch.zeros_like(st["q"])
        st["neff"] = torch.zeros((n, rows, hq), device="cuda")
        return st
    if kind == "append":
        n, tokens = case["seqs"], case["tokens"]
        lens = _uniform(gen, case["lo"], case["hi"], n)
        grow = _uniform(gen, max(1, tokens // 2), tokens, n)
        max_pages = (case["hi"] + tokens + PAGE - 1) // PAGE
        pages = n * (max_pages + 1)
        st["kv"] = _pool(gen, pages, hkv)
        st["table"], st["lens"] = _table(gen, lens, max_pages, pages), lens.int()
        st["grow"] = grow.int()
        new = torch.randn((2, n, tokens, hkv, DIM), generator=gen, device="cuda")
        st["k"], st["v"] = _unit(new).bfloat16().contiguous().unbind(0)
    elif kind == "beam":
        groups, beams = case["prompts"], case["beams"]
        n = groups * beams
        lens = _uniform(gen, case["lo"], case["hi"], groups)
        steps = 1 + int(seed) % 100  # tokens that each beam has written of its own
        whole = lens // PAGE         # a prompt's full pages are shared by its beams
        total = lens + steps
        max_pages = (case["hi"] + 101 + PAGE - 1) // PAGE
        shared = _table(gen, whole * PAGE, max_pages, max(1, int(whole.sum())))
        col = torch.arange(max_pages, device="cuda")
        each = ((total + PAGE - 1) // PAGE - whole).repeat_interleave(beams)
        first = int(whole.sum()) + torch.cumsum(each, 0) - each
        at = col - whole.repeat_interleave(beams)[:, None]
        table = torch.where((at >= 0) & (at < each[:, None]), first[:, None] + at, -1)
        table = torch.where(at < 0, shared.long().repeat_interleave(beams, 0), table)
        pages = groups * (case["hi"] // PAGE) + 5 * n
        perm = torch.randperm(pages, generator=gen, device="cuda")
        st["table"] = torch.where(table >= 0, perm[table.clamp(min=0)], -1).int().contiguous()
        st["lens"] = total.repeat_interleave(beams).int()
        st["kv"] = _pool(gen, pages, hkv)
        parent = torch.randint(beams, (groups, beams), generator=gen, device="cuda")
        parent += torch.arange(groups, device="cuda")[:, None] * beams
        st["src"] = parent.reshape(-1).int()
        st["grow"] = torch.ones(n, dtype=torch.int32, device="cuda")
    else:
        pages, n = case["pages"], case["seqs"]
        live = max(n, int(pages * case["live"]))
        share = 0.5 + torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
        count = (share / share.sum() * (live - n)).long() + 1
        r = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
        lens = count * PAGE - (r * PAGE).long()
        st["kv"] = _pool(gen, pages, hkv)
        st["table"] = _table(gen, lens, 3 * live // n + 2, pages)
        st["lens"] = lens.int()
    st["refs"] = _references(st["table"], st["kv"].shape[0])
    st["bounds"] = _bounds(st["kv"])
    return st


# ------------------------------------------------------------- plain forms ---

def _polar(raw, seen, values, n, u):
    """The mixing step of rows of raw products against their visible keys.

    raw [..., rows, keys] fp32, seen the same in truth values, values
    [..., keys, 64], n [..., rows] visible keys, u [..., rows, 64].  A row that
    sees nothing gives zeros."""
    count = n.clamp(min=1).float()
    wide = n.clamp(min=1).double()
    c = torch.where(n > L_TRAIN, S * (1 + ALPHA * torch.log(wide / L_TRAIN)), S).float()
    raw = torch.where(seen, raw, 0.0)
    top = torch.where(seen, raw, -math.inf).amax(-1)
    top = torch.where(n > 0, top, 0.0)
    weight = torch.exp((raw - top[..., None]) * c[..., None]) * seen
    acc = weight @ values
    total, square = weight.sum(-1), weight.square().sum(-1)
    neff = (total * total / square.clamp(min=1e-30)).clamp(min=1.0)
    neff = torch.minimum(neff, count)
    mean = raw.sum(-1) / count
    spread = (((raw - mean[..., None]) * seen).square().sum(-1) / count).sqrt()
    null = c * (mean + spread * torch.log(wide).mul(2).sqrt().float())
    gate = torch.sigmoid(BETA * (c * top - null))
    amount = gate * torch.tanh(torch.log(neff) / math.log(L_TRAIN))
    norm = acc.square().sum(-1).sqrt().clamp(min=1e-30)
    out = acc / norm[..., None] + amount[..., None] * u
    empty = n <= 0
    return torch.where(empty[..., None], 0.0, out), torch.where(empty, 0.0, neff)


def _plain_tree(st):
    q, table, lens, kv = st["q"].float(), st["table"].long(), st["lens"].long(), st["kv"]
    n, m, hq, _ = q.shape
    hkv, keys = kv.shape[2], table.shape[1] * PAGE
    g = hq // hkv
    pages = kv[table.clamp(min=0)].float()                 # [n, pages, 2, hkv, 64, 64]
    k, v = pages.permute(2, 0, 3, 1, 4, 5).reshape(2, n, hkv, keys, DIM)
    del pages
    k = torch.cat((k, st["k"].float().transpose(1, 2)), 2)
    v = torch.cat((v, st["v"].float().transpose(1, 2)), 2)
    node = torch.arange(m, device=q.device)
    drafted = (st["mask"][:, :, None] >> node & 1).bool() & (node < st["nodes"][:, None, None])
    cached = torch.arange(keys, device=q.device) < lens[:, None, None]
    seen = torch.cat((cached.expand(n, m, keys), drafted), -1)           # [n, m, keys + m]
    v = torch.where(seen.any(1)[:, None, :, None], v, 0.0)
    count = seen.sum(-1)
    rows = q.view(n, m, hkv, g, DIM).permute(0, 2, 1, 3, 4).reshape(n, hkv, m * g, DIM)
    raw = rows @ k.transpose(-1, -2)
    u = st["u"].view(1, hkv, 1, g, DIM).expand(n, hkv, m, g, DIM).reshape(n, hkv, m * g, DIM)
    out, neff = _polar(raw, seen.repeat_interleave(g, 1)[:, None], v,
                       count.repeat_interleave(g, 1)[:, None].expand(n, hkv, m * g), u)
    out = out.view(n, hkv, m, g, DIM).permute(0, 2, 1, 3, 4).reshape(n, m, hq, DIM)
    neff = neff.view(n, hkv, m, g).permute(0, 2, 1, 3).reshape(n, m, hq)
    real = node < st["nodes"][:, None]
    return (torch.where(real[:, :, None, None], out.bfloat16(), st["out"]),
            torch.where(real[:, :, None], neff, st["neff"]))


def _plain_sparse(st):
    q, table, lens, kv = st["q"].float(), st["table"].long(), st["lens"].long(), st["kv"]
    keep = st["case"]["keep"]
    n, hq, _ = q.shape
    hkv, max_pages = kv.shape[2], table.shape[1]
    g = hq // hkv
    have = (lens + PAGE - 1) // PAGE
    # A page's score is the largest product that keys within its bounds allow.
    edge = st["bounds"][table.clamp(min=0)].double()       # [n, pages, hkv, 2, 64]
    rows = q.view(n, hkv, g, DIM).double()
    score = torch.einsum("nhgd,nphd->nhgp", rows.clamp(min=0), edge[:, :, :, 1])
    score += torch.einsum("nhgd,nphd->nhgp", rows.clamp(max=0), edge[:, :, :, 0])
    score = score.float().amax(2)                          # [n, hkv, pages]
    page = torch.arange(max_pages, device=q.device)
    score = torch.where(page == have[:, None, None] - 1, math.inf, score)
    score = torch.where(page < have[:, None, None], score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True)[1]
    chosen = torch.full((n, hkv, keep), max_pages, device=q.device, dtype=torch.long)
    take = min(keep, max_pages)
    chosen[:, :, :take] = torch.where(page[:take] < have[:, None, None], order[:, :, :take],
                                      max_pages)
    chosen = torch.sort(chosen, -1)[0]
    valid = chosen < max_pages
    phys = table[:, None].expand(n, hkv, max_pages).gather(2, chosen.clamp(max=max_pages - 1))
    head = torch.arange(hkv, device=q.device)[:, None]
    phys = phys.clamp(min=0)
    k = kv[phys, 0, head].float().view(n, hkv, keep * PAGE, DIM)
    v = kv[phys, 1, head].float().view(n, hkv, keep * PAGE, DIM)
    at = chosen[..., None] * PAGE + torch.arange(PAGE, device=q.device)
    seen = (valid[..., None] & (at < lens[:, None, None, None])).view(n, hkv, 1, keep * PAGE)
    raw = q.view(n, hkv, g, DIM) @ k.transpose(-1, -2)
    v = torch.where(seen.transpose(-1, -2), v, 0.0)
    out, neff = _polar(raw, seen, v, seen.sum(-1).expand(n, hkv, g), st["u"].view(hkv, g, DIM))
    return (out.view(n, hq, DIM).bfloat16(), neff.reshape(n, hq),
            torch.where(valid, chosen, -1).int())


def _plain_reserve(kv, bounds, refs, table, lens, grow):
    """Room for `grow` more tokens in each row: new pages, the lowest free ids
    first, and a copy of its own for a partly filled page that others share
    (the last of its sharers keeps it where all of them are served here)."""
    n, max_pages = table.shape
    pages = refs.numel()
    old, part = lens.long(), lens.long() % PAGE
    fits = (grow >= 0) & (old + grow <= max_pages * PAGE)
    tail = (old // PAGE).clamp(max=max_pages - 1)[:, None]
    page = table.gather(1, tail)[:, 0].long()
    writes = fits & (grow > 0) & (part > 0)
    same = writes[:, None] & writes & (page[:, None] == page)
    shared = writes & (refs[page.clamp(min=0)] > 1)
    keeps = (same.sum(1) == refs[page.clamp(min=0)]) & ~torch.triu(same, 1).any(1)
    copy = shared & ~keeps
    have = (old + PAGE - 1) // PAGE
    extra = torch.where(fits, (old + grow + PAGE - 1) // PAGE - have, 0)
    need = extra + copy
    end = torch.cumsum(need, 0)
    free = torch.argsort((refs != 0).byte(), stable=True)
    served = fits & (end <= (refs == 0).sum())
    copy = copy & served
    first = end - need
    col = torch.arange(max_pages, device=table.device)
    k = first[:, None] + copy[:, None] + col - have[:, None]
    new = served[:, None] & (col >= have[:, None]) & (col < (have + extra)[:, None])
    own_copy = copy[:, None] & (col == tail)
    fresh = free[torch.where(new, k, torch.where(own_copy, first[:, None], 0)).clamp(0, pages - 1)]
    taken = new | own_copy
    ones = taken.reshape(-1).int()
    refs.index_add_(0, fresh.reshape(-1), ones)
    refs.index_add_(0, page.clamp(min=0), -copy.int())
    table.copy_(torch.where(taken, fresh.int(), table))
    to = torch.where(copy, table.gather(1, tail)[:, 0].long(), -1)
    rows = copy.nonzero()[:, 0]
    src, dst = page[rows], to[rows]
    kept = (torch.arange(PAGE, device=table.device) < part[rows, None])[:, None, None, :, None]
    kv[dst] = torch.where(kept, kv[src], kv[dst])
    bounds[dst] = bounds[src]
    granted = torch.where(served, grow, 0)
    lens += granted
    return granted


def _plain_append(kv, bounds, k, v, table, lens, counts):
    n, tokens, hkv, _ = k.shape
    t = torch.arange(tokens, device=k.device)
    row, t = (t < counts[:, None]).nonzero().unbind(1)
    at = (lens - counts).long()[row] + t
    page = table[row, at // PAGE].long()
    kv[page, 0, :, at % PAGE] = k[row, t]
    kv[page, 1, :, at % PAGE] = v[row, t]
    # The bounds of every page that got a token, over the page's valid rows.
    col = torch.arange(table.shape[1], device=k.device)
    first, last = (lens - counts) // PAGE, (lens - 1) // PAGE
    row, col = ((col >= first[:, None]) & (col <= last[:, None]) & (counts > 0)[:, None]
                ).nonzero().unbind(1)
    page = table[row, col].long()
    valid = torch.arange(PAGE, device=k.device) < (lens[row] - col * PAGE)[:, None]
    valid = valid[:, None, :, None]
    for part in torch.arange(page.numel(), device=k.device).split(8192):
        keys, ok = kv[page[part], 0].float(), valid[part]
        low = torch.where(ok, keys, math.inf).amin(2)
        high = torch.where(ok, keys, -math.inf).amax(2)
        bounds[page[part]] = torch.stack((low, high), 2).bfloat16()


def _plain_fork(refs, src_table, src_lens, src, table, lens):
    rows, length = src_table[src.long()], src_lens[src.long()]
    col = torch.arange(table.shape[1], device=table.device)
    used = col < ((length + PAGE - 1) // PAGE)[:, None]
    table.copy_(torch.where(used, rows, table))
    lens.copy_(length)
    refs.index_add_(0, rows.clamp(min=0).reshape(-1).long(), used.reshape(-1).int())


def _plain_free(refs, table, lens):
    col = torch.arange(table.shape[1], device=table.device)
    used = col < ((lens + PAGE - 1) // PAGE)[:, None]
    refs.index_add_(0, table.clamp(min=0).reshape(-1).long(), -used.reshape(-1).int())
    table.masked_fill_(used, -1)
    lens.zero_()


def _plain_compact(kv, bounds, refs, table, lens):
    live = refs > 0
    used = live.sum()
    ids = torch.arange(refs.numel(), device=refs.device)
    src = (live & (ids >= used)).nonzero()[:, 0]
    dst = (~live & (ids < used)).nonzero()[:, 0]
    for a, b in zip(src.split(4096), dst.split(4096)):
        kv[b] = kv[a]
    bounds[dst] = bounds[src]
    refs[dst] = refs[src]
    refs[src] = 0
    ids[src] = dst
    col = torch.arange(table.shape[1], device=table.device)
    inside = col < ((lens + PAGE - 1) // PAGE)[:, None]
    table.copy_(torch.where(inside, ids[table.clamp(min=0).long()].int(), table))
    return used.int().view(1)


# -------------------------------------------------------------------- run ---

def run(st):
    if own:
        return _run_own(st)
    kind = st["case"]["kind"]
    if kind == "tree":
        return _plain_tree(st)
    if kind == "sparse":
        return _plain_sparse(st)
    # The cache's bookkeeping starts from the same state in every pass; what
    # the pool's pages hold in the end depends on that state alone.
    kv, bounds = st["kv"], st["bounds"]
    refs, table, lens = st["refs"].clone(), st["table"].clone(), st["lens"].clone()
    if kind == "append":
        granted = _plain_reserve(kv, bounds, refs, table, lens, st["grow"])
        _plain_append(kv, bounds, st["k"], st["v"], table, lens, granted)
        return kv, bounds, refs, table, lens, granted
    if kind == "beam":
        new, new_lens = torch.full_like(table, -1), torch.zeros_like(lens)
        _plain_fork(refs, table, lens, st["src"], new, new_lens)
        _plain_free(refs, table, lens)
        granted = _plain_reserve(kv, bounds, refs, new, new_lens, st["grow"])
        return kv, bounds, refs, table, lens, new, new_lens, granted
    used = _plain_compact(kv, bounds, refs, table, lens)
    return kv, bounds, refs, table, used


def _run_own(st):
    import polar_attention_b200 as pa
    kind = st["case"]["kind"]
    if kind == "tree":
        return pa.decode_paged_tree(st["q"], st["k"], st["v"], st["mask"], st["kv"], st["table"],
                                    st["lens"], st["u"], st["out"], st["neff"],
                                    tree_lens=st["nodes"], s=S, alpha=ALPHA, L=L_TRAIN, beta=BETA)
    if kind == "sparse":
        return pa.decode_paged_sparse(st["q"], st["kv"], st["bounds"], st["table"], st["lens"],
                                      st["u"], st["case"]["keep"], st["out"], s=S, alpha=ALPHA,
                                      L=L_TRAIN, beta=BETA)
    cache = pa.PageCache(st["kv"], st["refs"].clone(), st["bounds"])
    table, lens = st["table"].clone(), st["lens"].clone()
    if kind == "append":
        granted = pa.cache_reserve(cache, table, lens, st["grow"])
        pa.cache_append(cache, st["k"], st["v"], table, lens, granted)
        return cache.kv_pages, cache.bounds, cache.refs, table, lens, granted
    if kind == "beam":
        new, new_lens = torch.full_like(table, -1), torch.zeros_like(lens)
        pa.cache_fork(cache, table, lens, st["src"], new, new_lens)
        pa.cache_free(cache, table, lens)
        granted = pa.cache_reserve(cache, new, new_lens, st["grow"])
        return cache.kv_pages, cache.bounds, cache.refs, table, lens, new, new_lens, granted
    used = pa.cache_compact(cache, table, lens)
    return cache.kv_pages, cache.bounds, cache.refs, table, used


# ------------------------------------------------------------------- work ---

def _mean_len(case):
    return (case["lo"] + case["hi"]) / 2


def work(case):
    kind, hkv = case["kind"], case["hkv"]
    token = 2 * hkv * DIM * 2  # bytes of one token's key and value rows
    if kind == "tree":
        n, m, hq = case["seqs"], case["nodes"], case["hq"]
        cached = n * _mean_len(case)
        nodes = 0.75 * m if m > 1 else 1
        rows = n * nodes * hq
        return {"bytes": cached * token + n * nodes * token + rows * (2 * DIM * 2 + 4),
                "flops": 4 * DIM * nodes * hq * (cached + n * nodes / 2)}
    if kind == "sparse":
        n, hq, keep = case["seqs"], case["hq"], case["keep"]
        have = n * _mean_len(case) / PAGE
        read = min(n * keep, have)
        return {"bytes": have * hkv * 2 * DIM * 2 + read * PAGE * token
                + n * hq * (2 * DIM * 2 + 4) + n * hkv * keep * 4,
                "flops": have * hq * 4 * DIM + read * PAGE * hq * 4 * DIM}
    page = PAGE * token
    if kind == "append":
        n, tokens = case["seqs"], case["tokens"]
        new = n * (0.75 * tokens if tokens > 1 else 1)
        reread = n * PAGE / 2 * token / 2 if case["hi"] else 0  # keys of the page begun before
        edges = (new / PAGE + n) * hkv * 2 * DIM * 2
        return {"bytes": 2 * new * token + reread + edges, "flops": new * hkv * DIM * 2}
    if kind == "beam":
        n = case["prompts"] * case["beams"]
        entries = n * _mean_len(case) / PAGE
        copied = n * 0.4  # rows whose tail page another row keeps
        return {"bytes": entries * 4 * 6 + copied * page, "flops": entries * 2}
    moved = case["pages"] * case["live"] * (1 - case["live"])
    return {"bytes": 2 * moved * page + case["pages"] * 8, "flops": case["pages"]}


# ------------------------------------------------------------------ exact ---

def _row64(raw, values, u, s, alpha):
    """One group of rows in 64 bits; raw [rows, keys], every key visible."""
    n = raw.shape[1]
    if n == 0:
        return torch.zeros_like(u), u.new_zeros(u.shape[0])
    c = s * (1 + alpha * math.log(n / L_TRAIN)) if n > L_TRAIN else s
    z = c * raw
    p = torch.softmax(z, 1)
    direction = p @ values
    direction = direction / torch.linalg.vector_norm(direction, dim=1, keepdim=True).clamp(min=1e-30)
    neff = 1 / (p * p).sum(1)
    null = z.mean(1) + z.std(1, correction=0) * math.sqrt(2 * math.log(n))
    gate = 1 / (1 + torch.exp(-BETA * (z.amax(1) - null)))
    return direction + (gate * torch.tanh(torch.log(neff) / math.log(L_TRAIN)))[:, None] * u, neff


def exact(case, seed):
    if case["kind"] not in ("tree", "sparse"):
        return None  # pages, references and tables are copies and whole numbers
    st = prepare(case, seed)
    q, kv, u = st["q"].double(), st["kv"], st["u"].double()
    hkv = kv.shape[2]
    g = q.shape[-2] // hkv
    s, alpha = float(torch.tensor(S)), float(torch.tensor(ALPHA))
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    neff = torch.zeros(q.shape[:-1], dtype=torch.float64, device="cuda")
    for i, length in enumerate(st["lens"].tolist()):
        have = -(-length // PAGE)
        ids = st["table"][i, :have].long()
        for h in range(hkv):
            heads = slice(h * g, h * g + g)
            if case["kind"] == "sparse":
                low, high = st["bounds"][ids, h].double().unbind(1)
                rows = q[i, heads]
                bound = torch.maximum(rows[:, None] * low, rows[:, None] * high).sum(-1)
                score = bound.float().amax(0).tolist()
                score[-1] = math.inf
                best = sorted(range(have), key=lambda p: (-score[p], p))[:case["keep"]]
                at = torch.tensor([p * PAGE + t for p in sorted(best) for t in range(PAGE)
                                   if p * PAGE + t < length], device="cuda")
                k, v = kv[ids[at // PAGE], :, h, at % PAGE].double().unbind(1)
                out[i, heads], neff[i, heads] = _row64(rows @ k.T, v, u[heads], s, alpha)
                continue
            k, v = kv[ids, :, h].double().transpose(0, 1).reshape(2, have * PAGE, DIM)[:, :length]
            k = torch.cat((k, st["k"][i, :, h].double()))
            v = torch.cat((v, st["v"][i, :, h].double()))
            raw = q[i, :, heads] @ k.T                     # [nodes, g, keys]
            nodes = int(st["nodes"][i])
            for t, bits in enumerate(st["mask"][i, :nodes].tolist()):
                at = [length + j for j in range(nodes) if bits >> j & 1]
                seen = torch.cat((torch.arange(length), torch.tensor(at, dtype=torch.long))).cuda()
                out[i, t, heads], neff[i, t, heads] = _row64(raw[t][:, seen], v[seen], u[heads], s,
                                                             alpha)
    return (out, neff, None) if case["kind"] == "sparse" else (out, neff)
