"""Cases of the operators around the paged K/V cache: the append of tokens to a pool of pages, the selection of pages by
their summaries, the decode attention over the pool, the fork of sequences (which also frees and cuts them) and the
compaction of the pool.  With `own` false run() computes each in elementary torch operations in 32 bits; with `own` true
it makes the calls a program makes of sparse_long_context_gb300.ops.

A cache is a pool of pages [N, Hkv, P, D], a table [B, Cap/P] that gives the page of the pool which holds a sequence's
logical page, the sequences' lengths and the number of sequences that hold each page.  A case that changes the table,
lengths or counts puts them back first, so that every pass finds the same ones.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
GOLDEN = 0.6180339887498949  # multiples of it, modulo one, spread evenly


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one conversation of a thousand tokens in a pool for long ones: latency counts
        dict(name="attend_short", op="attend", batch=1, hq=28, hkv=4, d=128, page=16, cap=32768, low=1000, high=1000,
             dtype="bf16", lists=0, sink=False),
        # dense decode of 32 contexts of 49k to 64k tokens whose pages lie anywhere in the pool
        dict(name="attend_dense_64k", op="attend", batch=32, hq=12, hkv=2, d=128, page=16, cap=65536, low=49000,
             high=65536, dtype="bf16", lists=0, sink=False),
        # the sparse step: 128 selected pages per KV head out of 64k tokens
        dict(name="attend_lists_64k", op="attend", batch=32, hq=12, hkv=2, d=128, page=16, cap=65536, low=60000,
             high=65536, dtype="bf16", lists=128, sink=False),
        # fp32, heads of 64 channels with a sink logit, very uneven lengths
        dict(name="attend_f32_uneven", op="attend", batch=7, hq=64, hkv=8, d=64, page=64, cap=20480, low=1, high=20000,
             dtype="f32", lists=0, sink=True),
        # one decoded token for each of 32 sequences, some of which begin a page; page summaries kept
        dict(name="append_decode", op="append", batch=32, hkv=2, d=128, page=16, cap=8192, pool=16384, new=1,
             dtype="bf16", summaries=True),
        # four prompts of up to 32k tokens into an empty cache
        dict(name="append_prompt", op="append", batch=4, hkv=8, d=128, page=64, cap=32768, pool=2080, new=32768,
             dtype="bf16", summaries=False),
        # the selection before a sparse step: 4096 pages a row, first page and last 64 tokens always taken
        dict(name="select_64k", op="select", batch=32, hq=12, hkv=2, d=128, page=16, cap=65536, low=60000, high=65536,
             dtype="bf16", k=128, first=1, last=64),
        # the selection of three short fp32 contexts with an odd budget
        dict(name="select_f32_short", op="select", batch=3, hq=5, hkv=1, d=64, page=32, cap=8192, low=2000, high=7777,
             dtype="f32", k=37, first=2, last=100),
        # a beam search's step: eight groups of four beams are reordered
        dict(name="fork_beams", op="fork", batch=32, hkv=4, d=128, page=16, cap=4096, prompts=8, low=1500, high=3000,
             dtype="bf16", summaries=False, beams=True),
        # sixteen prompts of 20k to 32k tokens, whose prefixes three further requests each share
        dict(name="fork_prefixes", op="fork", batch=64, hkv=2, d=128, page=16, cap=32768, prompts=16, low=20000, high=32768,
             dtype="bf16", summaries=True, beams=False),
        # a pool of a thousand small fp32 pages after many sequences have ended
        dict(name="compact_small", op="compact", batch=9, hkv=1, d=64, page=32, cap=4096, pool=1000, low=100, high=4000,
             dtype="f32", summaries=True),
        # a pool of a gigabyte with half of its pages in use
        dict(name="compact_pool", op="compact", batch=48, hkv=4, d=128, page=16, cap=8192, pool=32768, low=2500,
             high=8192, dtype="bf16", summaries=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "select", "fork", "compact"])
    hkv, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
    group = rng.choice([1, 2, 3, 5, 6, 7, 8])
    page = rng.choice([16, 16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    batch = _log(rng, 1, 48)
    room = (1 << 28) // (batch * hkv * d * (2 if dtype == "f32" else 1))  # tokens a sequence may have
    cap = -(-_log(rng, 512, max(1024, min(131072, room))) // 256) * 256
    low = _log(rng, 1, cap)
    high = rng.randint(low, cap)
    c = dict(op=op, batch=batch, hkv=hkv, d=d, page=page, cap=cap, dtype=dtype)
    if op == "attend":
        lists = rng.choice([0, 0, min(cap // page, _log(rng, 3, 300))])
        return c | dict(hq=group * hkv, low=low, high=high, lists=lists, sink=rng.random() < 0.4)
    if op == "append":
        new = 1 if rng.random() < 0.4 else _log(rng, 2, cap // 2)
        return c | dict(pool=batch * (cap // page) + rng.randint(1, 99), new=new, summaries=rng.random() < 0.5)
    if op == "select":  # a budget of at most half of the shortest context's pages
        c["page"] = page = page if cap // page >= 32 else 16
        k = min(220, _log(rng, 8, cap // page // 2))
        low = rng.randint(2 * k * page, cap)
        return c | dict(hq=group * hkv, low=low, high=rng.randint(low, cap), k=k, first=rng.choice([0, 1, 2]) if k > 11 else 0,
                        last=rng.choice([0, 50, 64, 128]) if k > 11 else 0)
    if op == "fork":
        prompts = max(1, batch // rng.choice([2, 3, 4, 8]))
        return c | dict(prompts=prompts, low=low, high=high, summaries=rng.random() < 0.5, beams=rng.random() < 0.5)
    used = sum(-(-n // page) for n in _lens(c | dict(low=low, high=high)))
    return c | dict(pool=used + rng.randint(1, 2 * used + 8), low=low, high=high, summaries=rng.random() < 0.5)


def _size(c):
    return 2 if c["dtype"] == "bf16" else 4


def work(case):
    c = case
    row = c["hkv"] * c["d"] * _size(c)  # bytes of a token's keys (or values)
    page = c["page"]
    if c["op"] == "append":
        start, new = _spans(c)
        n = sum(new)
        pages = sum(-(-(s + k) // page) - s // page for s, k in zip(start, new))
        fresh = sum(-(-(s + k) // page) - -(-s // page) for s, k in zip(start, new))
        b = 4 * n * row + 8 * fresh + 12 * c["batch"]
        if c["summaries"]:  # those of the pages begun before are read as well
            b += 2 * pages * row + 2 * (pages - fresh) * row
        return {"bytes": b, "flops": 2 * n * c["hkv"] * c["d"]}
    if c["op"] == "fork":
        lens, keep, parent, changed = _fork_plan(c)
        kept = sum(-(-keep[i] // page) for i in range(c["batch"]) if changed[i])
        part = sum(keep[i] % page for i in range(c["batch"]) if changed[i])
        return {"bytes": 12 * kept + 12 * c["batch"] + 4 * part * row, "flops": kept}
    lens = _lens(c)
    pages = sum(-(-n // page) for n in lens)
    if c["op"] == "compact":
        moved = pages * (c["pool"] - pages) // c["pool"]
        return {"bytes": 4 * moved * page * row + 8 * pages + 8 * c["pool"] + (4 * moved * row if c["summaries"] else 0),
                "flops": pages}
    heads = c["batch"] * c["hq"] * c["d"]
    if c["op"] == "select":
        return {"bytes": 2 * pages * row + 4 * pages + heads * _size(c) + 4 * c["batch"] * c["hkv"] * c["k"],
                "flops": 4 * pages * c["hq"] * c["d"]}
    kept = sum(min(n, c["lists"] * page) if c["lists"] else n for n in lens)
    return {"bytes": 2 * kept * row + 2 * heads * _size(c) + 4 * c["batch"] * c["hq"] + 4 * -(-kept // page),
            "flops": 4 * kept * c["hq"] * c["d"]}


# ------------------------------------------------------------------- the inputs

def _lens(c):
    """Lengths between `low` and `high`: the first at `low`, the last of several at `high`, the others anywhere between."""
    low, high, b = c["low"], c["high"], c.get("prompts", c["batch"])
    return [high if 0 < i == b - 1 else low + int((high - low) * (i * GOLDEN % 1.0)) for i in range(b)]


def _spans(c):
    """Start and count of the new tokens of each sequence; every fourth sequence begins a page."""
    room = c["cap"] - c["new"]
    start = [int(room * ((i + 1) * GOLDEN % 1.0)) for i in range(c["batch"])]
    start = [s // c["page"] * c["page"] if i % 4 == 1 else s for i, s in enumerate(start)]
    return start, [max(1, c["new"] - (i % 5) * c["new"] // 16) for i in range(c["batch"])]


def _fork_plan(c):
    """Lengths before, lengths after, parents, and which sequences are not left as they are."""
    b, n, some = c["batch"], c["prompts"], _lens(c)
    if c["beams"]:  # every sequence is a beam of its group: slot i is beam i // n of prompt i % n
        lens = [some[i % n] for i in range(b)]
        beams = [-(-(b - i) // n) for i in range(n)]
        parent = [i % n + n * (int((i + 1) * GOLDEN * 64) % beams[i % n]) for i in range(b)]
        keep = [lens[p] for p in parent]
    else:
        lens = [some[i] if i < n else 0 for i in range(b)]
        parent = [i if i < n else i % n for i in range(b)]
        keep = [some[i] if i < n else max(1, int(some[i % n] * (0.5 + 0.5 * (i * GOLDEN % 1.0)))) for i in range(b)]
    return lens, keep, parent, [parent[i] != i or keep[i] != lens[i] for i in range(b)]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _keys(g, shape, dtype):
    """Key-like values: channels of very different size, as projected keys have."""
    gain = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)


def _spread(g, lens, mp, page, pool):
    """A table for sequences of these lengths: pages anywhere in the pool, each held once."""
    count = (_ints(lens) + page - 1) // page
    l = torch.arange(mp, device="cuda")
    at = (torch.cumsum(count, 0) - count)[:, None] + l
    ids = torch.randperm(pool, generator=g, device="cuda")
    return torch.where(l < count[:, None], ids[at.clamp(max=pool - 1)], -1).to(torch.int32)


def prepare(case, seed):
    c, g = case, torch.Generator("cuda")
    g.manual_seed(seed * 7919 + 29)
    op, b, h, d, page, mp = c["op"], c["batch"], c["hkv"], c["d"], c["page"], c["cap"] // c["page"]
    dt = BF16 if c["dtype"] == "bf16" else F32
    s = {"case": dict(c)}
    if op == "append":
        lens, new = _spans(c)
    elif op == "fork":
        lens, keep, parent, _ = _fork_plan(c)
    else:
        lens = _lens(c)
    used = sum(-(-n // page) for n in lens)
    pool = c.get("pool", used + used // 8 + b + 1)  # with pages to spare
    if op == "fork" and c["beams"]:  # the beams of a group share its complete pages
        s["table"] = _spread(g, lens, mp, page, pool)
        l = torch.arange(mp, device="cuda")
        whole = l < (_ints(lens) // page)[:, None]
        group = torch.arange(b, device="cuda") % c["prompts"]
        s["table"] = torch.where(whole, s["table"][group], s["table"])
    else:
        s["table"] = _spread(g, lens, mp, page, pool)
    s["ctx"] = _ints(lens)
    s["refs"] = torch.bincount(s["table"][s["table"] >= 0].long(), minlength=pool).to(torch.int32)
    if op == "select":  # the selection reads the summaries only
        s["k_pages"] = torch.empty((pool, h, page, d), dtype=dt, device="cuda")
        s["v_pages"] = torch.empty_like(s["k_pages"])
    else:
        s["k_pages"] = _keys(g, (pool, h, page, d), dt)
        s["v_pages"] = torch.randn((pool, h, page, d), generator=g, device="cuda").to(dt)
    s["kmin"] = s["kmax"] = None
    if op == "select":
        # keys of a model whose cache was rounded to steps of 1/32: every score is exact in 32 bits, whatever the order of its
        # sum, so that pages at the border of the budget compare equal exactly where they are equal
        mid, wide = (_keys(g, (pool, h, d), F32) for _ in range(2))
        s["kmin"] = (torch.round((mid - wide.abs()).clamp(-7, 7) * 32) / 32).to(dt)
        s["kmax"] = (torch.round((mid + wide.abs()).clamp(-7, 7) * 32) / 32).to(dt)
        s["kmin"], s["kmax"] = torch.minimum(s["kmin"], s["kmax"]), torch.maximum(s["kmin"], s["kmax"])
        q = torch.randn((b, c["hq"], d), generator=g, device="cuda").clamp(-7, 7)
        s["q"] = (torch.round(q * 32) / 32).to(dt)
    elif c.get("summaries"):  # of the rows of each page that hold tokens
        rows = torch.zeros(pool, dtype=torch.int64, device="cuda")
        held = (s["ctx"][:, None] - page * torch.arange(mp, device="cuda")).clamp(0, page)
        rows[s["table"][held > 0].long()] = held[held > 0]
        off = torch.arange(page, device="cuda") >= rows[:, None]
        x = s["k_pages"].float()
        s["kmin"] = torch.where(rows[:, None, None] > 0, x.masked_fill(off[:, None, :, None], math.inf).amin(2), 0.0).to(dt)
        s["kmax"] = torch.where(rows[:, None, None] > 0, x.masked_fill(off[:, None, :, None], -math.inf).amax(2), 0.0).to(dt)
        del x
    if op == "attend":
        hq = c["hq"]
        # a query looks for a few of its sequence's tokens and has a random part
        at = (torch.rand((b, 4), generator=g, device="cuda") * s["ctx"][:, None]).long()
        phys = torch.gather(s["table"].long(), 1, at // page)
        found = s["k_pages"][phys, :, at % page].float().sum(1)  # [b, h, d]
        s["q"] = (torch.randn((b, h, hq // h, d), generator=g, device="cuda") + 0.5 * found[:, :, None]).view(b, hq, d).to(dt)
        s["sink"] = torch.randn(hq, generator=g, device="cuda") if c["sink"] else None
        s["lists"] = None
        if c["lists"]:  # as a selection leaves it: first page, newest page, the others anywhere; ascending, -1 padded
            np_row = (s["ctx"].view(b, 1, 1) + page - 1) // page
            i = torch.arange(mp, device="cuda")
            score = torch.rand((b, h, mp), generator=g, device="cuda")
            score = torch.where((i == 0) | (i == np_row - 1), torch.full_like(score, 2.0), score).masked_fill(i >= np_row, -1.0)
            top = torch.topk(score, c["lists"], dim=-1)
            idx = torch.where(top.values < 0, mp, top.indices).sort(-1).values
            s["lists"] = torch.where(idx >= mp, -1, idx).to(torch.int32).view(b * h, c["lists"]).contiguous()
        s["out"] = torch.empty((b, hq, d), dtype=dt, device="cuda")
        s["lse"] = torch.empty((b, hq), device="cuda")
    elif op == "append":
        kv = _keys(g, (b, c["new"], 2 * h, d), dt)  # the key and value heads of one projection's output
        s["k_new"], s["v_new"] = kv[:, :, :h], kv[:, :, h:]
        s["new_len"] = _ints(new)
    elif op == "select":
        s["idx"] = torch.empty((b * h, c["k"]), dtype=torch.int32, device="cuda")
    elif op == "fork":
        s["parent"], s["keep"] = _ints(parent), _ints(keep)
        s["done"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        s["moved"] = torch.empty(pool, dtype=torch.int32, device="cuda")
    if own:
        from sparse_long_context_gb300 import ops
        s["desc"] = ops.make_desc(b, c.get("hq", h), h, d, page, c["cap"], dt)
        s["cache"] = ops.PagedCache(s["desc"], s["k_pages"], s["v_pages"], kmin=s["kmin"], kmax=s["kmax"])
        s["cache"].load(s["table"], s["ctx"])
        s["saved"] = s["cache"].meta.clone()
        if op in ("attend", "select", "fork", "compact"):
            make = {"attend": ops.paged_attend_workspace, "select": ops.paged_select_workspace,
                    "fork": ops.paged_fork_workspace, "compact": ops.paged_compact_workspace}[op]
            s["workspace"] = make(s["desc"], s["cache"])
    return s


# ------------------------------------------------------------------- one pass

def run(s):
    return {"attend": _attend, "append": _append, "select": _select, "fork": _fork, "compact": _compact}[s["case"]["op"]](s)


def _attend(s):
    c = s["case"]
    if own:
        from sparse_long_context_gb300 import ops
        ops.paged_decode_attend(s["desc"], s["cache"], s["q"], page_idx=s["lists"], sink=s["sink"], out=s["out"],
                                lse=s["lse"], workspace=s["workspace"])
        return [s["out"], s["lse"]]
    b, h, d, page = c["batch"], c["hkv"], c["d"], c["page"]
    q = s["q"].view(b, h, -1, d).float() / math.sqrt(d)
    rows = torch.arange(page, device="cuda")
    if s["lists"] is None:
        at = s["table"].clamp(min=0).long()                                     # [b, mp]
        k = s["k_pages"][at].permute(0, 2, 1, 3, 4).reshape(b, h, -1, d).float()
        v = s["v_pages"][at].permute(0, 2, 1, 3, 4).reshape(b, h, -1, d).float()
        dead = (torch.arange(k.shape[2], device="cuda") >= s["ctx"][:, None])[:, None, None]
    else:
        pg = s["lists"].view(b, h, -1).long()
        at = torch.gather(s["table"].long()[:, None].expand(-1, h, -1), 2, pg.clamp(min=0)).clamp(min=0)
        head = torch.arange(h, device="cuda")[:, None]
        k = s["k_pages"][at, head].reshape(b, h, -1, d).float()
        v = s["v_pages"][at, head].reshape(b, h, -1, d).float()
        pos = pg[..., None] * page + rows
        dead = ((pg[..., None] < 0) | (pos >= s["ctx"].view(b, 1, 1, 1))).reshape(b, h, 1, -1)
        v = v.masked_fill(dead.transpose(2, 3), 0.0)
    x = torch.matmul(q, k.transpose(2, 3)).masked_fill_(dead, -math.inf)
    del k
    top = x.amax(-1, keepdim=True)
    if s["sink"] is not None:
        top = torch.maximum(top, s["sink"].view(1, h, -1, 1))
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(s["sink"].view(1, h, -1, 1) - top)
    return [torch.matmul(p / total, v).view(b, -1, d).to(s["q"].dtype), (top + total.log()).view(b, -1)]


def _append(s):
    c = s["case"]
    if own:
        from sparse_long_context_gb300 import ops
        s["cache"].meta.copy_(s["saved"])
        ops.paged_append(s["desc"], s["cache"], s["k_new"], s["v_new"], new_len=s["new_len"])
        return _state(s, s["cache"].ctx_len, s["cache"].table, s["cache"].refs)
    b, page, mp, pool = c["batch"], c["page"], c["cap"] // c["page"], s["refs"].shape[0]
    end = s["ctx"] + s["new_len"]
    had, need = (s["ctx"] + page - 1) // page, (end + page - 1) // page
    first = torch.cumsum(need - had, 0) - (need - had)
    free = torch.sort((s["refs"] != 0).to(torch.int8), stable=True).indices     # free pages first, in their order
    l = torch.arange(mp, device="cuda")
    fresh = (l >= had[:, None]) & (l < need[:, None])
    table = torch.where(fresh, free[(first[:, None] + l - had[:, None]).clamp(0, pool - 1)], s["table"]).to(torch.int32)
    refs = torch.bincount(table[table >= 0].long(), minlength=pool).to(torch.int32)
    seq, t = (torch.arange(c["new"], device="cuda") < s["new_len"][:, None]).nonzero(as_tuple=True)
    pos = s["ctx"].long()[seq] + t
    phys = table[seq, pos // page].long()
    s["k_pages"][phys, :, pos % page] = s["k_new"][seq, t]
    s["v_pages"][phys, :, pos % page] = s["v_new"][seq, t]
    if c["summaries"]:
        seq, lp = ((l >= (s["ctx"] // page)[:, None]) & (l < need[:, None])).nonzero(as_tuple=True)
        phys = table[seq, lp].long()
        off = (lp[:, None] * page + torch.arange(page, device="cuda") >= end[seq][:, None])[:, None, :, None]
        x = s["k_pages"][phys].float()
        s["kmin"][phys] = x.masked_fill(off, math.inf).amin(2).to(s["kmin"].dtype)
        s["kmax"][phys] = x.masked_fill(off, -math.inf).amax(2).to(s["kmin"].dtype)
    return _state(s, end, table, refs)


def _state(s, ctx, table, refs):
    out = {"k": s["k_pages"], "v": s["v_pages"], "ctx": ctx, "table": table, "refs": refs}
    if s["kmin"] is not None:
        out |= {"kmin": s["kmin"], "kmax": s["kmax"]}
    return out


def _select(s):
    c = s["case"]
    if own:
        from sparse_long_context_gb300 import ops
        ops.paged_select_pages(s["desc"], s["cache"], s["q"], c["k"], n_sink_pages=c["first"], n_local_tokens=c["last"],
                               out=s["idx"], workspace=s["workspace"])
        return s["idx"]
    b, h, d, page, k = c["batch"], c["hkv"], c["d"], c["page"], c["k"]
    at = s["table"].clamp(min=0).long()
    low, high = (s[n][at].permute(0, 2, 3, 1).float() for n in ("kmin", "kmax"))  # [b, h, d, mp]
    q = s["q"].view(b, h, -1, d).float()
    score = (torch.matmul(q.clamp(min=0), high) + torch.matmul(q.clamp(max=0), low)).amax(2)
    n = ((s["ctx"] + page - 1) // page).view(b, 1, 1)
    i = torch.arange(c["cap"] // page, device="cuda")
    first_last = torch.where(torch.tensor(c["last"] > 0, device="cuda"), (s["ctx"] - c["last"]).clamp(min=0) // page, n.view(-1))
    score = score.masked_fill((i < c["first"]) | (i >= first_last.view(b, 1, 1)), math.inf).masked_fill(i >= n, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k]
    order = torch.where(order >= n, c["cap"], order).sort(-1).values
    return torch.where(order < c["cap"], order, -1).to(torch.int32).view(b * h, k)


def _fork(s):
    c = s["case"]
    if own:
        from sparse_long_context_gb300 import ops
        s["cache"].meta.copy_(s["saved"])
        ops.paged_fork(s["desc"], s["cache"], s["parent"], keep_len=s["keep"], done=s["done"], workspace=s["workspace"])
        return _state(s, s["cache"].ctx_len, s["cache"].table, s["cache"].refs) | {"done": s["done"]}
    b, page, mp, pool = c["batch"], c["page"], c["cap"] // c["page"], s["refs"].shape[0]
    i, l = torch.arange(b, device="cuda"), torch.arange(mp, device="cuda")
    parent = s["parent"].long()
    length = torch.minimum(s["ctx"][parent], s["keep"])
    same = (parent == i) & (length == s["ctx"])
    whole, part = (length // page).long(), (length % page).long()
    rows = s["table"][parent]
    held = (l < whole[:, None]) | (same & (part > 0))[:, None] & (l == whole[:, None])
    holders = torch.bincount(rows[held].long(), minlength=pool)
    # a page that a sequence's cut leaves partial: its lowest user keeps it if nobody holds it whole, the others copy it
    cut = ~same & (part > 0)
    source = torch.where(cut, torch.gather(rows, 1, whole.clamp(max=mp - 1)[:, None])[:, 0].long(), pool)
    lowest = torch.full((pool + 1,), b, device="cuda").scatter_reduce(0, source, i, "amin")
    keeps = cut & (lowest[source] == i) & (torch.cat([holders, holders.new_ones(1)])[source] == 0)
    copies = cut & ~keeps
    free = torch.sort((s["refs"] != 0).to(torch.int8), stable=True).indices
    to = torch.where(keeps, source, free[(torch.cumsum(copies, 0) - copies.long()).clamp(max=pool - 1)])
    table = torch.where(held, rows, torch.where(cut[:, None] & (l == whole[:, None]), to[:, None], -1)).to(torch.int32)
    refs = torch.bincount(table[table >= 0].long(), minlength=pool).to(torch.int32)
    which = copies.nonzero()[:, 0]
    mine = (torch.arange(page, device="cuda") < part[which, None])[:, None, :, None]
    for pages in (s["k_pages"], s["v_pages"]):
        pages[to[which]] = torch.where(mine, pages[source[which]], pages[to[which]])
    if c["summaries"]:
        which = cut.nonzero()[:, 0]
        off = (torch.arange(page, device="cuda") >= part[which, None])[:, None, :, None]
        x = s["k_pages"][to[which]].float()
        s["kmin"][to[which]] = x.masked_fill(off, math.inf).amin(2).to(s["kmin"].dtype)
        s["kmax"][to[which]] = x.masked_fill(off, -math.inf).amax(2).to(s["kmin"].dtype)
    return _state(s, length, table, refs) | {"done": torch.ones_like(s["done"])}


def _compact(s):
    if own:
        from sparse_long_context_gb300 import ops
        s["cache"].meta.copy_(s["saved"])
        ops.paged_compact(s["desc"], s["cache"], moved=s["moved"], workspace=s["workspace"])
        return _state(s, s["cache"].ctx_len, s["cache"].table, s["cache"].refs) | {"moved": s["moved"]}
    used = s["refs"] > 0
    count, i = used.sum(), torch.arange(used.shape[0], device="cuda")
    old = (used & (i >= count)).nonzero()[:, 0]
    new = (~used & (i < count)).nonzero()[:, 0]
    moved = torch.where(used, i, -1)
    moved[old] = new
    s["k_pages"][new] = s["k_pages"][old]
    s["v_pages"][new] = s["v_pages"][old]
    if s["kmin"] is not None:
        s["kmin"][new] = s["kmin"][old]
        s["kmax"][new] = s["kmax"][old]
    table = torch.where(s["table"] >= 0, moved[s["table"].clamp(min=0).long()], -1).to(torch.int32)
    refs = torch.bincount(table[table >= 0].long(), minlength=used.shape[0]).to(torch.int32)
    return _state(s, s["ctx"], table, refs) | {"moved": moved.to(torch.int32)}


# ------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, one sequence after the other.  A selection gives whole numbers
    only."""
    c = case
    if c["op"] == "select":
        return None
    s = prepare(c, seed)
    if c["op"] == "attend":
        return _exact_attend(s)
    page = c["page"]
    k, v = s["k_pages"].double(), s["v_pages"].double()
    low, high = (s["kmin"].double(), s["kmax"].double()) if s["kmin"] is not None else (None, None)
    table, free = s["table"].tolist(), [p for p, n in enumerate(s["refs"].tolist()) if n == 0]

    def summed_up(p, n):
        if low is not None:
            low[p], high[p] = k[p, :, :n].amin(1), k[p, :, :n].amax(1)

    if c["op"] == "append":
        for i, (at, n) in enumerate(zip(*_spans(c))):
            begun, all_of = -(-at // page), -(-(at + n) // page)
            table[i][begun:all_of], free = free[:all_of - begun], free[all_of - begun:]
            pos = torch.arange(at, at + n, device="cuda")
            p = torch.tensor(table[i], device="cuda")[pos // page]
            k[p, :, pos % page], v[p, :, pos % page] = s["k_new"][i, :n].double(), s["v_new"][i, :n].double()
            if low is not None:
                full = torch.tensor(table[i][at // page:(at + n) // page], device="cuda").long()
                low[full], high[full] = k[full].amin(2), k[full].amax(2)
                if (at + n) % page:
                    summed_up(table[i][(at + n) // page], (at + n) % page)
    elif c["op"] == "fork":
        _, keep, parent, changed = _fork_plan(c)
        whole = {p for i in range(c["batch"]) for p in table[parent[i]][:keep[i] // page if changed[i] else -(-keep[i] // page)]}
        for i in range(c["batch"]):
            n = keep[i] % page
            if changed[i] and n:
                p = to = table[parent[i]][keep[i] // page]
                if p in whole:
                    to = free.pop(0)
                    k[to, :, :n], v[to, :, :n] = k[p, :, :n], v[p, :, :n]
                whole.add(p)
                summed_up(to, n)
    else:
        used = sorted(p for p, n in enumerate(s["refs"].tolist()) if n)
        late = [p for p in used if p >= len(used)]
        for p, to in zip(late, [p for p in free if p < len(used)]):
            k[to], v[to] = k[p], v[p]
            if low is not None:
                low[to], high[to] = low[p], high[p]
    none = {"k": k, "v": v, "ctx": None, "table": None, "refs": None}
    none |= {"kmin": low, "kmax": high} if low is not None else {}
    return none | ({"done": None} if c["op"] == "fork" else {"moved": None} if c["op"] == "compact" else {})


def _exact_attend(s):
    c = s["case"]
    b, h, d, page = c["batch"], c["hkv"], c["d"], c["page"]
    g = c["hq"] // h
    out = torch.zeros((b, c["hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((b, c["hq"]), dtype=torch.float64, device="cuda")
    for i, n in enumerate(_lens(c)):
        mine = s["table"][i, :-(-n // page)].long()
        for j in range(h):
            k, v = (s[name][mine, j].reshape(-1, d)[:n].double() for name in ("k_pages", "v_pages"))
            if s["lists"] is not None:
                p = s["lists"][i * h + j].long()
                t = (p[p >= 0][:, None] * page + torch.arange(page, device="cuda")).reshape(-1)
                k, v = k[t[t < n]], v[t[t < n]]
            x = s["q"][i, j * g:(j + 1) * g].double() @ k.T / math.sqrt(d)
            if s["sink"] is not None:
                x = torch.cat([x, s["sink"][j * g:(j + 1) * g, None].double()], 1)
            lse[i, j * g:(j + 1) * g] = torch.logsumexp(x, 1)
            out[i, j * g:(j + 1) * g] = torch.softmax(x, 1)[:, :n if s["lists"] is None else k.shape[0]] @ v
    return [out, lse]
