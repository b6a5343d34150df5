"""Cases of the operators around the 8-bit K/V cache: the per-head norm and rotation of queries and
keys, the append of tokens to the cache, the decode attention over it, and the eviction that keeps
it within a budget.  With `own` false run() computes each in elementary torch operations in 32
bits; with `own` true it makes the calls a program makes of sparse_long_context_gb300.ops.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
LEVELS = {"int8": 127.0, "e4m3": 448.0}  # largest code value of each format
GOLDEN = 0.6180339887498949               # multiples of it, modulo one, spread evenly


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of 32 sequences deep in a long context: latency counts
        dict(name="rope_decode", op="rope", tokens=32, hq=12, hkv=2, d=128, rot=128, inter=False, norm=True,
             dtype="bf16", theta=1e6, far=65536),
        # the projected queries and keys of a 32k prompt
        dict(name="rope_prompt", op="rope", tokens=32768, hq=28, hkv=4, d=128, rot=128, inter=False, norm=True,
             dtype="bf16", theta=1e6, far=32768),
        # fp32, interleaved pairs, half of the channels rotated, positions near a million, odd count
        dict(name="rope_f32_far", op="rope", tokens=4099, hq=4, hkv=1, d=64, rot=32, inter=True, norm=True,
             dtype="f32", theta=1e4, far=1 << 20),
        # one decoded token for each of 32 sequences, page summaries and weight sums kept current
        dict(name="append_decode", op="append", batch=32, hkv=2, d=128, cap=65536, block=64, fmt="int8", new=1,
             page=16, mass=True),
        # four prompts of up to 32k tokens into an empty cache
        dict(name="append_prompt", op="append", batch=4, hkv=8, d=128, cap=32768, block=64, fmt="e4m3", new=32768,
             page=16, mass=False),
        # a chunk of a prompt fed in pieces, small blocks, odd lengths, starting inside a block
        dict(name="append_chunk", op="append", batch=5, hkv=8, d=64, cap=4096, block=16, fmt="int8", new=1021,
             page=0, mass=False),
        # dense decode of 32 ragged contexts of up to 64k tokens
        dict(name="attend_dense_64k", op="attend", batch=32, hq=12, hkv=2, d=128, cap=65536, block=64, fmt="int8",
             low=49000, pages=0, page=16, sink=False, mass=False),
        # the sparse step: 128 pages of 16 tokens per KV head out of 64k tokens
        dict(name="attend_pages_64k", op="attend", batch=32, hq=12, hkv=2, d=128, cap=65536, block=64, fmt="e4m3",
             low=60000, pages=128, page=16, sink=False, mass=False),
        # one short conversation: latency counts
        dict(name="attend_short", op="attend", batch=1, hq=28, hkv=4, d=128, cap=1024, block=32, fmt="int8",
             low=1000, pages=0, page=16, sink=False, mass=False),
        # 128k contexts with a sink logit, summing every block's weight for a later eviction
        dict(name="attend_mass_128k", op="attend", batch=4, hq=64, hkv=8, d=64, cap=131072, block=64, fmt="e4m3",
             low=100000, pages=0, page=16, sink=True, mass=True),
        # prompts of 32k tokens cut to a 16k budget in a smaller cache
        dict(name="evict_prompt", op="evict", batch=8, hkv=4, d=128, cap=32768, block=64, fmt="int8", keep=256,
             sinks=1, recent=16, low=32000, page=0),
        # small caches, some of them still within the budget, page summaries moved along
        dict(name="evict_small", op="evict", batch=2, hkv=8, d=64, cap=4096, block=16, fmt="e4m3", keep=127, sinks=2,
             recent=5, low=1500, page=16),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "evict"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 5, 6, 7, 8])
    d = rng.choice([64, 128])
    fmt = rng.choice(["int8", "e4m3"])
    block = rng.choice([16, 32, 64, 128])
    if op == "rope":
        most = 32768 * 32 * 128 // ((group + 1) * hkv * d)
        return dict(op=op, tokens=_log(rng, 1, min(most, 40000)), hq=group * hkv, hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4]), inter=rng.random() < 0.5, norm=rng.random() < 0.8,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), theta=rng.choice([1e4, 5e5, 1e6]),
                    far=_log(rng, 64, 1 << 20))
    batch = _log(rng, 1, 32)
    most = max(512, min(131072, (1 << 27) // (batch * hkv * d)))
    cap = -(-_log(rng, 256, most) // 128) * 128
    if op == "append":
        new = 1 if rng.random() < 0.4 else _log(rng, 2, cap // 2)
        return dict(op=op, batch=batch, hkv=hkv, d=d, cap=cap, block=block, fmt=fmt, new=new,
                    page=rng.choice([0, 16, 64]), mass=rng.random() < 0.5)
    if op == "attend":
        page = rng.choice([16, 32, 64])
        pages = rng.choice([0, 0, min(cap // page, _log(rng, 4, 512))])
        return dict(op=op, batch=batch, hq=group * hkv, hkv=hkv, d=d, cap=cap, block=block, fmt=fmt,
                    low=_log(rng, 1, cap), pages=pages, page=page, sink=rng.random() < 0.4,
                    mass=pages == 0 and rng.random() < 0.4)
    keep = _log(rng, 8, max(8, cap // block - 1)) if cap // block > 9 else 1
    return dict(op=op, batch=batch, hkv=hkv, d=d, cap=cap, block=block, fmt=fmt, keep=keep,
                sinks=rng.choice([0, 1, 2]) if keep >= 8 else 0, recent=rng.choice([0, 1, 4]) if keep >= 8 else 0,
                low=_log(rng, 1, cap), page=rng.choice([0, 16]))


def work(case):
    c, op = case, case["op"]
    if op == "rope":
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["tokens"] * (c["hq"] + c["hkv"]) * c["d"]
        return {"bytes": 2 * n * e + 4 * c["tokens"], "flops": 8 * n}
    rows = c["batch"] * c["hkv"]
    if op == "append":
        start, new = _spans(c)
        n = sum(new) * c["hkv"]
        full = sum((s + k) // c["block"] - s // c["block"] for s, k in zip(start, new)) * c["hkv"]
        b = n * c["d"] * 4 + full * c["block"] * c["d"] * 2 + full * 8
        b += sum(s % c["block"] for s, k in zip(start, new) if (s + k) // c["block"] > s // c["block"]) * c["hkv"] * 4 * c["d"]
        b += sum((s + k) % c["block"] if (s + k) // c["block"] > s // c["block"] else k
                 for s, k in zip(start, new)) * c["hkv"] * 4 * c["d"]
        if c["page"]:
            b += sum((s + k - 1) // c["page"] - s // c["page"] + 1 for s, k in zip(start, new)) * c["hkv"] * 4 * c["d"]
        return {"bytes": b, "flops": 4 * n * c["d"]}
    lens = _lens(c)
    if op == "attend":
        q = c["batch"] * c["hq"] * c["d"] * 2
        kept = sum(min(n, c["pages"] * c["page"]) if c["pages"] else n for n in lens)
        tail = sum(n % c["block"] for n in lens) if not c["pages"] else 0
        b = kept * c["hkv"] * 2 * c["d"] + tail * c["hkv"] * 2 * c["d"] + 2 * q + c["batch"] * c["hq"] * 4
        b += kept // (c["page"] if c["pages"] else c["block"]) * c["hkv"] * 8
        b += sum(n // c["block"] for n in lens) * c["hkv"] * 8 if c["mass"] else 0
        return {"bytes": b, "flops": 4 * kept * c["hq"] * c["d"]}
    kept = sum(min(n // c["block"], c["keep"]) for n in lens) * c["hkv"]
    b = kept * (4 * c["block"] * c["d"] + 16 + 8) + sum(n // c["block"] for n in lens) * c["hkv"] * 4
    b += sum(n % c["block"] for n in lens) * c["hkv"] * 8 * c["d"]
    b += kept * (c["block"] // c["page"]) * 8 * c["d"] if c["page"] else 0
    return {"bytes": b, "flops": rows * c["cap"] // c["block"]}


# ------------------------------------------------------------------- the inputs

def _lens(c):
    """Context lengths between `low` and the capacity: the first at `low`, the last of several at the capacity, the
    others anywhere between."""
    low, high, b = c["low"], c["cap"], c["batch"]
    return [high if 0 < i == b - 1 else low + int((high - low) * (i * GOLDEN % 1.0)) for i in range(b)]


def _spans(c):
    """Start and count of the new tokens of each sequence.  Single tokens go anywhere; of chunks, the even sequences
    start on a block border and end anywhere, the odd ones start anywhere and end on a border (so that a pass
    can be repeated on the same tail buffer)."""
    start, new = [], []
    for i in range(c["batch"]):
        room = c["cap"] - c["new"]
        s = int(room * ((i + 1) * GOLDEN % 1.0))
        if c["new"] == 1:
            n = 1
            s = s // c["block"] * c["block"] + c["block"] - 1 if i % 4 == 1 and s // c["block"] * c["block"] + c["block"] <= c["cap"] else s
        elif i % 2 == 0:
            s = s // c["block"] * c["block"]
            n = c["new"] - (i % 5) * c["new"] // 16
        else:
            end = (s + c["new"]) // c["block"] * c["block"]
            n = end - s
            if n < 1:
                s, n = s // c["block"] * c["block"], c["new"]
        start.append(s)
        new.append(n)
    return start, new


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _keys(g, shape, dtype=F32):
    """Key-like values: channels of very different size, as projected keys have."""
    gain = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)


def _stored(g, rows, cap, d, block, fmt, keys):
    """A cache as an earlier append left it: codes and scales of normal values with a gain of their own for each block."""
    top = LEVELS[fmt]
    codes = torch.empty((rows, cap, d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, cap // block), device="cuda")
    for r in range(0, rows, 8):  # a few rows at a time
        n = min(8, rows - r)
        x = _keys(g, (n, cap, d), BF16) if keys else torch.randn((n, cap, d), generator=g, device="cuda").to(BF16)
        x = x.view(n, cap // block, block * d).float()
        amax = x.abs().amax(-1)
        y = x * top / amax[..., None]
        y = torch.round(y).to(torch.int8).view(torch.uint8) if fmt == "int8" else y.to(torch.float8_e4m3fn).view(torch.uint8)
        codes[r:r + n] = y.view(n, cap, d)
        scales[r:r + n] = amax / top
    return codes, scales


def prepare(case, seed):
    c, g = case, torch.Generator("cuda")
    g.manual_seed(seed * 7919 + 17)
    s = {"case": dict(c)}
    if c["op"] == "rope":
        dt = BF16 if c["dtype"] == "bf16" else F32
        wide = c["hq"] + 2 * c["hkv"]
        qkv = _keys(g, (c["tokens"], wide, c["d"])).to(dt)  # one projection's output: q, k and v heads
        s["q"], s["k"] = qkv[:, :c["hq"]], qkv[:, c["hq"]:c["hq"] + c["hkv"]]
        s["positions"] = torch.randint(0, c["far"], (c["tokens"],), generator=g, device="cuda").to(torch.int32) \
            if c["tokens"] < 4096 or c["far"] > c["tokens"] else torch.arange(c["tokens"], dtype=torch.int32, device="cuda")
        s["wq"] = (1 + 0.2 * torch.randn(c["d"], generator=g, device="cuda")).to(dt) if c["norm"] else None
        s["wk"] = (1 + 0.2 * torch.randn(c["d"], generator=g, device="cuda")).to(dt) if c["norm"] else None
        s["q_out"] = torch.empty((c["tokens"], c["hq"], c["d"]), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((c["tokens"], c["hkv"], c["d"]), dtype=dt, device="cuda")
        if own:
            from sparse_long_context_gb300 import ops
            s["rope"] = ops.make_rope(c["hq"], c["hkv"], c["d"], dt, rotary_dim=c["rot"], theta=c["theta"],
                                      interleaved=c["inter"], eps=1e-6)
        return s

    b, h, d, cap, block, fmt = c["batch"], c["hkv"], c["d"], c["cap"], c["block"], c["fmt"]
    page = c["page"] or 16
    nblk = cap // block
    if c["op"] == "append":
        s["k_codes"] = torch.zeros((b, h, cap, d), dtype=torch.uint8, device="cuda")
        s["v_codes"] = torch.zeros_like(s["k_codes"])
        s["k_scales"] = torch.zeros((b, h, nblk), device="cuda")
        s["v_scales"] = torch.zeros_like(s["k_scales"])
        start, new = _spans(c)
        kv = _keys(g, (b, c["new"], 2 * h, d), BF16)  # the key and value heads of one projection's output
        s["k_new"], s["v_new"] = kv[:, :, :h], kv[:, :, h:]
        s["ctx"], s["new_len"] = _ints(start), _ints(new)
        s["ctx_out"] = torch.zeros(b, dtype=torch.int32, device="cuda")
        s["mass"] = torch.rand((b, h, nblk), generator=g, device="cuda") if c["mass"] else None
        if c["page"]:
            s["kmin"] = (-torch.rand((b, h, cap // page, d), generator=g, device="cuda")).to(BF16)
            s["kmax"] = torch.rand((b, h, cap // page, d), generator=g, device="cuda").to(BF16)
    else:
        s["lens"] = _lens(c)
        s["ctx"] = _ints(s["lens"])
        k, ks = _stored(g, b * h, cap, d, block, fmt, True)
        v, vs = _stored(g, b * h, cap, d, block, fmt, False)
        s["k_codes"], s["v_codes"] = k.view(b, h, cap, d), v.view(b, h, cap, d)
        s["k_scales"], s["v_scales"] = ks.view(b, h, nblk), vs.view(b, h, nblk)
    s["k_tail"] = _keys(g, (b, h, block, d), BF16)
    s["v_tail"] = torch.randn((b, h, block, d), generator=g, device="cuda").to(BF16)

    if c["op"] == "attend":
        hq = c["hq"]
        # a query looks for a few of its row's tokens and has a random part
        at = torch.randint(0, max(1, c["low"] // block) * block if c["low"] >= block else 1, (b, h, 4, 1), generator=g, device="cuda")
        found = _values(torch.gather(s["k_codes"], 2, at.expand(-1, -1, -1, d)), fmt) * torch.gather(s["k_scales"], 2, at[..., 0] // block)[..., None]
        q = torch.randn((b, h, hq // h, d), generator=g, device="cuda") + found.sum(2, keepdim=True) * 0.5
        s["q"] = q.view(b, hq, d).to(BF16)
        s["sink"] = torch.randn(hq, generator=g, device="cuda") if c["sink"] else None
        s["pages"] = None
        if c["pages"]:  # as a selection leaves it: first page, newest page, the others anywhere; ascending, -1 padded
            np_row = (s["ctx"].view(b, 1, 1) + page - 1) // page
            i = torch.arange(cap // page, device="cuda")
            score = torch.rand((b, h, cap // page), generator=g, device="cuda")
            score = torch.where((i == 0) | (i == np_row - 1), torch.full_like(score, 2.0), score).masked_fill(i >= np_row, -1.0)
            top = torch.topk(score, c["pages"], dim=-1)
            idx = torch.where(top.values < 0, cap, top.indices).sort(-1).values
            s["pages"] = torch.where(idx >= cap, -1, idx).to(torch.int32).view(b * h, c["pages"]).contiguous()
        if c["mass"]:
            s["mass"] = 10 * torch.rand((b, h, nblk), generator=g, device="cuda")
            s["mass_out"] = torch.zeros_like(s["mass"])
        s["out"] = torch.empty((b, hq, d), dtype=BF16, device="cuda")
        s["lse"] = torch.empty((b, hq), device="cuda")
    if c["op"] == "evict":
        keep = c["keep"]
        s["mass"] = torch.rand((b, h, nblk), generator=g, device="cuda").pow(4) * 50  # a few blocks hold most of the weight
        cap2 = (keep + 1) * block
        s["to"] = {"k_codes": torch.zeros((b, h, cap2, d), dtype=torch.uint8, device="cuda"),
                   "v_codes": torch.zeros((b, h, cap2, d), dtype=torch.uint8, device="cuda"),
                   "k_scales": torch.zeros((b, h, keep + 1), device="cuda"),
                   "v_scales": torch.zeros((b, h, keep + 1), device="cuda"),
                   "k_tail": torch.zeros_like(s["k_tail"]), "v_tail": torch.zeros_like(s["v_tail"]),
                   "mass": torch.zeros((b, h, keep + 1), device="cuda")}
        s["ctx_out"] = torch.zeros(b, dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros((b * h, keep), dtype=torch.int32, device="cuda")
        if c["page"]:
            s["kmin"] = -torch.rand((b, h, cap // page, d), generator=g, device="cuda").to(BF16)
            s["kmax"] = torch.rand((b, h, cap // page, d), generator=g, device="cuda").to(BF16)
            s["to"]["kmin"] = torch.zeros((b, h, cap2 // page, d), dtype=BF16, device="cuda")
            s["to"]["kmax"] = torch.zeros_like(s["to"]["kmin"])
    if own:
        from sparse_long_context_gb300 import ops
        s["desc"] = ops.make_desc(b, c.get("hq", h), h, d, page, cap, BF16)
        names = ("k_codes", "v_codes", "k_scales", "v_scales", "k_tail", "v_tail")
        s["cache"] = ops.Kv8Cache(s["desc"], fmt, block, *(s[n] for n in names))
        if c["op"] == "attend":
            s["workspace"] = ops.kv8_attend_workspace(s["desc"], s["cache"], mass=c["mass"])
        if c["op"] == "evict":
            s["desc2"] = ops.make_desc(b, h, h, d, page, (keep + 1) * block, BF16)
            s["cache2"] = ops.Kv8Cache(s["desc2"], fmt, block, *(s["to"][n] for n in names))
    return s


# ------------------------------------------------------------------- one pass

def run(s):
    return {"rope": _rope, "append": _append, "attend": _attend, "evict": _evict}[s["case"]["op"]](s)


def _values(codes, fmt):
    """What stored codes stand for, apart from their block's scale."""
    return codes.view(torch.int8).float() if fmt == "int8" else codes.view(torch.float8_e4m3fn).float()


def _shown(codes, fmt):
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)


def _turned(x, weight, cos, sin, c):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    r, out = c["rot"], x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["inter"] else (x[..., :r // 2], x[..., r // 2:r])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    if c["inter"]:
        out[..., 0:r:2], out[..., 1:r:2] = lo, hi
    else:
        out[..., :r // 2], out[..., r // 2:r] = lo, hi
    return out


def _rope(s):
    c = s["case"]
    if own:
        from sparse_long_context_gb300 import ops
        ops.qk_norm_rope(s["rope"], s["q"], s["k"], s["positions"], q_weight=s["wq"], k_weight=s["wk"],
                         q_out=s["q_out"], k_out=s["k_out"])
        return [s["q_out"], s["k_out"]]
    f = c["theta"] ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
    angle = s["positions"].double()[:, None, None] * f  # 64 bits: far positions times fast frequencies
    cos, sin = angle.cos().float(), angle.sin().float()
    return [_turned(s["q"], s["wq"], cos, sin, c).to(s["q"].dtype), _turned(s["k"], s["wk"], cos, sin, c).to(s["k"].dtype)]


def _quantised(x, fmt):
    """Codes and scales of blocks x [..., block, D]."""
    top = LEVELS[fmt]
    amax = x.abs().amax((-1, -2))
    y = torch.where(amax[..., None, None] > 0, x * top / amax[..., None, None], torch.zeros_like(x))
    codes = torch.round(y).to(torch.int8).view(torch.uint8) if fmt == "int8" else y.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, amax / top


def _append(s):
    c = s["case"]
    if own:
        from sparse_long_context_gb300 import ops
        ops.kv8_append(s["desc"], s["cache"], s["k_new"], s["v_new"], s["ctx"], new_len=s["new_len"],
                       kmin=s.get("kmin"), kmax=s.get("kmax"), mass=s["mass"], ctx_out=s["ctx_out"])
        return _appended(s)
    b, h, d, block, fmt = c["batch"], c["hkv"], c["d"], c["block"], c["fmt"]
    end = s["ctx"] + s["new_len"]
    seq = torch.arange(b, device="cuda")
    first = s["ctx"] // block
    blk = first[:, None] + torch.arange(c["new"] // block + 2, device="cuda")  # the blocks that may be touched
    pos = blk[..., None] * block + torch.arange(block, device="cuda")          # [b, blocks, block]
    fresh = (pos >= s["ctx"][:, None, None]) & (pos < end[:, None, None])
    old = pos < s["ctx"][:, None, None]
    done = ((blk + 1) * block <= end[:, None]).nonzero(as_tuple=True)          # blocks that are complete now
    which = (pos - s["ctx"][:, None, None]).clamp(0, c["new"] - 1)
    touched = []
    for new, tail, codes, scales in ((s["k_new"], s["k_tail"], s["k_codes"], s["k_scales"]),
                                     (s["v_new"], s["v_tail"], s["v_codes"], s["v_scales"])):
        x = new[seq[:, None, None], which]                                      # [b, blocks, block, h, d]
        x = torch.where(old[..., None, None], tail.permute(0, 2, 1, 3)[:, None], x)
        x = x.permute(0, 1, 3, 2, 4)                                            # [b, blocks, h, block, d]
        y, sc = _quantised(x[done].float(), fmt)
        codes.view(b, h, -1, block, d)[done[0], :, blk[done]] = y
        scales[done[0], :, blk[done]] = sc
        touched.append(x)
    if s["mass"] is not None:
        s["mass"][done[0], :, blk[done]] = 0.0
    # the newest, partial block stays in the tail buffer
    last = (end // block - first).long().clamp(max=blk.shape[1] - 1)
    keep = (fresh[seq, last] & (blk[seq, last] == end // block)[:, None])[:, None, :, None]
    s["k_tail"].copy_(torch.where(keep, touched[0][seq, last], s["k_tail"]))
    s["v_tail"].copy_(torch.where(keep, touched[1][seq, last], s["v_tail"]))
    if c["page"]:
        page = c["page"]
        pg = (s["ctx"] // page)[:, None] + torch.arange(c["new"] // page + 2, device="cuda")
        pos = pg[..., None] * page + torch.arange(page, device="cuda")
        fresh = (pos >= s["ctx"][:, None, None]) & (pos < end[:, None, None])
        seen = fresh.any(-1).nonzero(as_tuple=True)
        x = s["k_new"][seq[:, None, None], (pos - s["ctx"][:, None, None]).clamp(0, c["new"] - 1)][seen].float()
        m = fresh[seen][..., None, None]
        low = x.masked_fill(~m, math.inf).amin(1)
        high = x.masked_fill(~m, -math.inf).amax(1)
        going = (pg[seen] * page < s["ctx"][seen[0]])[:, None, None]            # the page held tokens before
        was_low, was_high = s["kmin"][seen[0], :, pg[seen]].float(), s["kmax"][seen[0], :, pg[seen]].float()
        s["kmin"][seen[0], :, pg[seen]] = torch.where(going, torch.minimum(low, was_low), low).to(BF16)
        s["kmax"][seen[0], :, pg[seen]] = torch.where(going, torch.maximum(high, was_high), high).to(BF16)
    s["ctx_out"].copy_(end)
    return _appended(s)


def _appended(s):
    fmt = s["case"]["fmt"]
    out = {"k": _shown(s["k_codes"], fmt), "v": _shown(s["v_codes"], fmt), "ks": s["k_scales"], "vs": s["v_scales"],
           "kt": s["k_tail"], "vt": s["v_tail"], "ctx": s["ctx_out"]}
    if s["mass"] is not None:
        out["mass"] = s["mass"]
    if s["case"]["page"]:
        out |= {"kmin": s["kmin"], "kmax": s["kmax"]}
    return out


def _whole(codes, scales, tail, ctx, fmt, block):
    """The cache's values [b, h, cap, d] in 32 bits: complete blocks from the codes, the newest one from its tail."""
    b, h, cap, d = codes.shape
    x = _values(codes, fmt).view(b, h, cap // block, block, d) * scales[..., None, None]
    newest = (ctx // block).view(b, 1, 1, 1, 1)
    i = torch.arange(cap // block, device="cuda").view(1, 1, -1, 1, 1)
    return torch.where(i == newest, tail[:, :, None].float(), x).view(b, h, cap, d)


def _attend(s):
    c = s["case"]
    if own:
        from sparse_long_context_gb300 import ops
        ops.kv8_decode_attend(s["desc"], s["cache"], s["q"], s["ctx"], page_idx=s["pages"], sink=s["sink"],
                              mass_in=s.get("mass"), mass_out=s.get("mass_out"), out=s["out"], lse=s["lse"],
                              workspace=s["workspace"])
        return [s["out"], s["lse"]] + ([s["mass_out"]] if c["mass"] else [])
    b, h, d, block = c["batch"], c["hkv"], c["d"], c["block"]
    q = s["q"].view(b, h, -1, d).float() / math.sqrt(d)
    if s["pages"] is None:
        k = _whole(s["k_codes"], s["k_scales"], s["k_tail"], s["ctx"], c["fmt"], block)
        v = _whole(s["v_codes"], s["v_scales"], s["v_tail"], s["ctx"], c["fmt"], block)
        dead = (torch.arange(c["cap"], device="cuda") >= s["ctx"][:, None])[:, None, None]
    else:  # only the listed pages' tokens
        pos = (s["pages"].view(b, h, -1, 1).clamp(min=0) * c["page"] + torch.arange(c["page"], device="cuda")).view(b, h, -1).long()
        k, v = (_listed(s, pos, n) for n in ("k", "v"))
        dead = ((pos >= s["ctx"].view(b, 1, 1)) | (s["pages"].view(b, h, -1, 1) < 0).expand(-1, -1, -1, c["page"]).reshape(b, h, -1))[:, :, None]
    x = torch.matmul(q, k.transpose(2, 3)).masked_fill_(dead, -math.inf)
    del k
    top = x.amax(-1, keepdim=True)
    if s["sink"] is not None:
        top = torch.maximum(top, s["sink"].view(1, h, -1, 1))
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(s["sink"].view(1, h, -1, 1) - top)
    p = p / total
    out = torch.matmul(p, v).view(b, -1, d).to(BF16)
    lse = (top + total.log()).view(b, -1)
    if not c["mass"]:
        return [out, lse]
    each = p.sum(2).view(b, h, -1, block).sum(-1)
    full = torch.arange(c["cap"] // block, device="cuda") < (s["ctx"] // block)[:, None, None]
    return [out, lse, torch.where(full, s["mass"] + each, s["mass_out"])]


def _listed(s, pos, n):
    c = s["case"]
    d, block = c["d"], c["block"]
    wide = pos[..., None].expand(-1, -1, -1, d)
    x = _values(torch.gather(s[n + "_codes"], 2, wide), c["fmt"]) * torch.gather(s[n + "_scales"], 2, pos // block)[..., None]
    tail = torch.gather(s[n + "_tail"], 2, wide % block).float()
    return torch.where((pos // block == (s["ctx"] // block).view(-1, 1, 1))[..., None], tail, x)


def _evict(s):
    c, to = s["case"], s["to"]
    if own:
        from sparse_long_context_gb300 import ops
        ops.kv8_evict(s["desc"], s["cache"], s["ctx"], s["mass"], c["keep"], n_sink_blocks=c["sinks"],
                      n_recent_blocks=c["recent"], dst_desc=s["desc2"], dst=s["cache2"], ctx_out=s["ctx_out"],
                      mass_out=to["mass"], kept_idx=s["kept"], kmin=s.get("kmin"), kmax=s.get("kmax"),
                      kmin_out=to.get("kmin"), kmax_out=to.get("kmax"))
        return _evicted(s)
    b, h, d, block, keep = c["batch"], c["hkv"], c["d"], c["block"], c["keep"]
    n = (s["ctx"] // block).view(b, 1, 1)
    i = torch.arange(c["cap"] // block, device="cuda")
    forced = (i < c["sinks"]) | (i >= n - c["recent"])
    key = s["mass"].masked_fill(forced, math.inf).masked_fill(i >= n, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    order = torch.where(order >= n, c["cap"], order).sort(-1).values
    there = order < c["cap"]
    at = torch.where(there, order, 0)
    for name in ("k_codes", "v_codes"):
        x = torch.gather(s[name].view(b, h, -1, block * d), 2, at[..., None].expand(-1, -1, -1, block * d))
        new = to[name].view(b, h, keep + 1, block * d)
        new[:, :, :keep] = torch.where(there[..., None], x, new[:, :, :keep])
    for name in ("k_scales", "v_scales", "mass"):
        to[name][:, :, :keep] = torch.where(there, torch.gather(s[name], 2, at), to[name][:, :, :keep])
    for name in ("kmin", "kmax") if c["page"] else ():
        w = block // c["page"] * d
        x = torch.gather(s[name].view(b, h, -1, w), 2, at[..., None].expand(-1, -1, -1, w))
        new = to[name].view(b, h, keep + 1, w)
        new[:, :, :keep] = torch.where(there[..., None], x, new[:, :, :keep])
        # the pages that hold the newest, partial block move with it
        rest = torch.arange(block // c["page"], device="cuda") * c["page"] < (s["ctx"] % block).view(b, 1)
        src = (n * (block // c["page"]) + torch.arange(block // c["page"], device="cuda")).clamp(max=c["cap"] // c["page"] - 1)
        dst = torch.minimum(n, torch.tensor(keep, device="cuda")) * (block // c["page"]) + torch.arange(block // c["page"], device="cuda")
        moved = torch.gather(s[name], 2, src[..., None].expand(-1, h, -1, d))
        was = torch.gather(to[name], 2, dst[..., None].expand(-1, h, -1, d))
        to[name].scatter_(2, dst[..., None].expand(-1, h, -1, d), torch.where(rest[:, None, :, None], moved, was))
    part = (torch.arange(block, device="cuda") < (s["ctx"] % block)[:, None])[:, None, :, None]
    for name in ("k_tail", "v_tail"):
        to[name].copy_(torch.where(part, s[name], to[name]))
    s["kept"].copy_(torch.where(there, order, -1).view(b * h, keep))
    s["ctx_out"].copy_(torch.minimum(s["ctx"] // block, torch.tensor(keep, device="cuda")) * block + s["ctx"] % block)
    return _evicted(s)


def _evicted(s):
    c, to = s["case"], s["to"]
    out = {n: to[n] for n in ("k_scales", "v_scales", "k_tail", "v_tail", "mass")}
    out |= {"k": _shown(to["k_codes"], c["fmt"]), "v": _shown(to["v_codes"], c["fmt"]), "ctx": s["ctx_out"], "kept": s["kept"]}
    if c["page"]:
        out |= {"kmin": to["kmin"], "kmax": to["kmax"]}
    return out


# ------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, one head or sequence after the other."""
    c = case
    s = prepare(c, seed)
    if c["op"] == "rope":
        i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
        angle = torch.outer(s["positions"].to(torch.float64), torch.exp(-2 * i / c["rot"] * math.log(c["theta"])))
        turn = torch.polar(torch.ones_like(angle), angle)
        outs = []
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            y = x.to(torch.float64)
            for head in range(y.shape[1]):
                z = y[:, head]
                if w is not None:
                    z = z / torch.sqrt((z * z).sum(1, keepdim=True) / c["d"] + 1e-6) * w.to(torch.float64)
                first = torch.arange(0, c["rot"], 2, device="cuda") if c["inter"] else torch.arange(c["rot"] // 2, device="cuda")
                second = first + (1 if c["inter"] else c["rot"] // 2)
                pair = torch.complex(z[:, first], z[:, second]) * turn
                z = z.clone()
                z[:, first], z[:, second] = pair.real, pair.imag
                y[:, head] = z
            outs.append(y)
        return outs
    if c["op"] == "append":
        return _exact_append(s)
    if c["op"] == "attend":
        return _exact_attend(s)
    return _exact_evict(s)


def _exact_append(s):
    c = s["case"]
    block, top = c["block"], LEVELS[c["fmt"]]
    scales = {"k": s["k_scales"].double(), "v": s["v_scales"].double()}
    start, new = s["ctx"].tolist(), s["new_len"].tolist()
    for b in range(c["batch"]):
        for n in ("k", "v"):
            head = start[b] // block * block
            x = torch.cat([s[n + "_tail"][b].transpose(0, 1)[:start[b] - head], s[n + "_new"][b, :new[b]]]).double()
            full = x.shape[0] // block
            if full:
                biggest = x[:full * block].reshape(full, block, c["hkv"], c["d"]).abs().amax((1, 3))
                scales[n][b, :, head // block:head // block + full] = (biggest / top).T
    none = {"k": None, "v": None, "kt": None, "vt": None, "ctx": None, "mass": None, "kmin": None, "kmax": None}
    return none | {"ks": scales["k"], "vs": scales["v"]}


def _exact_attend(s):
    c = s["case"]
    b, h, d, block = c["batch"], c["hkv"], c["d"], c["block"]
    g = c["hq"] // h
    out = torch.zeros((b, c["hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((b, c["hq"]), dtype=torch.float64, device="cuda")
    mass = s["mass_out"].double() if c["mass"] else None
    for i in range(b):
        n = s["lens"][i]
        full = n // block
        for j in range(h):
            kv = []
            for name in ("k", "v"):
                x = _values(s[name + "_codes"][i, j, :full * block], c["fmt"]).double()
                x = x * s[name + "_scales"][i, j, :full].double().repeat_interleave(block)[:, None]
                kv.append(torch.cat([x, s[name + "_tail"][i, j, :n - full * block].double()]))
            if s["pages"] is not None:
                p = s["pages"][i * h + j].long()
                t = (p[p >= 0][:, None] * c["page"] + torch.arange(c["page"], device="cuda")).reshape(-1)
                t = t[t < n]
                kv = [x[t] for x in kv]
            x = s["q"][i, j * g:(j + 1) * g].double() @ kv[0].T / math.sqrt(d)
            if s["sink"] is not None:
                x = torch.cat([x, s["sink"][j * g:(j + 1) * g, None].double()], 1)
            lse[i, j * g:(j + 1) * g] = torch.logsumexp(x, 1)
            p = torch.softmax(x, 1)[:, :kv[1].shape[0]]
            out[i, j * g:(j + 1) * g] = p @ kv[1]
            if mass is not None:
                mass[i, j, :full] = s["mass"][i, j, :full].double() + p[:, :full * block].sum(0).view(full, block).sum(1)
    return [out, lse] + ([mass] if c["mass"] else [])


def _exact_evict(s):
    c = s["case"]
    got = {n: s["to"][n].double() for n in ("k_scales", "v_scales", "mass")}
    mass = s["mass"].double().tolist()
    for i in range(c["batch"]):
        n = s["lens"][i] // c["block"]
        for j in range(c["hkv"]):
            must = {x for x in range(n) if x < c["sinks"] or x >= n - c["recent"]}
            others = sorted((x for x in range(n) if x not in must), key=lambda x: (-mass[i][j][x], x))
            kept = sorted(list(must) + others[:c["keep"] - len(must)])
            for name, to in got.items():
                to[i, j, :len(kept)] = s[name][i, j, kept].double()
    return got | {n: None for n in ("k_tail", "v_tail", "k", "v", "ctx", "kept") + (("kmin", "kmax") if c["page"] else ())}
