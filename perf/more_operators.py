"""Measured cases of the paged KV cache: the page step (block tables and slot
maps from request lengths), the rotary write of new rows into the pages, and
attention of new rows over them.

A case names one operator, the requests' lengths (drawn from its own "mix", so
that they are the case's and not the inputs' seed's), heads and page size.  The
plain forms compute in 32 bits (angles in 64) with elementary torch operations
and round once at the end.
"""
import math
import random

import torch

own = False  # True: the library's calls; False: the plain forms

THETA = 10000.0


def listed():
    return [
        # the draft windows of a page batch of 16 ragged requests: each grows by a boundary token and 32 [M] rows
        {"name": "pages-windows", "op": "pages", "R": 16, "rows": 33, "kv_lo": 512, "kv_hi": 2900, "back": 0.0,
         "done": 0.0, "page": 16, "mix": 5},
        # a full serving batch between two steps: tokens appended, rejected suffixes rolled back, requests ended
        {"name": "pages-churn", "op": "pages", "R": 1000, "rows": 1, "kv_lo": 16, "kv_hi": 8192, "back": 0.2,
         "done": 0.1, "page": 16, "mix": 7},
        # prompts of 64 page images, prefilled together
        {"name": "pages-prompts", "op": "pages", "R": 64, "rows": 1537, "kv_lo": 0, "kv_hi": 0, "back": 0.0,
         "done": 0.0, "page": 64, "mix": 8},
        # one AR token of each of 64 requests
        {"name": "write-tokens", "op": "write", "R": 64, "rows": 1, "kv_lo": 256, "kv_hi": 8192, "Hq": 12, "Hkv": 4,
         "d": 128, "page": 16, "layout": "head", "mix": 9},
        # the verify windows of the page batch
        {"name": "write-windows", "op": "write", "R": 16, "rows": 33, "kv_lo": 512, "kv_hi": 2900, "Hq": 12, "Hkv": 4,
         "d": 128, "page": 16, "layout": "head", "mix": 5},
        # five long prompts, pages that keep a token's heads together
        {"name": "write-prompts", "op": "write", "R": 5, "rows": 2731, "kv_lo": 0, "kv_hi": 0, "Hq": 12, "Hkv": 4,
         "d": 128, "page": 64, "layout": "token", "mix": 11},
        # one request, one token: a region's AR step
        {"name": "attn-one-token", "op": "attn", "R": 1, "rows": 1, "chunks": 0, "chunk": 0, "kv_lo": 1097,
         "kv_hi": 1097, "kind": "verify", "Hq": 12, "Hkv": 4, "d": 128, "page": 16, "layout": "head", "mix": 1},
        # AR steps of 64 requests of very different lengths
        {"name": "attn-tokens", "op": "attn", "R": 64, "rows": 1, "chunks": 0, "chunk": 0, "kv_lo": 256,
         "kv_hi": 8192, "kind": "verify", "Hq": 12, "Hkv": 4, "d": 128, "page": 16, "layout": "head", "mix": 9},
        # the draft windows of the page batch: [M] rows that see the whole window
        {"name": "attn-draft-windows", "op": "attn", "R": 16, "rows": 33, "chunks": 0, "chunk": 0, "kv_lo": 545,
         "kv_hi": 2933, "kind": "draft", "Hq": 12, "Hkv": 4, "d": 128, "page": 16, "layout": "head", "mix": 5},
        # a verify window behind one very long context
        {"name": "attn-verify-long", "op": "attn", "R": 1, "rows": 33, "chunks": 0, "chunk": 0, "kv_lo": 131105,
         "kv_hi": 131105, "kind": "verify", "Hq": 12, "Hkv": 4, "d": 128, "page": 64, "layout": "token", "mix": 2},
        # two long prompts prefilled a chunk at a time: this chunk of 2,048 rows is their last one
        {"name": "attn-chunks", "op": "attn", "R": 2, "rows": 0, "chunks": 2, "chunk": 2048, "kv_lo": 8192,
         "kv_hi": 8192, "kind": "verify", "Hq": 12, "Hkv": 4, "d": 128, "page": 16, "layout": "head", "mix": 3},
        # single tokens of 38 requests beside odd chunks of two others, small heads
        {"name": "attn-mixed", "op": "attn", "R": 40, "rows": 1, "chunks": 2, "chunk": 1021, "kv_lo": 1100,
         "kv_hi": 4000, "kind": "verify", "Hq": 8, "Hkv": 2, "d": 64, "page": 32, "layout": "token", "mix": 4},
    ]


def _log_int(rng, lo, hi):
    if hi <= max(lo, 0):
        return lo
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def draw(rng):
    most = [work(c) for c in listed() if c["name"] in ("attn-verify-long", "attn-chunks")]
    while True:
        case = _draw(rng)
        w = work(case)
        if all(w[k] <= max(m[k] for m in most) for k in w):
            return case


def _draw(rng):
    op = rng.choice(["pages", "write", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    mix = rng.randrange(1 << 20)
    if op == "pages":
        R = _log_int(rng, 1, 1000)
        kv_hi = _log_int(rng, 16, 8192)
        rows = _log_int(rng, 1, max(1, 65536 // R)) if rng.random() < 0.5 else rng.randint(1, 33)
        return {"op": op, "R": R, "rows": rows, "kv_lo": rng.randint(0, kv_hi), "kv_hi": kv_hi,
                "back": round(rng.choice([0.0, 0.5 * rng.random()]), 3),
                "done": round(rng.choice([0.0, 0.3 * rng.random()]), 3), "page": page, "mix": mix}
    hkv = rng.randint(1, 4)
    heads = {"Hq": hkv * rng.randint(1, 6), "Hkv": hkv, "d": rng.choice([64, 128]), "page": page,
             "layout": rng.choice(["head", "token"]), "mix": mix}
    if op == "write":
        T = _log_int(rng, 1, 8192)
        R = _log_int(rng, 1, min(T, 64))
        return {"op": op, "R": R, "rows": max(1, T // R), "kv_lo": 0, "kv_hi": _log_int(rng, 16, 8192), **heads}
    chunks = rng.choice([0, 0, 1, 2])
    R = max(chunks, _log_int(rng, 1, 64))
    chunk = _log_int(rng, 34, 1200) if chunks else 0
    rows = 1 if chunks else rng.choice([1, rng.randint(2, 65)])
    kv_hi = _log_int(rng, 1300, 65536 // R if R < 16 else 4096)
    return {"op": op, "R": R, "rows": rows, "chunks": chunks, "chunk": chunk,
            "kv_lo": max(rows, chunk, rng.randint(1, kv_hi)), "kv_hi": kv_hi,
            "kind": rng.choice(["verify", "draft"]) if not chunks else "verify", **heads}


def _lens(case):
    """Each request's (held, start, end): positions held before, and of its rows."""
    rng = random.Random(case["mix"])
    out = []
    for r in range(case["R"]):
        kv = _log_int(rng, case["kv_lo"], case["kv_hi"])
        if case["op"] == "attn":  # kv_len counts the new rows
            n = case["chunk"] if r < case["chunks"] else case["rows"]
            out.append((kv, kv - n, kv))
            continue
        u = rng.random()
        if r and u < case.get("done", 0.0):  # (the first request goes on)
            out.append((kv, 0, 0))
        elif r and u < case.get("done", 0.0) + case.get("back", 0.0):
            kept = max(0, kv - rng.randint(1, 33))
            out.append((kv, kept, kept))
        else:
            out.append((kv, kv, kv + case["rows"]))
    return out


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float32)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    ps, lens = case["page"], _lens(case)
    pages = lambda n: -(-n // ps)
    R = len(lens)
    T = sum(e - s for _, s, e in lens)
    st = {"op": case["op"], "page": ps, "T": T, "lens": lens}
    width = max(pages(max(h, e)) for h, _, e in lens)
    n_pages = sum(pages(max(h, e)) for h, _, e in lens) + 16
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)  # pages in a long run's order
    own_pages = [pages(h) for h, _, _ in lens] if case["op"] == "pages" else [pages(max(h, e)) for h, _, e in lens]
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(width, device="cuda")[None, :] < i32(own_pages)[:, None]
    n_held = sum(own_pages)
    table[held] = order[:n_held]
    cu = [0]
    for _, s, e in lens:
        cu.append(cu[-1] + e - s)
    if case["op"] == "pages":
        st.update(held=i32([x[0] for x in lens]), start=i32([x[1] for x in lens]), end=i32([x[2] for x in lens]),
                  table=table, n_free=i32([n_pages - n_held]))
        st["free"] = torch.cat([order[n_held:], torch.full((n_held,), -1, dtype=torch.int32, device="cuda")])
        return st
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    cache = lambda: normal(n_pages, Hkv, ps, d).bfloat16() if case["layout"] == "head" else \
        normal(n_pages, ps, Hkv, d).bfloat16().transpose(1, 2)
    st["k_cache"], st["v_cache"] = cache(), cache()
    # q, k and v as the fused projection leaves them: head ranges of one row
    qkv = normal(T, Hq + 2 * Hkv, d).bfloat16()
    st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if case["op"] == "write":
        pos = torch.cat([torch.arange(s, e, device="cuda") for _, s, e in lens])
        req = torch.repeat_interleave(torch.arange(R, device="cuda"), i32([e - s for _, s, e in lens]), output_size=T)
        st["pos"] = pos.to(torch.int32)
        st["slots"] = (table[req, pos // ps] * ps + pos % ps).to(torch.int32)
        return st
    st.update(table=table, cu=i32(cu), kv_len=i32([x[2] for x in lens]), kind=case["kind"], scale=d ** -0.5)
    return st


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from self_speculative_block_gb300 import gocr
    if st["op"] == "pages":
        s = gocr.op_page_step(st["held"], st["start"], st["end"], st["table"], st["free"], st["n_free"], st["page"],
                              st["T"])
        return {"table": st["table"], "free": st["free"], "n_free": s.n_free, "held": s.held, "kv_len": s.kv_len,
                "cu": s.cu_rows, "pos": s.pos, "slots": s.slots}
    if st["op"] == "write":
        q = gocr.op_kv_write_paged(st["q"], st["k"], st["v"], st["pos"], st["slots"], st["k_cache"], st["v_cache"],
                                   theta=THETA)
        return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    o, lse = gocr.op_attention_paged(st["q"], st["k_cache"], st["v_cache"], st["table"], st["cu"], st["kv_len"],
                                     kind=gocr.FWD_DRAFT if st["kind"] == "draft" else gocr.FWD_VERIFY,
                                     scale=st["scale"])
    return {"o": o, "lse": lse}


def _run_plain(st):
    return {"pages": _plain_pages, "write": _plain_write, "attn": _plain_attn}[st["op"]](st)


def _plain_pages(st):
    ps, T, table, free = st["page"], st["T"], st["table"], st["free"]
    held, start, end = (st[n].long() for n in ("held", "start", "end"))
    dev, (R, width), n_free = table.device, table.shape, st["n_free"].long()
    have, want = (held + ps - 1) // ps, (end + ps - 1) // ps
    less, need = (have - want).clamp(min=0), (want - have).clamp(min=0)
    # pages that requests give back, onto the stack so that the first lies on top
    at = torch.arange(width, device=dev)[None, :]
    back = (at >= want[:, None]) & (at < have[:, None])
    n_back = less.sum()
    f = (torch.cumsum(less, 0) - less)[:, None] + at - want[:, None]
    free = free.clone()
    to = torch.where(back, n_free + n_back - 1 - f, len(free))
    free = torch.cat([free, free[:1]]).scatter_(0, to.flatten(), table.flatten())[:-1]
    # pages that requests need, from the top of the stack
    total = n_free + n_back
    upto = torch.cumsum(need, 0)
    served = (need == 0) | (upto <= total)
    new = (at >= have[:, None]) & (at < want[:, None]) & served[:, None]
    k = (upto - need)[:, None] + at - have[:, None]
    table = torch.where(new, free[(total - 1 - k).clamp(0, len(free) - 1)], table)
    # the rows' positions and slots
    n = end - start
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(n, 0)])
    req = torch.repeat_interleave(torch.arange(R, device=dev), n, output_size=T)
    pos = torch.arange(T, device=dev) - cu[req] + start[req]
    slots = table[req, pos // ps].long() * ps + pos % ps
    pos, slots = (torch.where(served[req], x, -1) for x in (pos, slots))
    taken = torch.where(served, upto, 0).amax()
    return {"table": table, "free": free, "n_free": (total - taken).to(torch.int32),
            "held": torch.where(served, end, held).to(torch.int32),
            "kv_len": torch.where(served, end, 0).to(torch.int32),
            "cu": cu.to(torch.int32), "pos": pos.to(torch.int32), "slots": slots.to(torch.int32)}


def _plain_write(st):
    ps, d = st["page"], st["q"].shape[2]
    inv = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device=st["q"].device) / d)
    ang = st["pos"].double()[:, None] * inv
    c, s = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]

    def turn(x):
        a, b = x[..., :d // 2].float(), x[..., d // 2:].float()
        return torch.cat([a * c - b * s, b * c + a * s], -1).to(x.dtype)
    slots = st["slots"].long()
    st["k_cache"][slots // ps, :, slots % ps] = turn(st["k"])
    st["v_cache"][slots // ps, :, slots % ps] = st["v"]
    return {"q": turn(st["q"]), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain_attn(st):
    q, ps = st["q"], st["page"]
    T, Hq, d = q.shape
    Hkv = st["k_cache"].shape[1]
    o = torch.empty((T, Hq, d), dtype=q.dtype, device=q.device)
    lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    t0 = 0
    for r, (_, p0, kv) in enumerate(st["lens"]):
        n = kv - p0
        if n == 0:
            continue
        rows = slice(t0, t0 + n)
        t0 += n
        at = st["table"][r, :-(-kv // ps)].long()
        k, v = (st[c][at].transpose(0, 1).reshape(Hkv, -1, d)[:, :kv].float() for c in ("k_cache", "v_cache"))
        x = q[rows].float().view(n, Hkv, -1, d).permute(1, 2, 0, 3).reshape(Hkv, -1, d)    # [Hkv, G n, d]
        s = (x @ k.transpose(1, 2)) * st["scale"]
        last = torch.arange(p0, kv, device=q.device)
        if st["kind"] == "draft":
            last[1:] = kv - 1
        hidden = torch.arange(kv, device=q.device)[None, :] > last.repeat(Hq // Hkv)[:, None]
        s.masked_fill_(hidden, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        y = (p @ v) / l
        o[rows] = y.view(Hq, n, d).transpose(0, 1).to(q.dtype)
        lse[:, rows] = (m + torch.log(l)).view(Hq, n)
    return {"o": o, "lse": lse}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    lens, ps = _lens(case), case["page"]
    T = sum(e - s for _, s, e in lens)
    if case["op"] == "pages":
        # three lengths in; held, kv_len and cu out; a page in and out for each that changes hands; pos and slots out
        moved = sum(abs(-(-h // ps) - -(-e // ps)) for h, _, e in lens)
        return {"bytes": 24 * len(lens) + 8 * moved + 8 * T, "flops": 4 * T}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "write":
        return {"bytes": 4 * T * (Hq + 2 * Hkv) * d + 8 * T, "flops": 3 * T * (Hq + Hkv) * d}
    keys = sum(kv for _, p0, kv in lens if kv > p0)
    if case["kind"] == "draft":
        pairs = sum((p0 + 1) + (kv - p0 - 1) * kv for _, p0, kv in lens if kv > p0)
    else:
        pairs = sum((kv - p0) * p0 + (kv - p0) * (kv - p0 + 1) // 2 for _, p0, kv in lens)
    b = keys * Hkv * d * 4 + T * Hq * (d * 4 + 4) + sum(4 * -(-kv // ps) + 8 for _, _, kv in lens)
    return {"bytes": b, "flops": 4 * pairs * Hq * d}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers only
    st = prepare(case, seed)
    ps, (T, Hq, d) = case["page"], st["q"].shape
    if case["op"] == "write":
        i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           st["pos"].double()[:, None] * torch.exp(i * (-2.0 * math.log(THETA) / d)))[:, None, :]

        def rotated(x):
            z = torch.complex(x[..., :d // 2].double(), x[..., d // 2:].double()) * turn
            return torch.cat([z.real, z.imag], -1)
        out = {"q": rotated(st["q"])}
        page, off = torch.div(st["slots"].long(), ps, rounding_mode="floor"), torch.remainder(st["slots"].long(), ps)
        for name, new in (("k_cache", rotated(st["k"])), ("v_cache", st["v"].double())):
            c = st[name].double()
            for h in range(c.shape[1]):
                c[:, h].index_put_((page, off), new[:, h])
            out[name] = c
        return out
    G = Hq // case["Hkv"]
    o = torch.zeros((T, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((Hq, T), dtype=torch.float64, device="cuda")
    t0 = 0
    for r, (_, p0, kv) in enumerate(_lens(case)):
        n = kv - p0
        key = torch.arange(kv, device="cuda")
        page = st["table"][r].long()[key // ps]
        row = torch.arange(n, device="cuda")
        last = p0 + row if case["kind"] != "draft" else torch.where(row == 0, p0, kv - 1)
        for h in range(Hq):
            k, v = (st[c][:, h // G][page, key % ps].double() for c in ("k_cache", "v_cache"))
            for a in range(0, n, 1024):
                b = min(n, a + 1024)
                s = st["q"][t0 + a:t0 + b, h].double() @ k.T * case["d"] ** -0.5
                s = torch.where(key[None, :] <= last[a:b, None], s, torch.full_like(s, -math.inf))
                lse[h, t0 + a:t0 + b] = torch.logsumexp(s, 1)
                o[t0 + a:t0 + b, h] = torch.softmax(s, 1) @ v
        t0 += n
    return {"o": o, "lse": lse}
