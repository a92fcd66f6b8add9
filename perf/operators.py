"""Measured cases of the training-side operators: the token embedding with its
gradient, causal attention over packed sequences with its gradient, and the
language-model head fused with the softmax cross entropy and its gradient.

A case names one operator, its sizes, its element type and its direction:
grad = False runs the forward call alone (scoring, prefill), grad = True the
forward call and the backward call after it, as one training step makes them.
The plain forms compute in 32 bits with elementary torch operations and round
once at the end.
"""
import math

import numpy as np
import torch

own = False  # True: the library's calls; False: the plain forms

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MASK = -1     # the id of an [M] row
IGNORE = -1   # the label of a row without a target


def listed():
    return [
        # the draft window of one decode round: a boundary token and 32 [M] rows
        {"name": "embed-window", "op": "embed", "T": 33, "H": 1536, "V": 65536, "mask": 0.97, "dtype": "bf16",
         "grad": False},
        # the tiny fp32 decoder, one odd packed row, trained
        {"name": "embed-tiny-f32-grad", "op": "embed", "T": 1999, "H": 256, "V": 1024, "mask": 0.2, "dtype": "f32",
         "grad": True},
        # a joint-training row of 10,240 packed tokens with two corrupted streams, a third of it [M]
        {"name": "embed-packed-grad", "op": "embed", "T": 10240, "H": 1536, "V": 65536, "mask": 0.33, "dtype": "bf16",
         "grad": True},
        # prompts of one page's 18 short text and formula regions, prefilled together
        {"name": "attn-regions", "op": "attn", "Hq": 12, "Hkv": 4, "d": 128, "dtype": "bf16", "grad": False,
         "lens": "73,95,51,120,73,1,88,64,17,95,140,33,73,109,60,5,81,122"},
        # 16 ragged prompts of the page batch, scaled to one packed prefill
        {"name": "attn-prompts", "op": "attn", "Hq": 12, "Hkv": 4, "d": 128, "dtype": "bf16", "grad": False,
         "lens": "512,1031,287,640,901,333,256,1200,777,129,480,655,390,512,64,25"},
        # the tiny decoder's heads, a few odd sequences, trained
        {"name": "attn-tiny-grad", "op": "attn", "Hq": 4, "Hkv": 2, "d": 64, "dtype": "bf16", "grad": True,
         "lens": "64,1,193,130,311"},
        # a packed training row of samples of text, formula and table regions
        {"name": "attn-packed-grad", "op": "attn", "Hq": 12, "Hkv": 4, "d": 128, "dtype": "bf16", "grad": True,
         "lens": "872,345,419,1097,601,287,95,512,873,444,1203,730,368,146,200"},
        # one long document as a single training sequence
        {"name": "attn-long-grad", "op": "attn", "Hq": 12, "Hkv": 4, "d": 128, "dtype": "bf16", "grad": True,
         "lens": "8192"},
        # scores of one verify window (33 rows) against the full vocabulary
        {"name": "ce-window", "op": "ce", "T": 33, "H": 1536, "V": 65536, "dtype": "bf16", "grad": False},
        # scores of the tokens of one ragged batch
        {"name": "ce-score", "op": "ce", "T": 2047, "H": 1536, "V": 65536, "dtype": "bf16", "grad": False},
        # the last odd rows of an epoch, a small vocabulary of odd size
        {"name": "ce-odd-grad", "op": "ce", "T": 193, "H": 512, "V": 8191, "dtype": "bf16", "grad": True},
        # a training step over the full vocabulary
        {"name": "ce-train", "op": "ce", "T": 4096, "H": 1536, "V": 65536, "dtype": "bf16", "grad": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "attn", "ce"])
    grad = rng.random() < 0.6
    if op == "embed":
        return {"op": op, "T": _log_int(rng, 1, 10240), "H": 8 * _log_int(rng, 8, 192), "V": _log_int(rng, 1000, 65536),
                "mask": round(rng.choice([0.0, rng.random() * 0.9]), 3), "dtype": rng.choice(["bf16", "f32"]),
                "grad": grad}
    if op == "attn":
        # (sequences of one token are among them, but not alone: their q and k gradients are zero)
        total = _log_int(rng, 16, 8192)
        n = min(total // 8, _log_int(rng, 1, 32))
        cuts = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        hkv = rng.randint(1, 4)
        return {"op": op, "Hq": hkv * rng.randint(1, 3), "Hkv": hkv, "d": rng.choice([64, 128]), "dtype": "bf16",
                "grad": grad, "lens": ",".join(map(str, lens))}
    return {"op": op, "T": _log_int(rng, 1, 4096), "H": 8 * _log_int(rng, 8, 192), "V": _log_int(rng, 1000, 65536),
            "dtype": "bf16", "grad": grad}


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    normal = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float32)
    uniform = lambda n: torch.rand((n,), generator=g, device="cuda", dtype=torch.float32)
    st = {"op": case["op"], "grad": case["grad"]}
    if case["op"] == "embed":
        T, H, V = case["T"], case["H"], case["V"]
        # token ids of text follow a Zipf law: log-uniform ranks
        ids = torch.exp(uniform(T) * math.log(V)).long().clamp(1, V) - 1
        st["ids"] = torch.where(uniform(T) < case["mask"], torch.full_like(ids, MASK), ids).to(torch.int32)
        st["embed"] = (0.02 * normal(V, H)).to(dt)
        st["mask_embed"] = (0.02 * normal(H)).to(dt)
        st["scale"] = math.sqrt(H)
        st["dy"] = (1e-3 * normal(T, H)).to(dt)
    elif case["op"] == "attn":
        lens, Hq, Hkv, d = _lens(case), case["Hq"], case["Hkv"], case["d"]
        T = sum(lens)
        # q, k and v as the fused projection leaves them: head ranges of one row
        qkv = normal(T, Hq + 2 * Hkv, d).to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        st["do"] = (1e-2 * normal(T, Hq, d)).to(dt)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        st["scale"] = d ** -0.5
    else:
        T, H, V = case["T"], case["H"], case["V"]
        labels = torch.exp(uniform(T) * math.log(V)).long().clamp(1, V) - 1
        w = 0.02 * normal(V, H)
        # normalised hidden rows that lean towards their targets, as a trained decoder's do
        x = normal(T, H) + 10.0 * w[labels]
        st["w"] = w.to(dt)
        st["x"] = (x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-6)).to(dt)
        no = uniform(T) < 0.1
        st["labels"] = torch.where(no, torch.full_like(labels, IGNORE), labels).to(torch.int32)
        # the weight of each row in the mean losses of the clean and the corrupted streams
        st["dloss"] = torch.where(uniform(T) < 0.5, 1.0, 2.0) / (1.5 * T)
    return st


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from self_speculative_block_gb300 import gocr
    if st["op"] == "embed":
        out = {"y": gocr.op_embed(st["ids"], st["embed"], st["mask_embed"], scale=st["scale"])}
        if st["grad"]:
            out["d_embed"], out["d_mask"] = gocr.op_embed_backward(st["dy"], st["ids"], st["embed"].shape[0],
                                                                   mask=True, scale=st["scale"])
        return out
    if st["op"] == "attn":
        o, lse = gocr.op_attention_packed(st["q"], st["k"], st["v"], st["cu"], scale=st["scale"])
        out = {"o": o, "lse": lse}
        if st["grad"]:
            out["dq"], out["dk"], out["dv"] = gocr.op_attention_packed_backward(
                st["do"], st["q"], st["k"], st["v"], o, lse, st["cu"], scale=st["scale"])
        return out
    loss, lse = gocr.op_linear_ce(st["x"], st["w"], st["labels"])
    out = {"loss": loss, "lse": lse}
    if st["grad"]:
        out["dx"], out["dw"] = gocr.op_linear_ce_backward(st["dloss"], st["x"], st["w"], st["labels"], lse)
    return out


def _run_plain(st):
    return {"embed": _plain_embed, "attn": _plain_attn, "ce": _plain_ce}[st["op"]](st)


def _plain_embed(st):
    ids, E, m = st["ids"].long(), st["embed"], st["mask_embed"]
    rows = torch.where((ids == MASK)[:, None], m.float(), E[ids.clamp(min=0)].float())
    out = {"y": (rows * st["scale"]).to(E.dtype)}
    if st["grad"]:
        V = E.shape[0]
        d = torch.zeros((V + 1, E.shape[1]), device=E.device)
        d.index_add_(0, torch.where(ids == MASK, torch.full_like(ids, V), ids), st["dy"].float())
        d *= st["scale"]
        out["d_embed"], out["d_mask"] = d[:V].to(E.dtype), d[V].to(E.dtype)
    return out


def _plain_attn(st):
    dt = st["q"].dtype
    T, Hq, d = st["q"].shape
    G = Hq // st["k"].shape[1]
    q, do = (st[n].float().transpose(0, 1) for n in ("q", "do"))                               # [Hq, T, d]
    k, v = (st[n].float().transpose(0, 1).repeat_interleave(G, 0) for n in ("k", "v"))         # [Hq, T, d]
    cu = st["cu"].long()
    row = torch.arange(T, device=q.device)
    seq = torch.repeat_interleave(torch.arange(len(cu) - 1, device=q.device), cu[1:] - cu[:-1], output_size=T)
    hidden = (seq[:, None] != seq[None, :]) | (row[None, :] > row[:, None])
    s = (q @ k.transpose(1, 2)) * st["scale"]
    s.masked_fill_(hidden, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    p /= l
    o = p @ v
    out = {"o": o.transpose(0, 1).to(dt).contiguous(), "lse": (m + torch.log(l))[..., 0]}
    if st["grad"]:
        dv = p.transpose(1, 2) @ do
        ds = p * (do @ v.transpose(1, 2) - (do * o).sum(-1, keepdim=True)) * st["scale"]
        dq = ds @ k
        dk = ds.transpose(1, 2) @ q
        out["dq"] = dq.transpose(0, 1).to(dt).contiguous()
        out["dk"] = dk.view(-1, G, T, d).sum(1).transpose(0, 1).to(dt).contiguous()
        out["dv"] = dv.view(-1, G, T, d).sum(1).transpose(0, 1).to(dt).contiguous()
    return out


def _plain_ce(st):
    x, w, labels = st["x"].float(), st["w"].float(), st["labels"].long()
    logits = x @ w.T
    m = logits.amax(1, keepdim=True)
    lse = (m + torch.log(torch.exp(logits - m).sum(1, keepdim=True)))[:, 0]
    some = labels >= 0
    at = labels.clamp(min=0)
    loss = torch.where(some, lse - logits.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    out = {"loss": loss, "lse": lse}
    if st["grad"]:
        g = torch.exp(logits - lse[:, None])
        g.scatter_add_(1, at[:, None], torch.full_like(g[:, :1], -1.0))
        g *= torch.where(some, st["dloss"], torch.zeros_like(lse))[:, None]
        out["dx"], out["dw"] = (g @ w).to(st["x"].dtype), (g.T @ x).to(st["w"].dtype)
    return out


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "embed":
        T, H, V = case["T"], case["H"], case["V"]
        # forward: the distinct table rows in, y out; backward: dy in, the dense table gradient out
        rank = np.arange(1.0, V + 1.0)
        p = (1.0 - case["mask"]) * np.log1p(1.0 / rank) / math.log(V)  # of an id, by the law of prepare()
        rows = min(T, float(-np.expm1(T * np.log1p(-np.minimum(p, 0.999))).sum()) + 1.0)
        b = T * 4 + (rows + T) * H * es
        if case["grad"]:
            b += T * 4 + T * H * es + (V + 1) * H * es
        return {"bytes": b, "flops": T * H * (2 if case["grad"] else 1)}
    if case["op"] == "attn":
        lens, Hq, Hkv, d = _lens(case), case["Hq"], case["Hkv"], case["d"]
        T = sum(lens)
        pairs = sum(n * (n + 1) // 2 for n in lens)
        b = T * ((2 * Hq + 2 * Hkv) * d * es + Hq * 4) + 4 * (len(lens) + 1)
        f = 4 * pairs * Hq * d
        if case["grad"]:
            b += T * ((4 * Hq + 4 * Hkv) * d * es + Hq * 4)  # q, k, v, o, do and lse in; dq, dk, dv out
            f += 10 * pairs * Hq * d
        return {"bytes": b, "flops": f}
    T, H, V = case["T"], case["H"], case["V"]
    b, f = (T + V) * H * es + T * 12, 2 * T * V * H
    if case["grad"]:
        b += 2 * (T + V) * H * es + T * 12
        f += 6 * T * V * H  # the logits again (they are not kept), dx and dw
    return {"bytes": b, "flops": f}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "embed":
        scale, E = st["scale"], st["embed"].double()
        table = torch.cat([st["mask_embed"].double()[None], E]) * scale  # row 1 + id
        at = st["ids"].long() + 1
        out = {"y": table[at]}
        if case["grad"]:
            order = torch.argsort(at, stable=True)
            run_sum = torch.cumsum(st["dy"].double()[order] * scale, 0)
            run_sum = torch.cat([torch.zeros_like(run_sum[:1]), run_sum])
            edge = torch.searchsorted(at[order].contiguous(), torch.arange(len(table) + 1, device=at.device))
            d = run_sum[edge[1:]] - run_sum[edge[:-1]]
            out["d_embed"], out["d_mask"] = d[1:], d[0]
        return out
    if case["op"] == "attn":
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        G = Hq // Hkv
        q, k, v, do = (st[n].double() for n in ("q", "k", "v", "do"))
        o, dq = torch.zeros_like(q), torch.zeros_like(q)
        dk, dv = torch.zeros_like(k), torch.zeros_like(v)
        lse = torch.zeros((Hq, q.shape[0]), dtype=torch.float64, device=q.device)
        t0 = 0
        for n in _lens(case):
            r = slice(t0, t0 + n)
            t0 += n
            seen = torch.tril(torch.ones((n, n), dtype=torch.bool, device=q.device))
            for h in range(Hq):
                s = (q[r, h] @ k[r, h // G].T * st["scale"]).where(seen, torch.tensor(-math.inf, dtype=q.dtype, device=q.device))
                lse[h, r] = torch.logsumexp(s, 1)
                p = torch.softmax(s, 1)
                o[r, h] = p @ v[r, h // G]
                if case["grad"]:
                    dp = do[r, h] @ v[r, h // G].T
                    ds = p * (dp - (p * dp).sum(1, keepdim=True)) * st["scale"]
                    dq[r, h] = ds @ k[r, h // G]
                    dk[r, h // G] += ds.T @ q[r, h]
                    dv[r, h // G] += p.T @ do[r, h]
        out = {"o": o, "lse": lse}
        if case["grad"]:
            out.update(dq=dq, dk=dk, dv=dv)
        return out
    x, w, labels = st["x"].double(), st["w"].double(), st["labels"].long()
    T = x.shape[0]
    loss, lse = torch.zeros(T, dtype=torch.float64, device=x.device), torch.zeros(T, dtype=torch.float64, device=x.device)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for t in range(0, T, 1024):
        r = slice(t, min(T, t + 1024))
        z = x[r] @ w.T
        lp = torch.log_softmax(z, 1)
        lse[r] = torch.logsumexp(z, 1)
        y = labels[r]
        some = (y >= 0).double()
        i = torch.arange(len(y), device=x.device)
        loss[r] = -lp[i, y.clamp(min=0)] * some
        if case["grad"]:
            g = torch.exp(lp)
            g[i, y.clamp(min=0)] -= 1.0
            g *= (some * st["dloss"][r].double())[:, None]
            dx[r] = g @ w
            dw += g.T @ x[r]
    out = {"loss": loss, "lse": lse}
    if case["grad"]:
        out.update(dx=dx, dw=dw)
    return out
