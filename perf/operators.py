"""Cases of the paged key-value cache operators: cache_append, paged_decode and cache_evict.

They serve the softmax-attention layers that stand between a hybrid model's KDA layers: a new
token's keys and values go into a paged cache, its queries attend to that cache, and the cache is
cut back to a budget by the attention weight that its entries have gathered.

The plain form computes in 32 bits (selections are exact in any width), `exact` in 64 bits,
sequence by sequence. Sizes: 32 query heads and head sizes 64 and 128 are this library's own, the
8K and 262144-token lengths, the 64 sequences of 128 to 16384 tokens, the batch of 256 sequences
and the quarter of the heads that one of four tensor-parallel GPUs holds come from its benchmark;
page sizes, key-value head counts and budgets are generic.
"""
import math
import random

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------- cases

def attend(name, io, n, lo, hi, hq, hkv, d, page, acc=False, gate=False, layout="token"):
    return {"name": name, "op": "attend", "io": io, "n": n, "lo": lo, "hi": hi, "hq": hq,
            "hkv": hkv, "d": d, "page": page, "acc": acc, "gate": gate, "layout": layout}


def append(name, io, n, lo, hi, t_lo, t_hi, hkv, d, page, layout="token"):
    return {"name": name, "op": "append", "io": io, "n": n, "lo": lo, "hi": hi, "t_lo": t_lo,
            "t_hi": t_hi, "hkv": hkv, "d": d, "page": page, "layout": layout}


def evict(name, io, n, lo, hi, keep, first, recent, hkv, d, page, layout="token"):
    return {"name": name, "op": "evict", "io": io, "n": n, "lo": lo, "hi": hi, "keep": keep,
            "first": first, "recent": recent, "hkv": hkv, "d": d, "page": page, "layout": layout}


def listed():
    return [
        # the first answer tokens of one short chat: nothing but latency
        attend("attend_one_short", "bf16", 1, 200, 200, 32, 8, 128, 16),
        # continuous batching: 64 requests of 128 to 16384 tokens, with the layer's output gate
        attend("attend_varlen_64", "bf16", 64, 128, 16384, 32, 8, 128, 64, gate=True),
        # one document of 262144 tokens on one of four tensor-parallel GPUs (8 of 32 heads)
        attend("attend_256k_tp4", "bf16", 1, 262144, 262144, 8, 2, 128, 64, layout="head"),
        # a batch held at a budget of 4096 entries: the weights are gathered for the eviction
        attend("attend_budget_acc", "bf16", 32, 3500, 4224, 32, 8, 128, 16, acc=True, gate=True),
        # fp32 model under test: tiny, no head sharing, an empty sequence, odd pages
        attend("attend_f32_tiny", "f32", 7, 0, 300, 2, 2, 64, 24),
        # fp32 with one key-value head for 16 query heads, weights gathered
        attend("attend_f32_shared_acc", "f32", 16, 1, 4096, 16, 1, 128, 32, acc=True,
               layout="head"),
        # one decode step of 256 sequences
        append("append_decode_256", "bf16", 256, 0, 512, 1, 1, 8, 128, 16),
        # prompts of up to 8192 tokens enter the cache, some behind a cached prefix
        append("append_prompts", "bf16", 8, 0, 1000, 1, 8192, 8, 128, 64, layout="head"),
        # the budgeted batch again, cut back to 4096 entries after up to 128 new tokens
        evict("evict_budget", "bf16", 32, 4000, 4224, 4096, 4, 256, 8, 128, 16),
        # a document of 262144 tokens cut to half after its prefill
        evict("evict_256k_half", "bf16", 1, 262144, 262144, 131072, 16, 1024, 8, 128, 64),
        # fp32, a head count and page size without a factor of two, an empty sequence
        evict("evict_f32_odd", "f32", 5, 0, 1000, 333, 1, 17, 3, 64, 7, layout="head"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _unnamed(case):
    del case["name"]
    return case


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "evict"])
    io = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([1, 7, 16, 16, 24, 32, 64, 64, 100, 128])
    layout = rng.choice(["token", "head"])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    row = hkv * d * ESIZE[io]
    if op == "attend":
        hq = hkv * rng.choice([1, 2, 3, 4, 4, 5, 8, 8, 12, 16, 32])
        acc, gate = rng.random() < 0.4, rng.random() < 0.5
        n = _log(rng, 1, 256)
        # the plain form's time goes with the query heads too: both bounds keep it below the
        # largest listed case's
        most = min(2 ** 30 // row, 2 ** 25 // hq) // n
        hi = _log(rng, 4, max(4, min(262144, most)))
        lo = rng.choice([0, 1, hi // 4, hi // 2, hi])
        return _unnamed(attend("", io, n, lo, hi, hq, hkv, d, page, acc, gate, layout))
    if op == "append":
        n = _log(rng, 1, 256)
        t_hi = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, 2 ** 26 // row // n))
        hi = _log(rng, 2, max(2, 2 ** 27 // row // n))
        return _unnamed(append("", io, n, 0, hi, rng.choice([0, 1, t_hi]), t_hi, hkv, d, page,
                               layout))
    n = _log(rng, 1, 256)
    hi = _log(rng, 16, max(16, min(262144, 2 ** 29 // row // n)))
    keep = max(4, int(hi * rng.uniform(0.3, 1.0)))
    first = rng.randint(0, min(16, keep // 4))
    recent = rng.randint(0, keep // 4)
    return _unnamed(evict("", io, n, rng.choice([0, hi // 2, hi]), hi, keep, first, recent, hkv, d,
                          page, layout))


def _lens(n, lo, hi, salt):
    """Lengths in [lo, hi], the same for every seed; both ends occur when there is room."""
    r = random.Random(n * 1000003 + lo * 8191 + hi * 131 + salt)
    lens = [r.randint(lo, hi) for _ in range(n)]
    lens[0] = hi
    if n > 1:
        lens[-1] = lo
    return lens


def _case_lens(c):
    old = _lens(c["n"], c["lo"], c["hi"], 1)
    new = _lens(c["n"], c["t_lo"], c["t_hi"], 2) if c["op"] == "append" else [0] * c["n"]
    return old, new


# ---------------------------------------------------------------- inputs

def _cache(c, pages, gen, dev):
    """K and V pages, viewed as [pages, page, hkv, d] over token-major or head-major memory."""
    shape = (pages, c["page"], c["hkv"], c["d"]) if c["layout"] == "token" else \
        (pages, c["hkv"], c["page"], c["d"])
    out = []
    for _ in range(2):
        t = torch.randn(shape, generator=gen, device=dev, dtype=DTYPE[c["io"]])
        out.append(t if c["layout"] == "token" else t.transpose(1, 2))
    return out


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    io = DTYPE[c["io"]]
    old, new = _case_lens(c)
    total = [a + b for a, b in zip(old, new)]
    need = [-(-t // c["page"]) for t in total]
    pages = sum(need) + 3
    max_pages = max(1, max(need))
    # every sequence owns its pages, spread over the pool; unused table entries hold -1
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((c["n"], max_pages), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = torch.tensor(perm[at:at + k], dtype=torch.int32)
        at += k
    slots = max(1, max(total))
    s = {"case": c, "table": table.to(dev),
         "lens": torch.tensor(old, dtype=torch.int32, device=dev), "slots": slots}
    s["k"], s["v"] = _cache(c, pages, gen, dev)
    n, hkv, d = c["n"], c["hkv"], c["d"]
    if c["op"] == "attend":
        s["q"] = torch.randn(n, c["hq"], d, generator=gen, device=dev, dtype=io)
        s["z"] = torch.randn(n, c["hq"], d, generator=gen, device=dev, dtype=io) if c["gate"] else None
        s["scale"] = d ** -0.5
        # every query looks at its sequence's first entry, as trained models do
        some = [i for i, x in enumerate(old) if x > 0]
        pull = 3.0 * s["q"].float().view(n, hkv, -1, d).mean(2)
        s["k"][s["table"][some, 0].long(), 0] += pull[some].to(io)
        if c["acc"]:      # weight gathered so far, as in the eviction
            s["acc"] = _weights((n, hkv, slots), gen, dev)
        s["o"] = torch.empty_like(s["q"])
        if own:
            from kimi_delta_attention_32_b200 import kda
            s["ws"] = torch.empty(kda.paged_decode_workspace_size(
                n, c["hq"], hkv, d, slots, with_acc=c["acc"]), dtype=torch.uint8, device=dev)
    elif c["op"] == "append":
        t = sum(new)
        s["k_new"] = torch.randn(t, hkv, d, generator=gen, device=dev, dtype=io)
        s["v_new"] = torch.randn(t, hkv, d, generator=gen, device=dev, dtype=io)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        s["cu_host"], s["cu"] = cu, torch.tensor(cu, dtype=torch.int32, device=dev)
        # tokens that each sequence has seen: more than the cache holds where some were evicted
        s["seen"] = s["lens"] + 5
        s["acc"] = _weights((n, hkv, slots), gen, dev)
        s["pos"] = torch.zeros(n, hkv, slots, dtype=torch.int32, device=dev)
    else:
        s["acc"] = _weights((n, hkv, slots), gen, dev)
        # an earlier cut left its survivors in mixed order and gaps in the positions; the tokens
        # since then, in the last eighth, are in order
        slot = torch.arange(slots, device=dev)
        order = torch.rand(n, hkv, slots, generator=gen, device=dev)
        fresh = slot >= (s["lens"].view(n, 1, 1) * 7 // 8)
        order = torch.where(fresh, 2.0 + slot, order)
        mixed = torch.argsort(order, dim=-1, stable=True)
        s["pos"] = torch.where(mixed >= c["first"], mixed + 100, mixed).to(torch.int32)
        s["seen"] = s["lens"] + 100
        s["acc_out"] = torch.zeros_like(s["acc"])
        s["pos_out"] = torch.zeros_like(s["pos"])
        if own:
            from kimi_delta_attention_32_b200 import kda
            s["ws"] = torch.empty(kda.cache_evict_workspace_size(n, hkv, slots, c["keep"]),
                                  dtype=torch.uint8, device=dev)
    return s


def _weights(shape, gen, dev):
    """Gathered attention weights: a few heavy entries, many small ones, some never looked at."""
    w = torch.exp(2.0 * torch.randn(shape, generator=gen, device=dev) - 3.0)
    return torch.where(torch.rand(shape, generator=gen, device=dev) < 0.02, torch.zeros_like(w), w)


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _own_attend, "append": _own_append, "evict": _own_evict}[op](state)
    return {"attend": _plain_attend, "append": _plain_append, "evict": _plain_evict}[op](state)


def _own_attend(s):
    from kimi_delta_attention_32_b200 import kda
    acc = s.get("acc")
    kda.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], scale=s["scale"], z=s["z"],
                     acc=acc, max_len=s["slots"], o=s["o"], workspace=s["ws"])
    return {"o": s["o"]} if acc is None else {"o": s["o"], "acc": acc}


def _own_append(s):
    from kimi_delta_attention_32_b200 import kda
    c = s["case"]
    kw = {"positions": s["seen"], "acc": s["acc"], "pos": s["pos"]}
    if c["t_lo"] == c["t_hi"]:        # the same number of tokens each: the padded form
        shape = (c["n"], c["t_hi"], c["hkv"], c["d"])
        kda.cache_append(s["k_new"].view(shape), s["v_new"].view(shape), s["k"], s["v"],
                         s["table"], s["lens"], **kw)
    else:
        kda.cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"],
                         cu_seqlens=s["cu"], cu_host=s["cu_host"], **kw)
    return {"k": s["k"], "v": s["v"], "acc": s["acc"], "pos": s["pos"]}


def _own_evict(s):
    from kimi_delta_attention_32_b200 import kda
    c = s["case"]
    lens = kda.cache_evict(s["k"], s["v"], s["table"], s["lens"], c["keep"], s["acc"], s["pos"],
                           positions=s["seen"], n_first=c["first"], n_recent=c["recent"],
                           acc_out=s["acc_out"], pos_out=s["pos_out"], workspace=s["ws"])
    return {"k": s["k"], "v": s["v"], "acc": s["acc_out"], "pos": s["pos_out"], "lens": lens}


def _plain_attend(s):
    c = s["case"]
    n, hkv, d = c["n"], c["hkv"], c["d"]
    g, S = c["hq"] // hkv, s["slots"]
    at = s["table"].clamp(min=0).long()
    k = s["k"][at].reshape(n, -1, hkv, d)[:, :S].permute(0, 2, 1, 3).float()     # [n, hkv, S, d]
    v = s["v"][at].reshape(n, -1, hkv, d)[:, :S].permute(0, 2, 1, 3).float()
    live = torch.arange(S, device=k.device) < s["lens"].view(n, 1, 1, 1)
    x = torch.matmul(s["q"].float().view(n, hkv, g, d), k.transpose(2, 3)) * s["scale"]
    x = torch.where(live, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    w = p / torch.where(l == 0, torch.ones_like(l), l)
    o = torch.matmul(w, v).view(n, c["hq"], d)
    if s["z"] is not None:
        o = o / (1 + torch.exp(-s["z"].float()))
    s["o"].copy_(o)
    if "acc" not in s:
        return {"o": s["o"]}
    s["acc"] += w.sum(2)
    return {"o": s["o"], "acc": s["acc"]}


def _plain_append(s):
    c = s["case"]
    new = s["cu"][1:] - s["cu"][:-1]
    seq = torch.repeat_interleave(torch.arange(c["n"], device=s["cu"].device), new.long(),
                                  output_size=s["cu_host"][-1])
    i = torch.arange(s["cu_host"][-1], device=s["cu"].device) - s["cu"][:-1].long()[seq]
    slot = s["lens"].long()[seq] + i
    page = s["table"].long()[seq, slot // c["page"]]
    s["k"][page, slot % c["page"]] = s["k_new"]
    s["v"][page, slot % c["page"]] = s["v_new"]
    s["acc"][seq, :, slot] = 0.0
    s["pos"][seq, :, slot] = (s["seen"].long()[seq] + i).int()[:, None]
    return {"k": s["k"], "v": s["v"], "acc": s["acc"], "pos": s["pos"]}


def _plain_evict(s):
    c = s["case"]
    n, hkv, S, keep = c["n"], c["hkv"], s["slots"], c["keep"]
    dev = s["acc"].device
    lens = s["lens"].view(n, 1, 1).long()
    slot = torch.arange(S, device=dev).expand(n, hkv, S)
    live = slot < lens
    pos = s["pos"].long()
    guarded = (pos < c["first"]) | (pos >= s["seen"].view(n, 1, 1).long() - c["recent"])
    key = torch.where(torch.isnan(s["acc"]), torch.full_like(s["acc"], -math.inf), s["acc"])
    # larger weights first, equal ones by slot; then the guarded ones before all, the dead behind
    order = torch.argsort(key, dim=-1, descending=True, stable=True)
    rank = torch.where(live, torch.where(guarded, 0, 1), 2).gather(-1, order)
    order = order.gather(-1, torch.argsort(rank, dim=-1, stable=True))
    place = torch.empty_like(order).scatter_(-1, order, slot.contiguous())
    kept = live & (place < keep)
    hole = live & ~kept & (slot < keep)
    tail = kept & (slot >= keep)
    seq, head, to = hole.nonzero(as_tuple=True)         # both in (sequence, head, slot) order
    frm = tail.nonzero(as_tuple=True)[2]
    table, page = s["table"].long(), c["page"]
    for t in (s["k"], s["v"]):
        t[table[seq, to // page], to % page, head] = t[table[seq, frm // page], frm % page, head]
    stay = kept & (slot < keep)
    for src, dst in ((s["acc"], s["acc_out"]), (s["pos"], s["pos_out"])):
        dst.copy_(torch.where(stay, src, dst))
        dst[seq, head, to] = src[seq, head, frm]
    return {"k": s["k"], "v": s["v"], "acc": s["acc_out"], "pos": s["pos_out"],
            "lens": torch.clamp(s["lens"], max=keep)}


# ---------------------------------------------------------------- what a pass needs

def work(case):
    c = case
    old, new = _case_lens(c)
    e, hkv, d = ESIZE[c["io"]], c["hkv"], c["d"]
    row = 2 * hkv * d * e                     # one token's keys and values
    table = 4 * sum(-(-x // c["page"]) for x in old) + 4 * c["n"]
    if c["op"] == "attend":
        t = sum(old)
        ends = c["n"] * c["hq"] * d * e * (3 if c["gate"] else 2)
        return {"bytes": t * row + ends + table + (8 * t * hkv if c["acc"] else 0),
                "flops": 4 * t * c["hq"] * d}
    if c["op"] == "append":
        t = sum(new)
        return {"bytes": 2 * t * row + 8 * t * hkv + 4 * c["n"], "flops": 0}
    total = 0.0
    for x in old:
        kept = min(x, c["keep"])
        total += 8 * kept * hkv + 4           # weights and positions written
        if x > c["keep"]:
            total += 8 * x * hkv              # and read
            behind = x - c["keep"]            # slots behind the budget: the recent ones stay kept
            recent = min(c["recent"], behind)
            free = max(1, x - c["first"] - c["recent"])
            share = (c["keep"] - c["first"] - c["recent"]) / free
            total += 2 * row * (recent + (behind - recent) * share)
        else:
            total += 8 * x * hkv
    return {"bytes": total, "flops": 0}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "evict": _exact_evict}[case["op"]](s)


def _rows(table_row, length, page):
    """Page and row of every slot of one sequence."""
    j = torch.arange(length, device=table_row.device)
    return table_row[(j // page)].long(), j % page


def _exact_attend(s):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    lens = s["lens"].tolist()
    o = torch.zeros(c["n"], c["hq"], c["d"], dtype=torch.float64, device=s["q"].device)
    acc = s["acc"].double() if "acc" in s else None
    for i, length in enumerate(lens):
        if length == 0:
            continue
        page, row = _rows(s["table"][i], length, c["page"])
        for h in range(c["hkv"]):
            keys = s["k"][page, row, h].double()
            vals = s["v"][page, row, h].double()
            w = torch.softmax(s["q"][i, h * g:(h + 1) * g].double() @ keys.T * s["scale"], -1)
            o[i, h * g:(h + 1) * g] = w @ vals
            if acc is not None:
                acc[i, h, :length] += w.sum(0)
    if s["z"] is not None:
        o = o * torch.sigmoid(s["z"].double())
    return {"o": o} if acc is None else {"o": o, "acc": acc}


def _exact_append(s):
    c = s["case"]
    k, v, acc = s["k"].double(), s["v"].double(), s["acc"].double()
    for i, length in enumerate(s["lens"].tolist()):
        a, b = s["cu_host"][i], s["cu_host"][i + 1]
        if a == b:
            continue
        page, row = _rows(s["table"][i], length + b - a, c["page"])
        k[page[length:], row[length:]] = s["k_new"][a:b].double()
        v[page[length:], row[length:]] = s["v_new"][a:b].double()
        acc[i, :, length:length + b - a] = 0
    return {"k": k, "v": v, "acc": acc, "pos": None}


def _exact_evict(s):
    import numpy as np
    c, keep = s["case"], s["case"]["keep"]
    k, v, out = s["k"].double(), s["v"].double(), s["acc_out"].double()
    acc, pos = s["acc"].cpu().numpy().astype(np.float64), s["pos"].cpu().numpy()
    seen = s["seen"].tolist()
    for i, length in enumerate(s["lens"].tolist()):
        page, row = _rows(s["table"][i], length, c["page"])
        for h in range(c["hkv"]):
            a, p = acc[i, h, :length], pos[i, h, :length]
            at = np.arange(length)
            if length > keep:
                guarded = (p < c["first"]) | (p >= seen[i] - c["recent"])
                best = np.lexsort((at, -np.nan_to_num(a, nan=-np.inf, posinf=np.inf), ~guarded))[:keep]
                kept = np.zeros(length, bool)
                kept[best] = True
                to = torch.from_numpy(at[:keep][~kept[:keep]]).to(k.device)
                frm = torch.from_numpy(at[keep:][kept[keep:]]).to(k.device)
                for t in (k, v):
                    t[page[to], row[to], h] = t[page[frm], row[frm], h]
                a = a.copy()
                a[to.cpu().numpy()] = a[frm.cpu().numpy()]
            m = min(length, keep)
            out[i, h, :m] = torch.from_numpy(a[:m]).to(out.device)
    return {"k": k, "v": v, "acc": out, "pos": None, "lens": None}
