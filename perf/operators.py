"""What is measured of the bounded-cache attention operators, and their plain forms.

Three operators work on one key-value cache that is kept within a budget while
a sequence is generated:

- prompt attention (``window_attn``): ragged sequences of new tokens attend
  their keys causally, within a sliding window and to the first few tokens
  (sinks) that stay visible;
- decode attention (``paged_attn``): one new token per sequence attends its
  paged cache, with the same window and sinks, and optionally adds the weight
  that each cell received (over all query heads) to a running mass;
- eviction (``cache_evict``): the cells of largest mass, the sinks and the most
  recent cells are kept, in order, and copied into new pages.

With ``own`` false, ``run`` is the plain form in elementary torch operations in
32 bits; with ``own`` true it makes the framework's calls.
"""

import math
import random

import torch

own = False

D = 128                                    # head dimension of the framework
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8}


# ---- cases --------------------------------------------------------------------

def _decode(nseq, max_len, nkv, group, page, kv, q, layout="nhd", window=-1, sinks=0, mass=False, ragged=True):
    return {"op": "decode", "nseq": nseq, "max_len": max_len, "nkv": nkv, "group": group, "page": page, "kv": kv,
            "q": q, "layout": layout, "window": window, "sinks": sinks, "mass": mass, "ragged": ragged}


def _prompt(nseq, max_q, context, nkv, group, dtype, window=-1, sinks=0, ragged=True):
    return {"op": "prompt", "nseq": nseq, "max_q": max_q, "context": context, "nkv": nkv, "group": group,
            "dtype": dtype, "window": window, "sinks": sinks, "ragged": ragged}


def _evict(nseq, max_len, budget, sinks, recent, nkv, page, kv, layout="nhd", ragged=True):
    return {"op": "evict", "nseq": nseq, "max_len": max_len, "budget": budget, "sinks": sinks, "recent": recent,
            "nkv": nkv, "page": page, "kv": kv, "layout": layout, "ragged": ragged}


def listed():
    return [
        # a single user's chat, a few hundred tokens in: latency is all
        dict(_decode(1, 700, 8, 4, 16, "bf16", "bf16", ragged=False), name="decode_one"),
        # a full serving batch of ordinary lengths
        dict(_decode(64, 8192, 8, 4, 16, "bf16", "bf16"), name="decode_batch"),
        # a few long contexts on the framework's own cache form: int8 cells, binary16 scales, fp32 queries
        dict(_decode(4, 131072, 2, 4, 64, "int8", "fp32"), name="decode_long_int8"),
        # long sequences of which a window and the first tokens are read; heads outside cells, odd group
        dict(_decode(48, 32768, 8, 7, 32, "fp16", "fp16", layout="hnd", window=1024, sinks=4), name="decode_window"),
        # the step that also keeps the running mass that eviction goes by
        dict(_decode(16, 16384, 8, 4, 16, "bf16", "bf16", mass=True), name="decode_mass"),
        # a short question
        dict(_prompt(1, 77, 0, 8, 4, "bf16", ragged=False), name="prompt_short"),
        # a batch of ragged prompts under a small window with sinks
        dict(_prompt(8, 2048, 0, 8, 4, "bf16", window=512, sinks=4), name="prompt_batch"),
        # a long document under a window
        dict(_prompt(1, 8192, 0, 8, 4, "bf16", window=1024, sinks=16, ragged=False), name="prompt_long"),
        # the same length with every earlier token visible
        dict(_prompt(1, 8192, 0, 8, 4, "fp16", ragged=False), name="prompt_full"),
        # the next chunks of prompts whose earlier tokens are there already
        dict(_prompt(4, 512, 15872, 8, 4, "bf16"), name="prompt_chunk"),
        # one sequence that ran a little over a small budget
        dict(_evict(1, 576, 512, 4, 64, 8, 16, "bf16", ragged=False), name="evict_one"),
        # long contexts cut to an eighth, int8 cells
        dict(_evict(2, 131072, 16384, 16, 1024, 8, 64, "int8"), name="evict_long_int8"),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("decode", "decode", "prompt", "prompt", "evict"))
    layout = rng.choice(("nhd", "hnd", "joint"))
    page = rng.choice((8, 16, 16, 32, 48, 64, 128))
    nkv = rng.choice((1, 2, 4, 8))
    if op == "decode":
        kv = rng.choice(("bf16", "fp16", "int8"))
        q = rng.choice(("fp32", "bf16", "fp16")) if kv == "int8" else kv
        group = rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16))
        nseq = _log_int(rng, 1, 128)
        # no more cells than the largest listed batch holds
        max_len = _log_int(rng, 1, min(131072, 4_000_000 // (nseq * nkv)))
        window = rng.choice((-1, -1, _log_int(rng, 1, 8192)))
        sinks = rng.choice((0, rng.randint(1, 64))) if window >= 0 else 0
        return _decode(nseq, max_len, nkv, group, page, kv, q, layout, window, sinks, rng.random() < 0.3)
    if op == "prompt":
        group = rng.choice((1, 2, 3, 4, 5, 7, 8))
        nseq = _log_int(rng, 1, 16)
        # padded score elements (sequences x heads x queries x keys) within the largest listed case's
        most = 32 * 8192 * 8192 // (nseq * nkv * group)
        max_q = _log_int(rng, 1, min(8192, math.isqrt(most)))
        context = rng.choice((0, 0, _log_int(rng, 1, 16384)))
        context = max(0, min(context, most // max_q - max_q))
        window = rng.choice((-1, _log_int(rng, 1, 4096), _log_int(rng, 16, 4096)))
        sinks = rng.choice((0, rng.randint(1, 64))) if window >= 0 else 0
        return _prompt(nseq, max_q, context, nkv, group, rng.choice(("bf16", "fp16")), window, sinks)
    nseq = _log_int(rng, 1, 32)
    max_len = _log_int(rng, 64, min(131072, 2_000_000 // (nseq * nkv)))
    budget = max(16, int(max_len * rng.uniform(0.1, 0.95)))
    sinks = rng.randint(0, min(16, budget // 4))
    recent = rng.randint(0, budget // 2)
    return _evict(nseq, max_len, budget, sinks, recent, nkv, page, rng.choice(("bf16", "fp16", "int8")), layout)


def _lengths(case, longest, salt):
    """The sequences' lengths, a property of the case: the longest once, the others spread from an eighth of it."""
    n = case["nseq"]
    if not case["ragged"]:
        return [longest] * n
    rng = random.Random("%d %d %d" % (n, longest, salt))
    rest = [rng.randint(min(longest, longest // 8 + 1), longest) for _ in range(n - 1)]
    at = rng.randint(0, n - 1)
    return rest[:at] + [longest] + rest[at:]


def _decode_visible(case, length):
    w = length if case["window"] < 0 else min(length, case["window"])
    return min(length, w + min(case["sinks"], length - w))


def _prompt_visible(window, sinks, nq, nk):
    """Visible (query, key) pairs of one sequence whose nq queries are the last of its nk tokens."""
    total = 0
    for pos in range(nk - nq, nk):
        w = pos + 1 if window < 0 else min(pos + 1, window)
        total += w + min(sinks, pos + 1 - w)
    return total


def work(case):
    if case["op"] == "decode":
        seen = [_decode_visible(case, n) for n in _lengths(case, case["max_len"], 1)]
        heads = case["nkv"] * case["group"]
        cell = 2 * D * DTYPES[case["kv"]].itemsize + (4 if case["kv"] == "int8" else 0)
        qo = case["nseq"] * heads * (2 * D * DTYPES[case["q"]].itemsize + 4)
        more = 8 * sum(_lengths(case, case["max_len"], 1)) if case["mass"] else 0
        return {"bytes": sum(seen) * case["nkv"] * cell + qo + more, "flops": 4 * D * heads * sum(seen)}
    if case["op"] == "prompt":
        nq = _lengths(case, case["max_q"], 2)
        nk = [a + b for a, b in zip(nq, _lengths(case, case["context"], 3))] if case["context"] else nq
        heads = case["nkv"] * case["group"]
        pairs = sum(_prompt_visible(case["window"], case["sinks"], a, b) for a, b in zip(nq, nk))
        moved = sum(nq) * heads * (2 * D * 2 + 4) + sum(nk) * case["nkv"] * 2 * D * 2
        return {"bytes": moved, "flops": 4 * D * heads * pairs}
    lens = _lengths(case, case["max_len"], 1)
    kept = sum(min(n, case["budget"]) for n in lens)
    cell = case["nkv"] * (2 * D * DTYPES[case["kv"]].itemsize + (4 if case["kv"] == "int8" else 0))
    return {"bytes": 4 * sum(lens) + kept * (2 * cell + 8), "flops": 0}


# ---- what a user's program has before the call --------------------------------

def _values(shape, kv, gen, dev):
    if kv == "int8":
        return torch.randint(-127, 128, shape, generator=gen, device=dev, dtype=torch.int8)
    return torch.randn(shape, generator=gen, device=dev, dtype=DTYPES[kv])


def _pool(npages, case, gen, dev):
    """Key and value pages [npages, page, nkv, D] in the case's memory order: cells outside heads, heads outside
    cells, or keys and values of a page side by side; and for int8 cells one binary16 scale per cell and head."""
    page, nkv, kv = case["page"], case["nkv"], case["kv"]
    if case["layout"] == "hnd":
        k, v = (_values((npages, nkv, page, D), kv, gen, dev).transpose(1, 2) for _ in range(2))
    elif case["layout"] == "joint":
        k, v = _values((npages, 2, page, nkv, D), kv, gen, dev).unbind(1)
    else:
        k, v = (_values((npages, page, nkv, D), kv, gen, dev) for _ in range(2))
    ks = vs = None
    if kv == "int8":
        # |key| near 1 and |value| near 1, the scales spread over a factor of four
        ks, vs = (torch.exp2(torch.rand((npages, page, nkv), generator=gen, device=dev) * 2 - 7.2).to(torch.float16)
                  for _ in range(2))
    return k, v, ks, vs


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    if case["op"] == "prompt":
        nq = _lengths(case, case["max_q"], 2)
        nk = [a + b for a, b in zip(nq, _lengths(case, case["context"], 3))] if case["context"] else nq
        dt, nkv, heads = DTYPES[case["dtype"]], case["nkv"], case["nkv"] * case["group"]
        starts = [torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=dev)
                  for n in (nq, nk)]
        return {"case": case, "q": torch.randn((sum(nq), heads, D), generator=gen, device=dev, dtype=dt),
                "k": torch.randn((sum(nk), nkv, D), generator=gen, device=dev, dtype=dt),
                "v": torch.randn((sum(nk), nkv, D), generator=gen, device=dev, dtype=dt),
                "cu_q": starts[0], "cu_k": starts[1], "max_q": max(nq), "max_k": max(nk)}
    lens = _lengths(case, case["max_len"], 1)
    page, nseq = case["page"], case["nseq"]
    cols = -(-case["max_len"] // page)
    new_cols = -(-case["budget"] // page) if case["op"] == "evict" else 0
    npages = nseq * (cols + new_cols)
    k, v, ks, vs = _pool(npages, case, gen, dev)
    order = torch.randperm(npages, generator=gen, device=dev).to(torch.int32)
    state = {"case": case, "k": k, "v": v, "ks": ks, "vs": vs,
             "table": order[:nseq * cols].view(nseq, cols),
             "lens": torch.tensor(lens, dtype=torch.int32, device=dev)}
    # earlier steps left each cell some weight: a few cells have much of it
    mass = torch.rand((nseq, cols * page), generator=gen, device=dev).pow(4) * 8
    if case["op"] == "evict":
        return dict(state, mass=mass, new_table=order[nseq * cols:].view(nseq, new_cols))
    q = torch.randn((nseq, case["nkv"] * case["group"], D), generator=gen, device=dev, dtype=DTYPES[case["q"]])
    return dict(state, q=q, mass=mass if case["mass"] else None,
                mass_out=torch.zeros_like(mass) if case["mass"] else None)


# ---- the plain forms ------------------------------------------------------------

def _cells(pages, scale, table, page):
    """The cells of every sequence in order, in 32 bits: [nseq, cells, nkv, D]."""
    x = pages[table.long()].float()
    if scale is not None:
        x = x * scale[table.long()].float()[..., None]
    return x.flatten(1, 2)


def _softmax_sums(logits, seen):
    """exp(logit - largest) of the visible cells, their sum and the log of the sum of all exp(logit)."""
    logits = torch.where(seen, logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(logits - top)
    total = e.sum(-1, keepdim=True)
    return e, total, (top + torch.log(total))[..., 0]


def _plain_decode(s):
    c, dev = s["case"], s["q"].device
    k = _cells(s["k"], s["ks"], s["table"], c["page"])
    v = _cells(s["v"], s["vs"], s["table"], c["page"])
    nseq, cells = k.shape[:2]
    at, n = torch.arange(cells, device=dev)[None], s["lens"][:, None]
    seen = at < n
    if c["window"] >= 0:
        seen = seen & ((at >= n - c["window"]) | (at < c["sinks"]))
    v = torch.where(seen[..., None, None], v, 0.0)
    q = s["q"].float().view(nseq, c["nkv"], c["group"], D)
    logits = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1 / math.sqrt(D))       # [nseq, nkv, group, cells]
    e, total, lse = _softmax_sums(logits, seen[:, None, None])
    p = e / torch.where(total == 0, 1.0, total)
    out = torch.matmul(p, v.transpose(1, 2))
    made = {"out": out.reshape(s["q"].shape).to(s["q"].dtype), "lse": lse.reshape(nseq, -1)}
    if c["mass"]:
        new = s["mass"] + p.sum((1, 2))
        made["mass"] = torch.where(at < n, new, s["mass_out"])
    return made


def _plain_prompt(s):
    c, dev = s["case"], s["q"].device
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cu_q.diff()[:, None], cu_k.diff()[:, None]
    iq, ik = torch.arange(s["max_q"], device=dev)[None], torch.arange(s["max_k"], device=dev)[None]
    tq = torch.where(iq < nq, cu_q[:-1, None] + iq, 0)                         # padded to [nseq, max_q]
    tk = torch.where(ik < nk, cu_k[:-1, None] + ik, 0)
    pos = (nk - nq + iq)[..., None]                                            # a query's place among the keys
    seen = (ik[:, None] <= pos) & (ik < nk)[:, None] & (iq < nq)[..., None]
    if c["window"] >= 0:
        seen = seen & ((ik[:, None] > pos - c["window"]) | (ik[:, None] < c["sinks"]))
    nseq, heads = nq.shape[0], c["nkv"] * c["group"]
    q = s["q"].float()[tq].view(nseq, -1, c["nkv"], c["group"], D).permute(0, 2, 3, 1, 4)
    k = s["k"].float()[tk].permute(0, 2, 3, 1)[:, :, None]
    v = s["v"].float()[tk].permute(0, 2, 1, 3)[:, :, None]
    logits = torch.matmul(q, k) * (1 / math.sqrt(D))                           # [nseq, nkv, group, max_q, max_k]
    e, total, lse = _softmax_sums(logits, seen[:, None, None])
    out = torch.matmul(e, v) / torch.where(total == 0, 1.0, total)
    # back to the packed rows: row t of the batch is row (sequence, place) of the padded form
    t = torch.arange(s["q"].shape[0], device=dev)
    seq = torch.searchsorted(cu_q[1:], t, right=True)
    row = t - cu_q[seq]
    out = out.reshape(nseq, heads, -1, D)[seq, :, row]
    return {"out": out.to(s["q"].dtype), "lse": lse.reshape(nseq, heads, -1)[seq, :, row]}


def _plain_evict(s):
    c, dev = s["case"], s["mass"].device
    page, budget = c["page"], c["budget"]
    nseq, cells = s["mass"].shape
    at, n = torch.arange(cells, device=dev)[None], s["lens"][:, None]
    forced = (at < c["sinks"]) | (at >= n - c["recent"])
    key = torch.where(at < n, torch.where(forced, math.inf, s["mass"]), -math.inf)
    best = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :budget]   # ties: the lowest cell first
    new_lens = s["lens"].clamp(max=budget)
    i = torch.arange(budget, device=dev)[None]
    keep = i < new_lens[:, None]
    if best.shape[1] < budget:
        best = torch.nn.functional.pad(best, (0, budget - best.shape[1]))
    kept = torch.sort(torch.where(keep, best, cells), dim=1).values
    src = torch.where(keep, kept, 0)
    new_page, new_slot = torch.gather(s["new_table"].long(), 1, (i // page).expand(nseq, -1)), (i % page).expand(nseq, -1)
    old_page = torch.where(keep, torch.gather(s["table"].long(), 1, src // page), new_page)
    old_slot = torch.where(keep, src % page, new_slot)
    for pool in (s["k"], s["v"], s["ks"], s["vs"]):
        if pool is not None:
            pool[new_page, new_slot] = pool[old_page, old_slot]
    mass = torch.zeros((nseq, s["new_table"].shape[1] * page), device=dev)
    mass[:, :budget] = torch.where(keep, torch.gather(s["mass"], 1, src), 0.0)
    return _evicted(s, torch.where(keep, kept, -1).to(torch.int32), new_lens, mass)


def _evicted(s, kept, new_lens, mass):
    made = {"kept": kept, "lens": new_lens, "mass": mass, "k": s["k"], "v": s["v"]}
    return made if s["ks"] is None else dict(made, ks=s["ks"], vs=s["vs"])


# ---- one pass --------------------------------------------------------------------

def run(state):
    c = state["case"]
    if not own:
        return {"decode": _plain_decode, "prompt": _plain_prompt, "evict": _plain_evict}[c["op"]](state)
    import sparse_attention_kv_qsa_gb300 as qsa
    if c["op"] == "decode":
        out, lse = qsa.paged_attn(state["q"], state["k"], state["v"], state["table"], state["lens"],
                                  k_scale_f16=state["ks"], v_scale_f16=state["vs"], window=c["window"],
                                  sinks=c["sinks"], mass=state["mass"], mass_out=state["mass_out"])
        return {"out": out, "lse": lse, "mass": state["mass_out"]} if c["mass"] else {"out": out, "lse": lse}
    if c["op"] == "prompt":
        out, lse = qsa.window_attn(state["q"], state["k"], state["v"], state["cu_q"], state["cu_k"], state["max_q"],
                                   window=c["window"], sinks=c["sinks"])
        return {"out": out, "lse": lse}
    kept, new_lens, mass = qsa.cache_evict(state["k"], state["v"], state["table"], state["lens"], state["mass"],
                                           state["new_table"], c["budget"], sinks=c["sinks"], recent=c["recent"],
                                           k_scale_f16=state["ks"], v_scale_f16=state["vs"])
    return _evicted(state, kept, new_lens, mass)


# ---- the definitions in 64 bits ----------------------------------------------------

def _attend64(q, k, v, seen):
    """One head group in 64 bits: q [g, m, D], k and v [n, D], seen [m, n] -> out [g, m, D], lse [g, m], p."""
    logits = (q @ k.T / math.sqrt(D)).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(logits, -1)
    p = torch.exp(logits - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    return p @ v, lse, p


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return None          # nothing is computed: cells are chosen and moved
    f64 = torch.float64
    group, nkv = case["group"], case["nkv"]
    if case["op"] == "prompt":
        out = torch.zeros(s["q"].shape, dtype=f64, device=s["q"].device)
        lse = torch.zeros(s["q"].shape[:2], dtype=f64, device=s["q"].device)
        cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
        for i in range(case["nseq"]):
            a, b, x, y = cu_q[i], cu_q[i + 1], cu_k[i], cu_k[i + 1]
            key = torch.arange(y - x, device=out.device)
            for r in range(a, b, 2048):
                e = min(b, r + 2048)
                place = torch.arange(r - a, e - a, device=out.device)[:, None] + (y - x) - (b - a)
                seen = key <= place
                if case["window"] >= 0:
                    seen &= (place - key < case["window"]) | (key < case["sinks"])
                for h in range(nkv):
                    hs = slice(h * group, (h + 1) * group)
                    o, l, _ = _attend64(s["q"][r:e, hs].to(f64).transpose(0, 1), s["k"][x:y, h].to(f64),
                                        s["v"][x:y, h].to(f64), seen)
                    out[r:e, hs], lse[r:e, hs] = o.transpose(0, 1), l.T
        return {"out": out, "lse": lse}
    out = torch.zeros(s["q"].shape, dtype=f64, device=s["q"].device)
    lse = torch.zeros(s["q"].shape[:2], dtype=f64, device=s["q"].device)
    mass = s["mass_out"].to(f64) if case["mass"] else None
    for i, n in enumerate(s["lens"].tolist()):
        cell = torch.arange(n, device=out.device)
        page, slot = s["table"][i].long()[cell // case["page"]], cell % case["page"]
        seen = torch.ones_like(cell, dtype=torch.bool)
        if case["window"] >= 0:
            seen = (n - 1 - cell < case["window"]) | (cell < case["sinks"])
        gained = torch.zeros(n, dtype=f64, device=out.device)
        for h in range(nkv):
            k, v = s["k"][page, slot, h].to(f64), s["v"][page, slot, h].to(f64)
            if s["ks"] is not None:
                k, v = k * s["ks"][page, slot, h].to(f64)[:, None], v * s["vs"][page, slot, h].to(f64)[:, None]
            hs = slice(h * group, (h + 1) * group)
            o, l, p = _attend64(s["q"][i, hs].to(f64)[:, None], k, v, seen[None])
            out[i, hs], lse[i, hs] = o[:, 0], l[:, 0]
            gained += p.sum((0, 1))
        if mass is not None:
            mass[i, :n] = s["mass"][i, :n].to(f64) + gained
    made = {"out": out, "lse": lse}
    return dict(made, mass=mass) if case["mass"] else made
