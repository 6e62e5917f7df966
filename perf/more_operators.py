"""What is measured of the paged serving step's operators, and their plain forms.

Three operators bring new tokens to a paged key-value cache and answer them
where many sequences continue one long text:

- rotation by position (``rotate``): pairs of a head's elements are turned by
  an angle that grows with the token's place, on one axis (text) or several
  (time, height and width of a video);
- append (``cache_append``): the new tokens' keys, rotated on the way, and
  values go to their cells of the paged cache (int8 cells with a binary16 scale
  each), and the queries beside them are rotated in the same call;
- attention over a shared prefix (``prefix_attn``): one new token per sequence
  attends the pages of the prefix that its group of sequences shares, and its
  own pages after it.

With ``own`` false, ``run`` is the plain form in elementary torch operations in
32 bits (angles in 64); with ``own`` true it makes the framework's calls.
"""

import math
import random

import torch

own = False

D = 128                                    # head dimension of the framework
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8}


# ---- cases --------------------------------------------------------------------

def _rotate(ntok, heads, others, dtype, pairs=64, axes=1, interleaved=False, inverse=False, far=4096):
    return {"op": "rotate", "ntok": ntok, "heads": heads, "others": others, "dtype": dtype, "pairs": pairs, "axes": axes,
            "interleaved": interleaved, "inverse": inverse, "far": far}


def _append(nseq, new, context, nkv, group, page, kv, x, layout="nhd", pairs=64, axes=1, interleaved=False, k_out=False,
            ragged=True):
    return {"op": "append", "nseq": nseq, "new": new, "context": context, "nkv": nkv, "group": group, "page": page,
            "kv": kv, "x": x, "layout": layout, "pairs": pairs, "axes": axes, "interleaved": interleaved, "k_out": k_out,
            "ragged": ragged}


def _prefix(groups, nseq, prefix, rest, nkv, group, page, kv, q, layout="nhd", ragged=True):
    return {"op": "prefix", "groups": groups, "nseq": nseq, "prefix": prefix, "rest": rest, "nkv": nkv, "group": group,
            "page": page, "kv": kv, "q": q, "layout": layout, "ragged": ragged}


def listed():
    return [
        # one new token's query heads, a slice of its fused projection, far into a text
        dict(_rotate(1, 32, 16, "bf16", far=1_000_000), name="rotate_one"),
        # a video's patches on three axes, queries of a fused projection
        dict(_rotate(16384, 24, 48, "bf16", axes=3), name="rotate_video"),
        # half of each head turned, neighbours as pairs, 32-bit values: the gradient's way back
        dict(_rotate(4097, 16, 0, "fp32", pairs=32, interleaved=True, inverse=True, far=131072), name="rotate_part_fp32"),
        # a single user's next token
        dict(_append(1, 1, 700, 8, 4, 16, "bf16", "bf16", ragged=False), name="append_one"),
        # a full serving batch's next tokens; heads outside cells, odd group
        dict(_append(256, 1, 250, 8, 7, 32, "fp16", "fp16", layout="hnd"), name="append_batch"),
        # ragged prompts read in: the rotated keys are also kept for the prompt's own attention
        dict(_append(8, 4096, 0, 8, 4, 16, "bf16", "bf16", k_out=True), name="append_prompt"),
        # image and text prompts to int8 cells, positions on three axes (their values are compared as binary16 numbers)
        dict(_append(4, 2048, 100, 8, 4, 64, "int8", "bf16", axes=3, interleaved=True), name="append_prompt_int8"),
        # a few samples of one short question: latency is all
        dict(_prefix(1, 4, 600, 40, 8, 4, 16, "bf16", "bf16"), name="prefix_short"),
        # a serving batch behind one system prompt
        dict(_prefix(1, 64, 4096, 1024, 8, 4, 16, "bf16", "bf16"), name="prefix_chat"),
        # many questions to one long document
        dict(_prefix(1, 32, 65536, 256, 8, 4, 16, "bf16", "bf16"), name="prefix_long"),
        # hundreds of samples of one problem: the products count, not the reading
        dict(_prefix(1, 512, 8192, 128, 2, 8, 32, "fp16", "fp16", layout="hnd"), name="prefix_many"),
        # several documents, each with its readers, in the framework's own form: int8 cells, 32-bit queries
        dict(_prefix(3, 40, 65536, 700, 2, 4, 64, "int8", "fp32"), name="prefix_groups_int8"),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("rotate", "append", "append", "prefix", "prefix", "prefix"))
    layout = rng.choice(("nhd", "hnd", "joint"))
    page = rng.choice((8, 16, 16, 24, 32, 48, 64, 128))
    nkv = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16))
    pairs = rng.choice((64, 64, 48, 32, 16, 8))
    axes = rng.choice((1, 1, 2, 3, 4))
    if op == "rotate":
        heads = _log_int(rng, 1, 64)
        dtype = rng.choice(("bf16", "fp16", "fp32"))
        # no more bytes than the largest listed one moves
        ntok = _log_int(rng, 1, 16384 * 24 * 2 // (heads * DTYPES[dtype].itemsize))
        return _rotate(ntok, heads, rng.choice((0, 2, 16)), dtype, pairs, axes, rng.random() < 0.5, rng.random() < 0.3,
                       _log_int(rng, 16, 1_000_000))
    if op == "append":
        kv = rng.choice(("bf16", "fp16", "int8"))
        x = rng.choice(("fp32", "bf16", "fp16")) if kv == "int8" else rng.choice((kv, kv, "fp32"))
        nseq = _log_int(rng, 1, 256)
        # tokens x heads within the listed prompts'
        most = 8 * 4096 * 48 // ((group + 2) * nkv * (2 if x == "fp32" else 1))
        new = rng.choice((1, _log_int(rng, 1, 8), _log_int(rng, 1, 4096)))
        new = max(1, min(new, most // nseq))
        context = rng.choice((0, rng.randint(0, 300)))
        return _append(nseq, new, context, nkv, group, page, kv, x, layout, pairs, axes, rng.random() < 0.5,
                       rng.random() < 0.3)
    kv = rng.choice(("bf16", "fp16", "int8"))
    q = rng.choice(("fp32", "bf16", "fp16")) if kv == "int8" else kv
    groups = rng.choice((1, 1, 2, 3, 5, 8))
    nseq = max(groups, _log_int(rng, 1, 512))
    # padded score elements and cells within the largest listed cases'
    most = min(32 * 32 * 65536 // (nseq * nkv * group), 65536 * 8 // (groups * nkv))
    prefix = _log_int(rng, 1, max(1, min(65536, most)))
    rest = _log_int(rng, 1, max(1, min(2048, 64 * 1024 * 8 // (nseq * nkv))))
    return _prefix(groups, nseq, prefix, rest, nkv, group, page, kv, q, layout)


def _lengths(n, longest, ragged, salt):
    """Lengths, a property of the case: the longest once, the others spread from an eighth of it."""
    if not ragged or longest == 0:
        return [longest] * n
    rng = random.Random("%d %d %d" % (n, longest, salt))
    rest = [rng.randint(min(longest, longest // 8 + 1), longest) for _ in range(n - 1)]
    at = rng.randint(0, n - 1)
    return rest[:at] + [longest] + rest[at:]


def _new_tokens(case):
    """New tokens of each sequence, and its length with them."""
    new = _lengths(case["nseq"], case["new"], case["ragged"] and case["new"] > 1, 1)
    return new, [a + b for a, b in zip(new, _lengths(case["nseq"], case["context"], case["ragged"], 2))]


def _members(case):
    """Sequences of each group."""
    n, g = case["nseq"], case["groups"]
    cuts = sorted(random.Random("%d %d" % (n, g)).sample(range(1, n), g - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [n])]


def _cell_bytes(kv):
    return 2 * D * DTYPES[kv].itemsize + (4 if kv == "int8" else 0)


def work(case):
    if case["op"] == "rotate":
        return {"bytes": case["ntok"] * (2 * case["heads"] * D * DTYPES[case["dtype"]].itemsize + 4 * case["axes"]),
                "flops": 6 * case["ntok"] * case["heads"] * case["pairs"]}
    if case["op"] == "append":
        tokens, size = sum(_new_tokens(case)[0]), DTYPES[case["x"]].itemsize
        heads = case["nkv"] * case["group"]
        moved = 2 * heads * D * size + case["nkv"] * (2 * D * size + _cell_bytes(case["kv"]))
        if case["k_out"]:
            moved += case["nkv"] * D * size
        return {"bytes": tokens * (moved + 4 * case["axes"]), "flops": 6 * tokens * (heads + case["nkv"]) * case["pairs"]}
    members, prefix = _members(case), _lengths(case["groups"], case["prefix"], case["ragged"], 3)
    rest = _lengths(case["nseq"], case["rest"], case["ragged"], 4)
    heads = case["nkv"] * case["group"]
    seen = sum(a * b for a, b in zip(members, prefix)) + sum(rest)
    return {"bytes": (sum(prefix) + sum(rest)) * case["nkv"] * _cell_bytes(case["kv"])
            + case["nseq"] * heads * (2 * D * DTYPES[case["q"]].itemsize + 4),
            "flops": 4 * D * heads * seen}


# ---- what a user's program has before the call --------------------------------

def _pool(npages, case, made, dev):
    """Key and value pages [npages, page, nkv, D] in the case's memory order: cells outside heads, heads outside
    cells, or keys and values of a page side by side."""
    page, nkv = case["page"], case["nkv"]
    if case["layout"] == "hnd":
        return tuple(made((npages, nkv, page, D)).transpose(1, 2) for _ in range(2))
    if case["layout"] == "joint":
        return made((npages, 2, page, nkv, D)).unbind(1)
    return made((npages, page, nkv, D)), made((npages, page, nkv, D))


def _rotation(case, ntok, far, gen, dev):
    """Frequencies from 1 down to 1e-5 or so, an axis for each in runs (time, height, width), and positions."""
    pairs, axes = case["pairs"], case["axes"]
    freqs = torch.pow(500000.0, -torch.arange(pairs, device=dev, dtype=torch.float64) / pairs).to(torch.float32)
    axis = (torch.arange(pairs, device=dev) * axes // pairs).to(torch.int32) if axes > 1 else None
    positions = torch.randint(0, far, (axes, ntok), generator=gen, device=dev, dtype=torch.int32)
    return {"freqs": freqs, "axis": axis, "positions": positions}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(shape, kind):
        return torch.randn(shape, generator=gen, device=dev, dtype=DTYPES[kind])

    def starts(n):
        return torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=dev)

    if case["op"] == "rotate":
        x = normal((case["ntok"], case["heads"] + case["others"], D), case["dtype"])[:, :case["heads"]]
        return dict(_rotation(case, case["ntok"], case["far"], gen, dev), case=case, x=x)
    page, nkv, kv, nseq = case["page"], case["nkv"], case["kv"], case["nseq"]
    heads = nkv * case["group"]
    if case["op"] == "append":
        new, lens = _new_tokens(case)
        ntok, cols = sum(new), -(-max(lens) // page)
        npages = nseq * cols
        k_pages, v_pages = _pool(npages, case, lambda s: torch.zeros(s, device=dev, dtype=DTYPES[kv]), dev)
        qkv = normal((ntok, heads + 2 * nkv, D), case["x"])
        state = {"case": case, "q": qkv[:, :heads], "k": qkv[:, heads:heads + nkv], "v": qkv[:, heads + nkv:],
                 "k_pages": k_pages, "v_pages": v_pages, "ks": None, "vs": None,
                 "table": torch.randperm(npages, generator=gen, device=dev).to(torch.int32).view(nseq, cols),
                 "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "cu": starts(new),
                 "k_out": torch.empty((ntok, nkv, D), device=dev, dtype=DTYPES[case["x"]]) if case["k_out"] else None}
        if kv == "int8":
            state["ks"], state["vs"] = (torch.zeros((npages, page, nkv), device=dev, dtype=torch.float16) for _ in range(2))
        return dict(state, **_rotation(case, ntok, 8192, gen, dev))
    prefix = _lengths(case["groups"], case["prefix"], case["ragged"], 3)
    rest = _lengths(nseq, case["rest"], case["ragged"], 4)
    members = _members(case)
    pcols, cols = -(-max(prefix) // page), -(-max(rest) // page)
    npages = case["groups"] * pcols + nseq * cols
    ks = vs = None
    if kv == "int8":
        k, v = _pool(npages, case, lambda s: torch.randint(-127, 128, s, generator=gen, device=dev, dtype=torch.int8), dev)
        # |key| near 1 and |value| near 1, the scales spread over a factor of four
        ks, vs = (torch.exp2(torch.rand((npages, page, nkv), generator=gen, device=dev) * 2 - 7.2).to(torch.float16)
                  for _ in range(2))
    else:
        k, v = _pool(npages, case, lambda s: normal(s, kv), dev)
    order = torch.randperm(npages, generator=gen, device=dev).to(torch.int32)
    return {"case": case, "q": normal((nseq, heads, D), case["q"]), "k": k, "v": v, "ks": ks, "vs": vs,
            "prefix_table": order[:case["groups"] * pcols].view(case["groups"], pcols),
            "prefix_lens": torch.tensor(prefix, dtype=torch.int32, device=dev), "cu": starts(members),
            "most": max(members), "table": order[case["groups"] * pcols:].view(nseq, cols),
            "lens": torch.tensor(rest, dtype=torch.int32, device=dev)}


# ---- the plain forms ------------------------------------------------------------

def _turned(x, s, inverse=False):
    """x [ntok, heads, D] in 32 bits, its pairs turned by position x frequency (the angle in 64 bits)."""
    c = s["case"]
    pairs = c["pairs"]
    position = s["positions"].double()
    if s["axis"] is not None:
        angle = position[s["axis"].long()].T * s["freqs"].double()
    else:
        angle = position[0][:, None] * s["freqs"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if inverse:
        sin = -sin
    x = x.float()
    if c["interleaved"]:
        a, b = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :pairs], x[..., pairs:2 * pairs]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., 2 * pairs:]), -1)


def _plain_rotate(s):
    return {"out": _turned(s["x"], s, s["case"]["inverse"]).to(s["x"].dtype)}


def _codes(x):
    """int8 codes and binary16 scales of the last dimension's rows."""
    scale = (x.abs().amax(-1) / 127.0).to(torch.float16)
    f = scale.float()[..., None]
    return torch.where(f > 0, torch.round(x / torch.where(f > 0, f, 1.0)), 0.0).clamp(-127, 127).to(torch.int8), scale


def _places(s):
    """The page and slot of every new token's cell."""
    cu, t = s["cu"].long(), torch.arange(s["q"].shape[0], device=s["q"].device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    cell = s["lens"].long()[seq] - cu[seq + 1] + t
    page = s["case"]["page"]
    return s["table"].long()[seq, cell // page], cell % page


def _plain_append(s):
    c = s["case"]
    k = _turned(s["k"], s)
    page, slot = _places(s)
    if c["kv"] == "int8":
        s["k_pages"][page, slot], s["ks"][page, slot] = _codes(k)
        s["v_pages"][page, slot], s["vs"][page, slot] = _codes(s["v"].float())
    else:
        s["k_pages"][page, slot] = k.to(s["k_pages"].dtype)
        s["v_pages"][page, slot] = s["v"].to(s["v_pages"].dtype)
    if c["k_out"]:
        s["k_out"].copy_(k)
    return _appended(s, _turned(s["q"], s).to(s["q"].dtype))


def _appended(s, q_out):
    """int8 cells as the values they stand for."""
    made = {"q": q_out, "k": s["k_pages"], "v": s["v_pages"]}
    if s["ks"] is not None:
        made = dict(made, k=s["k_pages"] * s["ks"][..., None], v=s["v_pages"] * s["vs"][..., None], ks=s["ks"], vs=s["vs"])
    return dict(made, k_out=s["k_out"]) if s["case"]["k_out"] else made


def _cells(pages, scale, table):
    """The cells of every row of the table in order, in 32 bits: [rows, cells, nkv, D]."""
    x = pages[table.long()].float()
    if scale is not None:
        x = x * scale[table.long()].float()[..., None]
    return x.flatten(1, 2)


def _sums(q, k, v, seen):
    """Largest logit, sum of exp(logit - largest), and that sum over the values, of q [n, nkv, rows, D] over
    k, v [n, cells, nkv, D] where `seen` [n, cells]."""
    logits = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1 / math.sqrt(D))
    logits = torch.where(seen[:, None, None], logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    return top, e.sum(-1, keepdim=True), torch.matmul(e, torch.where(seen[..., None, None], v, 0.0).transpose(1, 2))


def _plain_prefix(s):
    c, dev = s["case"], s["q"].device
    nkv, group, nseq = c["nkv"], c["group"], c["nseq"]
    q = s["q"].float().view(nseq, nkv, group, D)
    cu = s["cu"].long()
    # the groups' queries padded to [groups, most members], and back
    i = torch.arange(s["most"], device=dev)[None]
    member = torch.where(cu[:-1, None] + i < cu[1:, None], cu[:-1, None] + i, 0)
    rows = q[member].permute(0, 2, 1, 3, 4).flatten(2, 3)                       # [groups, nkv, most x group, D]
    k, v = _cells(s["k"], s["ks"], s["prefix_table"]), _cells(s["v"], s["vs"], s["prefix_table"])
    seen = torch.arange(k.shape[1], device=dev)[None] < s["prefix_lens"][:, None]
    t = torch.arange(nseq, device=dev)
    g = torch.searchsorted(cu[1:], t, right=True)
    first = tuple(x.unflatten(2, (s["most"], group))[g, :, t - cu[g]] for x in _sums(rows, k, v, seen))
    k, v = _cells(s["k"], s["ks"], s["table"]), _cells(s["v"], s["vs"], s["table"])
    second = _sums(q, k, v, torch.arange(k.shape[1], device=dev)[None] < s["lens"][:, None])
    top = torch.maximum(first[0], second[0])
    base = torch.where(top == -math.inf, 0.0, top)
    a, b = torch.exp(first[0] - base), torch.exp(second[0] - base)
    total = first[1] * a + second[1] * b
    out = (first[2] * a + second[2] * b) / torch.where(total == 0, 1.0, total)
    return {"out": out.reshape(s["q"].shape).to(s["q"].dtype), "lse": (top + torch.log(total)).reshape(nseq, -1)}


# ---- one pass --------------------------------------------------------------------

def run(state):
    c = state["case"]
    if not own:
        return {"rotate": _plain_rotate, "append": _plain_append, "prefix": _plain_prefix}[c["op"]](state)
    import sparse_attention_kv_qsa_gb300 as qsa
    if c["op"] == "rotate":
        return {"out": qsa.rotate(state["x"], state["positions"], state["freqs"], axis=state["axis"],
                                  interleaved=c["interleaved"], inverse=c["inverse"])}
    if c["op"] == "append":
        q_out, _ = qsa.cache_append(state["k"], state["v"], state["k_pages"], state["v_pages"], state["table"],
                                    state["lens"], cu=state["cu"], k_scale_f16=state["ks"], v_scale_f16=state["vs"],
                                    q=state["q"], positions=state["positions"], freqs=state["freqs"],
                                    axis=state["axis"], interleaved=c["interleaved"], k_out=state["k_out"])
        return _appended(state, q_out)
    out, lse = qsa.prefix_attn(state["q"], state["k"], state["v"], state["prefix_table"], state["prefix_lens"],
                               state["cu"], state["table"], state["lens"], k_scale_f16=state["ks"],
                               v_scale_f16=state["vs"])
    return {"out": out, "lse": lse}


# ---- the definitions in 64 bits ----------------------------------------------------

def _turned64(x, s, sign):
    """The pairs as complex numbers times exp(i sign angle), in 64 bits."""
    c, n = s["case"], s["case"]["pairs"]
    x = x.to(torch.float64)
    which = torch.zeros(n, dtype=torch.long, device=x.device) if s["axis"] is None else s["axis"].long()
    angle = torch.einsum("np,n->pn", s["positions"].to(torch.float64).index_select(0, which), s["freqs"].to(torch.float64))
    unit = torch.polar(torch.ones_like(angle), sign * angle)[:, None, :]
    both = x[..., :2 * n].unflatten(-1, (n, 2) if c["interleaved"] else (2, n))
    if not c["interleaved"]:
        both = both.transpose(-1, -2)
    both = torch.view_as_real(torch.view_as_complex(both.contiguous()) * unit)
    if not c["interleaved"]:
        both = both.transpose(-1, -2)
    out = x.clone()
    out[..., :2 * n] = both.flatten(-2)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "rotate":
        return {"out": _turned64(s["x"], s, -1.0 if case["inverse"] else 1.0)}
    page = case["page"]
    if case["op"] == "append":
        q, k, v = (_turned64(s["q"], s, 1.0), _turned64(s["k"], s, 1.0), s["v"].to(f64))
        made = {"q": q, "k": None, "v": None}
        if case["k_out"]:
            made["k_out"] = k
        if case["kv"] == "int8":
            return dict(made, ks=None, vs=None)     # codes and scales are roundings
        pools = [torch.zeros(s["k_pages"].shape, dtype=f64, device=k.device) for _ in range(2)]
        cu, lens = s["cu"].tolist(), s["lens"].tolist()
        for i, n in enumerate(lens):
            a, b = cu[i], cu[i + 1]
            cell = torch.arange(n - (b - a), n, device=k.device)
            at = s["table"][i].long()[cell // page]
            pools[0][at, cell % page], pools[1][at, cell % page] = k[a:b], v[a:b]
        return dict(made, k=pools[0], v=pools[1])
    group, nkv = case["group"], case["nkv"]
    out = torch.zeros(s["q"].shape, dtype=f64, device=s["q"].device)
    lse = torch.zeros(s["q"].shape[:2], dtype=f64, device=s["q"].device)
    cu, plens, lens = s["cu"].tolist(), s["prefix_lens"].tolist(), s["lens"].tolist()

    def cells(pages, scale, row, n, h):
        j = torch.arange(n, device=out.device)
        at = row.long()[j // page]
        x = pages[at, j % page, h].to(f64)
        return x if scale is None else x * scale[at, j % page, h].to(f64)[:, None]

    for i, n in enumerate(plens):
        for h in range(nkv):
            hs = slice(h * group, (h + 1) * group)
            pk, pv = (cells(x, y, s["prefix_table"][i], n, h) for x, y in ((s["k"], s["ks"]), (s["v"], s["vs"])))
            # a few sequences at once against the prefix, then each one's own cells
            for r in range(cu[i], cu[i + 1], 64):
                e = min(cu[i + 1], r + 64)
                shared = torch.einsum("sgd,nd->sgn", s["q"][r:e, hs].to(f64), pk) / math.sqrt(D)
                own_logits, own_values = [], []
                for t in range(r, e):
                    k, v = (cells(x, y, s["table"][t], lens[t], h) for x, y in ((s["k"], s["ks"]), (s["v"], s["vs"])))
                    own_logits.append(s["q"][t, hs].to(f64) @ k.T / math.sqrt(D))
                    own_values.append(v)
                ends = torch.stack([torch.logsumexp(x, -1) for x in own_logits])
                total = torch.logaddexp(torch.logsumexp(shared, -1), ends)
                lse[r:e, hs] = total
                out[r:e, hs] = torch.exp(shared - total[..., None]) @ pv
                for t in range(r, e):
                    out[t, hs] += torch.exp(own_logits[t - r] - total[t - r][:, None]) @ own_values[t - r]
    return {"out": out, "lse": lse}
