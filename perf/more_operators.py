"""Performance cases of the decoding operators: the visibility masks of drafted
token trees, attention of such trees over the 4-bit paged cache, sampling with
temperature, top-k, top-p and min-p from given random numbers, the walk down a
tree along the sampled tokens, and the move of the accepted tokens' keys and
values to the places behind the prefix.

``run(state)`` is one call of an operator: in plain torch operations where
``own`` is false, through ``bit_mixed_precision_amd.bq`` where it is true.
``exact`` computes the same outputs in 64 bits from the definitions.

A tree's nodes are ordered, parents[i] < i, node 0 the root (parent -1).  The
sequence's cache ends with its nodes: node i is key seq_len - nodes + i.  Bit j
of row i of a mask (word j / 32, bit j % 32) says that node i sees node j.

A page of the cache holds, for each kv head, PAGE tokens as
  K codes   [PAGE][D/2]               byte d/2 holds d even in its low nibble
  V codes   [PAGE/4][units][4][U]     U = 2 bytes (D = 64) or 4: unit u of a
                                      token holds d = 2Uu .. 2Uu + 2U - 1
  K params  [PAGE][2] fp16            scale, min: value = code * scale + min
  V params  [PAGE][2] fp16
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one conversation's small tree: latency counts
        {"name": "mask 1 x 25", "op": "mask", "batch": 1, "nodes": 25, "len": 700},
        # a serving batch's trees
        {"name": "mask 256 x 64", "op": "mask", "batch": 256, "nodes": 64, "len": 8192},
        # one short conversation
        {"name": "attn b1 8 nodes len 700", "op": "attn", "batch": 1, "nodes": 8, "len": 700, "ragged": False, "hq": 32, "hkv": 8, "d": 128, "page": 16, "window": 0, "dtype": "fp16"},
        # a serving batch of ragged lengths
        {"name": "attn b16 32 nodes len <= 8192", "op": "attn", "batch": 16, "nodes": 32, "len": 8192, "ragged": True, "hq": 32, "hkv": 8, "d": 128, "page": 16, "window": 0, "dtype": "bf16"},
        # a few long contexts with wide trees
        {"name": "attn b3 61 nodes len 30001", "op": "attn", "batch": 3, "nodes": 61, "len": 30001, "ragged": False, "hq": 64, "hkv": 8, "d": 128, "page": 64, "window": 0, "dtype": "fp16"},
        # one token of one conversation, every filter on
        {"name": "sample 1 x 32000", "op": "sample", "rows": 1, "vocab": 32000, "k": True, "p": True, "min": True, "greedy": 0.0, "dtype": "fp16"},
        # a decode batch by temperature and top-p
        {"name": "sample 64 x 131072", "op": "sample", "rows": 64, "vocab": 131072, "k": False, "p": True, "min": False, "greedy": 0.0, "dtype": "bf16"},
        # the nodes of many trees, each request with its own settings, an odd vocabulary
        {"name": "sample 487 x 100003", "op": "sample", "rows": 487, "vocab": 100003, "k": True, "p": True, "min": True, "greedy": 0.25, "dtype": "fp32"},
        # one conversation's tree
        {"name": "accept 1 x 25", "op": "accept", "batch": 1, "nodes": 25},
        # a serving batch's trees
        {"name": "accept 256 x 64", "op": "accept", "batch": 256, "nodes": 64},
        # one layer of a small batch
        {"name": "compact 1 layer 3 x 25", "op": "compact", "layers": 1, "batch": 3, "nodes": 25, "len": 700, "taken": 4, "hkv": 8, "d": 128, "page": 16, "dtype": "fp16"},
        # every layer's cache of a serving batch
        {"name": "compact 32 layers 64 x 64", "op": "compact", "layers": 32, "batch": 64, "nodes": 64, "len": 350, "taken": 5, "hkv": 8, "d": 128, "page": 16, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "sample", "sample", "sample", "mask", "accept", "compact"])
    if op == "sample":
        vocab = _log(rng, 1000, 131072)
        return {"op": op, "rows": max(1, min(_log(rng, 1, 487), 487 * 100003 // vocab)), "vocab": vocab, "k": rng.random() < 0.6,
                "p": rng.random() < 0.7, "min": rng.random() < 0.4, "greedy": rng.choice([0.0, 0.0, 0.25]),
                "dtype": rng.choice(["fp16", "bf16", "fp32"])}
    nodes = _log(rng, 1, 64)
    if op in ("mask", "accept"):
        case = {"op": op, "batch": _log(rng, 1, 256), "nodes": nodes}
        return {**case, "len": _log(rng, 64, 8192)} if op == "mask" else case
    d, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "compact":
        return {"op": op, "layers": _log(rng, 1, 32), "batch": _log(rng, 1, 64), "nodes": nodes, "len": _log(rng, 64, 350),
                "taken": rng.randint(1, max(1, min(5, nodes // 2))), "hkv": hkv, "d": d, "page": page, "dtype": dtype}
    hq = hkv * rng.choice([1, 3, 4, 8])
    length = _log(rng, 100, 30000)
    # tokens of all sequences: no more codes and no more products than the largest
    most = int(min(130000 * 8 * 128 / (hkv * d), 3 * 61 * 30001 * 64 * 128 / (hq * nodes * d)))
    length = max(nodes, min(length, most))
    return {"op": op, "batch": max(1, min(_log(rng, 1, 32), most // length)), "nodes": nodes, "len": length,
            "ragged": rng.random() < 0.6, "hq": hq, "hkv": hkv, "d": d, "page": page, "window": rng.choice([0, 0, 0, 1024]),
            "dtype": dtype}


def work(case):
    c = case
    words = -(-c.get("nodes", 1) // 32)
    if c["op"] == "mask":
        total = c["batch"] * c["nodes"]
        return {"bytes": 4 * total + 4 * c["batch"] + 4 * total * (words + 1), "flops": total}
    if c["op"] == "accept":
        total = c["batch"] * c["nodes"]
        return {"bytes": 12 * total + 4 * total + 8 * c["batch"], "flops": total}
    if c["op"] == "sample":
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": c["rows"] * (c["vocab"] * size + 28), "flops": 4 * c["rows"] * c["vocab"]}
    if c["op"] == "compact":
        moved = c["layers"] * c["batch"] * (c["taken"] - 1) * c["hkv"]
        read = c["layers"] * c["batch"] * c["taken"] * c["hkv"]
        return {"bytes": moved * 2 * (c["d"] + 8) + read * (c["d"] + 8 + 4 * c["d"]), "flops": 4 * read * c["d"]}
    seen, pairs = 0, 0
    for n in _lengths(c):
        prefix = n - c["nodes"]
        seen += min(prefix, c["window"]) + c["nodes"] if c["window"] else n
        pairs += c["nodes"] * (min(n, c["window"]) if c["window"] else n)
    return {"bytes": seen * c["hkv"] * (c["d"] + 8) + c["batch"] * c["nodes"] * (c["hq"] * (4 * c["d"] + 4) + 4 * words),
            "flops": 4 * c["d"] * c["hq"] * pairs}


def _lengths(c):
    """The sequences' lengths with their nodes: all `len`, or ragged from a third of it up."""
    if not c["ragged"]:
        return [max(c["len"], c["nodes"])] * c["batch"]
    return [max(c["nodes"], c["len"] - (c["len"] * 2 // 3) * ((7 * i) % 16) // 15 - i) for i in range(c["batch"])]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _trees(batch, nodes, g):
    """Parents int32 [batch, nodes]: each node hangs on one of the few nodes
    before the middle of those before it, as trees of the likeliest
    continuations do, or on the one right before it."""
    i = torch.arange(nodes, device="cuda")
    wide = (torch.rand(batch, nodes, generator=g, device="cuda") * ((i + 1) // 2)).long()
    chain = torch.rand(batch, nodes, generator=g, device="cuda") < 0.2
    parents = torch.where(chain, i - 1, wide.minimum(i - 1))
    return parents.clamp(min=0).masked_fill(i == 0, -1).to(torch.int32)


def _closure(parents):
    """[batch, nodes, nodes] bool: node i sees j, itself and its ancestors."""
    n = parents.shape[1]
    i = torch.arange(n, device=parents.device)
    see = ((parents[..., None] == i) | (i[:, None] == i)).float()
    for _ in range(max(1, (n - 1).bit_length())):  # paths of twice the length
        see = (torch.bmm(see, see) > 0).float()
    return see > 0


def _words(see):
    """Bits [rows, n] as int32 words [rows, ceil(n / 32)], the lowest first."""
    rows, n = see.shape
    w = -(-n // 32)
    bits = torch.zeros(rows, w * 32, dtype=torch.int64, device=see.device)
    bits[:, :n] = see
    v = (bits.view(rows, w, 32) << torch.arange(32, device=see.device)).sum(2)
    return torch.where(v >= 1 << 31, v - (1 << 32), v).to(torch.int32)


def _bits(mask, n):
    """The words back as bool [rows, n]."""
    return ((mask[..., None] >> torch.arange(32, device=mask.device)) & 1).bool().flatten(1)[:, :n]


def _quantize_tokens(x):
    """4-bit codes, scale and min (fp16) of each row of x (its last dimension)."""
    x = x.float()
    lo = x.amin(-1, keepdim=True).half().float()
    scale = ((x.amax(-1, keepdim=True) - lo) / 15).half().float()
    codes = torch.where(scale > 0, ((x - lo) / scale).round(), torch.zeros_like(x)).clamp(0, 15)
    return codes, scale, lo


def _unit(d):
    return 2 if d == 64 else 4


def _fill_cache(k, v, page):
    """Pages [pages, hkv, PAGE, D] of keys and values as the cache's bytes [pages, bytes]."""
    pages, hkv, _, d = k.shape
    parts, params = [], []
    for x, is_v in ((k, False), (v, True)):
        codes, scale, lo = _quantize_tokens(x)
        codes = codes.to(torch.uint8)
        b = codes[..., 0::2] | (codes[..., 1::2] << 4)
        if is_v:
            u = _unit(d)
            b = b.view(pages, hkv, page // 4, 4, d // 2 // u, u).transpose(3, 4)
        parts.append(b.reshape(pages, hkv, -1))
        params.append(torch.cat([scale, lo], -1).half().view(pages, hkv, -1).view(torch.uint8))
    return torch.cat(parts + params, 2).view(pages, -1)


def _page_values(raw, hkv, d, page):
    """Bytes of pages [n, page bytes] -> (k codes, v codes [n, hkv, PAGE, D], k and v params [n, hkv, PAGE, 2] fp16)."""
    n = raw.shape[0]
    raw = raw.view(n, hkv, page * (d + 8))
    kb = raw[..., : page * d // 2].reshape(n, hkv, page, d // 2)
    u = _unit(d)
    vb = raw[..., page * d // 2: page * d].reshape(n, hkv, page // 4, d // 2 // u, 4, u).transpose(3, 4).reshape(n, hkv, page, d // 2)
    kp = raw[..., page * d: page * d + 4 * page].contiguous().view(torch.float16).view(n, hkv, page, 2)
    vp = raw[..., page * d + 4 * page:].contiguous().view(torch.float16).view(n, hkv, page, 2)
    spread = lambda b: torch.stack([b & 15, b >> 4], -1).view(n, hkv, page, d)  # noqa: E731
    return spread(kb), spread(vb), kp, vp


def _tables(lens, page, seed):
    """A block table int32 [batch, most] of shuffled pages (-1 past a sequence's end), and how many there are."""
    most = max(-(-n // page) for n in lens)
    pages = sum(-(-n // page) for n in lens)
    blocks = torch.full((len(lens), most), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    at = 0
    for i, n in enumerate(lens):
        w = -(-n // page)
        blocks[i, :w] = order[at: at + w]
        at += w
    return blocks.cuda(), pages


def _random_cache(pages, hkv, d, page, T, g):
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    cache = torch.empty(pages, hkv * page * (d + 8), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (hkv * page * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        # keys carry a channel's own offset, as they do after a projection's bias
        cache[i: i + n] = _fill_cache((normal(n, hkv, page, d) + 0.5 * normal(1, hkv, 1, d)).to(T), normal(n, hkv, page, d).to(T), page)
    return cache


def prepare(case, seed):
    c, g = case, _generator(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    uniform = lambda *shape: torch.rand(*shape, generator=g, device="cuda")  # noqa: E731
    s = dict(c)
    if c["op"] == "sample":
        rows, vocab = c["rows"], c["vocab"]
        # the bulk of a vocabulary, and a few dozen tokens that stand out, more in some rows than in others
        x = normal(rows, vocab) * 2
        at = torch.randint(0, vocab, (rows, 64), generator=g, device="cuda")
        x += torch.zeros_like(x).scatter_reduce_(1, at, uniform(rows, 64) * (3 + 9 * uniform(rows, 1)), "amax")
        s["logits"] = x.to(DTYPES[c["dtype"]])
        s["u"] = uniform(rows)
        s["t"] = torch.where(uniform(rows) < c["greedy"], 0.0, 0.6 + 0.6 * uniform(rows))
        some = lambda: uniform(rows) < 0.75  # noqa: E731  requests that set what the others leave off
        s["top_k"] = torch.where(some(), torch.randint(1, 101, (rows,), generator=g, device="cuda"), 0).to(torch.int32) if c["k"] else None
        s["top_p"] = torch.where(some() | (not c["min"]), 0.8 + 0.18 * uniform(rows), 1.0) if c["p"] else None
        s["min_p"] = torch.where(some(), 0.02 + 0.08 * uniform(rows), 0.0) if c["min"] else None
        return s
    b, n = c["batch"], c["nodes"]
    parents = _trees(b, n, g)
    if c["op"] == "mask":
        s["parents"] = parents
        s["lens"] = torch.randint(n, n + c["len"], (b,), generator=g, device="cuda", dtype=torch.int32)
        return s
    if c["op"] == "accept":
        # tokens that differ within a tree; a model agrees with one of a node's children more often than not
        first = torch.randint(0, 30000, (b, 1), generator=g, device="cuda")
        tokens = (first + 7 * torch.arange(n, device="cuda")).to(torch.int32)
        child = torch.zeros(b, n, dtype=torch.int64, device="cuda")
        child.scatter_reduce_(1, parents.clamp(min=0).long(), torch.arange(n, device="cuda").expand(b, n), "amax")
        agree = (uniform(b, n) < 0.7) & (child > 0)
        s["parents"], s["tokens"] = parents, tokens
        s["sampled"] = torch.where(agree, tokens.gather(1, child), tokens + 3)
        return s
    T, hkv, d, page = DTYPES[c["dtype"]], c["hkv"], c["d"], c["page"]
    if c["op"] == "compact":
        lens = [n + max(1, c["len"] - 3 * i) for i in range(b)]
        s["blocks"], pages = _tables(lens, page, seed)
        s["cache"] = _random_cache(c["layers"] * pages, hkv, d, page, T, g).view(c["layers"], pages, -1)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        # accepted nodes from behind the places that they move to: a pass can be made again on the same cache
        later = uniform(b, n).masked_fill(torch.arange(n, device="cuda") < c["taken"], -1.0).topk(max(1, c["taken"] - 1), 1)[1].sort(1)[0]
        path = torch.cat([torch.zeros(b, 1, dtype=torch.int64, device="cuda"), later], 1)[:, : c["taken"]]
        s["path"] = torch.cat([path, torch.full((b, 2), -1, device="cuda")], 1).to(torch.int32)
        s["count"] = torch.full((b,), c["taken"], dtype=torch.int32, device="cuda")
        # where the accepted tokens stand afterwards, in every layer
        t = (s["lens"].long() - n)[:, None] + torch.arange(c["taken"], device="cuda")
        slots = (s["blocks"].long().gather(1, t // page) * page + t % page).view(-1)
        s["slots"] = (torch.arange(c["layers"], device="cuda")[:, None] * (pages * page) + slots).view(-1)
        return s
    lens = _lengths(c)
    s["blocks"], pages = _tables(lens, page, seed)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cache"] = _random_cache(pages, hkv, d, page, T, g)
    s["mask"] = _words(_closure(parents).view(b * n, n))
    s["x"] = (normal(b * n, c["hq"], d) * 1.5).to(T)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    return {"mask": _mask, "attn": _attn, "sample": _sample, "accept": _accept, "compact": _compact}[state["op"]](state)


def _mask(s):
    if own:
        from bit_mixed_precision_amd import bq
        return bq.tree_mask(s["parents"], s["lens"])
    n = s["nodes"]
    see = _closure(s["parents"])
    depth = see.sum(2) - 1
    return _words(see.flatten(0, 1)), (s["lens"][:, None] - n + depth).to(torch.int32).view(-1)


def _accept(s):
    if own:
        from bit_mixed_precision_amd import bq
        return bq.tree_accept(s["tokens"], s["parents"], s["sampled"])
    tokens, sampled, n = s["tokens"], s["sampled"], s["nodes"]
    i = torch.arange(n, device="cuda")
    parents = s["parents"].long()
    match = (parents >= 0) & (tokens == sampled.gather(1, parents.clamp(min=0)))
    # of the children that match, the first one is taken
    child = torch.where((parents[:, None, :] == i[:, None]) & match[:, None, :], i, n).amin(2)
    taken = match & (child.gather(1, parents.clamp(min=0)) == i) | (i == 0)
    on = (_closure(s["parents"]) & ~taken[:, None, :]).sum(2) == 0
    count = on.sum(1)
    last = torch.where(on, i, -1).amax(1)
    path = torch.where(on, i, n).sort(1)[0]
    return torch.where(path < n, path, -1).to(torch.int32), count.to(torch.int32), sampled.gather(1, last[:, None]).view(-1)


def _sample(s):
    if own:
        from bit_mixed_precision_amd import bq
        return bq.sample(s["logits"], s["u"], s["t"], s["top_k"], s["top_p"], s["min_p"])
    x = s["logits"].double()  # which token a number falls on is decided at borders between two sums
    rows, vocab = x.shape
    t = s["t"].double()[:, None]
    top = x.amax(1, keepdim=True)
    w = torch.where(x == top, 1.0, torch.exp((x - top) / torch.where(t > 0, t, 1.0)))
    order = x.sort(dim=1, descending=True, stable=True)[1]
    v = w.gather(1, order)
    rank = torch.arange(vocab, device="cuda")
    keep = torch.where(t > 0, vocab, 1) > rank
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep &= rank < torch.where(k > 0, k, vocab)
    if s["top_p"] is not None:
        v = v * keep
        keep &= (v.cumsum(1) - v < s["top_p"].double()[:, None] * v.sum(1, keepdim=True)) | (rank == 0) | (s["top_p"] >= 1)[:, None]
    if s["min_p"] is not None:
        keep &= v >= s["min_p"].double()[:, None]
    w = w * torch.zeros_like(keep).scatter(1, order, keep)
    sums = w.cumsum(1)
    total = sums[:, -1:]
    past = (sums > s["u"].double()[:, None] * total) & (w > 0)
    index = torch.where(past, rank, vocab).amin(1)
    index = torch.where(index < vocab, index, torch.where(w > 0, rank, -1).amax(1))
    return index.to(torch.int32), (w.gather(1, index[:, None]) / total).log().float().view(-1)


def _compact(s):
    """Moves the accepted tokens behind the prefix, in every layer, and reads them."""
    T, hkv, d, page, layers = DTYPES[s["dtype"]], s["hkv"], s["d"], s["page"], s["layers"]
    if own:
        from bit_mixed_precision_amd import bq
        bq.kv4_compact(s["cache"], s["blocks"], s["lens"], s["path"], s["count"], page, hkv, d, max_q_len=s["nodes"])
        return bq.kv4_read(s["cache"].flatten(0, 1), s["slots"], page, hkv, d, T)
    taken, u = s["taken"], _unit(d)
    pages = s["cache"].shape[1]
    prefix = (s["lens"].long() - s["nodes"])[:, None]
    table = s["blocks"].long()

    def places(t):  # (page over all layers, token in it) of keys [batch, taken]
        at = (torch.arange(layers, device="cuda")[:, None] * pages + table.gather(1, t // page).view(1, -1)).view(-1)
        return at, (t % page).view(1, -1).expand(layers, -1).reshape(-1)

    fp, ft = places(prefix + s["path"][:, :taken].long())
    tp, tt = places(prefix + torch.arange(taken, device="cuda"))
    raw = s["cache"].view(layers * pages, hkv, page * (d + 8))
    kb = raw[:, :, : page * d // 2].unflatten(2, (page, d // 2))
    vb = raw[:, :, page * d // 2: page * d].unflatten(2, (page // 4, d // 2 // u, 4, u))
    kp = raw[:, :, page * d: page * d + 4 * page].unflatten(2, (page, 4))
    vp = raw[:, :, page * d + 4 * page:].unflatten(2, (page, 4))
    k, v, kq, vq = kb[fp, :, ft], vb[fp, :, ft // 4, :, ft % 4], kp[fp, :, ft], vp[fp, :, ft]
    kb[tp, :, tt], vb[tp, :, tt // 4, :, tt % 4], kp[tp, :, tt], vp[tp, :, tt] = k, v, kq, vq
    rp, rt = s["slots"] // page, s["slots"] % page
    out = []
    for codes, par in ((kb[rp, :, rt], kp[rp, :, rt]), (vb[rp, :, rt // 4, :, rt % 4].flatten(2), vp[rp, :, rt])):
        par = par.contiguous().view(torch.float16).float()
        codes = torch.stack([codes & 15, codes >> 4], -1).flatten(2).float()
        out.append((codes * par[..., :1] + par[..., 1:]).to(T))
    return out[0], out[1]


def _attn(s):
    b, n, hq, hkv, d, page = s["batch"], s["nodes"], s["hq"], s["hkv"], s["d"], s["page"]
    if own:
        from bit_mixed_precision_amd import bq
        return bq.attn_kv4_tree(s["x"], s["cache"], s["blocks"], s["lens"], page, hkv, s["mask"], window=s["window"], return_lse=True)
    T = s["x"].dtype
    most = s["blocks"].shape[1]
    kc, vc, kp, vp = _page_values(s["cache"][s["blocks"].clamp(min=0).view(-1).long()], hkv, d, page)

    def dense(codes, par):
        par = par.float()
        x = codes.float() * par[..., :1] + par[..., 1:]
        return x.view(b, most, hkv, page, d).transpose(1, 2).reshape(b * hkv, most * page, d)

    x = s["x"].float().view(b, n, hkv, hq // hkv, d).transpose(1, 2).reshape(b * hkv, -1, d) / math.sqrt(d)
    scores = torch.bmm(x, dense(kc, kp).transpose(1, 2).contiguous()).view(b, hkv, n, hq // hkv, most * page)
    see = _bits(s["mask"], n).view(b, n, n)
    key = torch.arange(most * page, device="cuda")
    prefix = (s["lens"].long() - n)[:, None, None]
    node = (key - prefix).expand(b, n, -1)
    on = (node < 0) | (node < n) & see.gather(2, node.clamp(0, n - 1))
    if s["window"]:  # the last keys of those that a row sees
        on &= on.flip(2).cumsum(2).flip(2) <= s["window"]
    scores = scores.masked_fill(~on[:, None, :, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.bmm((p / total).view(b * hkv, -1, most * page), dense(vc, vp)).view(b, hkv, n, hq // hkv, d)
    lse = (top + total.log()).squeeze(-1).transpose(1, 2).reshape(b * n, hq)
    return o.transpose(1, 2).reshape(b * n, hq, d).to(T), lse


# --------------------------------------------------------------------------
# the definitions, in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("mask", "accept"):  # whole numbers
        return None
    s = prepare(case, seed)
    f = torch.float64
    if s["op"] == "sample":
        # the log of the probability with which the token is drawn, from the kept tokens in sorted order
        logp = torch.empty(s["rows"], dtype=f, device="cuda")
        for i in range(s["rows"]):
            x, t = s["logits"][i].to(f), float(s["t"][i])
            if t <= 0:
                logp[i] = 0.0
                continue
            y, order = torch.sort(-x, stable=True)
            y = -y
            if s["top_k"] is not None and int(s["top_k"][i]) > 0:
                y = y[: int(s["top_k"][i])]
            z = y / t
            if s["top_p"] is not None and float(s["top_p"][i]) < 1:
                before = torch.cumsum(torch.softmax(z, 0), 0)
                z = z[: 1 + int((before[:-1] < float(s["top_p"][i])).sum())]
            if s["min_p"] is not None and float(s["min_p"][i]) > 0:
                z = z[z >= z[0] + math.log(float(s["min_p"][i]))]
            kept, by_index = torch.sort(order[: z.numel()])
            z = z[by_index]
            log_q = z - torch.logsumexp(z, 0)
            at = torch.searchsorted(torch.cumsum(log_q.exp(), 0), s["u"][i].to(f).view(1), right=True)
            logp[i] = log_q[min(int(at), z.numel() - 1)]
        return None, logp

    hkv, d, page = s["hkv"], s["d"], s["page"]
    if s["op"] == "compact":
        layers, b, n, taken = s["layers"], s["batch"], s["nodes"], s["taken"]
        k, v = (torch.empty(layers, b, taken, hkv, d, dtype=f, device="cuda") for _ in range(2))
        for i in range(b):
            t = int(s["lens"][i]) - n + s["path"][i, :taken].long()
            for layer in range(layers):
                kc, vc, kp, vp = _page_values(s["cache"][layer, s["blocks"][i, t // page].long()], hkv, d, page)
                at = torch.arange(taken, device="cuda")
                for to, c, p in ((k, kc, kp), (v, vc, vp)):
                    c, p = c[at, :, t % page].to(f), p[at, :, t % page].to(f)
                    to[layer, i] = c * p[..., :1] + p[..., 1:]
        return k.view(-1, hkv, d), v.view(-1, hkv, d)

    b, n, hq = s["batch"], s["nodes"], s["hq"]
    out = torch.empty(b * n, hq, d, dtype=f, device="cuda")
    lse = torch.empty(b * n, hq, dtype=f, device="cuda")
    for i in range(b):
        length = int(s["lens"][i])
        ids = s["blocks"][i, : -(-length // page)].long()
        kc, vc, kp, vp = _page_values(s["cache"][ids], hkv, d, page)
        hide = torch.zeros(n, length, dtype=torch.bool, device="cuda")
        for j in range(n):
            hide[:, length - n + j] = (s["mask"][i * n: (i + 1) * n, j // 32].long() & (1 << (j % 32))) == 0
        if s["window"]:
            for r in range(n):
                seen = torch.nonzero(~hide[r]).view(-1)
                hide[r, seen[: -s["window"]]] = True
        for h in range(hkv):
            kk = (kc[:, h].to(f) * kp[:, h, :, 0, None].to(f) + kp[:, h, :, 1, None].to(f)).reshape(-1, d)[:length]
            vv = (vc[:, h].to(f) * vp[:, h, :, 0, None].to(f) + vp[:, h, :, 1, None].to(f)).reshape(-1, d)[:length]
            at = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            x = s["x"][i * n: (i + 1) * n, at].to(f).reshape(-1, d)
            z = torch.mm(x, kk.t().contiguous()) / math.sqrt(d)
            z = z.masked_fill(hide.repeat_interleave(hq // hkv, 0), float("-inf"))
            lse[i * n: (i + 1) * n, at] = torch.logsumexp(z, 1).view(n, -1)
            out[i * n: (i + 1) * n, at] = torch.mm(torch.softmax(z, 1), vv).view(n, -1, d)
    return out, lse
