"""The paged 4-bit K/V cache operators, as cases to be measured: attention over the cache, appending
to it, reading rows back, copying pages and compacting accepted draft tokens.

The cache holds K and V in the library's affine format (qmm_quantize's scheme at 4 bits): a row of
`dim` values is `dim/8` little-endian 32-bit words of codes and one fp16 scale and bias a group.
Arrays are [pages, kv_heads, page, ...]; a sequence's position p is row p % page of page
table[b, p // page].  A call's new tokens are the last ones of their sequences, sequence b's at rows
cu[b]..cu[b+1]-1 of the token axis.

Shapes are those of the 8B-class decoder that the library's benchmark takes its projections from
(4096 -> 4096 q/o and 4096 -> 1024 k/v: 32 query heads on 8 K/V heads of 128), and smaller and
larger heads around it.  Sequence lengths, new tokens and accepted counts follow from the case alone;
the values, the order of the pages and the masks from the seed.
"""
from __future__ import annotations

import math

import torch

own = False

LOG_MAX = 131072  # longest cache drawn


# ------------------------------------------------------------------------------------------ cases
def listed():
    model = dict(heads=32, kv_heads=8, dim=128)
    att = dict(op="attend", window=0, tree=False, **model)
    return [
        # one sequence decoding at the 1,024-token cache of the pages' step times: latency
        dict(name="attend 1 token over 1024", dtype="bf16", seqs=1, tokens=1, length=1024, group=64, page=64, **att),
        # a decode step of a serving batch, lengths from short to 16k
        dict(name="attend 32 ragged decodes", dtype="bf16", seqs=32, tokens=1, length=16384, group=64, page=64, **att),
        # draft trees of up to 6 tokens verified in one pass, small pages and groups
        dict(name="attend 8 draft trees", dtype="fp16", seqs=8, tokens=6, length=4099, group=32, page=16,
             **{**att, "tree": True}),
        # a chunk of a long prompt over what is cached already
        dict(name="attend a prompt chunk", dtype="bf16", seqs=1, tokens=1024, length=8191, group=128, page=64, **att),
        # the append of a decode step, and of a whole prompt (each read back through the cache)
        dict(name="append 64 decodes", op="append", dtype="bf16", seqs=64, tokens=1, length=2000, group=64, page=64,
             heads=32, kv_heads=8, dim=128),
        dict(name="append a prompt", op="append", dtype="fp16", seqs=1, tokens=8191, length=8191, group=64, page=64,
             heads=32, kv_heads=8, dim=128),
        # rows read back dense: a short prefix for a draft model, and whole caches on their way to another device
        dict(name="gather short prefixes", op="gather", dtype="bf16", seqs=6, tokens=100, length=700, group=64, page=16,
             heads=32, kv_heads=8, dim=128),
        dict(name="gather whole caches", op="gather", dtype="fp16", seqs=16, tokens=4097, length=4097, group=32, page=64,
             heads=32, kv_heads=8, dim=128),
        # the partly filled last pages of a few forked sequences, and a pool being defragmented
        dict(name="copy 4 pages", op="copy", pairs=4, pages=64, group=64, page=64, kv_heads=8, dim=128),
        dict(name="copy 1500 pages", op="copy", pairs=1500, pages=4096, group=64, page=64, kv_heads=8, dim=128),
        # accepted tokens of draft trees moved together: a small batch, and a large one of wide trees
        dict(name="compact 8 drafts", op="compact", seqs=8, tokens=6, length=1030, group=64, page=64, kv_heads=8, dim=128),
        dict(name="compact 256 drafts", op="compact", seqs=256, tokens=64, length=500, group=64, page=64, kv_heads=8,
             dim=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "append", "gather", "copy", "compact"])
    dim = rng.choice([64, 128, 128, 256])
    c = dict(op=op, dim=dim, group=rng.choice([g for g in (32, 64, 128) if g <= dim]), page=rng.choice([16, 32, 64, 128, 256]),
             kv_heads=rng.choice([1, 2, 4, 8]))
    if op == "copy":
        c.update(pairs=_log_int(rng, 1, 1024), pages=0)
        while _copy_bytes(c) > 200e6:
            c["pairs"] = c["pairs"] * 2 // 3
        c["pages"] = 2 * c["pairs"] + rng.randrange(1, 50)
        return c
    if op == "compact":
        c.update(seqs=_log_int(rng, 1, 256), tokens=_log_int(rng, 1, 64))
        c["length"] = c["tokens"] + _log_int(rng, 1, 400)
        return c
    c["dtype"] = rng.choice(["bf16", "fp16"])
    c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    c["seqs"] = _log_int(rng, 1, 64)
    if op in ("append", "gather"):
        c["tokens"] = _log_int(rng, 1, 8192)
        c["seqs"] = max(1, min(c["seqs"], 8192 // c["tokens"]))
        c["length"] = c["tokens"] + _log_int(rng, 1, 2000)
        return c
    c.update(window=0, tree=False)
    kind = rng.choice(["one", "one", "verify", "verify", "chunk"])
    if kind == "chunk":
        c["seqs"] = rng.choice([1, 1, 2, 3])
        c["tokens"] = _log_int(rng, 65, 1024)
    else:
        c["tokens"] = 1 if kind == "one" else rng.randrange(2, 17)
    c["length"] = c["tokens"] + _log_int(rng, 1, LOG_MAX)
    if kind == "verify":
        c["tree"] = rng.random() < 0.5
    if not c["tree"] and rng.random() < 0.25:
        c["window"] = _log_int(rng, 1, c["length"])
    top = listed()
    most = {k: max(work(x)[k] for x in top if x["op"] == "attend") for k in ("bytes", "flops")}
    padded = 32 * 16384 * 8 * 128  # values of K that the largest listed case's plain form holds
    while work(c)["bytes"] > most["bytes"] or work(c)["flops"] > most["flops"] or \
            c["seqs"] * c["length"] * c["kv_heads"] * dim > padded or \
            c["seqs"] * c["length"] * c["heads"] * c["tokens"] > 32 * 1024 * 8192:
        if c["seqs"] > 4:
            c["seqs"] //= 2
        c["length"] = c["tokens"] + (c["length"] - c["tokens"]) * 2 // 3
        if c["length"] == c["tokens"]:
            c["tokens"] = c["length"] = max(1, c["tokens"] // 2)
    c["window"] = min(c["window"], c["length"])
    return c


def _new_tokens(c):
    """New tokens of each sequence: all the same where there is one sequence or one token, else ragged."""
    n, t = c["seqs"], c["tokens"]
    return [t if b == 0 else 1 + (7 * b + 3) % t for b in range(n)]


def _lengths(c):
    """Tokens of each sequence, the new ones among them: the first is the longest, the others spread below it."""
    new = _new_tokens(c)
    return [c["length"] if b == 0 else max(new[b], 1 + int((b * 0.6180339887498949) % 1.0 * c["length"])) for b in range(c["seqs"])]


def _row_bytes(c):
    """Bytes of one position of one head, K or V: codes, scales and biases."""
    return c["dim"] // 2 + c["dim"] // c["group"] * 4


def _copy_bytes(c):
    return 2 * c["pairs"] * 2 * c["kv_heads"] * c["page"] * _row_bytes(c)


def work(c):
    if c["op"] == "copy":
        return {"bytes": _copy_bytes(c), "flops": 0}
    kv = 2 * c["kv_heads"]
    if c["op"] == "compact":
        return {"bytes": 2 * sum(_accepted(c)) * kv * _row_bytes(c), "flops": 0}
    new, lens = _new_tokens(c), _lengths(c)
    t = sum(new)
    if c["op"] == "gather":
        return {"bytes": t * kv * (_row_bytes(c) + 2 * c["dim"]), "flops": 0}
    if c["op"] == "append":  # the dense rows in, the cache rows out and in again, the dense rows out
        return {"bytes": t * kv * (2 * _row_bytes(c) + 4 * c["dim"]), "flops": 0}
    w = c["window"]
    rows = sum(min(n, w + q - 1) if w else n for q, n in zip(new, lens))  # cache rows that some query sees
    seen = sum(min(n - q + i + 1, w) if w else n - q + i + 1 for q, n in zip(new, lens) for i in range(q))
    if c["tree"]:  # the draft tokens of a tree are seen along its paths
        seen = sum((n - q) * q + q * (q + 1) // 2 for q, n in zip(new, lens))
    return {"bytes": rows * kv * _row_bytes(c) + t * c["heads"] * (4 * c["dim"] + 4), "flops": 4 * c["dim"] * c["heads"] * seen}


def _accepted(c):
    """Accepted draft tokens of each sequence (one at least: the first is always kept)."""
    return [1 + (5 * b + 2) % n for b, n in enumerate(_new_tokens(c))]


# ----------------------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _quantized(x, group):
    """Rows [..., dim] as the cache holds them: words of 8 codes, scales and biases."""
    v = x.float().unflatten(-1, (-1, group))
    lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    s = ((hi - lo) / torch.full_like(lo, 15.0)).half()
    b = lo.half()
    sf = s.float()
    q = torch.where(sf == 0, torch.zeros_like(v), ((v - b.float()) / sf).round().clamp(0, 15))
    q = q.flatten(-2).to(torch.int32).unflatten(-1, (-1, 8))
    shift = 4 * torch.arange(8, device=x.device, dtype=torch.int32)
    return (q << shift).sum(-1, dtype=torch.int64).to(torch.int32), s.squeeze(-1), b.squeeze(-1)


def _values(packed, scales, biases):
    """The values of such rows, in 32 bits."""
    shift = 4 * torch.arange(8, device=packed.device, dtype=torch.int32)
    q = ((packed.unsqueeze(-1) >> shift) & 15).flatten(-2).float()
    s, b = scales.float().unsqueeze(-1), biases.float().unsqueeze(-1)
    return (s * q.unflatten(-1, (scales.shape[-1], -1)) + b).flatten(-2)


def _pool(c, pages, g):
    """`pages` filled pages.  K has a few channels that stand out, as projected keys do; V has none."""
    dev, parts = "cuda", []
    shape = (c["kv_heads"], c["page"], c["dim"])
    loud = 1 + 3 * (torch.rand(c["kv_heads"], 1, c["dim"], device=dev, generator=g) < 0.04)
    step = max(1, (1 << 26) // math.prod(shape))
    for kind in range(2):
        got = []
        for p in range(0, pages, step):
            x = torch.randn((min(step, pages - p), *shape), device=dev, generator=g)
            got.append(_quantized((x * loud if kind == 0 else x).half(), c["group"]))
        parts += [torch.cat(a) for a in zip(*got)]
    return parts


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(int(seed))
    st = {"case": c}
    if c["op"] == "copy":
        st["arrays"] = _pool(c, c["pages"], g)
        at = torch.randperm(c["pages"], device=dev, generator=g).to(torch.int32)
        st["src"], st["dst"] = at[: c["pairs"]].clone(), at[c["pairs"]: 2 * c["pairs"]].clone()
        return _with_cache(st)
    new, lens, page = _new_tokens(c), _lengths(c), c["page"]
    need = [-(-n // page) for n in lens]
    total = sum(need) + 3
    st["arrays"] = _pool(c, total, g)
    order = torch.randperm(total, device=dev, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    where = [sum(need[:b]) for b in range(len(need))]
    host = order.cpu()
    for b, n in enumerate(need):
        table[b, :n] = host[where[b]: where[b] + n]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    st["table"], st["lens"] = table.to(dev), ints(lens)
    st["starts"] = ints([n - q for n, q in zip(lens, new)])
    st["cu"] = ints([sum(new[:b]) for b in range(len(new) + 1)])
    st["tokens"], st["longest"], st["most_new"] = sum(new), max(lens), max(new)
    if c["op"] == "compact":
        kept = _accepted(c)
        # the first token and a rising choice among the others
        rise = torch.rand(len(new), max(new), device=dev, generator=g).cpu()
        keep = [torch.cat([torch.zeros(1, dtype=torch.int64), 1 + rise[b, 1:n].argsort()[: k - 1].sort().values])
                for b, (n, k) in enumerate(zip(new, kept))]
        st["keep"] = torch.cat(keep).to(torch.int32).to(dev)
        st["cu_keep"] = ints([sum(kept[:b]) for b in range(len(kept) + 1)])
        return _with_cache(st)
    dt = _TYPES[c["dtype"]]
    st["dtype"] = dt
    if c["op"] == "gather":
        return _with_cache(st)
    # q, k and v of the new tokens are slices of one projection's output
    wide = (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
    qkv = torch.randn(st["tokens"], wide, device=dev, generator=g).to(dt).unflatten(-1, (-1, c["dim"]))
    st["q"], st["k"], st["v"] = qkv.split([c["heads"], c["kv_heads"], c["kv_heads"]], dim=1)
    if c["op"] == "attend":
        st["scale"], st["window"], st["tree"] = c["dim"] ** -0.5, c["window"], None
        if c["tree"]:  # each draft token sees itself and what a parent before it sees
            pick = torch.rand(st["tokens"], device=dev, generator=g).cpu().tolist()
            bits, r = [], 0
            for n in new:
                mine = [1]
                for i in range(1, n):
                    mine.append(mine[int(pick[r + i] * i)] | 1 << i)
                bits += mine
                r += n
            st["tree"] = torch.tensor(bits, dtype=torch.int64, device=dev)
    return _with_cache(st)


def _with_cache(st):
    """The handle that a program keeps for its cache: the six arrays and their format."""
    if own:
        import bit_quantized_gemm_qmm_b200 as qmm

        st["cache"] = qmm.KVCache(*st["arrays"], group=st["case"]["group"])
    return st


# ------------------------------------------------------------------------------------- plain forms
def _rows(table, page, seq, pos):
    """(page, row) of position `pos` of sequence `seq`, element by element."""
    return table[seq, pos // page].long(), pos % page


def _spread(cu, count, like):
    """For `count` rows behind one another, the sequence that each belongs to and its place in it."""
    r = torch.arange(count, device=like.device)
    seq = torch.searchsorted(cu.long(), r, right=True) - 1
    return seq, r - cu.long()[seq]


def _plain_gather(st):
    c = st["case"]
    seq, i = _spread(st["cu"], st["tokens"], st["table"])
    p, r = _rows(st["table"], c["page"], seq, st["starts"].long()[seq] + i)
    k = _values(*[a[p, :, r] for a in st["arrays"][:3]])
    v = _values(*[a[p, :, r] for a in st["arrays"][3:]])
    return {"k": k.to(st["dtype"]), "v": v.to(st["dtype"])}


def _plain_append(st):
    c = st["case"]
    seq, i = _spread(st["cu"], st["tokens"], st["table"])
    p, r = _rows(st["table"], c["page"], seq, st["starts"].long()[seq] + i)
    for a, x in zip(st["arrays"], _quantized(st["k"], c["group"]) + _quantized(st["v"], c["group"])):
        a[p, :, r] = x
    return _plain_gather(st)


def _plain_attend(st):
    c, q, dev = st["case"], st["q"], st["q"].device
    n, longest, most = c["seqs"], st["longest"], st["most_new"]
    hk, grp = c["kv_heads"], c["heads"] // c["kv_heads"]
    at = st["table"].long().clamp(min=0)
    # [seqs, kv_heads, positions, dim], padded to whole pages of the longest sequence
    k, v = (_values(*[a[at].transpose(1, 2).flatten(2, 3) for a in st["arrays"][j: j + 3]])[:, :, :longest] for j in (0, 3))
    seq, i = _spread(st["cu"], st["tokens"], q)
    wide = torch.zeros(n, most, c["heads"], c["dim"], device=dev)
    wide[seq, i] = q.float()
    wide = wide.unflatten(2, (hk, grp)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [seqs, kv_heads, grp * most, dim]
    lens, new = st["lens"].long(), (st["cu"][1:] - st["cu"][:-1]).long()
    pos = torch.arange(longest, device=dev)
    mine = (lens - new)[:, None] + torch.arange(most, device=dev)  # [seqs, most]
    if st["tree"] is None:
        sees = (pos <= mine[..., None]) & (pos < lens[:, None, None])
        if st["window"]:
            sees &= pos > mine[..., None] - st["window"]
    else:
        bits = torch.zeros(n, most, dtype=torch.int64, device=dev)
        bits[seq, i] = st["tree"]
        d = pos - (lens - new)[:, None, None]  # place among the new tokens
        sees = (d < 0) | ((d < new[:, None, None]) & ((bits[..., None] >> d.clamp(0, 63)) & 1).bool())
    sees = sees[:, None, None].expand(n, hk, grp, most, longest).reshape(n, hk, grp * most, longest)
    s = (wide @ k.transpose(-1, -2) * st["scale"]).masked_fill(~sees, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).squeeze(-1)
    back = lambda x: x.unflatten(2, (grp, most)).transpose(1, 3).transpose(2, 3)[seq, i].flatten(1, 2)  # noqa: E731
    return {"o": back(o).to(q.dtype), "lse": back(lse)}


def _plain_copy(st):
    for a in st["arrays"]:
        a[st["dst"].long()] = a[st["src"].long()]
    return list(st["arrays"])


def _plain_compact(st):
    c = st["case"]
    seq, j = _spread(st["cu_keep"], st["keep"].numel(), st["table"])
    base = st["starts"].long()[seq]
    fp, fr = _rows(st["table"], c["page"], seq, base + st["keep"].long())
    tp, tr = _rows(st["table"], c["page"], seq, base + j)
    for a in st["arrays"]:
        a[tp, :, tr] = a[fp, :, fr]
    return list(st["arrays"])


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "gather": _plain_gather, "copy": _plain_copy,
                "compact": _plain_compact}[op](st)
    import bit_quantized_gemm_qmm_b200 as qmm

    cache = st["cache"]
    if op == "attend":
        o, lse = qmm.kv_attention(cache, st["q"], st["table"], st["lens"], st["cu"], scale=st["scale"],
                                  window=st["window"], tree=st["tree"])
        return {"o": o, "lse": lse}
    if op in ("append", "gather"):
        if op == "append":
            qmm.kv_append(cache, st["k"], st["v"], st["table"], st["lens"], st["cu"])
        k, v = qmm.kv_gather(cache, st["table"], st["starts"], st["cu"], st["tokens"], st["dtype"])
        return {"k": k, "v": v}
    if op == "copy":
        qmm.kv_copy_pages(cache, st["src"], st["dst"])
    else:
        qmm.kv_compact(cache, st["table"], st["starts"], st["keep"], st["cu_keep"])
    return list(st["arrays"])  # rows are moved as they are: the arrays themselves


# ------------------------------------------------------------------------------------ in 64 bits
def _row64(words, scales, biases, dim):
    """Rows of codes as 64-bit values: code k of a row is bits 4k..4k+3 of its little-endian bit stream."""
    at = torch.arange(dim, device=words.device)
    w = words.long().index_select(-1, at // 8) & 0xFFFFFFFF
    code = (w // 16 ** (at % 8)) % 16
    per = dim // scales.shape[-1]
    return code.double() * scales.double().index_select(-1, at // per) + biases.double().index_select(-1, at // per)


def _encoded64(x, group):
    """What the cache holds for rows x, as values: the scheme's own roundings (the range, its fifteenth, the distance to
    the bias and the quotient to 32 bits, scale and bias to 16), each from a 64-bit result."""
    to32, to16 = (lambda t: t.float().double()), (lambda t: t.half().double())
    v = x.double().reshape(*x.shape[:-1], -1, group)
    lo, hi = v.min(-1, keepdim=True).values, v.max(-1, keepdim=True).values
    s, b = to16(to32(to32(hi - lo) / torch.tensor(15.0, dtype=torch.float64, device=x.device))), to16(lo)
    code = torch.floor(to32(to32(v - b) / torch.where(s == 0, torch.ones_like(s), s)) + 0.5)
    tie = to32(to32(v - b) / torch.where(s == 0, torch.ones_like(s), s))
    code = torch.where((tie % 1 == 0.5) & (code % 2 == 1), code - 1, code).clamp(0, 15)
    code = torch.where(s == 0, torch.zeros_like(code), code)
    return (code * s + b).reshape(x.shape)


def exact(c, seed):
    if c["op"] in ("copy", "compact"):
        return None  # nothing is computed
    st = prepare(c, seed)
    table, lens, new, page = st["table"].cpu(), _lengths(c), _new_tokens(c), c["page"]
    if c["op"] == "append":
        return {"k": _encoded64(st["k"], c["group"]), "v": _encoded64(st["v"], c["group"])}
    out_a, out_b, r = [], [], 0
    for b, (n, q) in enumerate(zip(lens, new)):
        pages = table[b, : -(-n // page)].long().to("cuda")
        k, v = ([x[pages].permute(1, 0, 2, 3).reshape(c["kv_heads"], -1, x.shape[-1])[:, :n] for x in st["arrays"][j: j + 3]]
                for j in (0, 3))
        if c["op"] == "gather":
            out_a.append(_row64(*[x[:, n - q:] for x in k], c["dim"]).transpose(0, 1))
            out_b.append(_row64(*[x[:, n - q:] for x in v], c["dim"]).transpose(0, 1))
            continue
        qs = st["q"][r: r + q].double()
        col, row = torch.arange(n, device="cuda"), torch.arange(n - q, n, device="cuda")
        if st["tree"] is not None:
            bit = torch.ones(q, n, dtype=torch.bool, device="cuda")
            for j in range(q):
                bit[:, n - q + j] = (st["tree"][r: r + q] // 2 ** j) % 2 == 1
        else:
            bit = col[None] <= row[:, None]
            if c["window"]:
                bit &= col[None] > row[:, None] - c["window"]
        o = torch.empty(q, c["heads"], c["dim"], dtype=torch.float64, device="cuda")
        lse = torch.empty(q, c["heads"], dtype=torch.float64, device="cuda")
        per = c["heads"] // c["kv_heads"]
        for h in range(c["kv_heads"]):
            kh, vh = _row64(*[x[h] for x in k], c["dim"]), _row64(*[x[h] for x in v], c["dim"])
            for j in range(h * per, (h + 1) * per):
                w = torch.where(bit, qs[:, j] @ kh.T * st["scale"], torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
                lse[:, j] = torch.logsumexp(w, -1)
                o[:, j] = torch.exp(w - lse[:, j, None]) @ vh
        out_a.append(o)
        out_b.append(lse)
        r += q
    return dict(zip(("o", "lse") if c["op"] == "attend" else ("k", "v"), (torch.cat(out_a), torch.cat(out_b))))
