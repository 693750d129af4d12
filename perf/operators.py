"""What is measured of the attention operators over a paged key-value cache, and their plain forms.

Three operators, each a step of one transformer layer between its q/k/v products and its output
product:

  append   the rotary position rotation of q and k (one axis, or time / height / width), the
           rotated q rounded to fp16, the rotated k and v written into their slots of the paged
           cache (fp16 rows, or Q8_0: int8 codes with one fp16 scale per 32 values)
  decode   attention of one new token of each sequence over the cache
  prefill  attention of the new tokens of each sequence (packed one after the other) over the
           cache, which holds them as its last rows

Attention of a query at position p over the keys j of its sequence, D values a head:

  s_j = cap * tanh(scale * q.k_j / cap)  (cap = 0: scale * q.k_j), minus slope_head * |p - j|
  visible(j) = first <= j < length and (j < prefix or (j <= p and p - j < window))
  out = sum_j softmax(s)_j v_j over the visible keys; zeros where none is visible

Cache layout: a pool holds n_pages pages; a page holds, for each kv head, page_size rows:
fp16 [page_size][D], or Q8_0 as int8 codes [page_size][D] followed by fp16 scales
[page_size][D / 32].  `run` computes the plain forms in 32-bit floats, or calls the library.
"""
import math

import numpy as np
import torch

own = False

HEADS = ((32, 8), (32, 32), (16, 2), (12, 4), (40, 8), (24, 1))
DIMS = (32, 64, 96, 128, 160, 256)
PAGES = (8, 16, 32, 64, 128, 256)


# ----------------------------------------------------------------------------------------
# the cases
# ----------------------------------------------------------------------------------------

def _append(name, type, heads, kv, dim, page, tokens, seqs, rot, layout, axes=1, fused=False):
    return {"name": name, "op": "append", "type": type, "heads": heads, "kv": kv, "dim": dim, "page": page,
            "tokens": tokens, "seqs": seqs, "rot": rot, "layout": layout, "axes": axes, "fused": fused}


def _attn(name, op, type, heads, kv, dim, page, seqs, shortest, longest, new=1, out="f32", cap=0.0, window=0,
          prefix=0, slopes=False, docs=1, empty=False):
    # shortest / longest: the sequences' lengths, the new tokens included; new: the most new
    # tokens of a sequence (prefill)
    return {"name": name, "op": op, "type": type, "heads": heads, "kv": kv, "dim": dim, "page": page, "seqs": seqs,
            "shortest": shortest, "longest": longest, "new": new, "out": out, "cap": cap, "window": window,
            "prefix": prefix, "slopes": slopes, "docs": docs, "empty": empty}


def listed():
    return [
        # a single decode step of a small model: one row of each head, all latency
        _append("append_one_token", "f16", 32, 8, 64, 16, 1, 1, 64, "adjacent"),
        # a decode batch into an 8-bit cache: one row of each of 61 sequences
        _append("append_batch_q8", "q8_0", 32, 8, 128, 64, 61, 61, 128, "halves"),
        # an image grid of a multimodal prompt, three position axes, part of each row rotated,
        # q, k and v in one fused buffer
        _append("append_grid_q8", "q8_0", 32, 8, 128, 32, 4095, 1, 96, "halves", axes=3, fused=True),
        # a long prompt's rows, the largest append of a prefill step
        _append("append_prompt", "f16", 32, 8, 128, 64, 8192, 3, 128, "adjacent", fused=True),
        # one chat turn of a small model: 77 cached tokens, all latency
        _attn("decode_short", "decode", "f16", 32, 8, 64, 16, 1, 77, 77),
        # an ordinary ragged serving batch
        _attn("decode_batch", "decode", "f16", 32, 8, 128, 64, 48, 100, 4000),
        # a large batch over an 8-bit cache, capped scores
        _attn("decode_batch_q8", "decode", "q8_0", 32, 8, 128, 128, 128, 500, 8191, cap=30.0),
        # one long document: few rows, the work is split over the length
        _attn("decode_long", "decode", "f16", 32, 8, 128, 64, 1, 130001, 130001),
        # a few drafted tokens verified against a short context, 64-wide heads
        _attn("prefill_draft", "prefill", "f16", 32, 8, 64, 16, 1, 709, 709, new=9, out="f16"),
        # ragged prompts, some with cached context, capped scores in a sliding window
        _attn("prefill_batch", "prefill", "f16", 32, 8, 128, 64, 6, 150, 1900, new=1001, out="f16", cap=50.0,
              window=1024),
        # a chunk of packed documents over an 8-bit cache, scores biased by distance
        _attn("prefill_docs_q8", "prefill", "q8_0", 32, 8, 128, 64, 2, 5000, 8000, new=2000, out="f16", slopes=True,
              docs=3),
        # a whole long prompt with a bidirectional prefix: bound by the matrix products
        _attn("prefill_long", "prefill", "f16", 32, 8, 128, 64, 1, 8192, 8192, new=8192, out="f16", prefix=500),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode", "prefill"))
    type = rng.choice(("f16", "q8_0"))
    heads, kv = rng.choice(HEADS)
    dim, page = rng.choice(DIMS), rng.choice(PAGES)
    if op == "append":
        most = min(8192, 8192 * 48 * 128 // ((heads + 2 * kv) * dim))
        tokens = _log(rng, 1, most)
        c = _append("", type, heads, kv, dim, page, tokens, min(tokens, _log(rng, 1, 64)),
                    rng.choice((dim, dim // 2, 3 * dim // 4)), rng.choice(("adjacent", "halves")), rng.choice((1, 1, 3)),
                    rng.random() < 0.5)
    elif op == "decode":
        seqs = _log(rng, 1, 128)
        most = max(64, min(131072, 8192 * 128 * 8 * 128 // (seqs * kv * dim)))
        longest = _log(rng, 1, most)
        c = _attn("", op, type, heads, kv, dim, page, seqs, _log(rng, 1, longest), longest, 1, rng.choice(("f32", "f16")),
                  rng.choice((0.0, 0.0, 30.0)), rng.choice((0, 0, _log(rng, 16, 4096))), rng.choice((0, _log(rng, 1, 64))),
                  rng.random() < 0.25, rng.choice((1, 1, 4)), rng.random() < 0.25)
    else:
        seqs = _log(rng, 1, 8)
        new = _log(rng, 1, 4096)
        most = max(new, min(16384, 8192 * 8192 * 32 * 128 // (seqs * new * heads * max(dim, 128)),
                            8192 * 128 * 8 * 128 // (seqs * kv * dim)))
        longest = _log(rng, new, most)
        c = _attn("", op, type, heads, kv, dim, page, seqs, _log(rng, 1, longest), longest, new, "f16",
                  rng.choice((0.0, 0.0, 50.0)), rng.choice((0, 0, _log(rng, 16, 4096))),
                  rng.choice((0, 0, _log(rng, 1, 1000))), rng.random() < 0.25, rng.choice((1, 1, 4)), rng.random() < 0.25)
    del c["name"]
    return c


# ----------------------------------------------------------------------------------------
# what a case fixes: lengths, new tokens, prefixes and document starts
# ----------------------------------------------------------------------------------------

def _lengths(case):
    """(lengths, new tokens) of the sequences, spread geometrically and shuffled."""
    n, lo, hi = case["seqs"], min(case["shortest"], case["longest"]), case["longest"]
    at = np.linspace(1.0, 0.0, n) if n > 1 else np.ones(1)
    order = np.random.RandomState(n).permutation(n)
    lens = np.round(lo * (hi / lo) ** at).astype(np.int64)[order]
    new = np.ones(n, np.int64) if case["op"] == "decode" else \
        np.minimum(np.maximum(np.round(case["new"] * at ** 0.5).astype(np.int64), 1)[order], lens)
    if case["empty"]:
        # a sequence without keys (decode), without new tokens (prefill)
        if case["op"] == "decode":
            lens[0] = 0
        elif n > 1:
            new[0] = 0
    return lens, new


def _rows(case):
    """(sequence, position, first visible key) of every query, packed."""
    lens, new = _lengths(case)
    seq = np.repeat(np.arange(len(lens)), new)
    begin = np.concatenate([[0], np.cumsum(new)])
    pos = np.arange(begin[-1]) - begin[seq] + (lens - new)[seq]
    size = np.maximum(1, -(-lens // case["docs"]))[seq]
    first = np.maximum(pos, 0) // size * size
    return lens, new, begin, seq, pos, first


def work(case):
    if case["op"] == "append":
        rows, kv, dim = case["tokens"], case["kv"], case["dim"]
        stored = 2 * kv * dim * (2 if case["type"] == "f16" else 1.0625)
        back = 2 * kv * dim * 2 if case["type"] == "q8_0" else 0  # the rows read back as fp16 values
        return {"bytes": rows * ((case["heads"] + 2 * kv) * dim * 4 + case["heads"] * dim * 2 + stored + back
                                 + (stored if back else 0) + 4 * case["axes"] + 8),
                "flops": rows * (case["heads"] + kv) * case["rot"] * 3}
    lens, new, begin, seq, pos, first = _rows(case)
    window = case["window"] or 1 << 40
    prefix = np.minimum(case["prefix"], lens)[seq]
    low = np.maximum(first, pos - window + 1)  # the causal part: [low, pos]
    early = np.maximum(0, np.minimum(prefix, low) - first)  # keys of the prefix before it
    late = np.maximum(0, prefix - np.maximum(first, pos + 1))  # and after it
    seen = early + np.maximum(0, pos + 1 - low) + late
    seen[lens[seq] == 0] = 0
    keys = 0
    for s in range(len(lens)):  # the keys that some query of the sequence sees
        if new[s] == 0 or lens[s] == 0:
            continue
        r = slice(begin[s], begin[s + 1])
        mark = np.zeros(lens[s] + 1, np.int64)
        p = np.minimum(prefix[r], lens[s])
        for a, b in ((low[r], pos[r] + 1), (np.minimum(first[r], p), p)):
            np.add.at(mark, a, 1)
            np.add.at(mark, np.maximum(a, b), -1)
        keys += int((np.cumsum(mark)[:-1] > 0).sum())
    row = case["dim"] * (2 if case["type"] == "f16" else 1.0625)
    return {"bytes": 2 * keys * case["kv"] * row + len(seq) * case["heads"] * case["dim"] * (2 + (4 if case["out"] == "f32" else 2)),
            "flops": 4 * int(seen.sum()) * case["heads"] * case["dim"]}


# ----------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------

BASE, AXIS_SPLIT = 500000.0, (0.25, 0.375, 0.375)


def _axis(case):
    """The position axis of each rotated pair: sections of the row, time first."""
    half = case["rot"] // 2
    if case["axes"] == 1:
        return None
    cuts = np.round(np.cumsum(AXIS_SPLIT) * half).astype(np.int64)
    return np.searchsorted(cuts, np.arange(half), side="right").clip(0, 2).astype(np.uint8)


def _pool(g, case, n_pages):
    """A pool of cached rows: N(0, 1) values around a mean of their own for each channel."""
    kv, dim, page = case["kv"], case["dim"], case["page"]
    mean = torch.randn((1, kv, 1, dim), device="cuda", generator=g)
    if case["type"] == "f16":
        x = torch.randn((n_pages, kv, page, dim), device="cuda", generator=g, dtype=torch.float16)
        return x.add_(mean.half())
    pool = torch.empty((n_pages, kv, page * dim // 16 * 17), dtype=torch.uint8, device="cuda")
    codes, scales = _planes(pool, case)
    x = torch.randn((n_pages, kv, page, dim), device="cuda", generator=g, dtype=torch.float16)
    codes.copy_(x.add_(mean.half()).mul_(36).round_().clamp_(-127, 127))
    scales.copy_((torch.rand(scales.shape, device="cuda", generator=g) + 0.5) / 36)
    return pool


def _planes(pool, case):
    """Views of a Q8_0 pool: codes [pages][kv][page][D], scales [pages][kv][page][D / 32]."""
    kv, dim, page = case["kv"], case["dim"], case["page"]
    codes = pool[..., :page * dim].view(torch.int8).unflatten(-1, (page, dim))
    scales = pool[..., page * dim:].view(torch.float16).unflatten(-1, (page, dim // 32))
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    kv, dim, page, heads = case["kv"], case["dim"], case["page"], case["heads"]
    state = {"case": case}
    if case["op"] == "append":
        n, seqs = case["tokens"], case["seqs"]
        share = np.diff(np.round(np.linspace(0, n, seqs + 1)).astype(np.int64))
        offset = (np.arange(seqs) * 37) % page  # each sequence continues a page that it has begun
        per = -(-(share + offset) // page)
        n_pages = int(per.sum()) + 3
        perm = torch.randperm(n_pages, device="cuda", generator=g)
        seq = np.repeat(np.arange(seqs), share)
        at = np.arange(n) - np.repeat(np.cumsum(share) - share, share)
        cell = torch.from_numpy(at + offset[seq]).cuda()
        table = torch.from_numpy((np.cumsum(per) - per)[seq]).cuda()
        state["slots"] = perm[table + cell // page] * page + cell % page
        where = torch.from_numpy(at).cuda() + torch.randint(0, 100000, (seqs,), device="cuda", generator=g)[
            torch.from_numpy(seq).cuda()]
        if case["axes"] == 3:  # frames of 24 x 32 patches
            where = torch.stack([where // 768, where // 32 % 24, where % 32])
        state["pos"] = where.reshape(case["axes"], n).to(torch.int32)
        x = torch.randn((n, (heads + 2 * kv) * dim), device="cuda", generator=g)
        parts = x.split([heads * dim, kv * dim, kv * dim], 1)
        if not case["fused"]:
            parts = [p.contiguous() for p in parts]
        state["q"], state["k"], state["v"] = (p.unflatten(1, (-1, dim)) for p in parts)
        state["q_out"] = torch.empty((n, heads, dim), dtype=torch.float16, device="cuda")
        # turns per position of each pair, as 64-bit fractions of a turn
        freq = BASE ** (-np.arange(case["rot"] // 2) * 2.0 / case["rot"]) / (2 * math.pi)
        state["turns"] = torch.from_numpy((freq * 2.0 ** 64).astype(np.uint64).view(np.int64)).cuda()
        axis = _axis(case)
        state["axis"] = torch.zeros(case["rot"] // 2, dtype=torch.int64, device="cuda") if axis is None else \
            torch.from_numpy(axis.astype(np.int64)).cuda()
    else:
        lens, new, begin, seq, pos, first = _rows(case)
        most = max(1, int(-(-lens.max() // page)))
        need = np.maximum(1, -(-lens // page))
        n_pages = int(need.sum()) + 2
        table = np.zeros((len(lens), most), np.int64)
        for s in range(len(lens)):
            table[s, :need[s]] = np.arange(need[s]) + need[:s].sum()
        perm = torch.randperm(n_pages, device="cuda", generator=g)
        state["pages"] = perm[torch.from_numpy(table).cuda()].to(torch.int32)
        state["lens"] = torch.from_numpy(lens).to("cuda", torch.int32)
        state["starts"] = torch.from_numpy(begin).to("cuda", torch.int32)
        state["first"] = torch.from_numpy(first).to("cuda", torch.int32) if case["docs"] > 1 else None
        state["prefix"] = torch.from_numpy(np.minimum(case["prefix"], lens)).to("cuda", torch.int32) if case["prefix"] \
            else None
        state["slopes"] = torch.exp2(-8.0 * (torch.arange(heads, device="cuda") + 1) / heads) if case["slopes"] else None
        state["q"] = torch.randn((int(begin[-1]), heads, dim), device="cuda", generator=g).mul_(1.5).half()
        state["out"] = torch.empty(state["q"].shape, dtype=torch.float32 if case["out"] == "f32" else torch.float16,
                                   device="cuda")
    state["kpool"], state["vpool"] = _pool(g, case, n_pages), _pool(g, case, n_pages)
    return state


# ----------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    return _plain_append(state) if state["case"]["op"] == "append" else _plain_attention(state)


def _own(state):
    """The library's calls, their arguments marshalled once as a program over fixed buffers does."""
    case = state["case"]
    if "step" not in state:
        from gguf_block_quantized_gb300 import syn
        cache = syn.KVCache(syn.F16 if case["type"] == "f16" else syn.Q8_0, case["kv"], case["dim"], case["page"],
                            state["kpool"], state["vpool"])
        if case["op"] == "append":
            rope = syn.Rope(case["rot"], BASE, layout=syn.ROPE_HALVES if case["layout"] == "halves" else syn.ROPE_ADJACENT,
                            axis=_axis(case))
            state["step"] = syn.prepare_kv_append(cache, rope, state["k"], state["v"], state["pos"], state["slots"],
                                                  state["q"], state["q_out"])
            if case["type"] == "q8_0":
                state["back"] = syn.prepare_kv_read(cache, state["slots"])
        else:
            more = {"cap": case["cap"], "window": case["window"], "slopes": state["slopes"], "prefix": state["prefix"],
                    "first": state["first"]}
            if case["op"] == "decode":
                state["step"] = syn.prepare_attn_decode(cache, state["q"], state["pages"], state["lens"], state["out"],
                                                        **more)
            else:
                state["step"] = syn.prepare_attn_prefill(cache, state["q"], state["starts"], state["pages"],
                                                         state["lens"], state["out"], **more)
    state["step"]()
    if case["op"] != "append":
        return {"out": state["out"]}
    if case["type"] == "f16":
        return {"q": state["q_out"], "k": state["kpool"], "v": state["vpool"]}
    k, v = state["back"]()
    return {"q": state["q_out"], "k": k, "v": v}


def _turned(x, cos, sin, rot, layout):
    if layout == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(state):
    case = state["case"]
    page, rot = case["page"], case["rot"]
    # position times turns wraps at whole turns in 64-bit integers; 24 bits of the rest are kept
    turns = (state["pos"].long()[state["axis"]].t() * state["turns"]) >> 40
    angle = turns.float()[:, None, :] * (2 * math.pi / 2 ** 24)
    cos, sin = torch.cos(angle), torch.sin(angle)
    q = _turned(state["q"], cos, sin, rot, case["layout"]).half()
    k = _turned(state["k"], cos, sin, rot, case["layout"])
    pages, cells = state["slots"] // page, state["slots"] % page
    if case["type"] == "f16":
        state["kpool"][pages, :, cells] = k.half()
        state["vpool"][pages, :, cells] = state["v"].half()
        return {"q": q, "k": state["kpool"], "v": state["vpool"]}
    return {"q": q, "k": _plain_q8(state["kpool"], k, pages, cells, case),
            "v": _plain_q8(state["vpool"], state["v"], pages, cells, case)}


def _plain_q8(pool, x, pages, cells, case):
    codes, scales = _planes(pool, case)
    x = x.unflatten(-1, (-1, 32))
    d = (x.abs().amax(-1) / 127).half()
    y = x / torch.where(d == 0, torch.ones_like(d), d).float()[..., None]
    c = (torch.sign(y) * torch.floor(y.abs() + 0.5)).clamp(-127, 127)
    codes[pages, :, cells] = c.flatten(-2).to(torch.int8)
    scales[pages, :, cells] = d
    back = codes[pages, :, cells].float().unflatten(-1, (-1, 32)) * scales[pages, :, cells].float()[..., None]
    return back.flatten(-2).half()


def _plain_rows(pool, pages, case):
    """The cached rows of every sequence, padded: [seqs, kv, longest, D] in 32 bits."""
    if case["type"] == "f16":
        x = pool[pages].float()
    else:
        codes, scales = _planes(pool, case)
        x = (codes[pages].float().unflatten(-1, (-1, 32)) * scales[pages].float()[..., None]).flatten(-2)
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attention(state):
    case, lens, q = state["case"], state["lens"], state["q"]
    heads, kv, dim = case["heads"], case["kv"], case["dim"]
    new = torch.diff(state["starts"]) if case["op"] == "prefill" else torch.ones_like(lens)
    most = case["new"] if case["op"] == "prefill" else 1
    row = torch.arange(most, device="cuda")
    at = (state["starts"][:-1, None] + row).clamp(max=q.shape[0] - 1).long()  # [seqs, most] into the packed rows
    pos = (lens - new)[:, None] + row
    key = torch.arange(state["pages"].shape[1] * case["page"], device="cuda")
    seen = (key <= pos[..., None])
    if case["window"]:
        seen = seen & (pos[..., None] - key < case["window"])
    if state["prefix"] is not None:
        seen = seen | (key < state["prefix"][:, None, None])
    if state["first"] is not None:
        seen = seen & (key >= state["first"][at][..., None])
    seen = (seen & (key < lens[:, None, None]))[:, None, None]  # [seqs, 1, 1, most, keys]
    pages = state["pages"].long()
    k = _plain_rows(state["kpool"], pages, case)
    g = heads // kv
    x = q[at].float().unflatten(2, (kv, g)).permute(0, 2, 3, 1, 4)  # [seqs, kv, g, most, D]
    s = torch.matmul(x.flatten(2, 3), k.transpose(2, 3)).unflatten(2, (g, most))
    s *= 1 / math.sqrt(dim)
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    if state["slopes"] is not None:
        s = s - state["slopes"].view(kv, g, 1, 1) * (pos[..., None] - key).abs()[:, None, None]
    s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)))
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total == 0, torch.ones_like(total), total)
    v = _plain_rows(state["vpool"], pages, case)
    # rows past a sequence's end are not its own
    v = torch.where((key < lens[:, None])[:, None, :, None], v, torch.zeros_like(v))
    y = torch.matmul(p.flatten(2, 3), v).unflatten(2, (g, most))  # [seqs, kv, g, most, D]
    seq = torch.searchsorted(state["starts"][1:].contiguous(), torch.arange(q.shape[0], device="cuda", dtype=torch.int32),
                             right=True)
    back = torch.arange(q.shape[0], device="cuda") - state["starts"][seq]
    y = y.permute(0, 3, 1, 2, 4)[seq, back].flatten(1, 2)
    return {"out": y.to(state["out"].dtype)}


# ----------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    return _exact_append(case, state) if case["op"] == "append" else _exact_attention(case, state)


def _exact_append(case, state):
    rot, page, n = case["rot"], case["page"], case["tokens"]
    axis = _axis(case)
    out = {}
    k = state["k"].double().clone()
    q = state["q"].double().clone()
    for i in range(rot // 2):
        f = BASE ** (-2.0 * i / rot)
        a = state["pos"][0 if axis is None else int(axis[i])].double() * f
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
        u, w = (i, i + rot // 2) if case["layout"] == "halves" else (2 * i, 2 * i + 1)
        for x in (q, k):
            xu, xw = x[..., u].clone(), x[..., w].clone()
            x[..., u] = xu * c - xw * s
            x[..., w] = xu * s + xw * c
    out["q"] = q
    for name, x, pool in (("k", k, state["kpool"]), ("v", state["v"].double(), state["vpool"])):
        if case["type"] == "f16":
            whole = pool.double().transpose(1, 2).flatten(0, 1)  # [slots, kv, D]
            whole[state["slots"]] = x
            out[name] = whole.view(-1, page, case["kv"], case["dim"]).transpose(1, 2).contiguous()
        else:
            b = x.reshape(n, case["kv"], -1, 32)
            d = (b.abs().amax(-1, keepdim=True) / 127).half().double()
            y = torch.where(d > 0, b / d, torch.zeros_like(b))
            c = torch.where(y < 0, torch.ceil(y - 0.5), torch.floor(y + 0.5)).clamp(-127, 127)
            out[name] = (c * d).reshape(x.shape)
    return out


def _exact_attention(case, state):
    lens, new, begin, seq, pos, first = _rows(case)
    heads, kv, dim, page = case["heads"], case["kv"], case["dim"], case["page"]
    g = heads // kv
    y = torch.zeros((len(seq), heads, dim), dtype=torch.float64, device="cuda")
    for s in range(len(lens)):
        n, m = int(lens[s]), int(new[s])
        if n == 0 or m == 0:
            continue
        mine = state["pages"][s, :-(-n // page)].long()
        j = torch.arange(n, device="cuda")
        for h in range(kv):
            def rows(pool):
                if case["type"] == "f16":
                    return pool[mine, h].double().reshape(-1, dim)[:n]
                flat = pool[mine, h]
                c = flat[:, :page * dim].contiguous().view(torch.int8).double().reshape(-1, dim // 32, 32)
                d = flat[:, page * dim:].contiguous().view(torch.float16).double().reshape(-1, dim // 32, 1)
                return (c * d).reshape(-1, dim)[:n]
            k, v = rows(state["kpool"]), rows(state["vpool"])
            step = max(1, 40_000_000 // (n * g))
            for a in range(0, m, step):
                b = min(m, a + step)
                r = slice(int(begin[s]) + a, int(begin[s]) + b)
                p = torch.from_numpy(pos[r]).cuda()[:, None]
                ok = (j <= p) & (p - j < (case["window"] or 1 << 40))
                ok = (ok | (j < min(case["prefix"], n))) & (j >= torch.from_numpy(first[r]).cuda()[:, None])
                x = state["q"][r, h * g:(h + 1) * g].double()
                z = torch.einsum("tgd,jd->tgj", x, k) / math.sqrt(dim)
                if case["cap"]:
                    z = torch.tanh(z / case["cap"]) * case["cap"]
                if case["slopes"]:
                    z = z - state["slopes"][h * g:(h + 1) * g].double()[:, None] * (p - j).abs().double()[:, None]
                z = torch.where(ok[:, None], z, torch.full_like(z, -math.inf))
                w = torch.softmax(z, -1).nan_to_num(0.0)
                y[r, h * g:(h + 1) * g] = torch.einsum("tgj,jd->tgd", w, v)
    return {"out": y}
