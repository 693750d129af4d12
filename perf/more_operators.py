"""What is measured of the operators of speculative decoding and beam search, and their plain forms.

  tree      attention of the drafted tokens of each sequence, nodes of a tree, over the paged cache that
            holds them as its last rows: a node sees the context and its own ancestors
  pages     the pages of a cache, counted by how many sequences hold them: beams forked and extended
            (a shared page that is written to is copied first), drafts accepted (extended, the accepted
            path's rows packed, the rest given back), long sequences packed, pages copied
  logprobs  the log probabilities of given tokens, the entropy and the most likely tokens of rows of logits

Tree attention of node i with parent(i) < i, or -1 on the context of c rows; depth d(i) from 0; position
p = c + d(i):

  visible(j < c) = j < prefix or p - j < window;  visible(c + a) = a is i or an ancestor, d(i) - d(a) < window
  s = cap * tanh(scale * q.k / cap) - slope_head * (p - position of the key),  out = softmax(s) v

Pages: refs counts the tables that hold each page (0: free); tables hold -1 where there is no page; pages
are taken lowest first.  Log probabilities: z = scale * cap * tanh(x / cap) over the allowed tokens,
logp = z - log sum exp z; alternatives by x, ties to the lowest token.

A pool holds n_pages pages of, for each kv head, page_size rows: fp16 [page_size][D], or Q8_0 as int8
codes [page_size][D] followed by fp16 scales [page_size][D / 32].  `run` computes the plain forms in
32-bit floats, or calls the library.
"""
import math

import numpy as np
import torch

own = False

HEADS = ((32, 8), (32, 32), (16, 2), (12, 4), (40, 8), (24, 1))
DIMS = (32, 64, 96, 128, 160, 256)
PAGES = (8, 16, 32, 64, 128, 256)
VOCABS = (128256, 32000, 50257, 151936, 9973, 777)


# ----------------------------------------------------------------------------------------
# the cases
# ----------------------------------------------------------------------------------------

def _tree(name, type, heads, kv, dim, page, seqs, shortest, longest, nodes, cap=0.0, window=0, prefix=0, slopes=False):
    # shortest / longest: the sequences' lengths, the drafts included; nodes: the most drafts of one
    return {"name": name, "op": "tree", "type": type, "heads": heads, "kv": kv, "dim": dim, "page": page, "seqs": seqs,
            "shortest": shortest, "longest": longest, "nodes": nodes, "cap": cap, "window": window, "prefix": prefix,
            "slopes": slopes}


def _pages(name, op, type, kv, dim, page, seqs, shortest, longest, new=1, beams=1, keep=0.5):
    # new: the most rows added to a sequence; beams: sequences that share a prompt; keep: share of the rows kept
    return {"name": name, "op": op, "type": type, "kv": kv, "dim": dim, "page": page, "seqs": seqs, "shortest": shortest,
            "longest": longest, "new": new, "beams": beams, "keep": keep}


def _logits(name, type, rows, vocab, ids, top, cap=0.0, mask=False, scales=False):
    return {"name": name, "op": "logprobs", "type": type, "rows": rows, "vocab": vocab, "ids": ids, "top": top,
            "cap": cap, "mask": mask, "scales": scales}


def listed():
    return [
        # a few drafted tokens of one chat turn on a small model: all latency
        _tree("tree_small", "f16", 32, 8, 64, 16, 1, 317, 317, 9),
        # an ordinary ragged serving batch, trees of up to 26 nodes
        _tree("tree_batch", "f16", 32, 8, 128, 64, 24, 190, 4000, 26),
        # a larger batch over an 8-bit cache, small trees, capped scores
        _tree("tree_batch_q8", "q8_0", 32, 8, 128, 128, 48, 500, 6001, 13, cap=30.0),
        # one long document, a large tree: the work is split over the length
        _tree("tree_long", "f16", 32, 8, 128, 64, 1, 120001, 120001, 64),
        # a step of beam search, 4 beams of a short prompt: tables alone but for a page's rows
        _pages("beam_small", "beam", "f16", 8, 64, 16, 4, 101, 101, 1, beams=4),
        # drafts of a serving batch accepted: few rows packed, the other pages given back
        _pages("accept_batch", "accept", "f16", 8, 128, 64, 64, 200, 4000, 26, keep=0.2),
        # long sequences packed to the rows an eviction keeps
        _pages("evict_long", "evict", "q8_0", 8, 128, 64, 3, 21001, 60001, keep=0.5),
        # sequences moved to other pages (swapped, or a pool made dense)
        _pages("copy_pages", "copy", "f16", 8, 128, 64, 24, 1000, 9000),
        # the distribution of one new token
        _logits("logprobs_one", "f32", 1, 128256, 1, 20),
        # a decode batch under grammars, each sequence with its temperature, capped logits
        _logits("logprobs_masked", "f32", 61, 50257, 1, 5, cap=30.0, mask=True, scales=True),
        # the drafted children of each node of a batch's trees
        _logits("logprobs_drafts", "f32", 600, 128256, 4, 8),
        # a prompt scored
        _logits("logprobs_prompt", "f16", 4095, 128256, 1, 1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "tree", "beam", "accept", "evict", "copy", "logprobs", "logprobs"))
    type = rng.choice(("f16", "q8_0"))
    heads, kv = rng.choice(HEADS)
    dim, page = rng.choice(DIMS), rng.choice(PAGES)
    if op == "tree":
        seqs, nodes = _log(rng, 1, 64), _log(rng, 1, 128)
        most = min(120000, 120000 * 8 * 128 // (seqs * kv * dim), 120000 * 64 * 32 // (seqs * nodes * heads))
        longest = _log(rng, nodes, max(2 * nodes, most))
        c = _tree("", type, heads, kv, dim, page, seqs, _log(rng, 1, longest), longest, nodes, rng.choice((0.0, 0.0, 30.0)),
                  rng.choice((0, 0, 0, _log(rng, 4, 4096))), rng.choice((0, 0, _log(rng, 1, 64))), rng.random() < 0.2)
    elif op == "logprobs":
        vocab = rng.choice(VOCABS)
        c = _logits("", rng.choice(("f32", "f16")), _log(rng, 1, min(4095, 600 * 128256 // vocab)), vocab, rng.choice((0, 1, 1, 3, 8)),
                    rng.choice((0, 1, 5, 20, 50)), rng.choice((0.0, 0.0, 30.0)), rng.random() < 0.3, rng.random() < 0.3)
    else:
        seqs = _log(rng, 1, 64)
        beams = rng.choice((1, 2, 4, 8)) if op == "beam" else 1
        most = max(40, min(30000, 120000 * 8 * 128 // (seqs * kv * dim)))
        longest = _log(rng, 10, most)
        c = _pages("", op, type, kv, dim, page, max(1, seqs // beams) * beams, _log(rng, 5, longest), longest,
                   1 if op == "beam" else _log(rng, 1, 64), beams, round(rng.uniform(0.05, 0.95), 2))
    del c["name"]
    return c


# ----------------------------------------------------------------------------------------
# what a case fixes: lengths and numbers of new rows
# ----------------------------------------------------------------------------------------

def _lengths(case):
    """(lengths, new rows) of the sequences, spread geometrically and shuffled; of a beam search's, of its prompts'."""
    n, lo, hi = case["seqs"], min(case["shortest"], case["longest"]), case["longest"]
    n = n // case["beams"] if "beams" in case else n
    at = np.linspace(1.0, 0.0, n) if n > 1 else np.ones(1)
    order = np.random.RandomState(n).permutation(n)
    lens = np.round(lo * (hi / lo) ** at).astype(np.int64)[order]
    most = case["nodes"] if case["op"] == "tree" else case["new"]
    new = np.maximum(np.round(most * at ** 0.5).astype(np.int64), 1)[order]
    if case["op"] == "tree":
        new = np.minimum(new, lens)
    return lens, new


def _row_bytes(case):
    return case["dim"] * (2 if case["type"] == "f16" else 1.0625)


def work(case):
    if case["op"] == "logprobs":
        n, size = case["rows"] * case["vocab"], 4 if case["type"] == "f32" else 2
        return {"bytes": n * size + (n / 8 if case["mask"] else 0) + case["rows"] * (8 * case["ids"] + 8 * case["top"] + 4),
                "flops": 6 * n}
    lens, new = _lengths(case)
    kv, page = case["kv"], case["page"]
    if case["op"] == "tree":
        context = lens - new
        window = case["window"] or 1 << 40
        depth = np.log2(new + 1)
        seen = np.minimum(context, window) + np.minimum(case["prefix"], np.maximum(context - window, 0))
        rows = int(new.sum()) * case["heads"] * case["dim"]
        return {"bytes": 2 * int((seen + new).sum()) * kv * _row_bytes(case) + 4 * rows,
                "flops": 4 * case["heads"] * case["dim"] * float((new * (np.minimum(context, window) + depth)).sum())}
    row = 2 * kv * _row_bytes(case)  # a token's key and value rows
    pages = -(-lens // page)
    if case["op"] == "beam":
        shared = (lens % page).sum() * case["beams"]
        return {"bytes": float(2 * row * shared + 4 * 4 * pages.sum() * case["beams"]), "flops": 0}
    if case["op"] == "accept":
        kept = np.maximum(1, np.round(case["keep"] * new))
        return {"bytes": float(2 * row * (kept - 1).sum() + 4 * len(lens) * (4 + pages.max()) + 8 * new.sum()), "flops": 0}
    if case["op"] == "evict":
        return {"bytes": float(2 * row * np.round(case["keep"] * lens).sum()), "flops": 0}
    return {"bytes": float(2 * row * page * pages.sum()), "flops": 0}


# ----------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------

def _pool(g, case, n_pages):
    """A pool of cached rows: N(0, 1) values around a mean of their own for each channel."""
    kv, dim, page = case["kv"], case["dim"], case["page"]
    mean = torch.randn((1, kv, 1, dim), device="cuda", generator=g)
    x = torch.randn((n_pages, kv, page, dim), device="cuda", generator=g, dtype=torch.float16).add_(mean.half())
    if case["type"] == "f16":
        return x
    pool = torch.empty((n_pages, kv, page * dim // 16 * 17), dtype=torch.uint8, device="cuda")
    codes, scales = _planes(pool, case)
    codes.copy_(x.mul_(36).round_().clamp_(-127, 127))
    scales.copy_((torch.rand(scales.shape, device="cuda", generator=g) + 0.5) / 36)
    return pool


def _planes(pool, case):
    """Views of a Q8_0 pool: codes [pages][kv][page][D], scales [pages][kv][page][D / 32]."""
    kv, dim, page = case["kv"], case["dim"], case["page"]
    codes = pool[..., :page * dim].view(torch.int8).unflatten(-1, (page, dim))
    scales = pool[..., page * dim:].view(torch.float16).unflatten(-1, (page, dim // 32))
    return codes, scales


def _parents(rand, new):
    """A tree of drafts for each sequence: its first token, then each under one of the later half of those before."""
    out = []
    for n in new:
        i = np.arange(n)
        low = np.maximum(i // 2 - 1, 0)
        out.append(np.where(i == 0, -1, low + np.floor(rand.rand(n) * np.maximum(i - low, 1)).astype(np.int64)))
    return np.concatenate(out)


def _cuda(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rand = np.random.RandomState(int(seed) % (1 << 32))
    state = {"case": case}
    if case["op"] == "logprobs":
        n, vocab = case["rows"], case["vocab"]
        x = torch.randn((n, vocab), device="cuda", generator=g).mul_(2.5)
        likely = torch.randint(0, vocab, (n, 6), device="cuda", generator=g)  # what the model leans to
        x.scatter_add_(1, likely, torch.rand((n, 6), device="cuda", generator=g) * 12)
        state["logits"] = x if case["type"] == "f32" else x.half()
        ids = torch.randint(0, vocab, (n, case["ids"]), device="cuda", generator=g)
        if case["ids"]:
            ids[:, 0] = likely[:, 0]
        if case["ids"] > 1:  # nodes of fewer children
            ids.masked_fill_(torch.rand(ids.shape, device="cuda", generator=g) < 0.2, -1)
        state["ids"] = ids.to(torch.int32)
        state["mask"] = state["scales"] = None
        if case["mask"]:  # grammars: some allow much, some a few tokens, one row none
            words = -(-vocab // 32)
            share = torch.rand((n, 1), device="cuda", generator=g) ** 4
            share[n // 2] = 0 if n > 2 else 1
            on = torch.rand((n, words * 32), device="cuda", generator=g) < share
            bits = on.view(n, words, 32).long() << torch.arange(32, device="cuda")
            state["mask"] = bits.sum(-1).to(torch.int32)
        if case["scales"]:
            state["scales"] = 0.5 + torch.rand(n, device="cuda", generator=g)
        return state
    lens, new = _lengths(case)
    page = case["page"]
    if case["op"] == "tree":
        need = np.maximum(1, -(-lens // page))
        table = np.zeros((len(lens), need.max()), np.int64)
        for s in range(len(lens)):
            table[s, :need[s]] = np.arange(need[s]) + need[:s].sum()
        n_pages = int(need.sum()) + 2
        perm = torch.randperm(n_pages, device="cuda", generator=g)
        heads, dim = case["heads"], case["dim"]
        state["pages"] = perm[_cuda(table, torch.int64)].to(torch.int32)
        state["lens"] = _cuda(lens)
        state["starts"] = _cuda(np.concatenate([[0], np.cumsum(new)]))
        state["parents"] = _cuda(_parents(rand, new))
        state["prefix"] = _cuda(np.minimum(case["prefix"], lens)) if case["prefix"] else None
        state["slopes"] = torch.exp2(-8.0 * (torch.arange(heads, device="cuda") + 1) / heads) if case["slopes"] else None
        state["q"] = torch.randn((int(new.sum()), heads, dim), device="cuda", generator=g).mul_(1.5).half()
        state["out"] = torch.empty_like(state["q"])
        state["kpool"], state["vpool"] = _pool(g, case, n_pages), _pool(g, case, n_pages)
        return state
    _prepare_pages(case, state, g, rand, lens, new)
    return state


def _prepare_pages(case, state, g, rand, lens, new):
    """Sequences (beams of a prompt share its pages), free pages among theirs, and the rows to keep."""
    page, beams, seqs = case["page"], case["beams"], case["seqs"]
    lens, new = np.repeat(lens, beams), np.repeat(new, beams)
    held = -(-lens // page)
    most = int((held + 1 + -(-new // page)).max())
    n_pages = int(held.sum() + (2 + -(-new // page)).sum()) * (2 if case["op"] in ("beam", "copy") else 1)
    perm = rand.permutation(n_pages)
    table = np.full((seqs, most), -1, np.int64)
    taken = 0
    for s in range(seqs):
        lead = s % beams == 0
        # beams share the pages of their prompt: all but their last two
        same = 0 if lead else max(0, int(held[s]) - 2)
        table[s, :same] = table[s - s % beams, :same]
        table[s, same:held[s]] = perm[taken:taken + held[s] - same]
        taken += int(held[s]) - same
    refs = np.bincount(table[table >= 0], minlength=n_pages)
    state["refs"], state["pages"], state["lens"] = _cuda(refs), _cuda(table), _cuda(lens)
    state["starts"] = _cuda(np.concatenate([[0], np.cumsum(new)]))
    state["new_lens"] = torch.empty(seqs, dtype=torch.int32, device="cuda")
    state["kept_lens"] = torch.empty(seqs, dtype=torch.int32, device="cuda")
    if case["op"] == "beam":
        # each beam goes on from one of its group's
        state["from"] = _cuda(np.arange(seqs) // beams * beams + rand.randint(0, beams, seqs))
        state["none"] = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        state["new_pages"] = torch.full((seqs, most), -1, dtype=torch.int32, device="cuda")
    elif case["op"] in ("accept", "evict"):
        whole = new if case["op"] == "accept" else lens
        base = lens if case["op"] == "accept" else np.zeros_like(lens)
        kept = np.maximum(1, np.round(case["keep"] * whole).astype(np.int64))
        rows = []
        for n, k in zip(whole, kept):  # the first row stays, as an accepted path's root does
            rows.append(np.sort(np.concatenate([[0], 1 + rand.permutation(int(n) - 1)[:int(k) - 1]])))
        state["base"], state["rows"] = _cuda(base), _cuda(np.concatenate(rows))
        state["row_starts"] = _cuda(np.concatenate([[0], np.cumsum(kept)]))
    else:
        state["src"] = _cuda(table[table >= 0])
        state["dst"] = _cuda(perm[taken:2 * taken])
    state["slots"] = torch.empty(int(new.sum()), dtype=torch.int64, device="cuda")
    state["kpool"], state["vpool"] = _pool(g, case, n_pages), _pool(g, case, n_pages)


# ----------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_logprobs(state) if op == "logprobs" else _plain_tree(state) if op == "tree" else _plain_pages(state)


def _own(state):
    """The library's calls, their arguments marshalled once as a program over fixed buffers does."""
    case = state["case"]
    if "steps" not in state:
        from gguf_block_quantized_gb300 import syn
        if case["op"] == "logprobs":
            state["steps"] = [syn.prepare_logprobs(state["logits"], state["ids"] if case["ids"] else None, n_top=case["top"],
                                                   cap=case["cap"], scales=state["scales"], mask=state["mask"])]
        else:
            cache = syn.KVCache(syn.F16 if case["type"] == "f16" else syn.Q8_0, case["kv"], case["dim"], case["page"],
                                state["kpool"], state["vpool"])
            state["steps"] = _steps(syn, cache, case, state)
    for step in state["steps"]:
        got = step()
    if case["op"] == "tree":
        return {"out": state["out"]}
    if case["op"] != "logprobs":
        return _pages_out(state)
    out = {"entropy": got.entropy}
    if case["ids"]:
        out["logprob"] = got.logprob
    if case["top"]:
        out["top"], out["top_logprob"] = got.top, got.top_logprob
    return out


def _steps(syn, cache, case, state):
    if case["op"] == "tree":
        return [syn.prepare_attn_tree(cache, state["q"], state["starts"], state["parents"], state["pages"], state["lens"],
                                      state["out"], cap=case["cap"], window=case["window"], slopes=state["slopes"],
                                      prefix=state["prefix"])]
    if case["op"] == "beam":
        return [syn.prepare_kv_trim(cache, state["refs"], state["new_pages"], state["none"]),
                syn.prepare_kv_fork(cache, state["refs"], state["from"], state["pages"], state["lens"], state["new_pages"],
                                    state["new_lens"]),
                syn.prepare_kv_extend(cache, state["refs"], state["new_pages"], state["new_lens"], state["kept_lens"],
                                      state["slots"], state["starts"])]
    compact = syn.prepare_kv_compact(cache, state["refs"], state["pages"], state["base"], state["row_starts"], state["rows"],
                                     state["kept_lens"]) if "rows" in state else None
    if case["op"] == "accept":
        return [syn.prepare_kv_extend(cache, state["refs"], state["pages"], state["lens"], state["new_lens"], state["slots"],
                                      state["starts"]),
                compact, syn.prepare_kv_trim(cache, state["refs"], state["pages"], state["kept_lens"])]
    return [compact] if case["op"] == "evict" else [syn.prepare_kv_copy(cache, cache, state["src"], state["dst"])]


def _pages_out(state):
    """The pools' bits, and the tables, counts, lengths and slots of the calls that write them."""
    case = state["case"]
    bits = torch.int16 if case["type"] == "f16" else torch.uint8
    out = {"k": state["kpool"].view(bits), "v": state["vpool"].view(bits)}
    if case["op"] == "beam":
        out |= {"pages": state["new_pages"], "lens": state["kept_lens"], "refs": state["refs"], "slots": state["slots"]}
    elif case["op"] == "accept":
        out |= {"pages": state["pages"], "lens": state["kept_lens"], "refs": state["refs"], "slots": state["slots"]}
    elif case["op"] == "evict":
        out["lens"] = state["kept_lens"]
    return out


# ---- pages -----------------------------------------------------------------------------

def _plain_pages(state):
    case = state["case"]
    if case["op"] == "copy":
        src, dst = state["src"].long(), state["dst"].long()
        for pool in (state["kpool"], state["vpool"]):
            pool[dst] = pool[src]
    elif case["op"] == "beam":
        _plain_trim(state, state["new_pages"], state["none"])
        _plain_fork(state)
        _plain_extend(state, state["new_pages"], state["new_lens"], state["kept_lens"])
    else:
        if case["op"] == "accept":
            _plain_extend(state, state["pages"], state["lens"], state["new_lens"])
        _plain_compact(state)
        if case["op"] == "accept":
            _plain_trim(state, state["pages"], state["kept_lens"])
    return _pages_out(state)


def _plain_trim(state, pages, lens):
    column = torch.arange(pages.shape[1], device="cuda")
    gone = (column >= -(-lens[:, None] // state["case"]["page"])) & (pages >= 0)
    state["refs"].index_add_(0, pages.clamp(min=0).flatten(), -gone.flatten().int())
    pages.masked_fill_(gone, -1)


def _plain_fork(state):
    pages, lens, source = state["pages"], state["lens"], state["from"].long()
    state["new_lens"].copy_(lens[source])
    column = torch.arange(pages.shape[1], device="cuda")
    held = column < -(-state["new_lens"][:, None] // state["case"]["page"])
    state["new_pages"].copy_(torch.where(held, pages[source], torch.full_like(pages, -1)))
    state["refs"].index_add_(0, state["new_pages"].clamp(min=0).flatten(), held.flatten().int())


def _plain_extend(state, pages, lens, new_lens):
    """Rows lens .. lens + new - 1 of every sequence in pages of its own, taken lowest first."""
    page, refs = state["case"]["page"], state["refs"]
    width, n_pages = pages.shape[1], refs.shape[0]
    start, old = state["starts"].long(), lens.long()
    new = torch.diff(start)
    column = torch.arange(width, device="cuda")
    first, end = old // page, -(-(old + new) // page)
    fits = end <= width
    used = (column >= first[:, None]) & (column < end[:, None]) & fits[:, None] & (new > 0)[:, None]
    at = pages.clamp(min=0).long()
    shared = used & (pages >= 0) & (refs[at] > 1)
    order = torch.arange(pages.numel(), device="cuda").view_as(at)
    # a page whose holders all write in this call stays with the last of them
    writers = torch.zeros_like(refs).index_add_(0, at.flatten(), shared.flatten().int())
    last = torch.full((n_pages,), -1, dtype=torch.int64, device="cuda").scatter_reduce_(
        0, at.flatten(), torch.where(shared, order, torch.full_like(order, -1)).flatten(), "amax")
    kept = shared & (writers[at] == refs[at]) & (last[at] == order)
    free = torch.cumsum((refs == 0).long(), 0)
    missing = used & (pages < 0)
    enough = (missing | (shared & ~kept)).sum() <= free[-1]
    take = missing | (shared & ~(kept & enough))
    demand = take.sum(1)
    done = fits & (enough | (torch.cumsum(demand, 0) <= free[-1]) | (demand == 0))
    take = take & done[:, None]
    rank = torch.cumsum(take.flatten().long(), 0).view_as(at)
    got = torch.searchsorted(free, rank).clamp(max=n_pages - 1)
    away = take & shared
    refs.index_add_(0, at.flatten(), -away.flatten().int())
    refs.index_add_(0, torch.where(take, got, torch.zeros_like(got)).flatten(), take.flatten().int())
    # the rows of a first page that was shared
    mine = torch.arange(pages.shape[0], device="cuda")
    f = first.clamp(max=width - 1)
    moved = away[mine, f]
    src = at[mine, f]
    dst = torch.where(moved, got[mine, f], src)
    row = torch.arange(page, device="cuda")
    move = (moved[:, None] & (row < (old % page)[:, None])).view(-1, 1, page, 1)
    for plane in _all_planes(state):
        plane[dst] = torch.where(move, plane[src], plane[dst])
    pages.copy_(torch.where(take, got.to(torch.int32), pages))
    new_lens.copy_(old + torch.where(done, new, torch.zeros_like(new)))
    token = torch.arange(state["slots"].shape[0], device="cuda")
    s = torch.searchsorted(start[1:].contiguous(), token, right=True)
    at_row = old[s] + token - start[s]
    slot = pages[s, (at_row // page).clamp(max=width - 1)].long() * page + at_row % page
    state["slots"].copy_(torch.where(done[s], slot, torch.full_like(slot, -1)))


def _all_planes(state):
    """The pools as [pages][kv][page][values]."""
    pools = (state["kpool"], state["vpool"])
    return pools if state["case"]["type"] == "f16" else _planes(pools[0], state["case"]) + _planes(pools[1], state["case"])


def _plain_compact(state):
    page, pages = state["case"]["page"], state["pages"].long()
    start, rows, base = state["row_starts"].long(), state["rows"].long(), state["base"].long()
    i = torch.arange(rows.shape[0], device="cuda")
    s = torch.searchsorted(start[1:].contiguous(), i, right=True)
    to, come = base[s] + i - start[s], base[s] + rows
    for plane in _all_planes(state):
        plane[pages[s, to // page], :, to % page] = plane[pages[s, come // page], :, come % page]
    state["kept_lens"].copy_(base + torch.diff(start))


# ---- tree attention --------------------------------------------------------------------

def _plain_rows(pool, pages, case):
    """The cached rows of every sequence, padded: [seqs, kv, longest, D] in 32 bits."""
    if case["type"] == "f16":
        x = pool[pages].float()
    else:
        codes, scales = _planes(pool, case)
        x = (codes[pages].float().unflatten(-1, (-1, 32)) * scales[pages].float()[..., None]).flatten(-2)
    return x.transpose(1, 2).flatten(2, 3)


def _plain_tree(state):
    case, lens, q = state["case"], state["lens"].long(), state["q"]
    heads, kv, dim, most = case["heads"], case["kv"], case["dim"], case["nodes"]
    start = state["starts"].long()
    new = torch.diff(start)
    node = torch.arange(most, device="cuda")
    at = (start[:-1, None] + node).clamp(max=q.shape[0] - 1)  # [seqs, most] into the packed nodes
    up = torch.where(node < new[:, None], state["parents"].long()[at], torch.full_like(at, -1))
    # powers of (identity + parent) count walks to each ancestor: positive where there is one
    step = (up[..., None] == node).double() + torch.eye(most, device="cuda", dtype=torch.float64)
    above = torch.linalg.matrix_power(step, most) > 0  # [seqs, most, most]: node, its ancestors and itself
    depth = above.sum(-1) - 1
    context = (lens - new)[:, None]
    key = torch.arange(state["pages"].shape[1] * case["page"], device="cuda")
    # the key's position: its row, or its node's depth past the context
    draft = key - context  # [seqs, keys]
    among = (draft >= 0) & (draft < new[:, None])
    there = draft.clamp(0, most - 1)
    key_pos = torch.where(among, context + torch.gather(depth, 1, there), key)
    pos = context + depth
    far = pos[..., None] - key_pos[:, None]  # [seqs, most, keys]
    near = far < (case["window"] or 1 << 40)
    seen = (draft < 0)[:, None] & near
    if state["prefix"] is not None:
        seen = seen | ((draft < 0) & (key < state["prefix"][:, None]))[:, None]
    seen = seen | (among[:, None] & near & torch.gather(above, 2, there[:, None].expand(-1, most, -1)))
    pages = state["pages"].long()
    k = _plain_rows(state["kpool"], pages, case)
    g = heads // kv
    x = q[at].float().unflatten(2, (kv, g)).permute(0, 2, 3, 1, 4)  # [seqs, kv, g, most, D]
    s = torch.matmul(x.flatten(2, 3), k.transpose(2, 3)).unflatten(2, (g, most))
    s *= 1 / math.sqrt(dim)
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    if state["slopes"] is not None:
        s = s - state["slopes"].view(kv, g, 1, 1) * far[:, None, None]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)))
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total == 0, torch.ones_like(total), total)
    v = _plain_rows(state["vpool"], pages, case)
    y = torch.matmul(p.flatten(2, 3), v).unflatten(2, (g, most))  # [seqs, kv, g, most, D]
    token = torch.arange(q.shape[0], device="cuda")
    seq = torch.searchsorted(start[1:].contiguous(), token, right=True)
    state["out"].copy_(y.permute(0, 3, 1, 2, 4)[seq, token - start[seq]].flatten(1, 2))
    return {"out": state["out"]}


# ---- log probabilities -----------------------------------------------------------------

def _plain_logprobs(state):
    case = state["case"]
    x = state["logits"].float()
    vocab = x.shape[1]
    if state["mask"] is not None:
        on = (state["mask"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        x = x.masked_fill(on.flatten(1)[:, :vocab] == 0, -math.inf)
    z = case["cap"] * torch.tanh(x / case["cap"]) if case["cap"] else x
    if case["cap"]:
        z = torch.where(x == -math.inf, x, z)
    if state["scales"] is not None:
        z = z * state["scales"][:, None]
    top = z.amax(1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)  # (a row without a token)
    d = z - top
    e = torch.exp(d)
    total = e.sum(1)
    log_total = torch.log(torch.where(total == 0, torch.ones_like(total), total))
    some = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1)
    out = {"entropy": log_total - some / torch.where(total == 0, torch.ones_like(total), total)}
    if case["ids"]:
        ids = state["ids"].long()
        got = torch.gather(d, 1, ids.clamp(min=0)) - log_total[:, None]
        out["logprob"] = torch.where(ids < 0, torch.zeros_like(got), got)
    if case["top"]:
        # a whole number that orders by value, then lowest token first
        b = (x + 0.0).view(torch.int32)
        key = ((b ^ ((b >> 31) & 0x7FFFFFFF)).long() << 32) - torch.arange(vocab, device="cuda")
        token = torch.topk(key, case["top"], 1).indices
        got = torch.gather(d, 1, token) - log_total[:, None]
        out["top"] = torch.where(got == -math.inf, torch.full_like(token, -1), token).to(torch.int32)
        out["top_logprob"] = got
    return out


# ----------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "logprobs":
        return _exact_logprobs(case, prepare(case, seed))
    if case["op"] == "tree":
        return _exact_tree(case, prepare(case, seed))
    return None  # whole numbers and copies


def _exact_tree(case, state):
    lens, new = _lengths(case)
    heads, kv, dim, page = case["heads"], case["kv"], case["dim"], case["page"]
    g, begin = heads // kv, np.concatenate([[0], np.cumsum(new)])
    parents = state["parents"].cpu().numpy()
    y = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    for s in range(len(lens)):
        n, m = int(lens[s]), int(new[s])
        c = n - m
        up = parents[begin[s]:begin[s + 1]]
        depth, chain = np.zeros(m, np.int64), np.zeros((m, m), bool)
        for i in range(m):
            if up[i] >= 0:
                depth[i] = depth[up[i]] + 1
                chain[i] = chain[up[i]]
            chain[i, i] = True
        where = np.concatenate([np.arange(c), c + depth])  # each key's position
        far = torch.from_numpy(c + depth[:, None] - where[None]).cuda()
        ok = np.concatenate([np.ones((m, c), bool), chain], 1)
        ok = torch.from_numpy(ok).cuda() & (far < (case["window"] or 1 << 40))
        ok[:, :min(case["prefix"], c)] = True
        mine = state["pages"][s, :-(-n // page)].long()
        for h in range(kv):
            def rows(pool):
                flat = pool[mine, h]
                if case["type"] == "f16":
                    return flat.double().reshape(-1, dim)[:n]
                codes = flat[:, :page * dim].contiguous().view(torch.int8).double().reshape(-1, dim // 32, 32)
                scale = flat[:, page * dim:].contiguous().view(torch.float16).double().reshape(-1, dim // 32, 1)
                return (codes * scale).reshape(-1, dim)[:n]
            x = state["q"][begin[s]:begin[s + 1], h * g:(h + 1) * g].double()
            z = torch.einsum("tgd,jd->tgj", x, rows(state["kpool"])) / math.sqrt(dim)
            if case["cap"]:
                z = torch.tanh(z / case["cap"]) * case["cap"]
            if case["slopes"]:
                z = z - state["slopes"][h * g:(h + 1) * g].double()[:, None] * far.double()[:, None]
            w = torch.softmax(torch.where(ok[:, None], z, torch.full_like(z, -math.inf)), -1)
            y[begin[s]:begin[s + 1], h * g:(h + 1) * g] = torch.einsum("tgj,jd->tgd", w, rows(state["vpool"]))
    return {"out": y}


def _exact_logprobs(case, state):
    """A few hundred rows at a time, by the library's own log_softmax in 64 bits."""
    vocab, parts = case["vocab"], []
    for a in range(0, case["rows"], 256):
        x = state["logits"][a:a + 256].double()
        z = x
        if case["cap"]:
            z = torch.tanh(z / case["cap"]) * case["cap"]
        if case["scales"]:
            z = z * state["scales"][a:a + 256].double()[:, None]
        if case["mask"]:
            words = state["mask"][a:a + 256].long() & 0xFFFFFFFF
            token = torch.arange(vocab, device="cuda")
            z = torch.where((words[:, token // 32] >> (token % 32)) % 2 == 1, z, torch.full_like(z, -math.inf))
        empty = (z == -math.inf).all(1)
        lp = torch.log_softmax(z, 1)
        lp[empty] = -math.inf
        p = lp.exp()
        part = {"entropy": -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)}
        if case["ids"]:
            ids = state["ids"][a:a + 256].long()
            part["logprob"] = torch.where(ids < 0, torch.zeros(ids.shape, dtype=torch.float64, device="cuda"),
                                          torch.gather(lp, 1, ids.clamp(min=0)))
        if case["top"]:
            part["top_logprob"] = torch.topk(lp, case["top"], 1).values
        parts.append(part)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
