"""Plain forms of the calls on a cache's pages (Python lists and numpy), as their definitions read."""
import numpy as np


def fork(refs, pages, lens, page, source):
    refs, width = refs.copy(), pages.shape[1]
    new_pages, new_lens = np.full((len(source), width), -1, np.int32), np.zeros(len(source), np.int32)
    for i, s in enumerate(source):
        if s < 0:
            continue
        new_lens[i] = min(lens[s], width * page)
        for j in range(-(-int(new_lens[i]) // page)):
            new_pages[i, j] = pages[s, j]
            refs[pages[s, j]] += 1
    return refs, new_pages, new_lens


def trim(refs, pages, lens, page):
    refs, pages = refs.copy(), pages.copy()
    for s, n in enumerate(lens):
        for j in range(-(-int(n) // page), pages.shape[1]):
            if pages[s, j] >= 0:
                refs[pages[s, j]] -= 1
                pages[s, j] = -1
    return refs, pages


def extend(refs, pages, lens, new, page):
    """-> refs, pages, lens, slots, {(sequence): (page copied from, page copied to, rows)}."""
    refs, pages, lens = refs.copy(), pages.copy(), [int(n) for n in lens]
    width = pages.shape[1]
    fits = [-(-(n + m) // page) <= width for n, m in zip(lens, new)]
    items = [(s, j) for s in range(len(lens)) if fits[s] and new[s] for j in range(lens[s] // page, -(-(lens[s] + new[s]) // page))]
    holders = {}
    for it in items:
        if pages[it] >= 0 and refs[pages[it]] > 1:
            holders.setdefault(int(pages[it]), []).append(it)
    kept = {its[-1] for p, its in holders.items() if len(its) == refs[p]}
    shared = {it for its in holders.values() for it in its}
    needy = [it for it in items if pages[it] < 0 or it in shared]
    free = [p for p in range(len(refs)) if refs[p] == 0]
    done = list(fits)
    if len([it for it in needy if it not in kept]) <= len(free):
        needy = [it for it in needy if it not in kept]
    else:
        total = 0
        for s in range(len(lens)):
            mine = sum(it[0] == s for it in needy)
            total += mine
            done[s] = fits[s] and (mine == 0 or total <= len(free))
        needy = [it for it in needy if done[it[0]]]
    moves = {}
    for it, p in zip(needy, free):
        s, j = it
        if it in shared:
            refs[pages[it]] -= 1
            if j == lens[s] // page:
                moves[s] = (int(pages[it]), p, lens[s] % page)
        pages[it] = p
        refs[p] = 1
    slots, out = [], np.array(lens, np.int32)
    for s, (n, m) in enumerate(zip(lens, new)):
        slots += [int(pages[s, (n + i) // page]) * page + (n + i) % page if done[s] else -1 for i in range(m)]
        out[s] = n + m if done[s] else n
    return refs, pages, out, np.array(slots, np.int64), moves
