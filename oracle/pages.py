"""Oracle for the pool of a cache's pages: plain Python, one entry at a time.

TEST INFRASTRUCTURE ONLY: the tests may use this module; the product path
never does.

A pool is a dict of lists: table (rows of entries, -1 where there is no page),
refs (entries that name each page), stack (pages that none names, the next one
to be handed out last).  The calls change it as include/hpc_decode.h says of
hpc_kv_free, hpc_kv_extend, hpc_kv_fork and hpc_kv_compact.
"""

from __future__ import annotations

PAGE = 64


def pages_of(tokens: int) -> int:
    return -(-tokens // PAGE)


def new(B: int, max_pages: int, num_pages: int) -> dict:
    return dict(table=[[-1] * max_pages for _ in range(B)], refs=[0] * num_pages,
                stack=list(range(num_pages - 1, -1, -1)))


def free(pool: dict, rows, keep=None) -> None:
    back = []
    for i, r in enumerate(rows):
        row = pool["table"][r]
        for j in range(pages_of(keep[i] if keep else 0), len(row)):
            p, row[j] = row[j], -1
            if p >= 0:
                pool["refs"][p] -= 1
                if p not in back:
                    back.append(p)
    pool["stack"] += [p for p in back if pool["refs"][p] == 0][::-1]


def extend(pool: dict, rows, lens) -> bool:
    """False where the stack has not enough: nothing has changed then."""
    want = []
    for r, L in zip(rows, lens):
        want += [(r, j) for j in range(pages_of(L))
                 if pool["table"][r][j] < 0 and (r, j) not in want]
    if len(want) > len(pool["stack"]):
        return False
    for r, j in want:
        p = pool["stack"].pop()
        pool["table"][r][j] = p
        pool["refs"][p] += 1
    return True


def fork(pool: dict, src, dst, lens):
    """The copies [(from, to)], or None where the stack has not enough."""
    if sum(L % PAGE > 0 for L in lens) > len(pool["stack"]):
        return None
    copies = []
    for a, b, L in zip(src, dst, lens):
        for j in range(L // PAGE):
            p = pool["table"][a][j]
            pool["table"][b][j] = p
            pool["refs"][p] += 1
        if L % PAGE:
            p = pool["stack"].pop()
            pool["table"][b][L // PAGE] = p
            pool["refs"][p] = 1
            copies.append((pool["table"][a][L // PAGE], p))
    return copies


def compact(pool: dict):
    refs = pool["refs"]
    live = sum(r > 0 for r in refs)
    far = [p for p in range(live, len(refs)) if refs[p] > 0]
    holes = [p for p in range(live) if refs[p] == 0]
    to = dict(zip(far, holes))
    pool["table"] = [[to.get(p, p) for p in row] for row in pool["table"]]
    for a, b in to.items():
        refs[b], refs[a] = refs[a], 0
    pool["stack"] = list(range(len(refs) - 1, live - 1, -1))
    return list(to.items())
