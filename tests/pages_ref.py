"""The page operations, sequence by sequence, on the host."""
from __future__ import annotations

import torch

from paged_ref import inv_freq


def fork(parents, grow, lens, table, page, ref):
    """(new table, new ref, new lens, src, dst, what was wrong) of lists; what the header says."""
    P, pages = len(table[0]), len(ref)
    wrong, ref = set(), list(ref)
    rows = []
    for r, row in enumerate(table):
        held = []
        for e in row:
            if e < 0:
                break
            if e >= pages:
                wrong.add("page")
                break
            held.append(e)
        rows.append(held)
        for e in held:
            ref[e] -= 1
    new, fresh, src, dst, seen, out_lens = [], [], [], [], set(), []
    for b, p in enumerate(parents):
        if p >= len(table):
            wrong.add("argument")
            p = -1
        n = max(lens[p], 0) if p >= 0 else 0
        held = rows[p] if p >= 0 else []
        if len(held) * page < n:
            wrong.add("page")
        elder = p >= 0 and p not in seen
        seen.add(p)
        mine = list(held) if elder else held[:n // page]
        for e in mine:
            ref[e] += 1
        copies = p >= 0 and not elder and n % page > 0 and n // page < len(held)
        new.append(mine)
        g = grow[b] if grow is not None else 0
        if g < 0:
            wrong.add("argument")
            g = 0
        want = -(-(n + g) // page)
        if want > P:
            wrong.add("capacity")
        fresh.append(min(want, P))
        src.append(held[n // page] if copies else -1)
        dst.append(n // page if copies else -1)
        out_lens.append(n)
    free = [i for i, c in enumerate(ref) if c == 0]
    for b, mine in enumerate(new):
        while len(mine) < fresh[b]:
            if not free:
                wrong.add("capacity")
                break
            mine.append(free.pop(0))
            ref[mine[-1]] = 1
        if dst[b] >= 0:
            dst[b] = mine[dst[b]] if dst[b] < len(mine) else -1
            src[b] = src[b] if dst[b] >= 0 else -1
    table = [mine + [-1] * (P - len(mine)) for mine in new]
    return table, ref, out_lens, src, dst, wrong


def turned(x, shift, rope, start, rd, interleaved=False):
    """fp64 x [..., d] with [start, start + rd) turned forward by `shift` positions."""
    f, _ = inv_freq(rope, rd)
    a = shift.double()[..., None] * f
    c, s = torch.cos(a), torch.sin(a)
    y = x.clone()
    part = x[..., start:start + rd]
    if interleaved:
        x0, x1 = part[..., 0::2], part[..., 1::2]
        y[..., start:start + rd:2], y[..., start + 1:start + rd:2] = x0 * c - x1 * s, x0 * s + x1 * c
    else:
        x0, x1 = part[..., :rd // 2], part[..., rd // 2:]
        y[..., start:start + rd] = torch.cat([x0 * c - x1 * s, x0 * s + x1 * c], dim=-1)
    return y
