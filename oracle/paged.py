"""Plain float64 oracle of the paged KV cache: page accounting, slot map and
attention of ragged chunks, written from their definitions with Python lists
and NumPy.  Shares no code with the library."""
from __future__ import annotations

import math
from typing import List, Optional, Tuple

import numpy as np


def pages(n: int, page_size: int) -> int:
    return -(-n // page_size)


def resize(cur: List[int], new: List[int], table: np.ndarray, page_size: int, free: List[int],
           max_new: int) -> dict:
    """One request after the other over a Python list used as the stack.
    Returns lens, cu, slots, table, free (the stack's contents)."""
    width = table.shape[1]
    table = table.copy()
    stack = list(free)
    B = len(cur)

    def fits(b):
        return (cur[b] >= 0 and new[b] >= 0 and pages(cur[b], page_size) <= width and
                pages(new[b], page_size) <= width)

    released = []
    for b in range(B):
        if fits(b):
            released += [int(table[b, c]) for c in range(pages(new[b], page_size),
                                                         pages(cur[b], page_size))]
    stack += released[::-1]
    lens, cu, slots = [], [0], []
    room = len(stack)      # pages that the sequences so far have not asked for
    asked = 0              # new tokens asked for so far
    for b in range(B):
        tok = max(0, new[b] - cur[b]) if cur[b] >= 0 and new[b] >= 0 else 0
        need = 0
        if fits(b):
            need = max(0, pages(new[b], page_size) - pages(cur[b], page_size))
        room -= need
        asked += tok
        served = fits(b) and (need == 0 or room >= 0) and (tok == 0 or asked <= max_new)
        if served:
            for c in range(pages(cur[b], page_size), pages(cur[b], page_size) + need):
                table[b, c] = stack.pop()
        lens.append(new[b] if served else cur[b])
        for p in range(cur[b], cur[b] + tok):
            if len(slots) < max_new:
                slots.append(int(table[b, p // page_size]) * page_size + p % page_size
                             if served else -1)
        cu.append(len(slots))
    slots += [-1] * (max_new - len(slots))
    return {"lens": lens, "cu": cu, "slots": slots, "table": table, "free": stack}


def visible(pos: int, ctx: int, block: int) -> int:
    """Keys [0, n) that the row at position pos sees."""
    if block == 0:
        return ctx
    if pos < 0:
        return 0
    return min(ctx, (pos // block + 1) * block)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, ctx: int, block: int,
           scale: Optional[float] = None) -> Tuple[np.ndarray, np.ndarray, np.ndarray, np.ndarray]:
    """One sequence: q [n][H][Dh], k and v [ctx][Hkv][Dh], float64.  Returns
    (o, lse, a, s): the outputs, the log-sum-exp, sum_j p_j |v_j| (what a
    relative error of the probabilities can move o by) and the largest
    sum_d |q_d k_d| * scale over the visible keys (what the scores' rounding
    is relative to)."""
    n, H, Dh = q.shape
    g = H // k.shape[1] if ctx else 1
    scale = 1.0 / math.sqrt(Dh) if scale is None else scale
    o = np.zeros((n, H, Dh))
    a = np.zeros((n, H, Dh))
    lse = np.full((n, H), -np.inf)
    mag = np.zeros((n, H))
    for i in range(n):
        m = visible(ctx - n + i, ctx, block)
        if m == 0:
            continue
        for h in range(H):
            kk, vv = k[:m, h // g], v[:m, h // g]
            s = kk @ q[i, h] * scale
            top = s.max()
            e = np.exp(s - top)
            tot = e.sum()
            o[i, h] = e @ vv / tot
            a[i, h] = e @ np.abs(vv) / tot
            lse[i, h] = top + math.log(tot)
            mag[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return o, lse, a, mag
