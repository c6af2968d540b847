"""Oracles of a prompt's way into the cache: page assignment and release, rotary positions and causal
attention over packed prompts, in numpy, from their definitions.  Test infrastructure; shares
nothing with the CUDA library."""
from __future__ import annotations

import math

import numpy as np


def _ceil(a, b):
    return -(-int(a) // int(b))


def page_assign(lens, cu, table, free, num_free, page, rows, num_pages):
    """(table, new_lens, slots, positions, num_free, flags) after the step; inputs are not changed."""
    BAD_PAGE, BAD_CONTEXT, BAD_QLEN, POOL = 0x1, 0x2, 0x4, 0x1000
    table, lens, cu = table.copy(), [int(x) for x in lens], [int(x) for x in cu]
    slots, pos = np.full(rows, -1, np.int64), np.zeros(rows, np.int32)
    new = np.array(lens, np.int32).reshape(-1)
    left, flags, out = min(max(int(num_free), 0), len(free)), 0, False
    if lens and (cu[0] < 0 or cu[-1] > rows or any(b < a for a, b in zip(cu[:-1], cu[1:]))):
        return table, new, slots, pos, left, BAD_QLEN
    for r, n in enumerate(lens):
        a, b = cu[r], cu[r + 1]
        end = n + b - a
        if n < 0 or end > 2**31 - 1 or _ceil(end, page) > table.shape[1]:
            flags |= BAD_CONTEXT
            pos[a:b] = (n + np.arange(b - a)).astype(np.int32)
            continue
        at = n + np.arange(b - a)
        pos[a:b] = at
        have, want = _ceil(n, page), _ceil(end, page)
        if want > have and (out or want - have > left):
            out, flags = True, flags | POOL
            continue
        for c in range(have, want):
            left -= 1
            table[r, c] = free[left]
        for i, p in zip(range(a, b), at):
            pg = int(table[r, p // page])
            if 0 <= pg < num_pages:
                slots[i] = pg * page + p % page
            else:
                flags |= BAD_PAGE
        new[r] = end
    return table, new, slots, pos, left, flags


def page_release(lens, new, table, free, num_free, page, num_pages):
    """(free, num_free, flags) after the pages behind the new lengths have been given back."""
    BAD_PAGE, BAD_CONTEXT, POOL = 0x1, 0x2, 0x1000
    free = free.copy()
    top, flags, full = min(max(int(num_free), 0), len(free)), 0, False
    for r, (n, m) in enumerate(zip(lens, new)):
        if n < 0 or m < 0 or _ceil(n, page) > table.shape[1]:
            flags |= BAD_CONTEXT
            continue
        back = [int(table[r, c]) for c in range(_ceil(m, page), _ceil(n, page))]
        if back and (full or top + len(back) > len(free)):
            full, flags = True, flags | POOL
            continue
        for pg in back:
            flags |= 0 if 0 <= pg < num_pages else BAD_PAGE
            free[top] = pg
            top += 1
    return free, top, flags


def rope(x, positions, radians, half, inverse=False, scale=1.0):
    """x fp64 [T, H, D]; radians: fp64 per position of each pair."""
    turn = np.exp(1j * (-1.0 if inverse else 1.0) * np.mod(
        np.asarray(positions, np.longdouble)[:, None] * np.asarray(radians, np.longdouble)[None], 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))
    ).astype(np.float64)) * scale
    n = len(radians)
    i = np.arange(n)
    one, two = (i, i + n) if half else (2 * i, 2 * i + 1)
    y = np.array(x, np.float64)
    z = (y[..., one] + 1j * y[..., two]) * turn[:, None]
    y[..., one], y[..., two] = z.real, z.imag
    return y


def prompt_attn(q, k, v, cu, sm_scale):
    """fp64 (out, lse, sum of weights * |v|, largest sm_scale * sum |q k| of a row); rows of no sequence are 0."""
    T, hq, D = q.shape
    G = hq // k.shape[1]
    out, mag = np.zeros((T, hq, D)), np.zeros((T, hq, D))
    lse, terms = np.zeros((T, hq)), np.zeros((T, hq))
    for a, b in zip(cu[:-1], cu[1:]):
        a, b = int(a), int(b)
        if b <= a:
            continue
        tril = np.tril(np.ones((b - a, b - a), bool))
        for h in range(hq):
            qq, kk, vv = q[a:b, h], k[a:b, h // G], v[a:b, h // G]
            x = np.where(tril, sm_scale * (qq @ kk.T), -math.inf)
            top = x.max(1, keepdims=True)
            w = np.exp(x - top)
            z = w.sum(1, keepdims=True)
            w /= z
            out[a:b, h], mag[a:b, h] = w @ vv, w @ np.abs(vv)
            lse[a:b, h] = (top + np.log(z))[:, 0]
            terms[a:b, h] = np.where(tril, sm_scale * (np.abs(qq) @ np.abs(kk).T), 0).max(1)
    return out, lse, mag, terms
