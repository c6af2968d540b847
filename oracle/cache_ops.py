"""Plain fp64 / integer oracles of the cache operators: attention mass, eviction, compaction,
beam selection and beam reordering, written from their definitions with loops over requests
and numpy over positions.

TEST INFRASTRUCTURE ONLY, like oracle.py: no code is shared with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from . import oracle as O

_E4M3 = None


def rows_f64(cache, scale, one=1.0):
    """Cache rows (uint8 e4m3 codes or uint16 bf16 bits, any shape [..., D]) as doubles."""
    global _E4M3
    if cache.dtype == np.uint8:
        if _E4M3 is None:
            _E4M3 = np.array([O.dec_e4m3(c) for c in range(256)])
        x = _E4M3[cache]
    else:
        x = (cache.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    if scale is not None:
        x = x * scale.astype(np.float64)[..., None]
    return x * one


def keys_of(p, r, h, n=None):
    """K rows [n, D] of request r, KV head h, in position order (doubles)."""
    n = int(p.context_lens[r]) if n is None else n
    pages = p.block_table[r, :-(-n // p.page_size)]
    sc = None if p.k_scale is None else p.k_scale[pages, h].reshape(-1)[:n]
    k = p.k_cache[pages, h].reshape(-1, p.head_dim)[:n]
    return rows_f64(k, sc, p.k_scale_scalar)


def attn_mass(p, lse, mass, decay, u=0.0):
    """The mass after a step over synth.Problem p with this lse [rows, Hq] and mass
    [B, Hkv, stride]; and, element by element, how far an fp32 evaluation may be from it.

    The bound follows the arithmetic: a score's 128 products are exact and are added with at
    most one unit (2^-23) of error each, relative to the sum of their magnitudes; the query may be
    represented to 2^-22 of its group's largest element (u = 2^-22, or 0 where it is exact); the fold
    of the scales, the lse in base 2 and their difference round once each (2^-24 of the largest
    of them, three roundings); exp2 is off by 2^-22 of itself; 16 q_len weights and the carried mass are
    added with 2^-24 of the sum each."""
    q = (p.q.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    out, tol = mass.astype(np.float64), np.zeros(mass.shape)
    for r in range(p.num_seqs):
        L, row0, ql = int(p.context_lens[r]), int(p.cu_seqlens_q[r]), int(p.q_lens[r])
        if ql == 0:
            continue
        for h in range(p.num_kv_heads):
            k = keys_of(p, r, h)
            old = decay * mass[r, h, :L].astype(np.float64) if decay else np.zeros(L)
            old[L - ql:] = 0
            w, e = np.zeros(L), np.zeros(L)
            for t in range(ql):
                cut = L - ql + t + 1
                for g in range(p.group_size):
                    j = h * p.group_size + g
                    if lse[row0 + t, j] == -np.inf:
                        continue
                    x, y = q[row0 + t, j], float(lse[row0 + t, j])
                    s = k[:cut] @ x * p.sm_scale
                    wt = np.exp(s - y)
                    mag = np.abs(k[:cut]) @ np.abs(x) * p.sm_scale
                    grp = np.abs(q[row0 + t, h * p.group_size:(h + 1) * p.group_size]).max()
                    d = 128 * 2.0 ** -23 * mag + u * grp * np.abs(k[:cut]).sum(1) * p.sm_scale
                    d += 3 * 2.0 ** -24 * (np.abs(s) + abs(y)) + 2.0 ** -22
                    w[:cut] += wt
                    e[:cut] += wt * d
            out[r, h, :L] = old + w
            tol[r, h, :L] = 1.01 * e + (16 * ql + 2) * 2.0 ** -24 * (w + old)
    return out, tol


def evict_select(mass, lens, budget, first, recent):
    B, H, _ = mass.shape
    keep = np.full((B, H, budget), -1, np.int32)
    new = np.zeros(B, np.int32)
    for r in range(B):
        L = int(lens[r])
        new[r] = min(L, budget)
        for h in range(H):
            if L <= budget:
                keep[r, h, :L] = np.arange(L)
                continue
            mid = list(range(first, L - recent))
            val = lambda i: (1, 0.0) if np.isnan(mass[r, h, i]) else (0, -float(mass[r, h, i]))  # noqa: E731
            best = sorted(mid, key=lambda i: (val(i), i))[:budget - first - recent]
            keep[r, h] = np.array(list(range(first)) + sorted(best) + list(range(L - recent, L)), np.int32)
    return keep, new


def kv_compact(keep, new_lens, src_table, dst_table, arrays, page_size, mass=None, mass_out=None):
    """New copies of `arrays` ([num_pages, Hkv, page_size, ...]) and of mass_out."""
    out = [a.copy() for a in arrays]
    mo = None if mass_out is None else mass_out.copy()
    for r in range(keep.shape[0]):
        for h in range(keep.shape[1]):
            for i in range(int(new_lens[r])):
                s = int(keep[r, h, i])
                for a, o in zip(arrays, out):
                    o[dst_table[r, i // page_size], h, i % page_size] = a[src_table[r, s // page_size], h, s % page_size]
                if mo is not None:
                    mo[r, h, i] = mass[r, h, s]
    return out, mo


def beam_select(logits, scores, eos=-1, finished=None, lengths=None, penalty=0.0):
    """(tokens, parents, totals fp64, finished, lengths) of one step; logits [N, W, V] doubles.
    Every candidate is ranked: rank, then beam, then token."""
    N, W, V = logits.shape
    res = [np.zeros((N, W), d) for d in (np.int32, np.int32, np.float64, np.uint8, np.int32)]
    for n in range(N):
        cand = []
        for b in range(W):
            x, cum = logits[n, b], float(scores[n, b])
            done = finished is not None and bool(finished[n, b])
            ln = 0 if lengths is None else int(lengths[n, b])
            ln = ln if done else ln + 1
            with np.errstate(all="ignore"):
                m = x.max()
                lse = m + np.log(np.exp(x - m).sum())
            tot = np.full(V, -np.inf)
            if not (np.isnan(cum) or cum == -np.inf):
                if done:
                    tot[eos] = cum
                elif np.isfinite(lse):
                    tot = cum + (x - lse)
            with np.errstate(over="ignore"):
                norm = np.float64(max(ln, 1)) ** penalty
            rank = np.where(np.isinf(tot), tot, tot / norm) + 0.0
            order = np.lexsort((np.arange(V), -rank))[:W]
            cand += [(-rank[v], b, int(v), tot[v], ln, done) for v in order]
        cand.sort(key=lambda c: c[:3])
        for j, (_, b, v, total, ln, done) in enumerate(cand[:W]):
            for a, val in zip(res, (v, b, total, done or (eos >= 0 and v == eos), ln)):
                a[n, j] = val
    return res


def beam_reorder(parents, lens, table, arrays, page_size):
    """(new table, new copies of arrays) after the beams followed their parents."""
    N, W = parents.shape
    out, made = table.copy(), [a.copy() for a in arrays]
    for n in range(N):
        L = int(lens[n * W])
        full, part = L // page_size, L % page_size
        childless = [b for b in range(W) if b not in parents[n]]
        seen = set()
        for j in range(W):
            p = int(parents[n, j])
            out[n * W + j, :full] = table[n * W + p, :full]
            if part:
                giver = p if p not in seen else childless.pop(0)
                seen.add(p)
                page = table[n * W + giver, full]
                out[n * W + j, full] = page
                if giver != p:
                    for a, o in zip(arrays, made):
                        o[page, :, :part] = a[table[n * W + p, full], :, :part]
    return out, made
