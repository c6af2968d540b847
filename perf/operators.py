"""The life of a paged KV cache between two decode steps, as cases that can be timed and compared.

Five operators: attention mass accumulated per cached token (`attn_mass`), the selection of
the tokens that a bounded cache keeps (`evict_select`), the move of the kept tokens to the
front of their pages (`kv_compact`), beam search's selection over beams and vocabulary
(`beam_select`) and the reordering of the beams' block tables, last pages and states
(`beam_reorder`).  With `own` false `run` computes them in elementary torch operations; with
`own` true it makes the calls a user of the library makes.
"""
import math

import numpy as np
import torch

own = False

G, D = 16, 128                 # query heads per KV head, head_dim
DEV = "cuda"
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one short request on small pages: the latency of a call in a tiny decode step
        dict(name="mass_small", op="mass", reqs=4, heads=1, lo=1, hi=300, page=16, kv="token", qlo=1, qhi=1),
        # the dense decode batch: 32 requests of 8192 tokens, one new token each
        dict(name="mass_8k", op="mass", reqs=32, heads=1, lo=8192, hi=8192, page=128, kv="token", qlo=1, qhi=1),
        # long contexts with one scale for the cache, the largest decode batch
        dict(name="mass_128k", op="mass", reqs=8, heads=1, lo=131072, hi=131072, page=128, kv="scalar", qlo=1, qhi=1),
        # speculative decode over a bf16 cache: ragged query lengths and contexts
        dict(name="mass_ragged_bf16", op="mass", reqs=31, heads=1, lo=1024, hi=32768, page=128, kv="bf16", qlo=1, qhi=4),
        # a few short contexts a little over their budget
        dict(name="select_small", op="select", reqs=4, heads=1, lo=300, hi=1000, budget=257, first=4, recent=64),
        # long contexts cut to an eighth
        dict(name="select_128k", op="select", reqs=8, heads=2, lo=100000, hi=131072, budget=16384, first=4, recent=1024),
        # a decode batch that has grown by one page-sized slack, moved into fresh pages
        dict(name="compact_8k", op="compact", reqs=32, heads=1, lo=8700, hi=9216, budget=8192, page=128, kv="token", inplace=False),
        # two short prompts cut in place, every kept token moving: odd sizes on small pages
        dict(name="compact_inplace", op="compact", reqs=8, heads=1, lo=16001, hi=32767, budget=4095, page=32, kv="token", inplace=True),
        # one request with four beams over a small vocabulary in fp32, odd row length
        dict(name="beam_small", op="beams", reqs=1, beams=4, vocab=32001, logits="f32", penalty=0.0),
        # a full batch of beams over a large vocabulary
        dict(name="beam_large", op="beams", reqs=32, beams=8, vocab=131072, logits="bf16", penalty=0.7),
        # four beams on small pages, no state beside the cache
        dict(name="reorder_small", op="reorder", reqs=1, beams=4, lo=300, hi=300, page=16, heads=1, kv="token", state=0),
        # a full batch of beams with their attention mass beside the cache
        dict(name="reorder_large", op="reorder", reqs=32, beams=8, lo=8000, hi=8190, page=128, heads=1, kv="token", state=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mass", "mass", "select", "compact", "beams", "reorder"])
    page = rng.choice([16, 32, 64, 128])
    heads = rng.choice([1, 1, 1, 2, 4])
    if op == "mass":
        hi = _log(rng, 1, 131072)
        reqs = max(1, min(_log(rng, 1, 48), 800000 // (hi * heads)))
        qhi = rng.choice([1, 1, 1, 2, 3, 4, 8])
        if hi * reqs * heads > 260000:
            qhi = min(qhi, 2)
        return dict(op="mass", reqs=reqs, heads=heads, lo=rng.randint(max(1, hi // 4), hi), hi=hi, page=page,
                    kv=rng.choice(["token", "token", "scalar", "bf16"]), qlo=1, qhi=min(qhi, max(1, hi // 4)))
    if op == "select":
        hi = _log(rng, 2, 131072)
        budget = max(1, int(hi * rng.uniform(0.05, 0.95)))
        first = rng.randint(0, min(8, budget // 4))
        return dict(op="select", reqs=_log(rng, 1, max(2, min(64, 1000000 // (hi * heads)))), heads=heads, lo=rng.randint(1, hi), hi=hi,
                    budget=budget, first=first, recent=rng.randint(0, budget // 2))
    if op == "compact":
        budget = _log(rng, 1, 16384)
        lo = 2 * budget + rng.randint(0, 64)
        hi = lo + rng.randint(0, budget)
        return dict(op="compact", reqs=max(1, min(_log(rng, 1, 48), 250000 // (budget * heads))), heads=heads, lo=lo, hi=hi, budget=budget,
                    page=page, kv=rng.choice(["token", "scalar", "bf16"]), inplace=rng.random() < 0.5)
    beams = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 32])
    if op == "beams":
        vocab = _log(rng, 40, 200000)
        return dict(op="beams", reqs=_log(rng, 1, max(2, min(64, 20000000 // (beams * vocab)))), beams=beams, vocab=vocab,
                    logits=rng.choice(["bf16", "f32"]), penalty=rng.choice([0.0, 0.6, 1.0]))
    hi = _log(rng, 1, 8192)
    return dict(op="reorder", reqs=_log(rng, 1, max(2, 200 // beams)), beams=beams, lo=max(1, hi // 2), hi=hi, page=page, heads=heads,
                kv=rng.choice(["token", "scalar", "bf16"]), state=rng.choice([0, 0, hi + 7]))


# ----------------------------------------------------------------------------- inputs

def _lens(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _tables(g, rows, hi, page, spare=0):
    """Distinct pages for `rows` rows of up to `hi` tokens (and `spare` pages more per row), in random order."""
    npg = -(-hi // page) + spare
    pages = torch.randperm(rows * npg, generator=g, device=DEV).to(torch.int32)
    return pages.view(rows, npg), rows * npg


def _cache(g, pages, heads, page, kv):
    """N(0, 1) rows as the cache holds them: (codes or bf16 values, scales or None, scale of the whole cache)."""
    x = torch.randn(pages, heads, page, D, generator=g, device=DEV)
    if kv == "bf16":
        return x.to(torch.bfloat16), None, 1.0
    if kv == "scalar":
        s = 0.0078125 + 0.01 * torch.rand(1, generator=g, device=DEV).item()
        return (x / s).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), None, s
    sc = x.abs().amax(-1) / E4M3_MAX
    return (x / sc[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), sc.contiguous(), 1.0


def _wide(cache, dt=torch.float32):
    """The values that cache bytes stand for."""
    return (cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache).to(dt)


def _rows(cu, qmax):
    """[reqs, qmax] query rows of each request (clamped), and which of them it has."""
    t = torch.arange(qmax, device=cu.device)[None, :]
    r = cu[:-1, None].long() + t
    return r.clamp(max=int(cu.shape[0]) * qmax), t < (cu[1:] - cu[:-1])[:, None]


def _scores(s, dt):
    """sm_scale q . k of every (request, KV head, query row, query head, position), -inf past the row's cutoff."""
    kc, bt, L, cu, qmax, heads = s["k"], s["table"], s["lens"], s["cu"], s["qmax"], s["heads"]
    n, page = L.numel(), kc.shape[2]
    k = _wide(kc[bt.long()], dt)
    if s["k_scale"] is not None:
        k = k * s["k_scale"][bt.long()].to(dt)[..., None]
    k = (k * s["k_one"]).permute(0, 2, 1, 3, 4).reshape(n, heads, -1, D)
    rows, has = _rows(cu, qmax)
    rows = rows.clamp(max=s["q"].shape[0] - 1)
    q = s["q"].to(dt)[rows].view(n, qmax, heads, G, D).permute(0, 2, 1, 3, 4).reshape(n, heads, qmax * G, D)
    x = (q @ k.transpose(-1, -2)).view(n, heads, qmax, G, -1) * s["sm"]
    pos = torch.arange(x.shape[-1], device=x.device)
    ql = cu[1:] - cu[:-1]
    cut = (L - ql)[:, None] + torch.arange(qmax, device=x.device)[None, :] + 1
    ok = (pos[None, None, :] < cut[..., None]) & has[..., None]
    return x.masked_fill(~ok[:, None, :, None, :], -math.inf), rows, has, ql


def _prepare_mass(c, g):
    """A decode step that has just run: its queries, cache and log-sum-exp, and the mass of the steps before."""
    n, heads = c["reqs"], c["heads"]
    lens = _lens(g, n, c["lo"], c["hi"])
    ql = torch.minimum(_lens(g, n, c["qlo"], c["qhi"]), lens)
    cu = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    cu[1:] = ql.cumsum(0).to(torch.int32)
    table, pages = _tables(g, n, c["hi"], c["page"])
    k, ks, one = _cache(g, pages, heads, c["page"], c["kv"])
    rows = int(cu[-1])
    s = dict(op="mass", heads=heads, lens=lens, cu=cu, table=table, k=k, k_scale=ks, k_one=one, qmax=int(ql.max()), sm=1.0 / math.sqrt(D),
             decay=0.96875, q=torch.randn(rows, heads * G, D, generator=g, device=DEV).to(torch.bfloat16))
    x, at, has, _ = _scores(s, torch.float32)
    lse = torch.logsumexp(x, -1).permute(0, 2, 1, 3).reshape(n, s["qmax"], heads * G)
    s["lse"] = lse[has].contiguous()
    width = table.shape[1] * c["page"]
    s["mass"] = torch.rand(n, heads, width, generator=g, device=DEV).pow(8) * 4
    s["out"] = torch.zeros(n, heads, width, device=DEV)
    return s


def _prepare_select(c, g):
    """Accumulated mass as decode leaves it: a heavy tail over six orders, and tokens that nothing looked at."""
    n, heads = c["reqs"], c["heads"]
    mass = torch.exp(2.5 * torch.randn(n, heads, c["hi"], generator=g, device=DEV))
    mass[torch.rand(mass.shape, generator=g, device=DEV) < 0.05] = 0.0
    return dict(op="select", mass=mass, lens=_lens(g, n, c["lo"], c["hi"]), budget=c["budget"], first=c["first"], recent=c["recent"])


def _prepare_compact(c, g):
    """Caches and a kept set.  Into fresh pages: any positions.  In place: positions at or past the budget, so that
    every kept token moves and a second pass over the same state does the same work on the same values."""
    n, heads, page, budget = c["reqs"], c["heads"], c["page"], c["budget"]
    lens = _lens(g, n, c["lo"], c["hi"])
    width = -(-c["hi"] // page)
    fresh = 0 if c["inplace"] else -(-budget // page)
    table, pages = _tables(g, n, c["hi"], page, fresh)
    rank = torch.rand(n, heads, c["hi"], generator=g, device=DEV)
    pos = torch.arange(c["hi"], device=DEV)
    rank = rank.masked_fill(pos >= lens[:, None, None], 2.0)
    if c["inplace"]:
        rank = rank.masked_fill(pos < budget, 2.0)
    new = torch.minimum(lens - budget if c["inplace"] else lens, torch.full_like(lens, budget))
    kept = rank.argsort(-1)[..., :budget]
    kept = kept.masked_fill(torch.arange(budget, device=DEV) >= new[:, None, None], c["hi"]).sort(-1).values
    keep = kept.masked_fill(torch.arange(budget, device=DEV) >= new[:, None, None], -1).to(torch.int32)
    k, ks, _ = _cache(g, pages, heads, page, c["kv"])
    v, vs, _ = _cache(g, pages, heads, page, c["kv"])
    mass = torch.rand(n, heads, c["hi"], generator=g, device=DEV)
    return dict(op="compact", keep=keep.contiguous(), new=new, table=table[:, :width].contiguous(),
                dst=None if c["inplace"] else table[:, width:].contiguous(), k=k, v=v, k_scale=ks, v_scale=vs, mass=mass,
                mass_out=mass if c["inplace"] else torch.zeros(n, heads, budget, device=DEV))


def _prepare_beams(c, g):
    """Logits of a language model (most of the mass on a few hundred tokens), beams some of which have ended."""
    n, w, v = c["reqs"], c["beams"], c["vocab"]
    x = 2.0 * torch.randn(n, w, v, generator=g, device=DEV)
    x += 6.0 * (torch.rand(n, w, v, generator=g, device=DEV) < 200.0 / v)
    return dict(op="beams", logits=x.to(torch.bfloat16) if c["logits"] == "bf16" else x, eos=2 % v, penalty=c["penalty"],
                scores=-20.0 + 3.0 * torch.randn(n, w, generator=g, device=DEV),
                finished=(torch.rand(n, w, generator=g, device=DEV) < 0.15).to(torch.uint8),
                lengths=torch.randint(1, 200, (n, w), generator=g, device=DEV, dtype=torch.int32))


def _prepare_reorder(c, g):
    """Beams whose histories share most of their pages and end in a page of their own."""
    n, w, page, heads = c["reqs"], c["beams"], c["page"], c["heads"]
    lens = _lens(g, n, c["lo"], c["hi"]).repeat_interleave(w)
    table, pages = _tables(g, n * w, c["hi"], page, 1)
    full = (lens // page)[:, None].long()
    col = torch.arange(table.shape[1], device=DEV)
    first = table.view(n, w, -1)[:, :1].expand(n, w, -1).reshape(n * w, -1)
    table = torch.where(col[None] < full, first, table).contiguous()
    parents = torch.randint(0, w, (n, w), generator=g, device=DEV, dtype=torch.int32)
    k, ks, _ = _cache(g, pages, heads, page, c["kv"])
    v, vs, _ = _cache(g, pages, heads, page, c["kv"])
    s = dict(op="reorder", parents=parents, lens=lens, table=table, table_out=torch.empty_like(table), k=k, v=v, k_scale=ks, v_scale=vs,
             state=None, state_out=None)
    if c["state"]:
        s["state"] = torch.rand(n * w, heads, c["state"], generator=g, device=DEV)
        s["state_out"] = torch.empty_like(s["state"])
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    made = {"mass": _prepare_mass, "select": _prepare_select, "compact": _prepare_compact, "beams": _prepare_beams, "reorder": _prepare_reorder}
    return made[case["op"]](case, g)


# -------------------------------------------------------------------- the plain forms

def _mass(s):
    """mass_out[p] = (p older than the step's rows ? decay mass[p] : 0) + sum over rows and heads of exp(score - lse)."""
    x, rows, has, ql = _scores(s, torch.float32)
    n, qmax, heads = x.shape[0], s["qmax"], s["heads"]
    lse = s["lse"][rows].view(n, qmax, heads, G).permute(0, 2, 1, 3)
    w = torch.exp(x - lse[..., None]).sum((2, 3))
    pos = torch.arange(w.shape[-1], device=w.device)
    old = pos[None, :] < (s["lens"] - ql)[:, None]
    out = torch.where(old[:, None, :], s["decay"] * s["mass"], torch.zeros_like(w)) + w
    return torch.where((pos[None, :] < s["lens"][:, None])[:, None, :], out, torch.zeros_like(out))


def _select(s):
    """The first and the most recent positions, then the largest mass (lowest position first among equals), ascending."""
    mass, L, budget = s["mass"], s["lens"], s["budget"]
    pos = torch.arange(mass.shape[-1], device=mass.device)
    n = L[:, None, None]
    rank = mass.masked_fill((pos < s["first"]) | (pos >= n - s["recent"]), math.inf).masked_fill(pos >= n, -1.0)
    width = min(budget, mass.shape[-1])
    kept = rank.sort(dim=-1, descending=True, stable=True).indices[..., :width]
    new = L.clamp(max=budget)
    beyond = torch.arange(width, device=mass.device) >= new[:, None, None]
    kept = kept.masked_fill(beyond, mass.shape[-1]).sort(-1).values.masked_fill(beyond, -1).to(torch.int32)
    keep = torch.full((*mass.shape[:2], budget), -1, dtype=torch.int32, device=mass.device)
    keep[..., :width] = kept
    return {"keep": keep, "new_lens": new}


def _values(x):
    return x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x


def _caches(s):
    return {"k": _values(s["k"]), "v": _values(s["v"])} | ({} if s["k_scale"] is None else {"k_scale": s["k_scale"], "v_scale": s["v_scale"]})


def _compact(s):
    """Slot i of every (request, KV head) takes what slot keep[i] holds."""
    page = s["k"].shape[2]
    b, h, i = (torch.arange(s["keep"].shape[-1], device=DEV)[None, None, :].expand_as(s["keep"]) < s["new"][:, None, None]).nonzero(as_tuple=True)
    src = s["keep"][b, h, i].long()
    dst = s["table"] if s["dst"] is None else s["dst"]
    sp, dp = s["table"][b, src // page].long(), dst[b, i // page].long()
    so, do = src % page, i % page
    s["k"][dp, h, do] = s["k"][sp, h, so]
    s["v"][dp, h, do] = s["v"][sp, h, so]
    if s["k_scale"] is not None:
        s["k_scale"][dp, h, do] = s["k_scale"][sp, h, so]
        s["v_scale"][dp, h, do] = s["v_scale"][sp, h, so]
    s["mass_out"][b, h, i] = s["mass"][b, h, src]
    return _caches(s) | {"mass": s["mass_out"]}


def _beams(s):
    """The best continuations by (score + log softmax) / length ** penalty, in 64 bits: neighbours may lie 1e-6 apart.  A
    beam that has ended goes on with the end token alone, at its score and length."""
    x, eos = s["logits"].double(), s["eos"]
    n, w, v = x.shape
    top = x.amax(-1, keepdim=True)
    lp = x - top - torch.exp(x - top).sum(-1, keepdim=True).log()
    done = s["finished"].bool()[..., None]
    tok = torch.arange(v, device=x.device)
    lp = torch.where(done, torch.where(tok == eos, 0.0, -math.inf).double(), lp)
    total = s["scores"].double()[..., None] + lp
    length = s["lengths"].long() + (~s["finished"].bool()).long()
    rank = total / length.clamp(min=1).double().pow(s["penalty"])[..., None]
    best = rank.view(n, w * v).sort(dim=-1, descending=True, stable=True).indices[:, :w]
    parent, token = best // v, best % v
    ended = s["finished"].gather(1, parent).bool() | (token == eos)
    return {"tokens": token.to(torch.int32), "parents": parent.to(torch.int32), "scores": total.view(n, w * v).gather(1, best).float(),
            "finished": ended.to(torch.uint8), "lengths": length.gather(1, parent).to(torch.int32)}


def _reorder(s):
    """Rows of the block table and of the state follow their parents; a parent's last, partial page goes to its first
    child, and further children take copies in the last pages of beams without children."""
    par, page = s["parents"].long(), s["k"].shape[2]
    n, w = par.shape
    same = (par[:, :, None] == par[:, None, :]).tril(-1).any(-1)
    alive = torch.zeros(n, w, dtype=torch.bool, device=DEV).scatter_(1, par, True)
    dead = alive.int().sort(dim=-1, stable=True).indices
    giver = torch.where(same, dead.gather(1, (same.int().cumsum(-1) - 1).clamp(min=0).long()), par)
    base = torch.arange(n, device=DEV)[:, None] * w
    src, giver, L = (base + par).view(-1), (base + giver).view(-1), s["lens"].long()
    full, part = L // page, L % page
    col = torch.arange(s["table"].shape[1], device=DEV)[None]
    mine = s["table"][giver, full]
    out = torch.where(col < full[:, None], s["table"][src], s["table"])
    out = torch.where((col == full[:, None]) & (part > 0)[:, None], mine[:, None], out)
    s["table_out"].copy_(out)
    r = (same.view(-1) & (part > 0)).nonzero()[:, 0]
    a, b = s["table"][src[r], full[r]].long(), mine[r].long()
    live = torch.arange(page, device=DEV)[None] < part[r][:, None]
    for x in (s["k"], s["v"]) + (() if s["k_scale"] is None else (s["k_scale"], s["v_scale"])):
        m = live[:, None, :, None] if x.dim() == 4 else live[:, None, :]
        x[b] = torch.where(m, x[a], x[b])
    if s["state"] is not None:
        s["state_out"].copy_(s["state"][src])
    return _caches(s) | {"table": s["table_out"]} | ({} if s["state"] is None else {"state": s["state_out"]})


def _call(s):
    from paged_fp8_kv_04_gb300 import binding as B
    if s["op"] == "mass":
        return B.attn_mass(s["q"], s["k"], s["table"], s["lens"], s["cu"], s["lse"], s["mass"], out=s["out"], k_scale=s["k_scale"],
                           k_scale_scalar=s["k_one"], max_q_len=s["qmax"], sm_scale=s["sm"], decay=s["decay"])
    if s["op"] == "select":
        keep, new = B.evict_select(s["mass"], s["lens"], budget=s["budget"], first=s["first"], recent=s["recent"])
        return {"keep": keep, "new_lens": new}
    if s["op"] == "compact":
        B.kv_compact(s["keep"], s["new"], s["table"], s["k"], s["v"], dst_block_table=s["dst"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                     mass=s["mass"], mass_out=s["mass_out"])
        return _caches(s) | {"mass": s["mass_out"]}
    if s["op"] == "beams":
        tokens, parents, scores, finished, lengths = B.beam_select(s["logits"], s["scores"], eos=s["eos"], finished=s["finished"],
                                                                   lengths=s["lengths"], length_penalty=s["penalty"])
        return {"tokens": tokens, "parents": parents, "scores": scores, "finished": finished, "lengths": lengths}
    B.beam_reorder(s["parents"], s["lens"], s["table"], s["table_out"], s["k"], s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                   states=[] if s["state"] is None else [(s["state"], s["state_out"])])
    return _caches(s) | {"table": s["table_out"]} | ({} if s["state"] is None else {"state": s["state_out"]})


def run(state):
    if own:
        return _call(state)
    return {"mass": _mass, "select": _select, "compact": _compact, "beams": _beams, "reorder": _reorder}[state["op"]](state)


# ------------------------------------------------------- what a pass cannot do without

def _token_bytes(kv):
    return {"token": D + 4, "scalar": D, "bf16": 2 * D}[kv]


def work(case):
    c, n = case, case["reqs"]
    if c["op"] == "mass":
        heads, L, rows = c["heads"], (c["lo"] + c["hi"]) / 2, n * (c["qlo"] + c["qhi"]) / 2
        return {"bytes": n * heads * L * (_token_bytes(c["kv"]) + 8) + rows * heads * G * (2 * D + 4) + 4 * n * L / c["page"],
                "flops": 2.0 * D * G * rows * heads * L}
    if c["op"] == "select":
        # every mass is read once, and compared at least once with what decides whether it stays
        cells = n * c["heads"] * (c["lo"] + c["hi"]) / 2
        return {"bytes": 4 * cells + 4 * n * c["heads"] * c["budget"], "flops": cells}
    if c["op"] == "compact":
        return {"bytes": n * c["heads"] * c["budget"] * (4.0 * _token_bytes(c["kv"]) + 12), "flops": 0}
    if c["op"] == "beams":
        cells = float(n * c["beams"] * c["vocab"])
        return {"bytes": cells * (2 if c["logits"] == "bf16" else 4) + 38 * n * c["beams"], "flops": 3 * cells}
    rows, pages = n * c["beams"], (c["lo"] + c["hi"]) / 2 / c["page"]
    # about a third of the beams share a parent with an earlier one, and half a page goes to each
    copies = max(0.0, n * (c["beams"] * (1 - 1 / c["beams"]) ** c["beams"])) * c["page"] / 2 * c["heads"]
    return {"bytes": 8.0 * rows * (pages + 2) + 4 * copies * _token_bytes(c["kv"]) + 8.0 * rows * c["heads"] * c["state"], "flops": 0}


# ----------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"mass": _exact_mass, "select": _exact_select, "compact": _exact_compact, "beams": _exact_beams, "reorder": _exact_reorder}[case["op"]](s)


def _exact_mass(s):
    out = torch.zeros(s["mass"].shape, dtype=torch.float64, device=DEV)
    L, cu, page = s["lens"].tolist(), s["cu"].tolist(), s["k"].shape[2]
    for b, n in enumerate(L):
        ql = cu[b + 1] - cu[b]
        pages = s["table"][b, : -(-n // page)].long()
        for h in range(s["heads"]):
            k = _wide(s["k"][pages, h], torch.float64)
            if s["k_scale"] is not None:
                k = k * s["k_scale"][pages, h].double()[..., None]
            k = k.reshape(-1, D)[:n] * s["k_one"]
            m = s["mass"][b, h, :n].double() * s["decay"]
            m[n - ql:] = 0
            for t in range(ql):
                row, cut = cu[b] + t, n - ql + t + 1
                w = torch.exp(k[:cut] @ s["q"][row, h * G:(h + 1) * G].double().T * s["sm"] - s["lse"][row, h * G:(h + 1) * G].double())
                m[:cut] += w.sum(-1)
            out[b, h, :n] = m
    return out


def _exact_select(s):
    mass, L = s["mass"].cpu().numpy(), s["lens"].tolist()
    keep = np.full((*mass.shape[:2], s["budget"]), -1, dtype=np.int32)
    for b, n in enumerate(L):
        for h in range(mass.shape[1]):
            if n <= s["budget"]:
                keep[b, h, :n] = np.arange(n)
                continue
            lo, hi = s["first"], n - s["recent"]
            middle = np.arange(lo, hi)
            order = np.lexsort((middle, -mass[b, h, lo:hi].astype(np.float64)))[: s["budget"] - s["first"] - s["recent"]]
            keep[b, h] = np.concatenate([np.arange(lo), np.sort(middle[order]), np.arange(hi, n)])
    return {"keep": keep, "new_lens": np.minimum(np.array(L, dtype=np.int32), s["budget"]).astype(np.int32)}


def _exact_compact(s):
    page = s["k"].shape[2]
    dst = s["table"] if s["dst"] is None else s["dst"]
    names = [n for n in ("k", "v", "k_scale", "v_scale") if s[n] is not None]
    out = {n: s[n].clone() for n in names}
    mass = s["mass_out"].clone()
    for b, n in enumerate(s["new"].tolist()):
        to = torch.arange(n, device=DEV)
        for h in range(s["k"].shape[1]):
            at = s["keep"][b, h, :n].long()
            for name in names:
                rows = s[name][:, h]
                out[name][:, h][dst[b][to // page].long(), to % page] = rows[s["table"][b][at // page].long(), at % page]
            mass[b, h, :n] = s["mass"][b, h][at]
    return {n: _values(x) for n, x in out.items()} | {"mass": mass}


def _exact_beams(s):
    x = s["logits"].double().cpu().numpy()
    n, w, v = x.shape
    if x.size > 40_000_000:
        return None
    prev, done, length = s["scores"].double().cpu().numpy(), s["finished"].cpu().numpy() != 0, s["lengths"].cpu().numpy()
    got = {k: [] for k in ("tokens", "parents", "scores", "finished", "lengths")}
    for b in range(n):
        found = []
        for j in range(w):
            if done[b, j]:
                found.append((prev[b, j] / max(1, length[b, j]) ** s["penalty"], j, s["eos"], prev[b, j], length[b, j]))
                continue
            lp = x[b, j] - np.logaddexp.reduce(x[b, j])
            for t in np.argsort(-x[b, j], kind="stable")[:w]:
                found.append(((prev[b, j] + lp[t]) / max(1, length[b, j] + 1) ** s["penalty"], j, int(t), prev[b, j] + lp[t], length[b, j] + 1))
        found.sort(key=lambda f: (-f[0], f[1], f[2]))
        if len(found) < w:
            return None
        for _, j, t, total, ln in found[:w]:
            for k, val in zip(got, (t, j, total, int(done[b, j] or t == s["eos"]), ln)):
                got[k].append(val)
    kinds = {"tokens": np.int32, "parents": np.int32, "scores": np.float64, "finished": np.uint8, "lengths": np.int32}
    return {k: np.array(val, dtype=kinds[k]).reshape(n, w) for k, val in got.items()}


def _exact_reorder(s):
    page, par, L = s["k"].shape[2], s["parents"].tolist(), s["lens"].tolist()
    w = len(par[0])
    table = s["table"].cpu().numpy()
    out = table.copy()
    names = [n for n in ("k", "v", "k_scale", "v_scale") if s[n] is not None]
    made = {n: s[n].clone() for n in names}
    for b, ps in enumerate(par):
        full, part = divmod(L[b * w], page)
        free = [j for j in range(w) if j not in ps]
        seen = set()
        for j, p in enumerate(ps):
            out[b * w + j, :full] = table[b * w + p, :full]
            if not part:
                continue
            to = table[b * w + p, full]
            if p in seen:
                src, to = int(to), int(table[b * w + free.pop(0), full])
                for name in names:
                    made[name][to, :, :part] = s[name][src, :, :part]
            seen.add(p)
            out[b * w + j, full] = to
    got = {n: _values(x) for n, x in made.items()} | {"table": torch.from_numpy(out)}
    if s["state"] is not None:
        got["state"] = torch.stack([s["state"][b * w + p] for b, ps in enumerate(par) for p in ps])
    return got
