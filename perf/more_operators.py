"""A prompt's way into the paged KV cache, as cases that can be timed and compared.

Four operators: pages given to requests that grow, with the slots and positions of their new tokens
(`page_assign`), pages taken back from requests that shrank or ended (`page_release`), rotary positions of
queries and keys (`rope`) and causal attention over whole packed prompts (`prompt_attn`).  With `own` false `run`
computes them in elementary torch operations; with `own` true it makes the calls a user of the library makes.
"""
import math

import numpy as np
import torch

own = False

D = 128                        # head_dim
DEV = "cuda"


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step: one new token for each of 32 requests, every 128th of which opens a page
        dict(name="assign_decode", op="assign", reqs=32, lo=1, hi=8191, qlo=1, qhi=1, page=128, pad=0, room=1.0),
        # speculative decode in a padded batch on small pages
        dict(name="assign_ragged", op="assign", reqs=31, lo=0, hi=32767, qlo=0, qhi=6, page=16, pad=7, room=1.0),
        # 32 prompts of 8192 tokens at once, and a pool that runs out before the last ones
        dict(name="assign_prefill", op="assign", reqs=32, lo=0, hi=0, qlo=8192, qhi=8192, page=16, pad=0, room=0.9),
        # a few short requests that end or shrink
        dict(name="release_small", op="release", reqs=4, lo=1, hi=300, keep=64, page=16),
        # long contexts that were cut to a budget
        dict(name="release_evicted", op="release", reqs=32, lo=100000, hi=131072, keep=16384, page=16),
        # the new tokens of a decode batch
        dict(name="rope_decode", op="rope", tokens=32, heads=1, group=16, rot=128, half=True, type="bf16", far=131072, scaling="none",
             packed=False, inverse=False),
        # prompts of 8192 tokens, rotated out of the buffer that the projections left
        dict(name="rope_prefill", op="rope", tokens=16384, heads=1, group=16, rot=128, half=True, type="bf16", far=8192, scaling="none",
             packed=True, inverse=False),
        # neighbouring pairs in half of the head, fp32, far positions of a stretched context, rotated back
        dict(name="rope_far", op="rope", tokens=1999, heads=4, group=5, rot=64, half=False, type="f32", far=1000000, scaling="yarn",
             packed=False, inverse=True),
        # a handful of short prompts: the latency of a call
        dict(name="prompt_short", op="prompt", reqs=4, lo=1, hi=300, heads=1, group=16, packed=False, pad=0),
        # one prompt as long as the chunks that prefill takes
        dict(name="prompt_2k", op="prompt", reqs=1, lo=2048, hi=2048, heads=1, group=16, packed=False, pad=0),
        # a packed batch of uneven prompts, several KV heads, rows behind the last one
        dict(name="prompt_packed", op="prompt", reqs=13, lo=200, hi=4001, heads=4, group=4, packed=True, pad=33),
        # a long prompt
        dict(name="prompt_32k", op="prompt", reqs=1, lo=32768, hi=32768, heads=1, group=16, packed=False, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["assign", "release", "rope", "prompt", "prompt"])
    page = rng.choice([16, 32, 64, 128])
    if op == "assign":
        qhi = rng.choice([1, 1, _log(rng, 2, 8192)])
        reqs = _log(rng, 1, max(2, min(2000, 262144 // qhi)))
        hi = _log(rng, 1, 32768)
        return dict(op="assign", reqs=reqs, lo=rng.randint(0, hi), hi=hi, qlo=rng.randint(0, qhi), qhi=qhi, page=page,
                    pad=rng.choice([0, 0, rng.randint(1, 64)]), room=rng.choice([1.0, 1.0, round(rng.uniform(0.3, 1.0), 3)]))
    if op == "release":
        hi = _log(rng, 1, 131072)
        return dict(op="release", reqs=_log(rng, 1, max(2, min(2000, 4000000 // hi))), lo=rng.randint(0, hi), hi=hi, keep=rng.randint(0, hi), page=page)
    heads, group = rng.choice([1, 1, 1, 2, 4]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 16, 32])
    if op == "rope":
        rot = rng.choice([128, 128, 64, 2 * rng.randint(1, 64)])
        return dict(op="rope", tokens=_log(rng, 1, max(2, min(20000, 270000 // (heads * (group + 1))))), heads=heads, group=group, rot=rot,
                    half=rng.random() < 0.6, type=rng.choice(["bf16", "bf16", "f32"]), far=_log(rng, 2, 1000000),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), packed=rng.random() < 0.5, inverse=rng.random() < 0.2)
    hi = _log(rng, 1, 24000)
    reqs = max(1, min(_log(rng, 1, 64), 40000 // hi, 260000 // (hi * heads * group), 16000000000 // (hi * hi * heads * group)))
    return dict(op="prompt", reqs=reqs, lo=rng.randint(max(1, hi // 8), hi), hi=hi, heads=heads, group=group, packed=rng.random() < 0.5,
                pad=rng.choice([0, 0, rng.randint(1, 200)]))


# ----------------------------------------------------------------------------- inputs

def _lens(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _even(g, n, lo, hi):
    """Lengths over the range in pairs of the same sum, in random order: whatever the seed, there are as many tokens."""
    one = _lens(g, n // 2, lo, hi)
    both = torch.cat([one, lo + hi - one, one.new_full((n % 2,), (lo + hi) // 2)])
    return both[torch.randperm(n, generator=g, device=DEV)]


def _pages(lens, page):
    return (lens + page - 1) // page


def _cu(lens):
    return torch.cat([lens.new_zeros(1), lens.cumsum(0).to(torch.int32)])


def _prepare_assign(c, g):
    """Contexts that hold pages of a pool, the rest of the pool as a stack of free pages, and the new tokens' counts."""
    n, page = c["reqs"], c["page"]
    lens, ql = _lens(g, n, c["lo"], c["hi"]), _even(g, n, c["qlo"], c["qhi"])
    width = -(-(c["hi"] + c["qhi"]) // page) + 1
    have, want = _pages(lens, page), _pages(lens + ql, page)
    used, need = int(have.sum()), int((want - have).sum())
    free = int(need * c["room"]) if c["room"] < 1.0 else need + 13
    ids = torch.randperm(used + free, generator=g, device=DEV).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV)[None] < have[:, None]] = ids[:used]
    stack = torch.full((used + free,), -1, dtype=torch.int32, device=DEV)
    stack[:free] = ids[used:]
    rows = int(ql.sum()) + c["pad"]
    return dict(op="assign", lens=lens, cu=_cu(ql), table=table, free=stack, num_free=torch.tensor([free], dtype=torch.int32, device=DEV),
                left=torch.zeros(1, dtype=torch.int32, device=DEV), page=page, pages=used + free, rows=rows)


def _prepare_release(c, g):
    """Contexts of which some end, some are cut to a budget and some stay, over a pool with a few free pages."""
    n, page = c["reqs"], c["page"]
    lens = _lens(g, n, c["lo"], c["hi"])
    new = torch.where(torch.rand(n, generator=g, device=DEV) < 0.2, torch.zeros_like(lens), lens.clamp(max=c["keep"]))
    width = max(1, -(-c["hi"] // page))
    have = _pages(lens, page)
    used, free = int(have.sum()), 29
    ids = torch.randperm(used + free, generator=g, device=DEV).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV)[None] < have[:, None]] = ids[:used]
    stack = torch.full((n * width + free,), -1, dtype=torch.int32, device=DEV)
    stack[:free] = ids[used:]
    return dict(op="release", lens=lens, new=new, table=table, free=stack, num_free=torch.tensor([free], dtype=torch.int32, device=DEV),
                left=torch.zeros(1, dtype=torch.int32, device=DEV), page=page, pages=used + free)


# A context stretched by 8 from one of 4096 tokens, and the base of the rotation.
BASE, FACTOR, TRAINED = 10000.0, 8.0, 4096


def _angles(rot, scaling):
    """Radians per position of each pair, in 64 bits, and what scales the rotated values."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    w = BASE ** (-2.0 * i / rot)
    if scaling == "linear":
        return w / FACTOR, 1.0
    if scaling == "ntk":
        return (BASE * FACTOR ** (rot / (rot - 2.0) if rot > 2 else 1.0)) ** (-2.0 * i / rot), 1.0
    if scaling == "yarn":
        # pairs that turn more than 32 times within the trained length stay, those below one turn are stretched
        def pair(turns):
            return rot * math.log(TRAINED / (turns * 2.0 * math.pi)) / (2.0 * math.log(BASE))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return w / FACTOR * ramp + w * (1.0 - ramp), 0.1 * math.log(FACTOR) + 1.0
    return w, 1.0


def _split(g, tokens, heads, group, dtype, packed):
    """Queries, keys and values as three tensors, or as views of the buffer that one projection wrote."""
    hq = heads * group
    if not packed:
        return [torch.randn(tokens, h, D, generator=g, device=DEV).to(dtype) for h in (hq, heads, heads)]
    x = torch.randn(tokens, (hq + 2 * heads) * D, generator=g, device=DEV).to(dtype)
    return [y.view(tokens, -1, D) for y in x.split([hq * D, heads * D, heads * D], dim=1)]


def _prepare_rope(c, g):
    dtype = torch.bfloat16 if c["type"] == "bf16" else torch.float32
    q, k, _ = _split(g, c["tokens"], c["heads"], c["group"], dtype, c["packed"])
    angles, scale = _angles(c["rot"], c["scaling"])
    s = dict(op="rope", q=q, k=k, positions=_lens(g, c["tokens"], 0, c["far"] - 1), rot=c["rot"], half=c["half"], inverse=c["inverse"],
             angles=angles.to(DEV), scale=scale, q_out=torch.empty(q.shape, dtype=dtype, device=DEV),
             k_out=torch.empty(k.shape, dtype=dtype, device=DEV))
    if own:
        from paged_fp8_kv_04_gb300 import binding as B
        s["freqs"], s["scale"] = B.rope_frequencies(c["rot"], base=BASE, scaling=None if c["scaling"] == "none" else c["scaling"],
                                                    factor=FACTOR, original_len=TRAINED, device=DEV)
    return s


def _prepare_prompt(c, g):
    lens = _even(g, c["reqs"], c["lo"], c["hi"])
    tokens = int(lens.sum()) + c["pad"]
    q, k, v = _split(g, tokens, c["heads"], c["group"], torch.bfloat16, c["packed"])
    return dict(op="prompt", q=q, k=k, v=v, cu=_cu(lens), sm=1.0 / math.sqrt(D), out=torch.zeros(q.shape, dtype=torch.bfloat16, device=DEV),
                lse=torch.zeros(q.shape[:2], device=DEV))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"assign": _prepare_assign, "release": _prepare_release, "rope": _prepare_rope, "prompt": _prepare_prompt}[case["op"]](case, g)


# -------------------------------------------------------------------- the plain forms

def _assign(s):
    """Requests take pages off the stack's top, in order, as long as the pool lasts; their tokens' slots follow."""
    L, page, cu = s["lens"].long(), s["page"], s["cu"].long()
    ql = cu[1:] - cu[:-1]
    have, want = _pages(L, page), _pages(L + ql, page)
    need = want - have
    upto = need.cumsum(0)
    served = (need == 0) | (upto <= s["num_free"].long())
    col = torch.arange(s["table"].shape[1], device=DEV)[None]
    rank = (upto - need)[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < want[:, None]) & served[:, None]
    top = (s["num_free"].long() - 1 - rank).clamp(min=0, max=s["free"].numel() - 1)
    s["table"].copy_(torch.where(fresh, s["free"][top], s["table"]))
    row = torch.arange(s["rows"], device=DEV)
    r = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    live = r < L.numel()
    r = r.clamp(max=L.numel() - 1)
    pos = L[r] + row - cu[r]
    slot = s["table"][r, pos // page].long() * page + pos % page
    return {"table": s["table"], "new_lens": torch.where(served, L + ql, L).to(torch.int32), "slots": torch.where(live & served[r], slot, -1),
            "positions": torch.where(live, pos, 0).to(torch.int32), "num_free": (s["num_free"] - torch.where(served, need, 0).sum()).to(torch.int32)}


def _release(s):
    """The pages behind each request's new length go onto the stack, request by request, in the table's order."""
    page = s["page"]
    col = torch.arange(s["table"].shape[1], device=DEV)[None]
    gone = (col >= _pages(s["new"], page)[:, None]) & (col < _pages(s["lens"], page)[:, None])
    ids = s["table"][gone]
    at = s["num_free"].long() + torch.arange(ids.numel(), device=DEV)
    s["free"][at] = ids
    return {"free": s["free"], "num_free": s["num_free"] + ids.numel()}


def _turn(x, cos, sin, rot, half):
    x = x.float()
    y = x[..., :rot]
    a, b = (y[..., : rot // 2], y[..., rot // 2:]) if half else (y[..., 0::2], y[..., 1::2])
    c, d = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([c, d], -1) if half else torch.stack([c, d], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _rope(s):
    """Pair i of a token at position p turns by p * angles[i], computed in 64 bits."""
    a = s["positions"].double()[:, None] * s["angles"][None]
    cos, sin = (torch.cos(a) * s["scale"]).float()[:, None], (torch.sin(a) * s["scale"]).float()[:, None]
    if s["inverse"]:
        sin = -sin
    return {n: _turn(s[n], cos, sin, s["rot"], s["half"]).to(s[n].dtype) for n in ("q", "k")}


def _prompt(s):
    """softmax(sm q k) v over each sequence's own earlier tokens, some query rows at a time."""
    heads = s["k"].shape[1]
    hq = s["q"].shape[1]
    cu = s["cu"].tolist()
    for a, b in zip(cu[:-1], cu[1:]):
        k = s["k"][a:b].float().permute(1, 2, 0)
        v = s["v"][a:b].float().permute(1, 0, 2)
        step = max(1, 200_000_000 // ((b - a) * hq)) if b > a else 1
        for t0 in range(a, b, step):
            t1 = min(b, t0 + step)
            n, end = t1 - t0, t1 - a
            q = s["q"][t0:t1].float().view(n, heads, hq // heads, D).permute(1, 2, 0, 3).reshape(heads, -1, D)
            x = ((q @ k[:, :, :end]) * s["sm"]).view(heads, hq // heads, n, end)
            seen = torch.arange(end, device=DEV)[None] <= (t0 - a) + torch.arange(n, device=DEV)[:, None]
            x = x.masked_fill(~seen, -math.inf)
            top = x.amax(-1, keepdim=True)
            x = torch.exp(x - top)
            z = x.sum(-1, keepdim=True)
            o = ((x.view(heads, -1, end) @ v[:, :end]).view(heads, hq // heads, n, D) / z).permute(2, 0, 1, 3)
            s["out"][t0:t1] = o.reshape(n, hq, D).to(torch.bfloat16)
            s["lse"][t0:t1] = (top + z.log())[..., 0].permute(2, 0, 1).reshape(n, hq)
    return {"out": s["out"], "lse": s["lse"]}


def _call(s):
    from paged_fp8_kv_04_gb300 import binding as B
    if s["op"] == "assign":
        new, slots, positions = B.page_assign(s["lens"], s["cu"], s["table"], s["free"], s["num_free"], page_size=s["page"], num_pages=s["pages"],
                                              num_rows=s["rows"], num_free_out=s["left"])
        return {"table": s["table"], "new_lens": new, "slots": slots, "positions": positions, "num_free": s["left"]}
    if s["op"] == "release":
        B.page_release(s["lens"], s["new"], s["table"], s["free"], s["num_free"], page_size=s["page"], num_pages=s["pages"], num_free_out=s["left"])
        return {"free": s["free"], "num_free": s["left"]}
    if s["op"] == "rope":
        q, k = B.rope(s["q"], s["k"], s["positions"], s["freqs"], layout="half" if s["half"] else "pairs", inverse=s["inverse"],
                      scale=s["scale"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    out, lse = B.prompt_attn(s["q"], s["k"], s["v"], s["cu"], sm_scale=s["sm"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _call(state)
    return {"assign": _assign, "release": _release, "rope": _rope, "prompt": _prompt}[state["op"]](state)


# ------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "assign":
        rows = c["reqs"] * (c["qlo"] + c["qhi"]) / 2
        pages = rows / c["page"]
        # lengths in and out, a page read and entered for each new one, slot and position of every row
        return {"bytes": 12 * c["reqs"] + 8 * pages + 12 * (rows + c["pad"]), "flops": 4 * rows}
    if c["op"] == "release":
        mean = (c["lo"] + c["hi"]) / 2
        pages = c["reqs"] * (mean - 0.8 * min(mean, c["keep"])) / c["page"]
        return {"bytes": 8 * c["reqs"] + 8 * pages, "flops": 2 * c["reqs"]}
    if c["op"] == "rope":
        size = 2 if c["type"] == "bf16" else 4
        rows = c["tokens"] * c["heads"] * (c["group"] + 1)
        return {"bytes": 2.0 * rows * D * size + 4 * c["tokens"], "flops": 3.0 * rows * c["rot"]}
    n, lo, hi, hq = c["reqs"], c["lo"], c["hi"], c["heads"] * c["group"]
    mean, square = (lo + hi) / 2, (lo * lo + lo * hi + hi * hi) / 3
    return {"bytes": n * mean * (4.0 * D * (hq + c["heads"]) + 4 * hq), "flops": 4.0 * D * hq * n * (square + mean) / 2}


# ----------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"assign": _exact_assign, "release": _exact_release, "rope": _exact_rope, "prompt": _exact_prompt}[case["op"]](s)


def _exact_assign(s):
    page, cu, lens, free = s["page"], s["cu"].tolist(), s["lens"].tolist(), s["free"].tolist()
    table, left, gone = s["table"].cpu().numpy().copy(), int(s["num_free"]), False
    slots, positions = np.full(s["rows"], -1, dtype=np.int64), np.zeros(s["rows"], dtype=np.int32)
    new = np.array(lens, dtype=np.int32)
    for r, n in enumerate(lens):
        a, b = cu[r], cu[r + 1]
        at = n + np.arange(b - a)
        positions[a:b] = at
        have, want = math.ceil(n / page), math.ceil((n + b - a) / page)
        if want > have:
            gone = gone or want - have > left
            if gone:
                continue
            for p in range(have, want):
                left -= 1
                table[r, p] = free[left]
        slots[a:b] = table[r, at // page].astype(np.int64) * page + at % page
        new[r] = n + b - a
    return {"table": table, "new_lens": new, "slots": slots, "positions": positions, "num_free": np.array([left], dtype=np.int32)}


def _exact_release(s):
    page, table, free, top = s["page"], s["table"].tolist(), s["free"].tolist(), int(s["num_free"])
    for r, (n, m) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        for p in range(math.ceil(m / page), math.ceil(n / page)):
            free[top] = table[r][p]
            top += 1
    return {"free": np.array(free, dtype=np.int32), "num_free": np.array([top], dtype=np.int32)}


def _exact_rope(s):
    rot, sign = s["rot"], -1.0 if s["inverse"] else 1.0
    at = s["positions"].cpu().numpy().astype(np.longdouble)[:, None] * s["angles"].cpu().numpy().astype(np.longdouble)[None]
    z = torch.from_numpy(np.exp(1j * sign * np.mod(at, 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))).astype(np.float64)) * s["scale"]).to(DEV)
    got = {}
    for name in ("q", "k"):
        y = s[name].double().clone()
        i = torch.arange(rot // 2, device=DEV)
        one, two = (i, i + rot // 2) if s["half"] else (2 * i, 2 * i + 1)
        w = torch.complex(y[..., one], y[..., two]) * z[:, None]
        y[..., one], y[..., two] = w.real, w.imag
        got[name] = y
    return got


def _exact_prompt(s):
    hq, heads = s["q"].shape[1], s["k"].shape[1]
    cu = s["cu"].tolist()
    if sum((b - a) ** 2 for a, b in zip(cu[:-1], cu[1:])) * hq * 2.0 * D > 6e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for a, b in zip(cu[:-1], cu[1:]):
        for h in range(hq):
            k, v = (s[n][a:b, h // (hq // heads)].double() for n in ("k", "v"))
            q = s["q"][a:b, h].double() * s["sm"]
            for t in range(0, b - a, 2048):
                e = min(b - a, t + 2048)
                x = q[t:e] @ k[:e].T
                x += torch.full((e - t, e), -math.inf, dtype=torch.float64, device=DEV).triu(t + 1)
                z = torch.logsumexp(x, -1)
                out[a + t:a + e, h] = torch.exp(x - z[:, None]) @ v[:e]
                lse[a + t:a + e, h] = z
    return {"out": out, "lse": lse}
