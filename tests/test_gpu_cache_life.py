"""The cache operators together, as a serving loop uses them (needs a GPU): decode, attention
mass, eviction and compaction, decode on; and beam search over the paged cache, against an
oracle that keeps every beam's whole history apart."""
import dataclasses

import numpy as np
import pytest
import torch

from cache_util import dev, host
from gpu_util import compare
from oracle import cache_ops as C
from oracle import oracle as O
from paged_fp8_kv_04_gb300 import binding as B
from paged_fp8_kv_04_gb300 import device as dv
from paged_fp8_kv_04_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _grow(p, budget, slack):
    """Problem p's block tables widened for `slack` more tokens per request."""
    ps, n = p.page_size, p.num_seqs
    width = -(-(int(p.context_lens.max()) + slack) // ps)
    pool = np.random.default_rng(1).permutation(n * width).astype(np.int32).reshape(n, width)
    arrays = {}
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        a = getattr(p, name)
        if a is None:
            continue
        b = np.zeros((n * width,) + a.shape[1:], a.dtype)
        for r in range(n):
            for g in range(-(-int(p.context_lens[r]) // ps)):
                b[pool[r, g]] = a[p.block_table[r, g]]
        arrays[name] = b
    return dataclasses.replace(p, block_table=pool, **arrays)


@pytest.mark.parametrize("page,heads", [(16, 2), (128, 1)])
def test_decode_with_a_bounded_cache(page, heads):
    """Requests decode token by token; whenever one holds budget + slack tokens all are cut to the budget.
    Every decode is checked against the oracle's attention over the very tokens that each
    KV head has kept, and every selection against the oracle's on the device's mass."""
    budget, slack, steps = 96, 24, 60
    rng = np.random.default_rng(page)
    p = _grow(synth.make_problem(31, num_seqs=3, context_lens=[90, 50, 110], q_lens=[1] * 3, page_size=page,
                                 num_kv_heads=heads, scale_mode="per_token"), budget, budget)
    d = dv.to_device(p)
    kc, vc, ks, vs, table = d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"], d["block_table"]
    width, Hq = table.shape[1] * page, heads * 16
    # the oracle's cache: per (request, head) the codes and scales kept, in order
    kept = [[[(p.k_cache[p.block_table[r, i // page], h, i % page].copy(), p.k_scale[p.block_table[r, i // page], h, i % page],
               p.v_cache[p.block_table[r, i // page], h, i % page].copy(), p.v_scale[p.block_table[r, i // page], h, i % page])
              for i in range(int(p.context_lens[r]))] for h in range(heads)] for r in range(3)]
    lens = p.context_lens.astype(np.int32).copy()
    mass = torch.full((3, heads, width), float("nan"), device="cuda")
    plan = B.Plan(num_kv_heads=heads, page_size=page, max_batch=3, max_context_len=width, out_dtype="f32")
    cu = dev(np.arange(4, dtype=np.int32))
    status, first, cuts = torch.zeros(1, dtype=torch.int32, device="cuda"), True, 0
    for step in range(steps):
        # a new token for every request, written by the library
        x = synth.bf16_bits(rng.standard_normal((3, heads, 128), dtype=np.float32))
        y = synth.bf16_bits(rng.standard_normal((3, heads, 128), dtype=np.float32))
        tb = host(table)
        slots = np.array([int(tb[r, lens[r] // page]) * page + lens[r] % page for r in range(3)], np.int64)
        B.kv_quantize_write(dev(x), dev(y), dev(slots), kc, vc, ks, vs)
        cache = [host(t) for t in (kc, ks, vc, vs)]
        for r in range(3):
            for h in range(heads):
                at = (int(tb[r, lens[r] // page]), h, int(lens[r]) % page)
                kept[r][h].append(tuple(np.copy(c[at]) for c in cache))
        lens += 1
        q = synth.bf16_bits(rng.standard_normal((3, Hq, 128), dtype=np.float32))
        ctx, lse = dev(lens), torch.empty(3, Hq, device="cuda")
        out = plan.decode(dev(q), kc, vc, table, ctx, k_scale=ks, v_scale=vs, lse=lse)
        B.attn_mass(dev(q), kc, table, ctx, cu, lse, mass, max_q_len=1, k_scale=ks, decay=0.0 if first else 0.9, status=status)
        first = False
        # the oracle's attention over what is kept
        want = np.zeros((3, Hq, 128))
        for r in range(3):
            for h in range(heads):
                k = C.rows_f64(np.stack([t[0] for t in kept[r][h]]), np.array([t[1] for t in kept[r][h]]))
                v = C.rows_f64(np.stack([t[2] for t in kept[r][h]]), np.array([t[3] for t in kept[r][h]]))
                for g in range(16):
                    qq = (q[r, h * 16 + g].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
                    s = k @ qq / np.sqrt(128.0)
                    w = np.exp(s - s.max())
                    want[r, h * 16 + g] = w @ v / w.sum()
        compare(host(out), want, f"step {step}")
        m = host(mass)
        for r in range(3):
            assert np.isfinite(m[r, :, :lens[r]]).all() and np.all(m[r, :, :lens[r]] >= 0)
            # the step's weights alone sum to 16 per KV head, the carried ones to at most 16 / (1 - 0.9)
            assert np.all(m[r, :, :lens[r]].sum(-1) <= 161.0) and np.all(m[r, :, :lens[r]].sum(-1) >= 15.9)
        if lens.max() >= budget + slack:
            keep, new = B.evict_select(mass, ctx, budget=budget, first=4, recent=16, status=status)
            want_keep, want_new = C.evict_select(m, lens, budget, 4, 16)
            assert np.array_equal(host(keep), want_keep) and np.array_equal(host(new), want_new)
            B.kv_compact(keep, new, table, kc, vc, k_scale=ks, v_scale=vs, mass=mass, status=status)
            for r in range(3):
                for h in range(heads):
                    kept[r][h] = [kept[r][h][i] for i in want_keep[r, h, :want_new[r]]]
            lens = want_new.astype(np.int32)
            cuts += 1
    torch.cuda.synchronize()
    assert cuts >= 2 and int(status[0]) == 0 and plan.device_status() == 0


def _beam_problem(rng, W, prompt, page, heads, steps):
    npg = -(-(prompt + steps) // page)
    pages = rng.permutation(W * npg).astype(np.int32).reshape(W, npg)
    shape = (W * npg, heads, page, 128)
    return pages, [np.zeros(shape, np.uint8), np.zeros(shape, np.uint8), np.zeros(shape[:3], np.float32), np.zeros(shape[:3], np.float32)]


@pytest.mark.parametrize("W,page,heads,prompt", [(4, 16, 1, 21), (3, 32, 2, 32), (8, 128, 1, 130)])
def test_beam_search_over_the_paged_cache(W, page, heads, prompt):
    """A prompt cached once, spread over W beams, then steps of select, reorder, write and decode.  Token
    embeddings and the output projection are random; every beam's history (tokens, and the codes
    and scales written for them) is kept apart on the host and decoded by the oracle."""
    rng = np.random.default_rng(W + page)
    steps, V, Hq = 12, 301, heads * 16
    table_h, arrays = _beam_problem(rng, W, prompt, page, heads, steps + 1)
    emb = [synth.bf16_bits(rng.standard_normal((V, heads, 128), dtype=np.float32)) for _ in range(2)]  # K and V of a token
    qs = synth.bf16_bits(rng.standard_normal((steps + 1, W, Hq, 128), dtype=np.float32))
    proj = torch.from_numpy(rng.standard_normal((Hq * 128, V)).astype(np.float32)).cuda() * 0.05
    kc, vc, ks, vs = (dev(a) for a in arrays)
    table, other = dev(table_h), torch.empty(table_h.shape, dtype=torch.int32, device="cuda")
    prompt_tokens = rng.integers(0, V, size=prompt)

    def write(tokens, slots):
        B.kv_quantize_write(dev(emb[0][tokens]), dev(emb[1][tokens]), dev(np.asarray(slots, np.int64)), kc, vc, ks, vs)

    write(prompt_tokens, [int(table_h[0, i // page]) * page + i % page for i in range(prompt)])
    lens = np.full(W, prompt, np.int32)
    history = torch.zeros(W, steps, dtype=torch.int32, device="cuda")
    spare = torch.empty_like(history)
    # the prompt is spread: every beam continues beam 0
    B.beam_reorder(dev(np.zeros((1, W), np.int32)), dev(lens), table, other, kc, vc, k_scale=ks, v_scale=vs)
    table, other = other, table
    scores = torch.full((1, W), -float("inf"), device="cuda")
    scores[0, 0] = 0.0
    finished, lengths = torch.zeros(1, W, dtype=torch.uint8, device="cuda"), torch.zeros(1, W, dtype=torch.int32, device="cuda")
    plan = B.Plan(num_kv_heads=heads, page_size=page, max_batch=W, max_context_len=prompt + steps + 1, out_dtype="f32")
    beams = [list(prompt_tokens) for _ in range(W)]          # the oracle's histories
    eos = 7
    one = {}

    def token_rows(t):  # codes and scales of a token, by the oracle's quantiser
        if t not in one:
            a = [np.zeros((1, heads, 16, 128), np.uint8), np.zeros((1, heads, 16, 128), np.uint8),
                 np.zeros((1, heads, 16), np.float32), np.zeros((1, heads, 16), np.float32)]
            O.kv_quantize_write(emb[0][[t]], emb[1][[t]], np.zeros(1, np.int64), *a)
            one[t] = [x[0, :, 0] for x in a]
        return one[t]

    def problem(q):
        """The beams as separate requests with pages of their own."""
        L = len(beams[0])
        npg = -(-L // page)
        arr = [np.zeros((W * npg,) + s, d) for s, d in (((heads, page, 128), np.uint8), ((heads, page, 128), np.uint8),
                                                       ((heads, page), np.float32), ((heads, page), np.float32))]
        for b in range(W):
            for i, t in enumerate(beams[b]):
                for a, x in zip(arr, token_rows(int(t))):
                    a[b * npg + i // page, :, i % page] = x
        return synth.Problem(num_seqs=W, num_kv_heads=heads, group_size=16, head_dim=128, page_size=page, kv_dtype="fp8",
                             scale_mode="per_token", q=q, k_cache=arr[0], v_cache=arr[1], k_scale=arr[2], v_scale=arr[3],
                             k_scale_scalar=1.0, v_scale_scalar=1.0, block_table=np.arange(W * npg, dtype=np.int32).reshape(W, npg),
                             context_lens=np.full(W, L, np.int32), cu_seqlens_q=np.arange(W + 1, dtype=np.int32), uniform_q_len=1,
                             selected=None, num_selected=None, sm_scale=1.0 / np.sqrt(128.0))

    for step in range(steps):
        out = plan.decode(dev(qs[step]), kc, vc, table, dev(lens), k_scale=ks, v_scale=vs)
        want, _ = O.decode(problem(qs[step]))
        compare(host(out), want, f"step {step}")
        logits = (out.view(W, -1) @ proj).view(1, W, V)
        before = [host(t).copy() for t in (scores, finished, lengths)]
        tokens, parents, scores, finished, lengths = B.beam_select(logits, scores, eos=eos, finished=finished, lengths=lengths,
                                                                  length_penalty=0.6)
        wt, wp, ws, wf, wl = C.beam_select(host(logits).astype(np.float64), before[0], eos, before[1], before[2], 0.6)
        tk, pr = host(tokens), host(parents)
        assert np.array_equal(tk, wt) and np.array_equal(pr, wp) and np.array_equal(host(finished), wf)
        assert np.array_equal(host(lengths), wl)
        B.beam_reorder(parents, dev(lens), table, other, kc, vc, k_scale=ks, v_scale=vs, states=[(history, spare)])
        table, other, history, spare = other, table, spare, history
        history[:, step] = tokens[0]
        tb = host(table)
        write(tk[0], [int(tb[b, lens[b] // page]) * page + lens[b] % page for b in range(W)])
        lens += 1
        beams = [beams[int(pr[0, b])] + [int(tk[0, b])] for b in range(W)]
        assert np.array_equal(host(history)[:, :step + 1], np.array([b[prompt:] for b in beams]))
        # a page that still takes tokens belongs to one beam alone
        last = tb[:, lens[0] // page] if lens[0] % page else tb[:, lens[0] // page - 1]
        if lens[0] % page:
            assert len(set(last.tolist())) == W
    assert plan.device_status() == 0


def test_beams_are_evicted_into_fresh_pages():
    """Beams share their prompt's pages, so their caches are cut into pages of their own."""
    rng = np.random.default_rng(5)
    W, page, L, budget = 4, 16, 150, 64
    npg, new_npg = -(-L // page), -(-budget // page)
    shared = rng.permutation(60).astype(np.int32)
    table = np.concatenate([np.repeat(shared[None, :npg - 1], W, 0), shared[npg - 1:npg - 1 + W, None]], 1).astype(np.int32)
    fresh = (60 + rng.permutation(W * new_npg)).astype(np.int32).reshape(W, new_npg)
    n = 60 + W * new_npg
    x = rng.standard_normal((n, 1, page, 128), dtype=np.float32)
    k, ksc = synth.quantize_per_token(x)
    v, vsc = synth.quantize_per_token(x[::-1].copy())
    q = synth.bf16_bits(rng.standard_normal((W, 16, 128), dtype=np.float32))
    kc, vc, ks, vs = (dev(a) for a in (k, v, ksc, vsc))
    lens, cu = dev(np.full(W, L, np.int32)), dev(np.arange(W + 1, dtype=np.int32))
    plan = B.Plan(page_size=page, max_batch=W, max_context_len=L, out_dtype="f32")
    lse = torch.empty(W, 16, device="cuda")
    plan.decode(dev(q), kc, vc, dev(table), lens, k_scale=ks, v_scale=vs, lse=lse)
    mass = B.attn_mass(dev(q), kc, dev(table), lens, cu, lse, torch.empty(W, 1, npg * page, device="cuda"), max_q_len=1,
                       k_scale=ks, decay=0.0)
    keep, new = B.evict_select(mass, lens, budget=budget, first=2, recent=8)
    moved = torch.zeros(W, 1, budget, device="cuda")
    B.kv_compact(keep, new, dev(table), kc, vc, dst_block_table=dev(fresh), k_scale=ks, v_scale=vs, mass=mass, mass_out=moved)
    out = plan.decode(dev(q), kc, vc, dev(fresh), new, k_scale=ks, v_scale=vs)
    assert np.array_equal(host(kc)[:60], k[:60]) and np.array_equal(host(vs)[:60], vsc[:60])   # the shared pages are as they were
    kp = host(keep)
    for b in range(W):
        at = kp[b, 0]
        rows = [C.rows_f64(a[table[b][at // page], 0, at % page], s[table[b][at // page], 0, at % page]) for a, s in ((k, ksc), (v, vsc))]
        qq = (q[b].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        s = qq @ rows[0].T / np.sqrt(128.0)
        w = np.exp(s - s.max(-1, keepdims=True))
        compare(host(out)[b:b + 1], (w @ rows[1] / w.sum(-1, keepdims=True))[None], f"beam {b}")
        assert np.array_equal(host(moved)[b, 0], host(mass)[b, 0][at])


def test_caches_beyond_four_gigabytes():
    """Pages whose bytes lie past 2^32: mass, compaction and reordering address them, and give
    what they give on a small cache."""
    page, pages = 128, (1 << 18) + 400          # 2^25 rows of 128 bytes, and more
    p = synth.make_problem(41, num_seqs=2, context_lens=[700, 640], q_lens=[1, 2], page_size=page)
    lse = O.decode(p)[1].astype(np.float32)
    used = p.num_pages
    where = torch.from_numpy((pages - 1 - np.arange(used) * 3).astype(np.int32)).cuda()    # high pages, apart

    def spread(a):
        big = torch.empty((pages,) + a.shape[1:], dtype=dev(a).dtype, device="cuda")
        big[where.long()] = dev(a)
        return big

    small = [dev(a) for a in (p.k_cache, p.v_cache, p.k_scale, p.v_scale)]
    big = [spread(a) for a in (p.k_cache, p.v_cache, p.k_scale, p.v_scale)]
    bt = dev(p.block_table)
    bt_big = torch.where(bt >= 0, where[bt.clamp(min=0).long()], bt)
    args = [dev(x) for x in (p.context_lens, p.cu_seqlens_q, lse)]
    m = [B.attn_mass(dev(p.q), c[0], t, *args, torch.zeros(2, 1, 700, device="cuda"), max_q_len=2, decay=0.0, k_scale=c[2])
         for c, t in ((small, bt), (big, bt_big))]
    assert torch.equal(m[0], m[1])
    keep, new = B.evict_select(m[0], args[0], budget=300, first=4, recent=32)
    for c, t in ((small, bt), (big, bt_big)):
        B.kv_compact(keep, new, t, c[0], c[1], k_scale=c[2], v_scale=c[3])
    for a, b in zip(small, big):
        assert torch.equal(a, b[where.long()])
    lens = torch.full((2,), 300, dtype=torch.int32, device="cuda")
    parents = torch.ones(1, 2, dtype=torch.int32, device="cuda")
    outs = []
    for c, t in ((small, bt), (big, bt_big)):
        o = torch.empty_like(t)
        B.beam_reorder(parents, lens, t, o, c[0], c[1], k_scale=c[2], v_scale=c[3])
        outs.append(o)
    assert torch.equal(outs[1], torch.where(outs[0] >= 0, where[outs[0].clamp(min=0).long()], outs[0]))
    for a, b in zip(small, big):
        assert torch.equal(a, b[where.long()])


def test_calls_on_a_stream_of_their_own():
    """stream=: the call and its outputs belong to that stream."""
    rng = np.random.default_rng(6)
    s = torch.cuda.Stream()
    logits, scores = torch.randn(2, 4, 5001, device="cuda"), torch.randn(2, 4, device="cuda")
    mass, lens = torch.rand(3, 2, 900, device="cuda"), dev(np.array([900, 500, 3], np.int32))
    a, b = B.beam_select(logits, scores), B.evict_select(mass, lens, budget=200, recent=9)
    s.wait_stream(torch.cuda.current_stream())
    x, y = B.beam_select(logits, scores, stream=s), B.evict_select(mass, lens, budget=200, recent=9, stream=s)
    s.synchronize()
    assert torch.equal(a[0], x[0]) and torch.equal(a[2], x[2]) and torch.equal(b[0], y[0]) and torch.equal(b[1], y[1])


def test_bindings_refuse_wrong_tensors():
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.zeros(8, 1, 16, 128, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(8, 1, 16, device="cuda")
    t, keep, new = torch.zeros(2, 4, **i32), torch.zeros(2, 1, 8, **i32), torch.zeros(2, **i32)
    mass = torch.zeros(2, 1, 64, device="cuda")
    bad = [
        lambda: B.kv_compact(keep, new, t, k, k.float(), k_scale=sc, v_scale=sc),
        lambda: B.kv_compact(keep, new, t, k, k.clone(), k_scale=sc),
        lambda: B.kv_compact(keep.long(), new, t, k, k.clone()),
        lambda: B.kv_compact(keep, new, t, k, k.clone(), dst_block_table=t + 4, mass=mass),
        lambda: B.kv_compact(keep, new, t, k, k.clone(), mass_out=mass),
        lambda: B.kv_compact(keep, new, t, k.bfloat16(), k.bfloat16(), k_scale=sc, v_scale=sc),
        lambda: B.evict_select(mass, new, budget=0),
        lambda: B.evict_select(mass, new, budget=4, first=3, recent=2),
        lambda: B.evict_select(mass, new.cpu(), budget=4),
        lambda: B.evict_select(mass[:, :, ::2], new, budget=4),
        lambda: B.beam_select(torch.zeros(2, 3, 9, device="cuda").half(), torch.zeros(2, 3, device="cuda")),
        lambda: B.beam_select(torch.zeros(2, 3, 9, device="cuda").transpose(0, 1), torch.zeros(3, 2, device="cuda")),
        lambda: B.beam_select(torch.zeros(2, 3, 9, device="cuda"), torch.zeros(2, 4, device="cuda")),
        lambda: B.beam_select(torch.zeros(2, 3, 9, device="cuda"), torch.zeros(2, 3, device="cuda"), length_penalty=1.0),
        lambda: B.beam_select(torch.zeros(2, 33, 9, device="cuda"), torch.zeros(2, 33, device="cuda")),
        lambda: B.beam_reorder(torch.zeros(1, 2, **i32), new, t, t, k, k.clone()),
        lambda: B.beam_reorder(torch.zeros(1, 2, **i32), new, t, torch.zeros_like(t), k, k.clone(), states=[(mass, mass)]),
        lambda: B.beam_reorder(torch.zeros(1, 2, **i32), new, t, torch.zeros_like(t), k, k.clone(), states=[(mass[:1], mass[:1].clone())]),
        lambda: B.beam_reorder(torch.zeros(1, 2, **i32), new, t, torch.zeros_like(t), k, k.clone(), states=[(mass, mass.clone())] * 5),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, B.PaError)):
            call()
            pytest.fail(f"call {i} was accepted")


def test_calls_on_two_streams_at_once():
    """The operators keep nothing between calls and share no workspace: two streams running them side by
    side give what one gives."""
    def work(seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        p = synth.make_problem(60 + seed, num_seqs=3, context_lens=[900, 2000, 4000], q_lens=[1, 2, 1], page_size=32)
        d = dv.to_device(p)
        lse = dev(O.decode(p)[1].astype(np.float32))
        logits = torch.randn(3, 4, 40000, generator=g, device="cuda")
        scores = torch.randn(3, 4, generator=g, device="cuda")
        parents = torch.randint(0, 3, (1, 3), generator=g, device="cuda", dtype=torch.int32)
        lens = torch.full((3,), 500, dtype=torch.int32, device="cuda")

        def run():
            c = [d[k].clone() for k in ("k_cache", "v_cache", "k_scale", "v_scale")]
            m = B.attn_mass(d["q"], c[0], d["block_table"], d["context_lens"], d["cu_seqlens_q"], lse,
                            torch.zeros(3, 1, 4000, device="cuda"), max_q_len=2, sm_scale=p.sm_scale, decay=0.0, k_scale=c[2])
            keep, new = B.evict_select(m, d["context_lens"], budget=700, first=4, recent=64)
            B.kv_compact(keep, new, d["block_table"], c[0], c[1], k_scale=c[2], v_scale=c[3], mass=m)
            table = torch.empty_like(d["block_table"])
            B.beam_reorder(parents, lens, d["block_table"], table, c[0], c[1], k_scale=c[2], v_scale=c[3])
            t = B.beam_select(logits, scores)
            return [m[:, :, :700].clone(), keep, new, table, *c, *t[:3]]
        return run

    runs = [work(1), work(2)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(runs[i]())
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        for g in many:
            for a, b in zip(w, g):
                assert torch.equal(a, b)


def test_empty_batches_enqueue_nothing():
    """No requests, or none with rows in this step: the outputs exist, and nothing is touched."""
    k = torch.full((4, 1, 16, 128), 7, dtype=torch.uint8, device="cuda")
    v = k.clone()
    scale = torch.ones(4, 1, 16, device="cuda")

    def ints(*shape):
        return torch.zeros(shape, dtype=torch.int32, device="cuda")

    def floats(*shape):
        return torch.zeros(shape, device="cuda")

    q = torch.zeros(0, 16, 128, dtype=torch.bfloat16, device="cuda")
    none = floats(0, 1, 64)
    assert B.attn_mass(q, k, ints(0, 4), ints(0), ints(1), floats(0, 16), none, max_q_len=1, k_scale=scale).shape == (0, 1, 64)
    idle = torch.full((2, 1, 64), 3.0, device="cuda")
    B.attn_mass(q, k, ints(2, 4), ints(2), ints(3), floats(0, 16), idle, max_q_len=1, k_scale=scale, decay=0.5)
    assert torch.all(idle == 3.0)
    keep, new = B.evict_select(none, ints(0), budget=8)
    assert keep.shape == (0, 1, 8) and new.shape == (0,)
    B.kv_compact(keep, new, ints(0, 4), k, v, k_scale=scale, v_scale=scale)
    B.kv_compact(keep, new, ints(0, 4), k, v, dst_block_table=ints(0, 2), mass=none, mass_out=floats(0, 1, 8))
    out = B.beam_select(floats(0, 4, 1000), floats(0, 4), eos=2, finished=torch.zeros(0, 4, dtype=torch.uint8, device="cuda"),
                        lengths=ints(0, 4), length_penalty=0.6)
    assert [tuple(x.shape) for x in out] == [(0, 4)] * 5
    B.beam_reorder(ints(0, 4), ints(0), ints(0, 4), ints(0, 4), k, v, k_scale=scale, v_scale=scale,
                   states=[(floats(0, 32), floats(0, 32))])
    torch.cuda.synchronize()
    assert torch.all(k == 7) and torch.all(v == 7)
