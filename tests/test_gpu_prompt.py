"""pa_prompt_attn against its definition in 64 bits (needs a GPU).

Bounds.  With w the exact weights of a row (sum 1), x its scores and A = sum_i w_i |v_i|:
 - a score is 128 products of bf16 (exact in fp32) added in fp32 by the tensor core, eight instructions of 16 terms each of
   which may cut the sum to a unit of its last place: within e = 2^-18 of the sum of the terms' magnitudes; the scale, the
   exponent's subtraction and 2^x add 2^-21 of the score's size and 2^-21: d = 2 e terms + 2^-21 (2 + |x|) on a weight, relative;
 - the weights of the second product are rounded to bf16 (2^-8 at most), their sum is not; sums of n terms in fp32 over
   n / 16 instructions: n 2^-26;
so an fp32 output is within (2^-8 + 2 d + n 2^-26) A of the exact one, a bf16 output half a step (2^-8) further, and the lse
within d + 2^-22 (|lse| + 2)."""
import math

import numpy as np
import pytest
import torch

from cache_util import word
from oracle import prompt_ops as C
from paged_fp8_kv_04_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _f64(x):
    return x.double().cpu().numpy()


def _cu(lens, first=0):
    return np.r_[first, first + np.cumsum(lens)].astype(np.int32)


def _inputs(g, T, heads, group, scale=1.0):
    mk = lambda h: torch.randn(T, h, 128, generator=g, device="cuda")  # noqa: E731
    return (mk(heads * group) * scale).bfloat16(), mk(heads).bfloat16(), mk(heads).bfloat16()


SENTINEL = 1234.0


def _call(q, k, v, cu, sm=None, f32=False, flags=0):
    st = word()
    out = torch.full(q.shape, SENTINEL, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], SENTINEL, device="cuda")
    o, l = B.prompt_attn(q, k, v, torch.from_numpy(np.asarray(cu, np.int32)).cuda(), sm_scale=sm, out=out, lse=lse, status=st)
    assert o is out and l is lse
    torch.cuda.synchronize()
    assert int(st) == flags, hex(int(st))
    return out, lse


def _compare(out, lse, q, k, v, cu, sm=None, f32=False):
    sm = 1.0 / math.sqrt(128.0) if sm is None else float(np.float32(sm))
    ref, rl, mag, terms = C.prompt_attn(_f64(q), _f64(k), _f64(v), cu, sm)
    rows = np.zeros(q.shape[0], bool)
    n = np.zeros(q.shape[0])
    for a, b in zip(cu[:-1], cu[1:]):
        rows[a:b] = True
        n[a:b] = np.arange(1, b - a + 1)
    d = 2 * 2.0**-18 * terms + 2.0**-21 * (2 + terms)
    tol = (2.0**-8 + 2 * d + n[:, None] * 2.0**-26)[..., None] * mag
    if not f32:
        tol = tol + 2.0**-8 * (np.abs(ref) + tol)
    err = np.abs(_f64(out) - ref)[rows]
    assert np.all(err <= tol[rows]), (float((err / tol[rows]).max()), np.argwhere(~(err <= tol[rows]))[:3])
    ltol = d + 2.0**-22 * (np.abs(rl) + 2)
    lerr = np.abs(_f64(lse) - rl)[rows]
    assert np.all(lerr <= ltol[rows]), float((lerr / ltol[rows]).max())
    assert bool((out[torch.from_numpy(~rows).cuda()] == SENTINEL).all()) and bool((lse[torch.from_numpy(~rows).cuda()] == SENTINEL).all())


@pytest.mark.parametrize("heads,group", [(1, 16), (1, 1), (2, 4), (4, 2), (1, 3), (2, 5), (1, 7), (1, 8), (3, 12), (1, 33), (1, 64), (1, 10)])
@pytest.mark.parametrize("lens", [[1], [2], [8], [9], [16], [17], [127, 1], [128], [129], [300, 0, 7, 64], [0, 0], [257, 383], [640, 1, 513], [900]])
def test_prompt(lens, heads, group):
    g = torch.Generator(device="cuda").manual_seed(sum(lens) * 100 + group)
    cu = _cu(lens)
    q, k, v = _inputs(g, max(int(cu[-1]), 1), heads, group)
    _compare(*_call(q, k, v, cu), q, k, v, cu)


@pytest.mark.parametrize("lens,heads,group", [([2048], 1, 16), ([1, 1300, 2049, 77], 2, 3), ([4099], 1, 2), ([3000, 5], 1, 6)])
def test_prompt_of_many_blocks(lens, heads, group):
    g = torch.Generator(device="cuda").manual_seed(len(lens))
    cu = _cu(lens, 5)
    q, k, v = _inputs(g, int(cu[-1]) + 70, heads, group)
    _compare(*_call(q, k, v, cu), q, k, v, cu)
    _compare(*_call(q, k, v, cu, f32=True), q, k, v, cu, f32=True)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("count,dead,n,heads,group", [(1, 1, 2, 1, 16), (1, 200, 700, 1, 16), (2, 128, 390, 1, 3), (1, 300, 1100, 2, 1), (90, 200, 400, 2, 16), (90, 130, 260, 4, 7)])
def test_prompt_scores_of_minus_infinity(count, dead, n, heads, group, f32):
    """The first keys of each sequence score -inf: weights of 0 for a row that attends others too, which is then as if they were
    not there; no row's else (0 / 0, and an lse of -inf)."""
    g = torch.Generator(device="cuda").manual_seed(n)
    cu = _cu([n] * count)
    q, k, v = _inputs(g, n * count, heads, group)
    q[..., 0] = q[..., 0].abs() + 0.5
    k.view(count, n, heads, 128)[:, :dead, :, 0] = -math.inf
    out, lse = _call(q, k, v, cu, f32=f32)
    for a in cu[:-1][:: max(1, count // 3)].tolist():
        assert bool(out[a : a + dead].isnan().all()) and bool((lse[a : a + dead] == -math.inf).all())
        at = slice(a + dead, a + n)
        _compare(out[at], lse[at], q[at], k[at], v[at], _cu([n - dead]), f32=f32)


@pytest.mark.parametrize("sm", [0.001, 0.5, 2.0])
def test_prompt_scales(sm):
    g = torch.Generator(device="cuda").manual_seed(11)
    cu = _cu([333, 130])
    q, k, v = _inputs(g, int(cu[-1]), 1, 5)
    _compare(*_call(q, k, v, cu, sm), q, k, v, cu, sm)


@pytest.mark.parametrize("group", [16, 3])
@pytest.mark.parametrize("kind", ["rising", "falling", "steps", "spike"])
def test_prompt_running_maximum(kind, group):
    """Scores that grow (or fall) by many powers of two from block to block, for some rows more than for others."""
    g = torch.Generator(device="cuda").manual_seed(12)
    n = 1100
    q, k, v = _inputs(g, n, 1, group)
    i = torch.arange(n, device="cuda", dtype=torch.float32)
    along = torch.randn(128, generator=g, device="cuda")
    along /= along.norm()
    size = {"rising": i / 4, "falling": (n - i) / 4, "steps": (i // 128 % 3) * 60, "spike": (i == 700) * 300.0}[kind]
    k = (k.float() * 0.2 + size[:, None, None] * along).bfloat16()
    q = (q.float() * 0.2 + (torch.rand(n, group, 1, generator=g, device="cuda") * 12) * along).bfloat16()
    cu = _cu([n])
    _compare(*_call(q, k, v, cu), q, k, v, cu)


def test_prompt_what_a_row_does_not_attend_has_no_effect():
    """Infinities and NaN in later tokens, other sequences and rows of no sequence: every other row bit for bit as before."""
    g = torch.Generator(device="cuda").manual_seed(13)
    for lens, heads, group in (([200, 131, 300], 2, 4), ([45, 700, 3], 1, 16), ([390, 390], 1, 3), ([500, 500], 1, 1)):
        cu = _cu(lens, 9)
        T = int(cu[-1]) + 140
        q, k, v = _inputs(g, T, heads, group)
        want, wl = _call(q, k, v, cu)
        for bad in (math.inf, -math.inf, math.nan):
            k2, v2, q2 = k.clone(), v.clone(), q.clone()
            a, b = int(cu[1]), int(cu[2])
            at = a + (b - a) * 2 // 3
            for x in (k2, v2):
                x[:9], x[int(cu[-1]):] = bad, bad
                x[at:b, :, ::3] = bad
            q2[:9], q2[int(cu[-1]):], q2[at:b] = bad, bad, bad
            out, lse = _call(q2, k2, v2, cu)
            same = torch.ones(T, dtype=torch.bool, device="cuda")
            same[at:b] = False
            assert torch.equal(out[same], want[same]) and torch.equal(lse[same], wl[same]), (lens, bad)


def test_prompt_infinities_that_a_row_attends():
    """An infinite or NaN value reaches exactly the rows and elements that attend it."""
    g = torch.Generator(device="cuda").manual_seed(14)
    for lens, group in (([180], 16), ([700], 4), ([300], 1)):
        cu = _cu(lens)
        q, k, v = _inputs(g, lens[0], 1, group)
        want, wl = _call(q, k, v, cu)
        n = lens[0]
        spots = [(n // 2, 5, math.inf), (n // 2 + 3, 77, -math.inf), (n - 1, 9, math.nan), (n // 2 + 7, 5, -math.inf), (1, 127, math.inf)]
        v2 = v.clone()
        for i, d, x in spots:
            v2[i, 0, d] = x
        out, lse = _call(q, k, v2, cu)
        assert torch.equal(lse, wl)
        clean = torch.ones_like(out, dtype=torch.bool)
        for i, d, x in spots:
            clean[i:, :, d] = False
        assert torch.equal(out[clean], want[clean])
        for d in (5, 77, 127):
            i, x = next((i, x) for i, e, x in spots if e == d)
            end = n // 2 + 7 if d == 5 else n
            # (a weight below what bf16 holds makes 0 * inf of it in a block that no row is cut in: not the case here)
            assert bool((out[i:end, :, d] == x).all()), (lens, d)
        assert bool(out[n // 2 + 7:, :, 5].isnan().all()) and bool(out[n - 1:, :, 9].isnan().all())


def test_prompt_bad_sequences_are_left_out():
    g = torch.Generator(device="cuda").manual_seed(15)
    q, k, v = _inputs(g, 300, 1, 4)
    cu = np.array([0, 100, 90, 200, 301], np.int32)   # the second runs backwards, the last past the rows
    out, lse = _call(q, k, v, cu, flags=0x4)
    for a, b in ((0, 100), (90, 200)):
        # rows 90 .. 99 belong to two: whichever came last
        s = slice(100, 200) if a else slice(0, 90)
        o, l = _call(q, k, v, [a, b])
        assert torch.equal(out[s], o[s]) and torch.equal(lse[s], l[s])
    assert bool((out[200:] == SENTINEL).all())
    out, _ = _call(q, k, v, [-5, 20, 40], flags=0x4)
    assert bool((out[:20] == SENTINEL).all()) and not bool((out[20:40] == SENTINEL).any())


def test_prompt_many_sequences():
    rng = np.random.default_rng(16)
    g = torch.Generator(device="cuda").manual_seed(16)
    for count, hi in ((384, 40), (385, 30), (4096, 9), (1000, 3)):
        cu = _cu(rng.integers(0, hi + 1, size=count), 3)
        q, k, v = _inputs(g, int(cu[-1]) + 8, 2, 2)
        _compare(*_call(q, k, v, cu), q, k, v, cu)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("count,lo,hi,heads,group", [(20, 0, 420, 4, 8), (32, 100, 300, 2, 16), (33, 1, 350, 3, 8), (128, 1, 90, 1, 33), (129, 0, 150, 2, 12), (600, 1, 40, 1, 16)])
def test_prompt_many_units(count, lo, hi, heads, group, f32):
    """More units than CTAs run at once, so that they come one after the other: ragged ends, empty sequences, odd groups."""
    rng = np.random.default_rng(count + f32)
    g = torch.Generator(device="cuda").manual_seed(count)
    cu = _cu(rng.integers(lo, hi + 1, size=count), 4)
    q, k, v = _inputs(g, int(cu[-1]) + 40, heads, group)
    _compare(*_call(q, k, v, cu, f32=f32), q, k, v, cu, f32=f32)


def test_prompt_many_units_and_what_they_do_not_attend():
    """Infinities and NaN of one sequence, of later tokens and of no sequence, among units that follow one another in a CTA; and where
    rows attend them."""
    rng = np.random.default_rng(21)
    g = torch.Generator(device="cuda").manual_seed(21)
    cu = _cu(rng.integers(60, 500, size=24), 7)
    T = int(cu[-1]) + 60
    q, k, v = _inputs(g, T, 4, 8)
    want, wl = _call(q, k, v, cu)
    for bad in (math.inf, math.nan):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        same = torch.ones(T, dtype=torch.bool, device="cuda")
        for s in range(0, 24, 2):
            a, b = int(cu[s]), int(cu[s + 1])
            at = a + (b - a) // 2
            for x in (k2, v2):
                x[at:b, :, 1::5] = bad
            q2[at:b], same[at:b] = bad, False
        for x in (q2, k2, v2):
            x[:7], x[int(cu[-1]):] = bad, bad
        out, lse = _call(q2, k2, v2, cu)
        assert torch.equal(out[same], want[same]) and torch.equal(lse[same], wl[same])
    v2, clean = v.clone(), torch.ones_like(want, dtype=torch.bool)
    for s in range(24):
        a, b = int(cu[s]), int(cu[s + 1])
        at = b - 1 - s
        v2[at, 3, 2 * s] = math.inf
        clean[at:b, 24:, 2 * s] = False
    out, lse = _call(q, k, v2, cu)
    assert torch.equal(out[clean], want[clean]) and torch.equal(lse, wl) and bool((out[~clean] == math.inf).all())


def test_prompt_many_units_running_maximum():
    g = torch.Generator(device="cuda").manual_seed(22)
    cu = _cu([700] * 12)
    n = int(cu[-1])
    q, k, v = _inputs(g, n, 2, 16)
    along = torch.nn.functional.normalize(torch.randn(128, generator=g, device="cuda"), dim=0)
    size = (torch.arange(n, device="cuda") % 700 // 100) * 40.0
    k = (k.float() * 0.2 + size[:, None, None] * along).bfloat16()
    q = (q.float() * 0.2 + (torch.rand(n, 32, 1, generator=g, device="cuda") * 12) * along).bfloat16()
    _compare(*_call(q, k, v, cu), q, k, v, cu)


def test_prompt_many_units_captured_with_new_lengths():
    """One graph, whose lengths change between replays from many units to few."""
    g = torch.Generator(device="cuda").manual_seed(23)
    q, k, v = _inputs(g, 9000, 2, 16)
    cu = torch.zeros(41, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        B.prompt_attn(q, k, v, cu, out=out, lse=lse)
        B.prompt_attn(q, k, v, cu, out=out, lse=lse)
    for lens in ([200] * 40, [9000] + [0] * 39, [0] * 40, [1] * 40, list(range(100, 300, 5)), [0] * 39 + [300]):
        c = _cu(lens)
        cu.copy_(torch.from_numpy(c))
        out.fill_(SENTINEL)
        lse.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        want, wl = _call(q, k, v, c)
        assert torch.equal(out, want) and torch.equal(lse, wl), lens[:3]
        if sum(lens) < 3000:
            _compare(out, lse, q, k, v, c)


@pytest.mark.parametrize("heads,group", [(2, 16), (3, 8), (1, 33)])
def test_prompt_units_that_are_split_and_in_turn(heads, group):
    """Buffers for many sequences that hold few tokens: CTAs take units in turn, and the longest are split.  The same as with
    buffers of their size, where every unit has a CTA of its own."""
    g = torch.Generator(device="cuda").manual_seed(24)
    q, k, v = _inputs(g, 9000, heads, group)
    tokens = 128 // group * 2
    for units in (100, 153, 170, 200, 250, 290):
        n = units * tokens // heads
        for lens in ([n], [n // 2, n - n // 2 - 9, 9], [n // 3, 0, n // 3, n // 4]):
            cu = _cu(lens + [0] * (32 - len(lens)))
            out, lse = _call(q, k, v, cu)
            t = int(cu[-1])
            small, sl = _call(q[:t], k[:t], v[:t], _cu(lens))
            assert torch.equal(out[:t], small) and torch.equal(lse[:t], sl), (units, lens)
            assert bool((out[t:] == SENTINEL).all())
            if units == 170:
                _compare(out, lse, q, k, v, cu)


@pytest.mark.parametrize("heads,group,lens", [(1, 16, [2432]), (1, 16, [4096]), (3, 8, [900, 1700]), (2, 16, [33, 1500])])
def test_prompt_split_units_before_others_are_the_same_every_time(heads, group, lens):
    """CTAs that have a split unit first and go on with others: the two slots, which join that unit's columns, go on at their own pace.
    Equal bits however often."""
    g = torch.Generator(device="cuda").manual_seed(27)
    cu = _cu(lens + [0] * 30)
    q, k, v = _inputs(g, max(int(cu[-1]), 160 * 2 * (128 // group) // heads), heads, group)
    want, wl = _call(q, k, v, cu)
    _compare(want, wl, q, k, v, cu)
    out, lse = torch.empty_like(q), torch.empty_like(wl)
    dcu, st = torch.from_numpy(cu).cuda(), word()
    wrong = torch.zeros(1, dtype=torch.int64, device="cuda")
    n = int(cu[-1])
    for _ in range(200):
        B.prompt_attn(q, k, v, dcu, out=out, lse=lse, status=st)
        wrong += (out[:n] != want[:n]).sum() + (lse[:n] != wl[:n]).sum()
    assert int(wrong) == 0 and int(st) == 0


def test_prompt_infinities_in_fp32_outputs():
    g = torch.Generator(device="cuda").manual_seed(25)
    for lens, heads, group in (([300, 41], 1, 16), ([90] * 30, 4, 8)):
        cu = _cu(lens)
        q, k, v = _inputs(g, int(cu[-1]), heads, group)
        want, wl = _call(q, k, v, cu, f32=True)
        v2, clean = v.clone(), torch.ones_like(want, dtype=torch.bool)
        for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
            v2[b - 20, 0, 100 - s] = -math.inf
            clean[b - 20:b, :group, 100 - s] = False
        out, lse = _call(q, k, v2, cu, f32=True)
        assert torch.equal(out[clean], want[clean]) and torch.equal(lse, wl) and bool((out[~clean] == -math.inf).all())


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("count", [3, 200])
@pytest.mark.parametrize("group,n,first,at", [(1, 256, 128, 131), (3, 168, 128, 150), (5, 150, 128, 128)])
def test_prompt_infinities_in_the_later_tiles_block_alone(group, n, first, at, count, f32):
    """Of the two tiles that a CTA has at a sequence's end the later one alone reads the block that begins at token `first`, and only
    that block holds what is not finite: rows before it are bit for bit as without it, those from there on attend it.  A CTA for each unit,
    and CTAs that take them in turn; several times."""
    g = torch.Generator(device="cuda").manual_seed(26)
    cu = _cu([n] * count)
    q, k, v = _inputs(g, n * count, 1, group)
    want, wl = _call(q, k, v, cu, f32=f32)
    v2 = v.clone().view(count, n, 128)
    v2[:, at, 7], v2[:, n - 2, 70] = math.inf, math.nan
    assert bool(v2[:, :first].isfinite().all())
    clean = torch.ones_like(want, dtype=torch.bool).view(count, n, group, 128)
    clean[:, at:, :, 7], clean[:, n - 2:, :, 70] = False, False
    clean = clean.view(want.shape)
    for _ in range(5):
        out, lse = _call(q, k, v2.view(v.shape), cu, f32=f32)
        assert torch.equal(out[clean], want[clean]) and torch.equal(lse, wl)
        assert bool((out.view(count, n, group, 128)[:, at:, :, 7] == math.inf).all())
        assert bool(out.view(count, n, group, 128)[:, n - 2:, :, 70].isnan().all())


def test_prompt_is_the_same_packed_or_alone_dense_or_a_view():
    g = torch.Generator(device="cuda").manual_seed(17)
    lens, heads, group = [333, 128, 1, 700], 2, 6
    cu = _cu(lens)
    T, hq = int(cu[-1]), heads * group
    buf = torch.randn(T, (hq + 2 * heads) * 128 + 24, generator=g, device="cuda").bfloat16()
    q, k, v = (x.unflatten(1, (-1, 128)) for x in buf[:, 16:-8].split([hq * 128, heads * 128, heads * 128], 1))
    out, lse = _call(q, k, v, cu)
    dense, dl = _call(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    assert torch.equal(out, dense) and torch.equal(lse, dl)
    for a, b in zip(cu[:-1], cu[1:]):
        one, ol = _call(q[a:b], k[a:b], v[a:b], [0, b - a])
        assert torch.equal(one, out[a:b]) and torch.equal(ol, lse[a:b])
    again, al = _call(q, k, v, cu)
    assert torch.equal(again, out) and torch.equal(al, lse)


def test_prompt_captured_and_on_two_streams():
    g = torch.Generator(device="cuda").manual_seed(18)
    calls = []
    for lens, heads, group in (([900, 30], 1, 16), ([64, 1200], 2, 4)):
        cu = _cu(lens)
        q, k, v = _inputs(g, int(cu[-1]), heads, group)
        calls.append((q, k, v, torch.from_numpy(cu).cuda(), _call(q, k, v, cu)))
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in calls]
    for (q, k, v, cu, _), s in zip(calls, streams):
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(3):
                B.prompt_attn(q, k, v, cu, out=out, lse=lse)
        graphs.append(graph)
        outs.append((out, lse))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (out, lse), (*_, (want, wl)) in zip(outs, calls):
        assert torch.equal(out, want) and torch.equal(lse, wl)
    # new lengths for the captured call, as a padded batch has them
    q, k, v, cu, _ = calls[0]
    cu.copy_(torch.tensor([0, 17, 400], dtype=torch.int32))
    outs[0][0].fill_(SENTINEL)
    graphs[0].replay()
    torch.cuda.synchronize()
    want, _ = _call(q, k, v, [0, 17, 400])
    assert torch.equal(outs[0][0], want)


def test_prompt_long():
    """Sampled rows of a prompt longer than any other test's, and rows far behind in a wide buffer."""
    g = torch.Generator(device="cuda").manual_seed(19)
    n = 20011
    q, k, v = _inputs(g, n, 1, 16)
    out, lse = _call(q, k, v, [0, n])
    rows = torch.tensor([0, 1, 127, 128, 8191, 12345, n - 2, n - 1], device="cuda")
    for t in rows.tolist():
        x = (q[t].double() @ k[:t + 1, 0].double().T) / math.sqrt(128.0)
        z = torch.logsumexp(x, -1)
        w = torch.exp(x - z[:, None])
        ref, mag = w @ v[:t + 1, 0].double(), w @ v[:t + 1, 0].double().abs()
        terms = ((q[t].double().abs() @ k[:t + 1, 0].double().abs().T) / math.sqrt(128.0)).amax(-1)
        d = 2 * 2.0**-18 * terms + 2.0**-21 * (2 + terms)
        tol = (2.0**-8 + 2 * d + t * 2.0**-26)[:, None] * mag
        tol = tol + 2.0**-8 * (ref.abs() + tol)
        assert bool(((out[t].double() - ref).abs() <= tol).all())
        assert bool(((lse[t].double() - z).abs() <= d + 2.0**-22 * (z.abs() + 2)).all())


def test_prompt_offsets_past_32_bits():
    """Rows whose elements lie beyond 2^31 of the buffers' start (8.6 GB a tensor)."""
    n, wide, g = 2**17 + 300, 2**14 + 512, torch.Generator(device="cuda").manual_seed(20)
    buf = torch.empty(n, wide, dtype=torch.bfloat16, device="cuda")
    last = slice(n - 260, n)
    buf[last, :768].normal_(generator=g)
    q, k, v = (buf[:, a:b].unflatten(1, (-1, 128)) for a, b in ((0, 512), (512, 640), (640, 768)))
    out = torch.empty(n, 4, 128, dtype=torch.bfloat16, device="cuda")
    B.prompt_attn(q, k, v, torch.tensor([n - 260, n], dtype=torch.int32, device="cuda"), out=out)
    want, _ = B.prompt_attn(*(x[last].contiguous() for x in (q, k, v)), torch.tensor([0, 260], dtype=torch.int32, device="cuda"))
    assert torch.equal(out[last], want)


def test_prompt_outputs_and_refusals():
    q, k = torch.zeros(8, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 2, 128, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    out, lse = B.prompt_attn(q, k, k, cu)
    assert out.dtype == torch.bfloat16 and out.shape == q.shape and lse is None
    out, lse = B.prompt_attn(q, k, k, cu, out_dtype="f32", want_lse=True)
    assert out.dtype == torch.float32 and lse.shape == (8, 4)
    out, lse = B.prompt_attn(q[:0], k[:0], k[:0], torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 128)
    for bad in (lambda: B.prompt_attn(q.half(), k, k, cu), lambda: B.prompt_attn(q, k.float(), k, cu), lambda: B.prompt_attn(q, k, k, cu.long()),
                lambda: B.prompt_attn(q, k, k, cu, out=torch.zeros_like(q).half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: B.prompt_attn(q[:, :3].contiguous(), k, k, cu), lambda: B.prompt_attn(q, k, k[:7], cu), lambda: B.prompt_attn(q, k, k[:, :1], cu),
                lambda: B.prompt_attn(q[0], k, k, cu), lambda: B.prompt_attn(q, k, k, cu[:0]), lambda: B.prompt_attn(q, k, k, cu, lse=torch.zeros(8, 3, device="cuda")),
                lambda: B.prompt_attn(q, k, k, cu.cpu()), lambda: B.prompt_attn(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, cu)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: B.prompt_attn(q, k, k, cu, out=q), lambda: B.prompt_attn(q, k, k, cu, sm_scale=-1.0),
                lambda: B.prompt_attn(*(x[..., :64].contiguous() for x in (q, k, k)), cu)):
        with pytest.raises(B.PaError):
            bad()
