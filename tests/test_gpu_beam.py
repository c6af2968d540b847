"""pa_beam_select and pa_beam_reorder against their definitions (needs a GPU).  Tokens, parents,
tables and bytes are equal; scores are rounded to fp32 once, after a log-sum-exp whose exponentials
are off by 2^-22 each and whose arguments by 2^-23 of their size."""
import numpy as np
import pytest
import torch

from cache_util import dev, host, same, word
from oracle import cache_ops as C
from paged_fp8_kv_04_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _logits(rng, N, W, V, dt, scale=3.0):
    x = torch.from_numpy((rng.standard_normal((N, W, V)) * scale).astype(np.float32)).to(dt)
    return x, x.double().numpy()


def _check(x, xd, scores, rtol_extra=0.0, **kw):
    N, W, V = xd.shape
    t = {k: dev(v) if isinstance(v, np.ndarray) else v for k, v in kw.items()}
    got = B.beam_select(x if x.is_cuda else x.cuda(), dev(scores), eos=t.get("eos", -1), finished=t.get("finished"),
                        lengths=t.get("lengths"), length_penalty=t.get("penalty", 0.0))
    want = C.beam_select(xd, scores, kw.get("eos", -1), kw.get("finished"), kw.get("lengths"), kw.get("penalty", 0.0))
    assert np.array_equal(host(got[0]), want[0]) and np.array_equal(host(got[1]), want[1])
    s, ws = host(got[2]).astype(np.float64), want[2]
    fin = np.isfinite(ws)
    assert np.array_equal(fin, np.isfinite(s)) and np.array_equal(s[~fin], ws[~fin])
    # the log-sum-exp: 2^-22 per exponential and 2^-23 of arguments up to their range, fp32 partial sums
    # of at most 2^12 terms (2^-24 each, at worst 2^-12 relative; the rows here stay below 2^-18); one rounding
    span = float(np.nanmax(np.where(np.isfinite(xd), np.abs(xd), 0))) * 2 + 1
    tol = 2.0 ** -18 + 2.0 ** -23 * span + 2.0 ** -24 * np.abs(ws[fin])
    assert np.all(np.abs(s[fin] - ws[fin]) <= tol), np.abs(s[fin] - ws[fin]).max()
    if kw.get("finished") is not None:
        assert np.array_equal(host(got[3]), want[3])
    if kw.get("lengths") is not None:
        assert np.array_equal(host(got[4]), want[4])
    return got


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [1, 2, 3, 4, 8, 17, 32])
@pytest.mark.parametrize("V", [1, 5, 33, 1000, 4097])
def test_small_vocabularies(dt, W, V):
    rng = np.random.default_rng(W * 10000 + V)
    x, xd = _logits(rng, 3, W, V, dt)
    _check(x, xd, (-5 + rng.standard_normal((3, W))).astype(np.float32))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,W,V", [(1, 4, 32001), (2, 8, 131072), (5, 5, 50001), (1, 1, 200000), (40, 2, 8191), (1, 32, 65537)])
def test_large_vocabularies(dt, N, W, V):
    rng = np.random.default_rng(V)
    x, xd = _logits(rng, N, W, V, dt)
    _check(x, xd, (-20 + 3 * rng.standard_normal((N, W))).astype(np.float32))


@pytest.mark.parametrize("penalty", [0.0, 0.6, 1.0, 2.5])
def test_finished_beams_and_length_penalty(penalty):
    rng = np.random.default_rng(7)
    x, xd = _logits(rng, 20, 6, 777, torch.float32)
    fin = (rng.random((20, 6)) < 0.4).astype(np.uint8)
    fin[3] = 1                                          # all have ended
    _check(x, xd, (-9 + 4 * rng.standard_normal((20, 6))).astype(np.float32), eos=5, finished=fin,
           lengths=rng.integers(0, 60, size=(20, 6)).astype(np.int32), penalty=penalty)


def test_the_end_token_ends_a_beam():
    x = torch.zeros(1, 2, 9)
    x[0, :, 4] = 9.0
    got = _check(x, x.double().numpy(), np.array([[-1.0, -1.5]], np.float32), eos=4, finished=np.zeros((1, 2), np.uint8),
                 lengths=np.array([[3, 8]], np.int32), penalty=1.0)
    assert host(got[3]).tolist() == [[1, 1]] and host(got[0]).tolist() == [[4, 4]]


@pytest.mark.parametrize("V", [3, 40, 5000])
def test_first_step_from_one_beam(V):
    """Beams that do not exist yet: their candidates come last, lowest beam and token first."""
    rng = np.random.default_rng(8)
    x, xd = _logits(rng, 4, 8, V, torch.bfloat16)
    s = np.full((4, 8), -np.inf, np.float32)
    s[:, 0] = 0
    _check(x, xd, s)
    s[2, 0] = -np.inf                                   # no beam at all
    _check(x, xd, s)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [64, 6000, 70000])
def test_ties_go_to_the_lowest_beam_and_token(dt, V):
    for build in (lambda x: x.zero_(), lambda x: x.copy_((torch.arange(V) % 3 == 1).float().expand_as(x)),
                  lambda x: x.copy_(torch.linspace(-4, 4, V).bfloat16().float().expand_as(x)),
                  lambda x: x.copy_(torch.linspace(4, -4, V).bfloat16().float().expand_as(x))):
        x = torch.empty(2, 5, V, dtype=dt)
        build(x)
        # powers of two apart, so that equal totals are equal in every evaluation
        _check(x, x.double().numpy(), np.array([[-2, -2, -2, -2, -2], [-64, -1, -1, -64, -1]], np.float32))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [12, 17, 32])
@pytest.mark.parametrize("V", [300, 6000, 40000])
def test_wide_beams_over_runs_of_equal_and_rising_logits(dt, W, V):
    """More elements reach the bound than are put in order at once."""
    scores = np.full((2, W), -2.0, np.float32)
    scores[1] = np.where(np.arange(W) % 3 == 1, -1.0, -64.0)
    for row in (torch.zeros(V), torch.linspace(-4, 4, V).bfloat16().float(), torch.linspace(4, -4, V).bfloat16().float(),
                (torch.arange(V) // 8 % 40).float() / 8):
        x = row.expand(2, W, V).to(dt).contiguous()
        _check(x, x.double().numpy(), scores)


def test_masked_infinite_and_nan_rows():
    rng = np.random.default_rng(9)
    x, _ = _logits(rng, 7, 3, 500, torch.float32)
    x[0, 1] = -np.inf                                   # a row with nothing allowed
    x[1, :, 7:] = -np.inf                               # few tokens allowed
    x[2, 0, 3] = np.nan
    x[3, 2, 5] = np.inf
    x[4] = -np.inf
    x[5, :, :] = torch.finfo(torch.float32).min         # the type's lowest value everywhere
    x[6, :, 2:] = torch.finfo(torch.float32).min
    with np.errstate(all="ignore"):
        _check(x, x.double().numpy(), (-3 + rng.standard_normal((7, 3))).astype(np.float32))


def test_strided_and_misaligned_rows():
    rng = np.random.default_rng(10)
    big = torch.from_numpy(rng.standard_normal((3, 4, 1030)).astype(np.float32))
    for dt in (torch.bfloat16, torch.float32):
        b = big.to(dt).cuda()
        for lo, V in ((0, 1000), (1, 1021), (3, 1027), (7, 511)):
            x = b[..., lo:lo + V]
            _check(x, x.double().cpu().numpy(), (-3 + rng.standard_normal((3, 4))).astype(np.float32))
            y = x.reshape(3, 4, V) if V == 1030 else b.view(12, 1030)[:, lo:lo + V]
            got = B.beam_select(y, dev(np.zeros((3, 4), np.float32)))
            assert torch.equal(got[0], B.beam_select(x, dev(np.zeros((3, 4), np.float32)))[0])


def test_in_place_outputs_and_graphs():
    rng = np.random.default_rng(11)
    x, xd = _logits(rng, 4, 4, 3001, torch.bfloat16)
    s0 = (-5 + rng.standard_normal((4, 4))).astype(np.float32)
    f0, l0 = (rng.random((4, 4)) < 0.3).astype(np.uint8), rng.integers(1, 9, size=(4, 4)).astype(np.int32)
    want = C.beam_select(xd, s0, 1, f0, l0, 0.5)
    xs, s, f, ln = x.cuda(), dev(s0), dev(f0), dev(l0)
    call = lambda: B.beam_select(xs, s, eos=1, finished=f, lengths=ln, length_penalty=0.5, scores_out=s, finished_out=f,  # noqa: E731
                                 lengths_out=ln)
    got = call()
    assert np.array_equal(host(got[0]), want[0]) and np.array_equal(host(f), want[3]) and np.array_equal(host(ln), want[4])
    second = call()
    torch.cuda.synchronize()
    a = [host(t).copy() for t in (second[0], second[1], s, f, ln)]
    for t, v in ((s, s0), (f, f0), (ln, l0)):
        t.copy_(dev(v))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    for t, v in ((s, s0), (f, f0), (ln, l0)):
        t.copy_(dev(v))
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for u, v in zip((got[0], got[1], s, f, ln), a):
        assert np.array_equal(host(u), v)


# -------------------------------------------------------------------------- reordering

def _problem(rng, N, W, L, page, heads, kv, spare=2):
    """Beams that share their full pages and have partial (and later) pages of their own."""
    stride = max(L) // page + 1 + spare
    pages = rng.permutation(N * W * stride).astype(np.int32)
    table = pages.reshape(N * W, stride).copy()
    for n in range(N):
        full = L[n] // page
        table[n * W:(n + 1) * W, :full] = table[n * W + rng.integers(0, W, size=W), :full]
    if kv == "bf16":
        arrays = [rng.integers(0, 1 << 16, size=(len(pages), heads, page, 128)).astype(np.uint16) for _ in range(2)]
    else:
        arrays = [rng.integers(0, 256, size=(len(pages), heads, page, 128)).astype(np.uint8) for _ in range(2)]
        if kv == "token":
            arrays += [rng.random((len(pages), heads, page)).astype(np.float32) for _ in range(2)]
    return table, arrays, np.repeat(np.array(L, np.int32), W)


def _reorder(parents, lens, table, arrays, states=(), status=None):
    d = [dev(a) for a in arrays]
    ks, vs = (d[2], d[3]) if len(d) == 4 else (None, None)
    out = torch.full(table.shape, -9, dtype=torch.int32, device="cuda")
    B.beam_reorder(dev(parents), dev(lens), dev(table), out, d[0], d[1], k_scale=ks, v_scale=vs, states=states, status=status)
    torch.cuda.synchronize()
    return host(out), [host(x) for x in d]


@pytest.mark.parametrize("kv", ["token", "scalar", "bf16"])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("W,heads", [(1, 1), (4, 2), (7, 1), (32, 1)])
def test_reorder_tables_pages_and_states(kv, page, W, heads):
    rng = np.random.default_rng(page + W)
    L = [0, 1, page - 1, page, page + 1, 5 * page + 7, 300]
    N = len(L)
    table, arrays, lens = _problem(rng, N, W, L, page, heads, kv)
    parents = rng.integers(0, W, size=(N, W)).astype(np.int32)
    parents[-1] = W - 1                                  # one beam takes all
    parents[-2] = np.arange(W)[::-1]                     # a permutation
    parents[-3] = 0                                      # a prompt spread over the beams
    want, made = C.beam_reorder(parents, lens, table, arrays, page)
    src = (np.arange(N)[:, None] * W + parents).reshape(-1)
    a = rng.random((N * W, heads, 37)).astype(np.float32)          # rows of 4-byte units
    b = rng.integers(0, 1 << 30, size=(N * W, 64)).astype(np.int32)  # of 16
    c = rng.integers(0, 255, size=(N * W, 13)).astype(np.uint8)      # of single bytes
    st, states = word(), [(dev(x), torch.zeros_like(dev(x))) for x in (a, b, c)]
    got, new = _reorder(parents, lens, table, arrays, states, st)
    assert int(st[0]) == 0
    assert np.array_equal(got, want)
    for x, y in zip(new, made):
        assert same(x, y)
    for x, (_, y) in zip((a, b, c), states):
        assert np.array_equal(host(y), x[src])


def test_reorder_keeps_flagged_requests():
    rng = np.random.default_rng(3)
    table, arrays, lens = _problem(rng, 5, 3, [40, 40, 40, 40, 40], 16, 1, "token")
    parents = np.zeros((5, 3), np.int32)
    parents[0, 1], parents[1, 2] = 3, -1
    lens[2 * 3 + 1] = 41
    lens[3 * 3:4 * 3] = 16 * table.shape[1] + 1
    ok = np.repeat([False, False, False, False, True], 3)
    want, made = C.beam_reorder(parents[4:], lens[12:], table[12:], arrays, 16)
    x = rng.random((15, 9)).astype(np.float32)
    st, state = word(), (dev(x), torch.zeros(15, 9, device="cuda"))
    got, new = _reorder(parents, lens, table, arrays, [state], st)
    assert int(st[0]) == B.DEV_BAD_BEAM | 0x2
    assert np.array_equal(got[12:], want) and np.array_equal(got[:12], table[:12])
    assert np.array_equal(host(state[1])[~ok], x[~ok])
    for a, b in zip(new, made):
        assert same(a, b)


def test_reorder_flags_bad_pages():
    rng = np.random.default_rng(4)
    table, arrays, lens = _problem(rng, 1, 3, [20], 16, 1, "token")
    table[2, 1] = 10 ** 6
    st = word()
    _, new = _reorder(np.zeros((1, 3), np.int32), lens, table, arrays, (), st)
    assert int(st[0]) == 0x1
    good, page = table[1, 1], table[0, 1]
    assert np.array_equal(new[0][good, :, :4], arrays[0][page, :, :4]) and np.array_equal(new[0][good, :, 4:], arrays[0][good, :, 4:])


# ------------------------------------------------- how exactly totals and ranks are computed

def test_length_penalties_are_exact_to_1e9():
    """Ended beams whose ranks lie within an fp32 step of each other: the order is fp64's wherever they differ by
    more than 1e-9 (relative), for lengths up to 2^31 - 1 and many penalties."""
    rng = np.random.default_rng(12)
    N = 4000
    n = np.stack([rng.integers(1, 600, size=N), rng.integers(1, 600, size=N)], 1)
    n[:50] = rng.integers(1, 2 ** 31 - 1, size=(50, 2))
    for p in (0.6, 1.0, 0.25, 2.0, 1.7):
        p32 = float(np.float32(p))
        t1 = (-1 - 40 * rng.random(N)).astype(np.float32)
        with np.errstate(over="ignore"):
            t2 = (t1 * (n[:, 1] / n[:, 0]) ** p32).astype(np.float32)
        rank = np.stack([t1 / n[:, 0].astype(np.float64) ** p32, t2 / n[:, 1].astype(np.float64) ** p32], 1)
        gap = (rank[:, 0] - rank[:, 1]) / np.abs(rank[:, 0])
        clear = np.abs(gap) > 1e-9
        assert clear.sum() > N // 2 and np.abs(gap).max() < 1e-6
        got = B.beam_select(torch.zeros(N, 2, 3, device="cuda"), dev(np.stack([t1, t2], 1)), eos=1,
                            finished=torch.ones(N, 2, dtype=torch.uint8, device="cuda"), lengths=dev(n.astype(np.int32)), length_penalty=p)
        assert np.array_equal((host(got[1])[:, 0] == 0)[clear], (gap > 0)[clear])


@pytest.mark.parametrize("shift", [0.0, 11.5, -7.25])
def test_logarithms_are_exact_to_1e9(shift):
    """A live beam over V equal logits has total score - ln V; against an ended beam at the nearest fp32
    number, the order is fp64's wherever they differ by more than 2e-9."""
    rng = np.random.default_rng(13)
    for V in list(range(1, 70)) + [100, 511, 512, 4099, 32771, 131072]:
        N = 64
        s1 = (-0.5 - 4 * rng.random(N)).astype(np.float32)
        total = s1.astype(np.float64) - np.log(V)
        s2 = total.astype(np.float32)
        gap = total - s2.astype(np.float64)
        clear = np.abs(gap) > 2e-9
        fin = np.zeros((N, 2), np.uint8)
        fin[:, 1] = 1
        got = B.beam_select(torch.full((N, 2, V), shift, device="cuda"), dev(np.stack([s1, s2], 1)), eos=0, finished=dev(fin))
        assert np.array_equal((host(got[1])[:, 0] == 0)[clear], (gap > 0)[clear]), V
