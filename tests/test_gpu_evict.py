"""pa_evict_select and pa_kv_compact against their definitions: every position and every byte
equal (needs a GPU)."""
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


def _fast_select(mass, L, budget, first, recent):
    """evict_select's oracle for long rows: numpy's stable sort over the middle."""
    B_, H, _ = mass.shape
    keep, new = np.full((B_, H, budget), -1, np.int32), np.minimum(L, budget).astype(np.int32)
    for r in range(B_):
        n = int(L[r])
        for h in range(H):
            if n <= budget:
                keep[r, h, :n] = np.arange(n)
                continue
            x = mass[r, h, first:n - recent].astype(np.float64)
            order = np.lexsort((np.arange(x.size), np.where(np.isnan(x), 0, -x), np.isnan(x)))
            mid = first + np.sort(order[:budget - first - recent])
            keep[r, h] = np.r_[0:first, mid, n - recent:n]
    return keep, new


def _select(mass, L, budget, first=0, recent=0, oracle=_fast_select):
    st = word()
    keep, new = B.evict_select(dev(mass), dev(np.asarray(L, np.int32)), budget=budget, first=first, recent=recent, status=st)
    wk, wn = oracle(mass, np.asarray(L), budget, first, recent)
    assert np.array_equal(host(new), wn)
    assert np.array_equal(host(keep), wk), np.argwhere(host(keep) != wk)[:4]
    assert int(st[0]) == 0


def _values(kind, rng, shape):
    x = rng.exponential(size=shape) * np.exp2(rng.uniform(-20, 4, size=shape))
    if kind == "ties":
        x = rng.integers(0, 3, size=shape).astype(np.float64)
    if kind == "equal":
        x[:] = 0.25
    if kind == "zeros":
        x = np.where(rng.random(shape) < 0.5, 0.0, -0.0)
    if kind == "odd":  # infinities, NaN, negatives, denormals
        pick = rng.integers(0, 8, size=shape)
        x = np.select([pick == 0, pick == 1, pick == 2, pick == 3, pick == 4],
                      [np.inf, -np.inf, np.nan, -x, 1e-42], x)
    return x.astype(np.float32)


@pytest.mark.parametrize("kind", ["tail", "ties", "equal", "zeros", "odd"])
def test_select_small_against_the_loop(kind):
    rng = np.random.default_rng(1)
    mass = _values(kind, rng, (6, 2, 140))
    L = [140, 139, 64, 33, 1, 0]
    for budget, first, recent in ((1, 0, 0), (1, 1, 0), (1, 0, 1), (32, 0, 0), (33, 4, 8), (64, 32, 32), (139, 3, 2), (140, 0, 0), (500, 0, 9)):
        _select(mass, L, budget, first, recent, C.evict_select)


@pytest.mark.parametrize("kind", ["tail", "ties", "equal", "odd"])
@pytest.mark.parametrize("n", [1025, 4096, 8193, 33000, 131072])
def test_select_lengths(kind, n):
    rng = np.random.default_rng(n)
    mass = _values(kind, rng, (3, 1, n + 3))
    L = [n, n - 1, (n + 1) // 2]
    for budget in (n // 8, n // 2 + 1, n - 1):
        _select(mass, L, budget, min(4, budget), min(64, budget // 2))


def test_select_very_long_rows():
    rng = np.random.default_rng(3)
    _select(_values("tail", rng, (1, 1, 900001)), [900001], 100000, 4, 1000)


@pytest.mark.parametrize("kind", ["tail", "ties", "odd"])
@pytest.mark.parametrize("n", [131073, 200000, 262144, 262145])
def test_select_rows_of_the_widest_clusters_and_beyond(kind, n):
    rng = np.random.default_rng(n)
    mass = _values(kind, rng, (2, 2, n))
    for budget in (1000, n // 2 + 1, n - 1):
        _select(mass, [n, n - 77777], budget, 4, 64)


def test_select_many_rows():
    rng = np.random.default_rng(4)
    mass = _values("tail", rng, (200, 3, 257))
    _select(mass, rng.integers(0, 258, size=200), 100, 2, 10)


def test_select_flags_bad_contexts():
    mass = np.ones((3, 1, 64), np.float32)
    st = word()
    keep, new = B.evict_select(dev(mass), dev(np.array([64, 65, -1], np.int32)), budget=16, status=st)
    assert int(st[0]) == 0x2 and host(new).tolist() == [16, 0, 0]
    assert np.all(host(keep)[1:] == -1) and host(keep)[0, 0].tolist() == list(range(16))


# ------------------------------------------------------------------------- compaction

def _cache(rng, pages, heads, page, kv):
    if kv == "bf16":
        k, v = (rng.integers(0, 1 << 16, size=(pages, heads, page, 128)).astype(np.uint16) for _ in range(2))
        return [k, v]
    k, v = (rng.integers(0, 256, size=(pages, heads, page, 128)).astype(np.uint8) for _ in range(2))
    if kv == "scalar":
        return [k, v]
    return [k, v] + [rng.random((pages, heads, page)).astype(np.float32) for _ in range(2)]


def _keeps(rng, B_, H, L, new, width):
    keep = np.full((B_, H, width), -1, np.int32)
    for r in range(B_):
        for h in range(H):
            keep[r, h, :new[r]] = np.sort(rng.choice(int(L[r]), size=int(new[r]), replace=False))
    return keep


def _compact(keep, new, table, dst, arrays, mass, mass_out, page, status=None):
    d = [dev(a) for a in arrays]
    ks, vs = (d[2], d[3]) if len(d) == 4 else (None, None)
    m = dev(mass)
    mo = m if dst is None else dev(mass_out)
    B.kv_compact(dev(keep), dev(new), dev(table), d[0], d[1], dst_block_table=dev(dst), k_scale=ks, v_scale=vs, mass=m,
                 mass_out=None if mass is None else mo, status=status)
    torch.cuda.synchronize()
    return [host(x) for x in d], None if mass is None else host(mo)


@pytest.mark.parametrize("kv", ["token", "scalar", "bf16"])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("heads", [1, 3])
def test_compact_moves_every_byte(kv, page, inplace, heads):
    rng = np.random.default_rng(page + heads)
    L = np.array([1, 15, 300, 1000, 777, 0], np.int32)
    new = np.array([1, 7, 129, 640, 777, 0], np.int32)   # one kept, odd, past a tile, several rounds, all, none
    B_, npg = len(L), -(-1000 // page)
    table = rng.permutation(B_ * npg * 2).astype(np.int32)
    src, dst = table[:B_ * npg].reshape(B_, npg), None if inplace else table[B_ * npg:].reshape(B_, npg)[:, :-(-777 // page)]
    arrays = _cache(rng, B_ * npg * 2, heads, page, kv)
    keep = _keeps(rng, B_, heads, L, new, 800)
    mass = rng.random((B_, heads, 1003)).astype(np.float32)
    mo = mass if inplace else np.full((B_, heads, 777), -3.0, np.float32)
    want, wm = C.kv_compact(keep, new, src, src if inplace else dst, arrays, page, mass, mo)
    st = word()
    got, gm = _compact(keep, new, src, dst, arrays, mass, mo, page, st)
    assert int(st[0]) == 0
    for a, b in zip(got, want):
        assert same(a, b)
    assert same(gm, wm)


@pytest.mark.parametrize("L,n", [(20000, 9001), (131072, 4096)])
def test_compact_long_in_place(L, n):
    """Many rounds: random kept sets, and one that shifts everything by a single slot."""
    rng = np.random.default_rng(L)
    page, npg = 32, L // 32
    table = rng.permutation(2 * npg).astype(np.int32).reshape(2, npg)
    arrays = _cache(rng, 2 * npg, 1, page, "token")
    keep = _keeps(rng, 2, 1, [L, L], [n, n], n)
    keep[1, 0] = np.arange(1, n + 1)
    new = np.array([n, n], np.int32)
    mass = rng.random((2, 1, L)).astype(np.float32)
    want, wm = C.kv_compact(keep, new, table, table, arrays, page, mass, mass)
    got, gm = _compact(keep, new, table, None, arrays, mass, None, page)
    for a, b in zip(got, want):
        assert same(a, b)
    assert same(gm, wm)


def test_compact_without_mass_and_with_shared_sources():
    """Two requests that share their pages are compacted into pages of their own."""
    rng = np.random.default_rng(9)
    page = 16
    src = np.repeat(rng.permutation(40)[:10].astype(np.int32)[None], 2, 0)
    dst = (40 + rng.permutation(8)).astype(np.int32).reshape(2, 4)
    arrays = _cache(rng, 48, 2, page, "token")
    new = np.array([50, 64], np.int32)
    keep = _keeps(rng, 2, 2, [160, 160], new, 64)
    want, _ = C.kv_compact(keep, new, src, dst, arrays, page)
    got, _ = _compact(keep, new, src, dst, arrays, None, None, page)
    for a, b in zip(got, want):
        assert same(a, b)


def test_compact_flags_and_skips_bad_entries():
    rng = np.random.default_rng(10)
    page = 16
    table = rng.permutation(24).astype(np.int32).reshape(4, 6)
    dst = (24 + rng.permutation(8)).astype(np.int32).reshape(4, 2)
    arrays = _cache(rng, 32, 1, page, "token")
    keep = np.tile(np.arange(0, 64, 2, dtype=np.int32), (4, 1, 1)).reshape(4, 1, 32)
    new = np.array([32, 32, 40, 32], np.int32)
    keep[0, 0, 5] = 96                 # past the table
    keep[0, 0, 6] = 95                 # not above the one before it, and neither is the next
    table2 = table.copy()
    table2[1, 0] = -4                  # positions 0 .. 15
    dst[3, 1] = 1000                   # slots 16 .. 31
    st = word()
    got, _ = _compact(keep, new, table2, dst, arrays, None, None, page, st)
    assert int(st[0]) == B.DEV_BAD_KEEP | 0x1
    want = [a.copy() for a in arrays]
    for r in (0, 1, 3):
        for i in range(32):
            s = int(keep[r, 0, i])
            if (r == 0 and i in (5, 6, 7)) or (r == 1 and s < 16) or (r == 3 and i >= 16):
                continue
            for a, o in zip(arrays, want):
                o[dst[r, i // page], 0, i % page] = a[table[r, s // page], 0, s % page]
    for a, b in zip(got, want):
        assert same(a, b)


def test_select_then_compact_in_a_graph():
    rng = np.random.default_rng(11)
    page, L = 32, 640
    table = rng.permutation(40).astype(np.int32).reshape(2, 20)
    arrays = _cache(rng, 40, 2, page, "token")
    mass = rng.random((2, 2, L)).astype(np.float32)
    lens = np.array([L, 500], np.int32)
    keep, new = C.evict_select(mass, lens, 300, 4, 32)
    want, wm = C.kv_compact(keep, new, table, table, arrays, page, mass, mass)
    base = [dev(a) for a in arrays] + [dev(mass)]
    d = [x.clone() for x in base]
    t, ln = dev(table), dev(lens)

    def step():
        k, n = B.evict_select(d[4], ln, budget=300, first=4, recent=32)
        B.kv_compact(k, n, t, d[0], d[1], k_scale=d[2], v_scale=d[3], mass=d[4])
        return n

    step()
    for x, y in zip(d, base):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n = step()
    for x, y in zip(d, base):
        x.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    assert host(n).tolist() == [300, 300]
    for a, b in zip(d, want + [wm]):
        assert same(host(a), b)
