"""pa_page_assign and pa_page_release against their definitions: every entry, slot and flag equal (needs a GPU)."""
import numpy as np
import pytest
import torch

from cache_util import dev, host, word
from oracle import prompt_ops as C
from paged_fp8_kv_04_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _case(rng, lens, ql, page, room=None, pad=0, width=None):
    """A pool whose pages lie in random order: (lens, cu, table, free, num_free, pages, rows)."""
    lens, ql = np.asarray(lens, np.int32), np.asarray(ql, np.int64)
    cu = np.r_[0, ql.cumsum()].astype(np.int32)
    have, want = -(-lens.astype(np.int64) // page), -(-(lens + ql) // page)
    width = width or int(want.max(initial=0)) + 1
    need = int((want - have).sum())
    left = need + 5 if room is None else int(need * room)
    ids = rng.permutation(int(have.sum()) + left + 3).astype(np.int32)
    table = np.full((len(lens), width), -7, np.int32)
    at = 0
    for r, n in enumerate(have):
        table[r, :n] = ids[at:at + n]
        at += n
    free = np.full(left + 9, -3, np.int32)
    free[:left] = ids[at:at + left]
    return lens, cu, table, free, left, len(ids), int(cu[-1]) + pad


def _assign(lens, cu, table, free, left, pages, rows, page, in_place=False, **kw):
    st = word()
    d = dict(lens=dev(lens), table=dev(table), free=dev(free), count=dev(np.array([left], np.int32)))
    out = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    new, slots, pos = B.page_assign(d["lens"], dev(cu), d["table"], d["free"], d["count"], page_size=page, num_pages=pages, num_rows=rows,
                                    num_free_out=None if in_place else out, new_lens=d["lens"] if in_place else None, status=st, **kw)
    t, wn, ws, wp, wl, flags = C.page_assign(lens, cu, table, free, left, page, rows, pages)
    assert np.array_equal(host(d["table"]), t)
    assert np.array_equal(host(new), wn)
    assert np.array_equal(host(pos), wp)
    assert np.array_equal(host(slots), ws), np.argwhere(host(slots) != ws)[:4]
    assert np.array_equal(host(d["free"]), free)
    assert int(d["count"] if in_place else out) == wl and (in_place or int(d["count"]) == left)
    assert int(st) == flags, (hex(int(st)), hex(flags))
    return flags


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("reqs,hi,qlo,qhi,pad", [(1, 0, 1, 1, 0), (1, 500, 0, 0, 3), (32, 8191, 1, 1, 0), (31, 3000, 0, 6, 7), (129, 700, 0, 90, 0), (700, 100, 1, 1, 40)])
def test_assign(page, reqs, hi, qlo, qhi, pad, in_place):
    rng = np.random.default_rng(reqs + page)
    for room in (None, 1.0, 0.7, 0.0):
        lens, ql = rng.integers(0, hi + 1, size=reqs), rng.integers(qlo, qhi + 1, size=reqs)
        _assign(*_case(rng, lens, ql, page, room, pad), page, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_assign_more_requests_than_threads(in_place):
    rng = np.random.default_rng(5)
    for reqs, qhi in ((1024, 3), (1025, 1), (3000, 20), (5000, 2)):
        lens, ql = rng.integers(0, 200, size=reqs), rng.integers(0, qhi + 1, size=reqs)
        for room in (None, 0.5, 0.99):
            _assign(*_case(rng, lens, ql, 16, room, 11), 16, in_place)


@pytest.mark.parametrize("reqs,q,page", [(1, 100003, 16), (3, 87381, 128), (32, 8192, 16), (9, 5001, 32)])
def test_assign_prompts(reqs, q, page):
    rng = np.random.default_rng(q)
    lens = rng.integers(0, 40, size=reqs)
    ql = np.full(reqs, q) - rng.integers(0, 30, size=reqs)
    for room in (None, 0.8):
        _assign(*_case(rng, lens, ql, page, room, 5), page)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("reqs,q,page", [(1, 16384, 16), (1, 16385, 16), (700, 24, 64), (2500, 11, 16), (5, 60001, 128)])
def test_assign_about_the_rows_of_one_cluster(reqs, q, page, in_place):
    rng = np.random.default_rng(q + page)
    lens = rng.integers(0, 70, size=reqs)
    ql = np.full(reqs, q) if reqs == 1 else q + rng.integers(-10, 11, size=reqs)
    for room in (None, 0.6):
        _assign(*_case(rng, lens, ql, page, room, 3), page, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_assign_many_rows_of_which_none_is_served(in_place):
    rng = np.random.default_rng(12)
    lens, cu, table, free, left, pages, rows = _case(rng, [3, 5], [20000, 9000], 16, None, 2)
    cu[1] = 31000
    assert _assign(lens, cu, table, free, left, pages, rows, 16, in_place) == 0x4


def test_assign_takes_lower_positions_from_the_top():
    lens, cu, table, free = np.array([15], np.int32), np.array([0, 40], np.int32), np.full((1, 4), 0, np.int32), np.array([4, 5, 6, 1], np.int32)
    d = dev(table)
    new, slots, pos = B.page_assign(dev(lens), dev(cu), d, dev(free), dev(np.array([4], np.int32)), page_size=16, num_pages=8, num_rows=40)
    assert host(d).tolist() == [[0, 1, 6, 5]] and int(new) == 55 and host(slots)[:2].tolist() == [15, 16] and host(slots)[17:19].tolist() == [6 * 16, 6 * 16 + 1]
    assert host(pos).tolist() == list(range(15, 55))


def test_assign_without_requests_or_rows():
    count, table = dev(np.array([3], np.int32)), torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    empty, cu, left = torch.zeros(0, dtype=torch.int32, device="cuda"), dev(np.zeros(1, np.int32)), word()
    new, slots, pos = B.page_assign(empty, cu, table, dev(np.arange(5, dtype=np.int32)), count, page_size=16, num_pages=9, num_rows=300, num_free_out=left)
    assert new.shape == (0,) and np.all(host(slots) == -1) and np.all(host(pos) == 0) and int(left) == 3
    new, slots, pos = B.page_assign(empty, cu, table, dev(np.arange(5, dtype=np.int32)), count, page_size=16, num_pages=9, num_rows=0)
    assert slots.shape == (0,) and int(count) == 3
    B.page_release(empty, empty, table, dev(np.arange(5, dtype=np.int32)), count, page_size=16, num_pages=9, num_free_out=left)
    assert int(left) == 3


def test_assign_flags_bad_requests_and_serves_the_others():
    rng = np.random.default_rng(9)
    lens, cu, table, free, left, pages, rows = _case(rng, [10, 40, 5, 0, 30], [20, 3, 70, 1, 9], 16, None, 2, 5)
    lens[1] = -4
    assert _assign(lens, cu, table, free, left, pages, rows, 16) == 0x2
    lens[1], lens[2] = 40, 75     # 75 + 70 tokens pass a table of five pages
    assert _assign(lens, cu, table, free, left, pages, rows, 16) == 0x2
    lens[2] = 2**31 - 20
    assert _assign(lens, cu, table, free, left, pages, rows, 16) == 0x2


@pytest.mark.parametrize("cu", [[0, 5, 3, 9], [-1, 2, 3, 4], [0, 2, 3, 11], [4, 3, 5, 6], [0, 2, 2**31 - 1, 3]])
def test_assign_serves_nobody_where_rows_do_not_ascend(cu):
    rng = np.random.default_rng(3)
    lens, _, table, free, left, pages, _ = _case(rng, [1, 2, 3], [5, 5, 5], 16)
    assert _assign(lens, np.array(cu, np.int32), table, free, left, pages, 10, 16) == 0x4


def test_assign_rows_before_the_first_request():
    rng = np.random.default_rng(4)
    lens, cu, table, free, left, pages, rows = _case(rng, [7, 0, 16], [30, 0, 2], 16)
    _assign(lens, cu + 6, table, free, left, pages, rows + 9, 16)


def test_assign_flags_bad_pages():
    rng = np.random.default_rng(6)
    lens, cu, table, free, left, pages, rows = _case(rng, [10, 20, 5], [20, 3, 30], 16)
    free[left - 1], free[left - 2] = -5, pages + 3   # entered as they stand
    assert _assign(lens, cu, table, free, left, pages, rows, 16) == 0x1
    free[left - 1], free[left - 2], table[1, 1] = 0, 1, pages
    assert _assign(lens, cu, table, free, left, pages, rows, 16) == 0x1


def test_assign_takes_the_count_as_within_the_stack():
    rng = np.random.default_rng(7)
    lens, cu, table, free, left, pages, rows = _case(rng, [0, 0], [40, 40], 16)
    free[:], pages = np.arange(len(free)), len(free)
    assert _assign(lens, cu, table, free, len(free) + 1000, pages, rows, 16) == 0
    assert _assign(lens, cu, table, free, -5, pages, rows, 16) == 0x1000


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("reqs,hi", [(1, 1), (4, 300), (33, 9000), (1500, 200), (8, 131072)])
def test_release(reqs, hi, page):
    rng = np.random.default_rng(reqs * page)
    for room in (10**9, 20, 0):
        lens = rng.integers(0, hi + 1, size=reqs).astype(np.int32)
        new = np.where(rng.random(reqs) < 0.3, 0, rng.integers(0, hi + 1, size=reqs)).astype(np.int32)  # some grow
        width = -(-hi // page) + 2
        pages = reqs * width
        table = rng.permutation(pages).astype(np.int32).reshape(reqs, width)
        left = int(rng.integers(0, 9))
        capacity = left + min(room, pages)
        free = np.full(max(capacity, 1), -3, np.int32)
        for in_place in (False, True):
            st, d, count, out = word(), dev(free), dev(np.array([left], np.int32)), word()
            dt = dev(table)
            B.page_release(dev(lens), dev(new), dt, d, count, page_size=page, num_pages=pages, num_free_out=None if in_place else out, status=st)
            wf, wl, flags = C.page_release(lens, new, table, free, left, page, pages)
            assert np.array_equal(host(d), wf) and int(count if in_place else out) == wl and int(st) == flags
            assert np.array_equal(host(dt), table)


def test_release_flags_bad_requests_and_pages():
    table = np.arange(12, dtype=np.int32).reshape(4, 3)
    table[0, 1] = 99
    lens, new = np.array([40, -1, 49, 48], np.int32), np.array([16, 0, 0, -2], np.int32)
    d, st, count = dev(np.full(20, -3, np.int32)), word(), dev(np.array([2], np.int32))
    B.page_release(dev(lens), dev(new), dev(table), d, count, page_size=16, num_pages=50, status=st)
    assert int(st) == 0x3 and int(count) == 4 and host(d)[:5].tolist() == [-3, -3, 99, 2, -3]


def test_pool_over_many_captured_steps():
    """Decode steps replayed from one graph, all state updated in place, then everything given back: no page is lost."""
    rng = np.random.default_rng(8)
    reqs, page, pages, width = 24, 16, 500, 12
    free = rng.permutation(pages).astype(np.int32)
    d = dict(lens=dev(np.zeros(reqs, np.int32)), table=dev(np.full((reqs, width), -1, np.int32)), free=dev(free), count=dev(np.array([pages], np.int32)))
    cu = dev(np.arange(reqs + 1, dtype=np.int32))
    slots, pos, st = torch.zeros(reqs + 3, dtype=torch.int64, device="cuda"), torch.zeros(reqs + 3, dtype=torch.int32, device="cuda"), word()

    def step():
        B.page_assign(d["lens"], cu, d["table"], d["free"], d["count"], page_size=page, num_pages=pages, new_lens=d["lens"], slot_mapping=slots, positions=pos,
                      status=st)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    B.torch_module()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    seen = set()
    for n in range(100):
        graph.replay()
        s = host(slots)
        assert np.all(host(d["lens"]) == n + 1) and np.all(s[reqs:] == -1) and np.all(host(pos)[:reqs] == n)
        assert len(set(s[:reqs].tolist())) == reqs and not seen & set(s[:reqs].tolist())
        seen |= set(s[:reqs].tolist())
    assert int(st) == 0 and int(d["count"]) == pages - reqs * 7
    zero = torch.zeros_like(d["lens"])
    B.page_release(d["lens"], zero, d["table"], d["free"], d["count"], page_size=page, num_pages=pages, status=st)
    assert int(d["count"]) == pages and sorted(host(d["free"]).tolist()) == list(range(pages)) and int(st) == 0


def test_paging_refuses_wrong_tensors():
    lens, cu, table = dev(np.zeros(3, np.int32)), dev(np.zeros(4, np.int32)), dev(np.zeros((3, 4), np.int32))
    free, count = dev(np.arange(8, dtype=np.int32)), dev(np.array([8], np.int32))
    kw = dict(page_size=16, num_pages=8)
    with pytest.raises(TypeError):
        B.page_assign(lens.long(), cu, table, free, count, num_rows=3, **kw)
    with pytest.raises(TypeError):
        B.page_assign(lens, cu, table, free, count, **kw)                       # no rows
    with pytest.raises(ValueError):
        B.page_assign(lens, cu[:3], table, free, count, num_rows=3, **kw)
    with pytest.raises(ValueError):
        B.page_assign(lens, cu, table.t(), free, count, num_rows=3, **kw)
    with pytest.raises(ValueError):
        B.page_assign(lens, cu, table, free, count, num_rows=-1, **kw)
    with pytest.raises(ValueError):
        B.page_assign(lens, cu, table, free, count, num_rows=3, slot_mapping=torch.zeros(4, dtype=torch.int64, device="cuda"), **kw)
    with pytest.raises(B.PaError):
        B.page_assign(lens, cu, table, free, count, num_rows=3, page_size=20, num_pages=8)
    with pytest.raises(B.PaError):
        B.page_assign(lens, cu, table, free, count, num_rows=3, new_lens=cu[:3], **kw)
    with pytest.raises(B.PaError):
        B.page_release(lens, lens, table, free, free[3:4], **kw)
    with pytest.raises(ValueError):
        B.page_release(lens, lens[:2], table, free, count, **kw)
