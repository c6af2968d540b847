"""pa_attn_mass against its fp64 definition, element by element, within the bound that
oracle/cache_ops.py derives from the arithmetic (needs a GPU)."""
import numpy as np
import pytest
import torch

from cache_util import dev, host, run_mass, word
from oracle import cache_ops as C
from oracle import oracle as O
from paged_fp8_kv_04_gb300 import binding as B
from paged_fp8_kv_04_gb300 import synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -22   # how exactly the query is held, relative to its group's largest element


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _check(p, decay=1.0, pad=5, seed=0, lse=None):
    rng = np.random.default_rng(seed)
    if lse is None:
        lse = O.decode(p)[1].astype(np.float32)
    L = int(p.context_lens.max())
    mass = rng.exponential(size=(p.num_seqs, p.num_kv_heads, L + pad)).astype(np.float32)
    want, tol = C.attn_mass(p, lse, mass, decay, U)
    st = word()
    for inplace in (True, False):
        m = dev(mass)
        out = None if inplace else torch.full_like(m, -7.0)
        got = host(run_mass(p, lse, m, decay, out=out, status=st))
        for r in range(p.num_seqs):
            n = int(p.context_lens[r]) if p.q_lens[r] else 0
            assert np.all(np.abs(got[r, :, :n] - want[r, :, :n]) <= tol[r, :, :n]), (
                r, inplace, np.abs(got[r, :, :n] - want[r, :, :n]).max())
            keep = mass[r, :, n:] if inplace else np.float32(-7.0)
            assert np.all(got[r, :, n:] == keep), (r, inplace, "positions past the context were written")
    assert int(st[0]) == 0
    return got


@pytest.mark.parametrize("kv,scale", [("fp8", "per_token"), ("fp8", "scalar"), ("bf16", "none")])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_modes_and_pages(kv, scale, page):
    p = synth.make_problem(11, num_seqs=5, context_lens=[1, 127, 128, 129, 700], q_lens=[1, 1, 1, 1, 1],
                           page_size=page, kv_dtype=kv, scale_mode=scale, num_kv_heads=2)
    _check(p, 0.75)


@pytest.mark.parametrize("kv,scale", [("fp8", "per_token"), ("bf16", "none")])
@pytest.mark.parametrize("ql", [[1, 0, 2, 5], [4, 8, 9, 3], [33, 16, 17, 64]])
def test_ragged_query_lengths(kv, scale, ql):
    p = synth.make_problem(12, num_seqs=4, context_lens=[64, 100, 257, 515], q_lens=ql, page_size=32,
                           kv_dtype=kv, scale_mode=scale, num_kv_heads=1)
    _check(p, 0.5)


def test_lengths_equal_to_the_query_and_empty_contexts():
    p = synth.make_problem(13, num_seqs=4, context_lens=[0, 3, 0, 8], q_lens=[0, 3, 0, 8], page_size=16)
    _check(p, 1.0)


def test_many_requests_and_heads():
    rng = np.random.default_rng(5)
    L = rng.integers(1, 400, size=60)
    p = synth.make_problem(14, num_seqs=60, context_lens=L, q_lens=rng.integers(0, 3, size=60).clip(max=L), page_size=16,
                           num_kv_heads=3)
    _check(p, 0.9)


@pytest.mark.parametrize("kv,scale", [("fp8", "per_token"), ("bf16", "none")])
@pytest.mark.parametrize("most", [1, 2, 9])
def test_more_short_requests_than_sms(kv, scale, most):
    """Many requests of a tile or two for every CTA, some of them without rows."""
    rng = np.random.default_rng(most)
    L = rng.integers(0, 200, size=900)
    ql = np.where(rng.random(900) < 0.2, 0, rng.integers(1, most + 1, size=900)).clip(max=L)
    p = synth.make_problem(24, num_seqs=900, context_lens=L, q_lens=ql, page_size=16, num_kv_heads=2, kv_dtype=kv,
                           scale_mode=scale)
    _check(p, 0.5)


def test_wide_magnitudes():
    """Key rows over 2^-3 .. 2^3 and query elements over 2^-2 .. 2^2."""
    p = synth.make_problem(15, num_seqs=3, context_lens=[90, 300, 513], q_lens=[1, 2, 1], page_size=64,
                           kv_mag_log2=3.0, q_mag_log2=2.0)
    _check(p, 0.9)


def test_zero_queries_and_zero_keys():
    p = synth.make_problem(16, num_seqs=2, context_lens=[50, 200], q_lens=[1, 2], page_size=16)
    p.q[0] = 0
    p.k_cache[p.block_table[1, :4]] = 0
    p.k_scale[p.block_table[1, :4]] = 0
    _check(p, 1.0)


def test_rows_without_keys_give_no_weight():
    p = synth.make_problem(17, num_seqs=2, context_lens=[40, 300], q_lens=[2, 1], page_size=16)
    lse = O.decode(p)[1].astype(np.float32)
    lse[0, 3:9] = -np.inf
    lse[2] = -np.inf
    got = _check(p, 0.25, lse=lse)
    assert np.isfinite(got[:, :, :40]).all()


def test_decay_zero_reads_no_mass():
    p = synth.make_problem(18, num_seqs=2, context_lens=[40, 300], q_lens=[1, 1], page_size=16)
    lse = O.decode(p)[1].astype(np.float32)
    zero = np.zeros((2, 1, 300), np.float32)
    want, tol = C.attn_mass(p, lse, zero, 0.0, U)
    m = torch.full((2, 1, 300), float("nan"), device="cuda")
    got = host(run_mass(p, lse, m, 0.0))
    for r, n in enumerate([40, 300]):
        assert np.all(np.abs(got[r, 0, :n] - want[r, 0, :n]) <= tol[r, 0, :n])


def test_unused_slots_of_a_page_hold_anything():
    """Codes and scales past the context are NaN: they reach nothing."""
    p = synth.make_problem(19, num_seqs=3, context_lens=[5, 130, 200], q_lens=[1, 2, 1], page_size=128)
    for r, L in enumerate([5, 130, 200]):
        last = p.block_table[r, (L - 1) // 128]
        p.k_cache[last, :, (L - 1) % 128 + 1:] = 0x7F
        p.k_scale[last, :, (L - 1) % 128 + 1:] = np.nan
    _check(p, 0.5)


def test_requests_share_pages():
    """Two requests over the same pages (a common prefix): the mass belongs to the request."""
    p = synth.make_problem(20, num_seqs=2, context_lens=[300, 300], q_lens=[1, 1], page_size=32)
    p.block_table[1] = p.block_table[0]
    _check(p, 0.5)


def test_flagged_requests_are_skipped():
    p = synth.make_problem(21, num_seqs=5, context_lens=[40, 60, 80, 100, 120], q_lens=[1, 1, 1, 1, 1], page_size=16)
    lse = O.decode(p)[1].astype(np.float32)
    mass = np.ones((5, 1, 120), np.float32)
    want, tol = C.attn_mass(p, lse, mass, 0.5, U)
    p.context_lens[1] = 121          # past the mass row
    p.context_lens[2] = -1
    p.block_table[3, 2] = 10 ** 6     # positions 32 .. 47
    st = word()
    got = host(run_mass(p, lse, dev(mass), 0.5, status=st))
    assert int(st[0]) == 0x1 | 0x2 | 0x4 or int(st[0]) == 0x1 | 0x2
    assert np.all(got[1] == 1) and np.all(got[2] == 1)
    for r, n in ((0, 40), (4, 120)):
        assert np.all(np.abs(got[r, 0, :n] - want[r, 0, :n]) <= tol[r, 0, :n])
    assert np.all(got[3, 0, 32:48] == 0.5)
    ok = np.r_[0:32, 48:100]
    assert np.all(np.abs(got[3, 0, ok] - want[3, 0, ok]) <= tol[3, 0, ok])


def test_bad_query_lengths_are_flagged():
    p = synth.make_problem(22, num_seqs=3, context_lens=[40, 60, 80], q_lens=[1, 3, 1], page_size=16)
    lse = O.decode(p)[1].astype(np.float32)
    st = word()
    got = host(run_mass(p, lse, dev(np.ones((3, 1, 80), np.float32)), 0.5, max_q_len=2, status=st))
    assert int(st[0]) == 0x4 and np.all(got[1] == 1) and np.all(got[0, 0, :39] >= 0.5)


def test_repeats_are_identical_and_streams_are_followed():
    p = synth.make_problem(23, num_seqs=4, context_lens=[1000, 2000, 3001, 5], q_lens=[1, 2, 1, 1], page_size=64)
    lse = O.decode(p)[1].astype(np.float32)
    m = dev(np.random.default_rng(0).exponential(size=(4, 1, 3001)).astype(np.float32))
    a = run_mass(p, lse, m, 0.5, out=torch.zeros_like(m))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run_mass(p, lse, m, 0.5, out=torch.zeros_like(m))
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_captured_steps_accumulate():
    """One captured call replayed three times equals three calls."""
    p = synth.make_problem(24, num_seqs=3, context_lens=[500, 129, 64], q_lens=[1, 1, 1], page_size=128)
    lse = O.decode(p)[1].astype(np.float32)
    t = [dev(x) for x in (p.q, p.k_cache, p.block_table, p.context_lens, p.cu_seqlens_q, lse)]
    ks = dev(p.k_scale)
    a, b = torch.ones((3, 1, 500), device="cuda"), torch.ones((3, 1, 500), device="cuda")
    call = lambda m: B.attn_mass(*t, m, max_q_len=1, sm_scale=p.sm_scale, decay=0.5, k_scale=ks)  # noqa: E731
    for _ in range(3):
        call(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(b)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_binding_refuses_what_the_library_cannot_see():
    p = synth.make_problem(25, num_seqs=2, context_lens=[40, 60], q_lens=[1, 1], page_size=16)
    lse = O.decode(p)[1].astype(np.float32)
    m = torch.zeros(2, 1, 60, device="cuda")
    with pytest.raises(TypeError):
        run_mass(p, lse, m.double())
    with pytest.raises(ValueError):
        run_mass(p, lse, torch.zeros(2, 1, 120, device="cuda")[..., ::2])
    with pytest.raises(ValueError):
        run_mass(p, lse[:1], m)
    with pytest.raises(ValueError):
        run_mass(p, lse, m.cpu())
    with pytest.raises(B.PaError):
        run_mass(p, lse, m, 2.0)
