"""Refusals of the operators on a prompt's way into the cache (checked before any device is touched: the
pointers are never dereferenced, and valid calls without work enqueue nothing), the rotary frequencies, and the
oracle's definitions against closed forms."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import prompt_ops as C
from paged_fp8_kv_04_gb300 import binding as B
from paged_fp8_kv_04_gb300 import build as libbuild
from test_cache_ops_host import _fill

OK, INVALID, UNSUP, CAP, RAGGED, ALIGN, CUDA, DEVDATA, WS = range(9)
X = 0x900000000


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.lib()


ASSIGN = dict(num_pages=64, num_seqs=0, num_rows=0, block_table_stride=8, page_size=16, free_capacity=64, num_free=X, num_free_out=X)


@pytest.mark.parametrize("over,want", [
    (dict(), OK), (dict(reserved=1), INVALID), (dict(num_seqs=-1), INVALID), (dict(num_rows=-1), INVALID),
    (dict(block_table_stride=0), INVALID), (dict(page_size=8), UNSUP), (dict(page_size=128), OK), (dict(free_capacity=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(num_pages=2**31), INVALID), (dict(num_pages=2**31 - 1), OK),
    (dict(cu_seqlens_q=None), INVALID), (dict(free_pages=None), INVALID), (dict(num_free=None), INVALID), (dict(num_free_out=None), INVALID),
    (dict(context_lens=None, block_table=None, new_lens=None, slot_mapping=None, positions=None), OK),
    (dict(num_seqs=2, context_lens=None), INVALID), (dict(num_seqs=2, block_table=None), INVALID), (dict(num_seqs=2, new_lens=None), INVALID),
    (dict(num_rows=2, slot_mapping=None), INVALID), (dict(status=None), OK),
    (dict(slot_mapping=0x100000004), ALIGN), (dict(positions=0x100000002), ALIGN), (dict(block_table=0x100000002), ALIGN), (dict(status=X + 1), ALIGN),
    # outputs that share bytes with what other CTAs read or write
    (dict(num_seqs=8, num_rows=8, context_lens=X, new_lens=X + 4), INVALID), (dict(num_seqs=8, cu_seqlens_q=X + 32, new_lens=X), INVALID),
    (dict(num_seqs=8, block_table=X - 100), INVALID), (dict(num_seqs=8, num_rows=8, slot_mapping=X + 64, positions=X + 124), INVALID),
    (dict(num_seqs=8, num_rows=8, slot_mapping=X, free_pages=X + 60), INVALID), (dict(num_free=X, num_free_out=X + 4, free_pages=X + 4), INVALID),
    (dict(num_seqs=8, block_table=X - 256, num_free_out=X - 4), INVALID), (dict(num_seqs=8, block_table=X - 300, free_pages=X - 48, num_free=X + 512, num_free_out=X + 512), INVALID),
])
def test_page_assign_refusals(lib, over, want):
    assert lib.pa_page_assign(ctypes.byref(_fill(B.PageAssignArgs, ASSIGN, over)), None) == want
    assert lib.pa_page_assign(None, None) == INVALID


RELEASE = dict(num_pages=64, num_seqs=0, block_table_stride=8, page_size=16, free_capacity=64, num_free=X, num_free_out=X)


@pytest.mark.parametrize("over,want", [
    (dict(), OK), (dict(reserved=1), INVALID), (dict(num_seqs=-1), INVALID), (dict(block_table_stride=0), INVALID), (dict(page_size=256), UNSUP),
    (dict(free_capacity=0), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=2**31), INVALID), (dict(free_pages=None), INVALID),
    (dict(num_free_out=None), INVALID), (dict(context_lens=None, new_lens=None, block_table=None), OK), (dict(num_seqs=1, new_lens=None), INVALID),
    (dict(free_pages=X + 2), ALIGN), (dict(new_lens=0x100000001), ALIGN),
    (dict(num_seqs=8, free_pages=X - 252), INVALID), (dict(num_seqs=8, free_pages=X + 64, block_table=X + 316), INVALID),
    (dict(num_seqs=8, free_pages=X + 64, context_lens=X + 64), INVALID), (dict(num_seqs=8, new_lens=X - 28), INVALID),
    (dict(num_seqs=8, num_free_out=X + 4, context_lens=X + 4), INVALID),
])
def test_page_release_refusals(lib, over, want):
    assert lib.pa_page_release(ctypes.byref(_fill(B.PageReleaseArgs, RELEASE, over)), None) == want
    assert lib.pa_page_release(None, None) == INVALID


FAR = {f: i << 44 for i, f in enumerate(("context_lens", "cu_seqlens_q", "block_table", "new_lens", "free_pages"), 1)}


@pytest.mark.parametrize("seqs", [2**30 + 1, 2**31 - 1])
def test_paging_of_more_requests_than_the_kernels_count(lib, seqs):
    assert lib.pa_page_assign(ctypes.byref(_fill(B.PageAssignArgs, ASSIGN, dict(FAR, num_seqs=seqs))), None) == INVALID
    far = {f: at for f, at in FAR.items() if f != "cu_seqlens_q"}
    assert lib.pa_page_release(ctypes.byref(_fill(B.PageReleaseArgs, RELEASE, dict(far, num_seqs=seqs))), None) == INVALID


ROPE = dict(q_stride=2048, k_stride=128, q_out_stride=2048, k_out_stride=128, num_tokens=0, num_q_heads=16, num_kv_heads=1, head_dim=128,
            rot_dim=128, dtype=0, layout=0, inverse=0, scale=1.0)
# one buffer of 18 heads: 16 queries, a key, a value
PACKED = dict(num_tokens=5, q=X, k=X + 4096, q_stride=2304, k_stride=2304)


@pytest.mark.parametrize("over,want", [
    (dict(), OK), (dict(reserved=1), INVALID), (dict(num_tokens=-1), INVALID), (dict(num_q_heads=0), INVALID), (dict(num_kv_heads=-1), INVALID),
    (dict(head_dim=64), UNSUP), (dict(rot_dim=0), INVALID), (dict(rot_dim=3), INVALID), (dict(rot_dim=130), INVALID), (dict(rot_dim=2), OK),
    (dict(dtype=2), INVALID), (dict(layout=2), INVALID), (dict(inverse=2), INVALID), (dict(inverse=1), OK), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q_stride=2047), INVALID), (dict(k_out_stride=127), INVALID), (dict(q_out_stride=2**41), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(k=None, k_out=None, num_kv_heads=0, k_stride=0, k_out_stride=0), OK),
    (dict(num_kv_heads=0), INVALID), (dict(positions=None), INVALID), (dict(freqs=None), INVALID), (dict(num_q_heads=70000, q_stride=2**24, q_out_stride=2**24), UNSUP),
    (dict(q=X + 1), ALIGN), (dict(q=X + 2), OK), (dict(q=X + 2, dtype=1), ALIGN), (dict(freqs=X + 4), ALIGN), (dict(positions=X + 2), ALIGN),
    # overlaps: in place is exact, rows of one buffer may interleave
    (dict(PACKED, q_out=X + 2), INVALID), (dict(PACKED, q_out=X + 4096), INVALID), (dict(PACKED, q_out=X, q_out_stride=2048), INVALID),
    (dict(PACKED, k_out=X + 4092, k_out_stride=2304), INVALID), (dict(PACKED, k_out=X + 4608 - 128, k_out_stride=2304), INVALID),
    (dict(num_tokens=3, q_out=X, k_out=X + 2 * 4096 + 4000), INVALID), (dict(num_tokens=3, q_out=X, positions=X + 12284), INVALID),
    (dict(num_tokens=3, k_out=X, freqs=X - 504), INVALID),
])
def test_rope_refusals(lib, over, want):
    assert lib.pa_rope(ctypes.byref(_fill(B.RopeArgs, ROPE, over)), None) == want
    assert lib.pa_rope(None, None) == INVALID


ATTN = dict(q_stride=2048, k_stride=128, v_stride=128, num_seqs=0, num_rows=0, num_kv_heads=1, group_size=16, head_dim=128, out_dtype=0, sm_scale=0.088)


@pytest.mark.parametrize("over,want", [
    (dict(), OK), (dict(reserved=1), INVALID), (dict(num_seqs=-1), INVALID), (dict(num_rows=-1), INVALID), (dict(num_seqs=4096), OK),
    (dict(num_seqs=4097), UNSUP), (dict(num_rows=2**24, q=1 << 40, k=2 << 40, v=3 << 40, out=4 << 40), OK), (dict(num_rows=2**24 + 1), UNSUP), (dict(num_kv_heads=0), INVALID),
    (dict(num_kv_heads=65, k_stride=65 * 128, v_stride=65 * 128, q_stride=2**18), UNSUP), (dict(group_size=0), INVALID),
    (dict(group_size=65, q_stride=2**16), UNSUP), (dict(group_size=64, q_stride=8192), OK), (dict(group_size=1), OK), (dict(head_dim=64), UNSUP),
    (dict(out_dtype=2), INVALID), (dict(out_dtype=1), OK), (dict(sm_scale=0.0), INVALID), (dict(sm_scale=float("inf")), INVALID),
    (dict(q_stride=2040), INVALID), (dict(k_stride=120), INVALID), (dict(q_stride=2049), ALIGN), (dict(v_stride=132), ALIGN),
    (dict(v_stride=2**39), INVALID), (dict(q=None), INVALID), (dict(v=None), INVALID), (dict(cu_seqlens=None), INVALID), (dict(out=None), INVALID),
    (dict(lse=None, status=None), OK), (dict(k=X + 8), ALIGN), (dict(out=X + 4), ALIGN), (dict(lse=X + 2), ALIGN),
    (dict(num_rows=4, num_seqs=1, out=X, q=X + 4 * 4096 - 16), INVALID), (dict(num_rows=4, num_seqs=1, out=X, out_dtype=1, v=X + 4 * 8192 - 16), INVALID),
    (dict(num_rows=4, num_seqs=1, lse=X, k=X + 240), INVALID), (dict(num_rows=4, num_seqs=1, lse=X, out=X + 240), INVALID),
    (dict(num_rows=4, num_seqs=1, lse=X, cu_seqlens=X + 252), INVALID),
])
def test_prompt_attn_refusals(lib, over, want):
    assert lib.pa_prompt_attn(ctypes.byref(_fill(B.PromptAttnArgs, ATTN, over)), None) == want
    assert lib.pa_prompt_attn(None, None) == INVALID


# ------------------------------------------------------------------------- frequencies

def _radians(rot, **kw):
    f, scale = B.rope_frequencies(rot, device="cpu", **kw)
    assert f.dtype == torch.int64 and f.shape == (rot // 2,)
    return np.array([(int(x) % 2**64) / 2.0**64 * 2.0 * math.pi for x in f]), scale


def test_frequencies_without_scaling():
    w, scale = _radians(128)
    assert scale == 1.0 and w[0] == pytest.approx(1.0, rel=1e-15)
    assert w == pytest.approx(10000.0 ** (-np.arange(64) / 64.0), rel=1e-13)


def test_frequencies_of_stretched_contexts():
    plain, _ = _radians(64, base=500000.0)
    linear, scale = _radians(64, base=500000.0, scaling="linear", factor=4.0)
    assert scale == 1.0 and linear * 4.0 == pytest.approx(plain, rel=1e-12)
    ntk, scale = _radians(64, base=500000.0, scaling="ntk", factor=4.0)
    assert scale == 1.0 and ntk[0] == pytest.approx(plain[0], rel=1e-14) and ntk[-1] * 4.0 == pytest.approx(plain[-1], rel=1e-12)
    yarn, scale = _radians(64, base=500000.0, scaling="yarn", factor=4.0, original_len=8192)
    turns = 8192 * plain / (2 * math.pi)
    assert scale == pytest.approx(1.0 + 0.1 * math.log(4.0))
    assert yarn[turns > 64] == pytest.approx(plain[turns > 64], rel=1e-12) and yarn[turns < 0.5] * 4.0 == pytest.approx(plain[turns < 0.5], rel=1e-12)
    assert np.all(yarn <= plain * (1 + 1e-12)) and np.all(yarn * 4.0 >= plain * (1 - 1e-12))
    assert _radians(2, scaling="ntk", factor=2.0)[0] == pytest.approx([1.0])


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=130), dict(rot_dim=64, scaling="other"), dict(rot_dim=64, base=1.0),
                                dict(rot_dim=64, base=math.inf), dict(rot_dim=64, scaling="linear", factor=0.5),
                                dict(rot_dim=64, scaling="yarn", factor=2.0, beta_fast=1.0, beta_slow=2.0), dict(rot_dim=64, scaling="yarn", factor=2.0, original_len=0)])
def test_frequencies_refused(kw):
    with pytest.raises(ValueError):
        B.rope_frequencies(device="cpu", **kw)


def test_layout_and_type_names_are_checked():
    with pytest.raises(ValueError):
        B.rope(None, None, None, None, layout="interleaved")
    with pytest.raises(ValueError):
        B.prompt_attn(None, None, None, None, out_dtype="f16")


# ------------------------------------------------------------- the oracle's definitions

def test_oracle_assigns_in_order_until_the_pool_is_empty():
    table = np.full((4, 4), -1, np.int32)
    table[1, 0] = 9
    free = np.array([5, 6, 7, 8], np.int32)
    # 17 new tokens: 2 pages; 3 more in a page that is there; 3 pages, of which 2 are left; 16: 1, but the pool is closed
    t, new, slots, pos, left, flags = C.page_assign([0, 4, 0, 0], [1, 18, 21, 55, 71], table, free, 4, 16, 75, 20)
    assert t.tolist() == [[8, 7, -1, -1], [9, -1, -1, -1], [-1] * 4, [-1] * 4]
    assert new.tolist() == [17, 7, 0, 0] and left == 2 and flags == 0x1000
    assert slots[0] == -1 and slots[1:17].tolist() == list(range(128, 144)) and slots[17] == 112 and slots[18:21].tolist() == [148, 149, 150]
    assert np.all(slots[21:] == -1) and pos[1:18].tolist() == list(range(17)) and pos[18:21].tolist() == [4, 5, 6] and np.all(pos[71:] == 0)


def test_oracle_release_undoes_an_assignment():
    rng = np.random.default_rng(0)
    free = rng.permutation(40).astype(np.int32)
    table = np.full((3, 12), -1, np.int32)
    t, new, *_, left, _ = C.page_assign([0, 0, 0], [0, 100, 101, 150], table, free, 40, 16, 150, 40)
    back, top, flags = C.page_release(new, [0, 0, 0], t, free, left, 16, 40)
    assert top == 40 and flags == 0 and sorted(back) == list(range(40))
    back, top, flags = C.page_release(new, [33, 1, 99], t, free, left, 16, 40)
    assert top == left + 7 - 3 and back[left:top].tolist() == t[0, 3:7].tolist()


def test_oracle_rope_closed_forms():
    x = np.random.default_rng(1).standard_normal((3, 2, 8))
    w = np.array([math.pi / 2, math.pi])
    y = C.rope(x, [0, 1, 2], w, True, scale=2.0)
    assert np.allclose(y[0, :, :4], 2 * x[0, :, :4]) and np.array_equal(y[..., 4:], x[..., 4:])
    assert np.allclose(y[1, :, 0], -2 * x[1, :, 2]) and np.allclose(y[1, :, 2], 2 * x[1, :, 0]) and np.allclose(y[1, :, 1], -2 * x[1, :, 1])
    z = C.rope(x, [0, 1, 2], w, False)
    assert np.allclose(z[1, :, 0], -x[1, :, 1]) and np.allclose(z[1, :, 1], x[1, :, 0]) and np.allclose(C.rope(z, [0, 1, 2], w, False, inverse=True), x)


def test_oracle_prompt_closed_forms():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((7, 4, 16)), rng.standard_normal((7, 2, 16)), rng.standard_normal((7, 2, 16))
    out, lse, mag, _ = C.prompt_attn(0 * q, k, v, [1, 4, 4, 6], 0.25)
    assert np.allclose(out[1], v[1].repeat(2, 0)) and np.allclose(out[3], v[1:4].mean(0).repeat(2, 0)) and np.allclose(out[5], v[4:6].mean(0).repeat(2, 0))
    assert np.allclose(lse[3], math.log(3)) and np.all(out[0] == 0) and np.all(out[6] == 0) and np.all(mag >= np.abs(out) - 1e-12)
    far = k.copy()
    far[3:] = np.nan
    assert np.allclose(C.prompt_attn(q, k, v, [0, 3], 0.25)[0][:3], C.prompt_attn(q, far, v, [0, 3], 0.25)[0][:3])
