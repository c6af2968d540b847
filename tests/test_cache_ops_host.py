"""Refusals of the cache operators (checked before any device is touched: the pointers are
never dereferenced, and valid calls without work enqueue nothing), and the oracle's definitions
against closed forms."""
import ctypes

import numpy as np
import pytest

from oracle import cache_ops as C
from paged_fp8_kv_04_gb300 import binding as B
from paged_fp8_kv_04_gb300 import build as libbuild
from paged_fp8_kv_04_gb300 import synth

OK, INVALID, UNSUP, CAP, RAGGED, ALIGN, CUDA, DEVDATA, WS = range(9)


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.lib()


def _fill(cls, base, over):
    a = cls()
    addr = 0x100000000
    for name, kind in cls._fields_:
        if kind is ctypes.c_void_p:
            addr += 0x10000000
            setattr(a, name, addr)
    for k, v in {**base, **over}.items():
        setattr(a, k, v)
    return a


MASS = dict(num_pages=64, num_seqs=0, num_rows=0, num_kv_heads=1, group_size=16, head_dim=128, page_size=128,
            kv_dtype=0, scale_mode=2, block_table_stride=8, mass_stride=1024, max_q_len=1, sm_scale=0.088, decay=1.0)


@pytest.mark.parametrize("over,want", [
    (dict(), OK), (dict(reserved=1), INVALID), (dict(num_seqs=-1), INVALID), (dict(num_rows=-1), INVALID),
    (dict(max_q_len=0), INVALID), (dict(max_q_len=65), UNSUP), (dict(max_q_len=64), OK),
    (dict(num_seqs=4097), UNSUP), (dict(group_size=8), UNSUP), (dict(head_dim=64), UNSUP),
    (dict(page_size=256), UNSUP), (dict(num_kv_heads=0), INVALID), (dict(num_kv_heads=65), UNSUP),
    (dict(kv_dtype=2), INVALID), (dict(kv_dtype=1), UNSUP), (dict(kv_dtype=1, scale_mode=0), OK),
    (dict(scale_mode=0), UNSUP), (dict(scale_mode=1, k_scale=None, k_scale_scalar=0.5), OK),
    (dict(scale_mode=1, k_scale_scalar=float("inf")), INVALID), (dict(scale_mode=1, k_scale_scalar=-1.0), INVALID),
    (dict(k_scale=None), INVALID), (dict(sm_scale=0.0), INVALID), (dict(sm_scale=float("nan")), INVALID),
    (dict(decay=-0.5), INVALID), (dict(decay=1.5), INVALID), (dict(decay=float("nan")), INVALID),
    (dict(mass=None), INVALID), (dict(mass=None, decay=0.0), OK), (dict(mass_out=None), INVALID),
    (dict(lse=None), INVALID), (dict(q=None), INVALID), (dict(block_table_stride=0), INVALID),
    (dict(mass_stride=0), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=1 << 25), CAP),
    (dict(q=0x100000008), ALIGN), (dict(k_cache=0x100000004), ALIGN), (dict(k_scale=0x100000004), ALIGN),
    (dict(lse=0x100000002), ALIGN), (dict(mass_out=0x100000002), ALIGN), (dict(status=None), OK),
    (dict(mass=0x900000000, mass_out=0x900000000), OK),
    (dict(num_seqs=2, num_rows=0, mass=0x900000000, mass_out=0x900000010), INVALID),
])
def test_attn_mass_refusals(lib, over, want):
    assert lib.pa_attn_mass(ctypes.byref(_fill(B.AttnMassArgs, MASS, over)), None) == want
    assert lib.pa_attn_mass(None, None) == INVALID


SELECT = dict(num_seqs=0, num_kv_heads=1, mass_stride=1024, budget=128, keep_first=4, keep_recent=64)


@pytest.mark.parametrize("over,want", [
    (dict(), OK), (dict(reserved=1), INVALID), (dict(num_seqs=-1), INVALID), (dict(num_seqs=65536), UNSUP),
    (dict(num_kv_heads=0), INVALID), (dict(num_kv_heads=65), UNSUP), (dict(mass_stride=0), INVALID),
    (dict(mass_stride=2**30 + 1), UNSUP), (dict(num_seqs=1024, num_kv_heads=64), UNSUP),
    (dict(budget=0), INVALID), (dict(keep_first=-1), INVALID), (dict(keep_recent=-1), INVALID),
    (dict(keep_first=64, keep_recent=65), INVALID), (dict(keep_first=64, keep_recent=64), OK),
    (dict(keep_first=2**31 - 1, keep_recent=2**31 - 1), INVALID), (dict(mass=None), INVALID),
    (dict(keep=None), INVALID), (dict(new_lens=0x100000000, context_lens=0x100000000), INVALID),
    (dict(mass=0x100000002), ALIGN), (dict(keep=0x100000001), ALIGN), (dict(status=None), OK),
])
def test_evict_select_refusals(lib, over, want):
    assert lib.pa_evict_select(ctypes.byref(_fill(B.EvictSelectArgs, SELECT, over)), None) == want
    assert lib.pa_evict_select(None, None) == INVALID


COMPACT = dict(num_pages=64, num_seqs=0, num_kv_heads=1, head_dim=128, page_size=128, kv_dtype=0, scale_mode=2,
               keep_stride=128, block_table_stride=8, dst_block_table_stride=4, mass_stride=1024, mass_out_stride=256)


@pytest.mark.parametrize("over,want", [
    (dict(), OK), (dict(reserved=1), INVALID), (dict(num_seqs=-1), INVALID), (dict(num_seqs=65536), UNSUP),
    (dict(head_dim=64), UNSUP), (dict(page_size=8), UNSUP), (dict(scale_mode=0), UNSUP), (dict(kv_dtype=5), INVALID),
    (dict(kv_dtype=1, scale_mode=0, k_scale=None, v_scale=None), OK), (dict(keep_stride=0), INVALID),
    (dict(block_table_stride=0), INVALID), (dict(dst_block_table_stride=0), INVALID), (dict(v_scale=None), INVALID),
    (dict(keep=None), INVALID), (dict(num_pages=1 << 25), CAP), (dict(mass_out=None), INVALID),
    (dict(mass=None, mass_out=None), OK), (dict(mass_out_stride=0), INVALID),
    # in place the mass moves in its own rows; into other pages it must not overlap them
    (dict(dst_block_table=None), INVALID),
    (dict(dst_block_table=None, dst_block_table_stride=0, mass=0x900000000, mass_out=0x900000000, mass_out_stride=1024), OK),
    (dict(dst_block_table=None, mass=0x900000000, mass_out=0x900000000), INVALID),
    (dict(num_seqs=1, mass=0x900000000, mass_out=0x900000100), INVALID),
    (dict(k_cache=0x100000008), ALIGN), (dict(v_scale=0x100000002), ALIGN), (dict(dst_block_table=0x100000002), ALIGN),
    (dict(keep=0x100000002), ALIGN),
])
def test_kv_compact_refusals(lib, over, want):
    assert lib.pa_kv_compact(ctypes.byref(_fill(B.KvCompactArgs, COMPACT, over)), None) == want
    assert lib.pa_kv_compact(None, None) == INVALID


BEAM = dict(logits_stride=1000, num_reqs=0, num_beams=4, vocab=1000, logits_dtype=0, eos_token=2)


@pytest.mark.parametrize("over,want", [
    (dict(), OK), (dict(reserved=1), INVALID), (dict(num_reqs=-1), INVALID), (dict(num_reqs=65536), UNSUP),
    (dict(num_beams=0), INVALID), (dict(num_beams=33), UNSUP), (dict(vocab=0), INVALID), (dict(logits_stride=999), INVALID),
    (dict(vocab=(1 << 24) + 1, logits_stride=1 << 25), UNSUP), (dict(logits_dtype=2), INVALID),
    (dict(eos_token=1000), INVALID), (dict(eos_token=-2), INVALID), (dict(eos_token=-1), INVALID),
    (dict(eos_token=-1, finished=None), OK), (dict(length_penalty=-1.0), INVALID),
    (dict(length_penalty=float("inf")), INVALID), (dict(lengths=None), INVALID),
    (dict(lengths=None, lengths_out=None), OK), (dict(lengths=None, lengths_out=None, length_penalty=1.0), INVALID),
    (dict(finished_out=None, lengths_out=None), OK), (dict(logits=None), INVALID), (dict(parents=None), INVALID),
    (dict(logits=0x100000001), ALIGN), (dict(logits=0x100000002), OK),
    (dict(logits=0x100000002, logits_dtype=1), ALIGN), (dict(tokens=0x100000002), ALIGN),
])
def test_beam_select_refusals(lib, over, want):
    assert lib.pa_beam_select(ctypes.byref(_fill(B.BeamSelectArgs, BEAM, over)), None) == want
    assert lib.pa_beam_select(None, None) == INVALID


REORDER = dict(num_pages=64, num_states=0, num_reqs=0, num_beams=4, num_kv_heads=1, head_dim=128, page_size=128,
               kv_dtype=0, scale_mode=2, block_table_stride=8)


def _states(a, *triples):
    a.num_states = len(triples)
    for i, (x, y, n) in enumerate(triples):
        a.state_in[i], a.state_out[i], a.state_bytes[i] = x, y, n
    return a


@pytest.mark.parametrize("over,want", [
    (dict(), OK), (dict(reserved=1), INVALID), (dict(num_reqs=-1), INVALID), (dict(num_beams=0), INVALID),
    (dict(num_beams=33), UNSUP), (dict(num_reqs=16384), UNSUP), (dict(num_states=5), INVALID),
    (dict(num_states=-1), INVALID), (dict(num_states=1), INVALID), (dict(head_dim=96), UNSUP),
    (dict(block_table_stride=0), INVALID), (dict(parents=None), INVALID), (dict(k_scale=None), INVALID),
    (dict(scale_mode=1, k_scale=None, v_scale=None), OK), (dict(k_cache=0x100000004), ALIGN),
    (dict(block_table_out=0x100000002), ALIGN), (dict(num_pages=1 << 25), CAP),
    (dict(num_reqs=1, block_table=0x900000000, block_table_out=0x900000040), INVALID),
])
def test_beam_reorder_refusals(lib, over, want):
    assert lib.pa_beam_reorder(ctypes.byref(_fill(B.BeamReorderArgs, REORDER, over)), None) == want
    assert lib.pa_beam_reorder(None, None) == INVALID


def test_beam_reorder_state_overlaps(lib):
    call = lambda reqs, *s: lib.pa_beam_reorder(ctypes.byref(_states(_fill(  # noqa: E731
        B.BeamReorderArgs, dict(REORDER, num_reqs=reqs), {}), *s)), None)
    x = 0x900000000
    assert call(0, (x, x + 4096, 64)) == OK
    assert call(0, (x, x + 4096, 0)) == INVALID
    assert call(1, (x, x, 64)) == INVALID                                     # in place
    assert call(1, (x, x + 128, 64)) == INVALID                               # in and out share rows
    assert call(1, (x, x + 4096, 64), (x + 8192, x + 4096, 64)) == INVALID    # two outputs share
    assert call(1, (x, x + 4096, 64), (x + 4096, x + 8192, 64)) == INVALID    # one's output is another's input


# Outputs that share bytes with what other CTAs of the call read or write: refused before any device is touched.

X = 0x900000000


@pytest.mark.parametrize("over", [
    dict(lse=X, mass_out=X + 8), dict(q=X, mass_out=X + 2 * 16 * 256 - 4), dict(context_lens=X + 4096, mass_out=X),
    dict(cu_seqlens_q=X, mass_out=X + 8), dict(block_table=X, mass_out=X + 60),
])
def test_attn_mass_refuses_overlaps(lib, over):
    assert lib.pa_attn_mass(ctypes.byref(_fill(B.AttnMassArgs, dict(MASS, num_seqs=2, num_rows=2), over)), None) == INVALID


@pytest.mark.parametrize("over", [
    dict(context_lens=X, new_lens=X), dict(context_lens=X, new_lens=X + 4), dict(context_lens=X + 28, new_lens=X),
    dict(mass=X, keep=X), dict(mass=X, keep=X + 8 * 4096 - 4), dict(mass=X + 8 * 512 - 4, keep=X), dict(mass=X, new_lens=X + 64),
    dict(context_lens=X, keep=X + 16), dict(keep=X, new_lens=X + 8 * 512 - 4),
])
def test_evict_select_refuses_overlaps(lib, over):
    assert lib.pa_evict_select(ctypes.byref(_fill(B.EvictSelectArgs, dict(SELECT, num_seqs=8), over)), None) == INVALID


@pytest.mark.parametrize("over", [
    dict(mass_out=X, keep=X + 8), dict(mass_out=X, new_lens=X + 2048 - 4), dict(mass_out=X, block_table=X),
    dict(mass_out=X + 12, dst_block_table=X),
    dict(dst_block_table=None, mass=X, mass_out=X, mass_out_stride=1024, keep=X + 8188),
])
def test_kv_compact_refuses_overlaps(lib, over):
    assert lib.pa_kv_compact(ctypes.byref(_fill(B.KvCompactArgs, dict(COMPACT, num_seqs=2), over)), None) == INVALID


@pytest.mark.parametrize("over", [
    dict(scores=X, scores_out=X + 4), dict(scores=X + 16, scores_out=X), dict(finished=X, finished_out=X + 1),
    dict(lengths=X, lengths_out=X + 16), dict(tokens=X, parents=X), dict(tokens=X, scores=X + 44), dict(parents=X, lengths=X),
    dict(scores_out=X, finished=X + 8), dict(tokens=X, finished_out=X), dict(lengths_out=X, scores=X), dict(scores_out=X, lengths_out=X),
    dict(logits=X, tokens=X + 11 * 2000 + 1996), dict(logits=X, scores_out=X), dict(logits=X, finished_out=X + 5000),
    dict(logits=X, lengths_out=X + 8, logits_stride=1 << 62),
])
def test_beam_select_refuses_overlaps(lib, over):
    assert lib.pa_beam_select(ctypes.byref(_fill(B.BeamSelectArgs, dict(BEAM, num_reqs=3), over)), None) == INVALID


@pytest.mark.parametrize("over", [
    dict(parents=X, block_table_out=X), dict(context_lens=X + 96, block_table_out=X), dict(block_table=X, block_table_out=X + 4),
])
def test_beam_reorder_refuses_overlaps(lib, over):
    assert lib.pa_beam_reorder(ctypes.byref(_fill(B.BeamReorderArgs, dict(REORDER, num_reqs=1), over)), None) == INVALID


@pytest.mark.parametrize("name", ["parents", "context_lens", "block_table", "block_table_out"])
def test_beam_reorder_refuses_states_over_its_tables(lib, name):
    call = lambda s: lib.pa_beam_reorder(ctypes.byref(_states(_fill(  # noqa: E731
        B.BeamReorderArgs, dict(REORDER, num_reqs=1), {name: X}), s)), None)
    assert call((X + (1 << 20), X + 8, 64)) == INVALID
    if name == "block_table_out":
        assert call((X + 124, X + (1 << 20), 64)) == INVALID


# ------------------------------------------------------------------------ the oracle

def test_oracle_mass_sums_to_the_rows():
    """Every query row spreads a mass of one per head over its attended positions."""
    p = synth.make_problem(3, num_seqs=3, context_lens=[1, 40, 77], q_lens=[1, 3, 2], page_size=16, num_kv_heads=2)
    from oracle import oracle as O
    _, lse = O.decode(p)
    m, tol = C.attn_mass(p, lse, np.zeros((3, 2, 80), np.float32), 1.0)
    for r, ql in enumerate([1, 3, 2]):
        assert np.allclose(m[r].sum(-1), 16 * ql, rtol=1e-12)
    # 16 heads of weight <= 1, 128 additions of 2^-23, score magnitudes below 16: 16 * 2^-12
    assert tol.max() < 2.0 ** -8


def test_oracle_evict_select_closed_forms():
    mass = np.arange(20, dtype=np.float32).reshape(1, 1, 20)
    keep, new = C.evict_select(mass, [20], 6, 2, 1)
    assert keep[0, 0].tolist() == [0, 1, 16, 17, 18, 19] and new.tolist() == [6]
    keep, _ = C.evict_select(np.zeros((1, 1, 9), np.float32), [9], 4, 0, 1)
    assert keep[0, 0].tolist() == [0, 1, 2, 8]
    keep, new = C.evict_select(mass, [3], 6, 2, 1)
    assert keep[0, 0].tolist() == [0, 1, 2, -1, -1, -1] and new.tolist() == [3]


def test_oracle_beam_select_closed_forms():
    x = np.log(np.array([[[0.5, 0.3, 0.2], [0.1, 0.8, 0.1]]]))
    t, p, s, f, _ = C.beam_select(x, np.array([[0.0, np.log(0.5)]]))
    assert t.tolist() == [[0, 1]] and p.tolist() == [[0, 1]] and np.allclose(np.exp(s), [[0.5, 0.4]])
    t, p, s, f, ln = C.beam_select(x, np.array([[-1.0, -1.5]]), eos=2, finished=np.array([[1, 0]]),
                                   lengths=np.array([[4, 4]]), penalty=0.0)
    assert t.tolist() == [[2, 1]] and p.tolist() == [[0, 1]] and f.tolist() == [[1, 0]] and ln.tolist() == [[4, 5]]
    t, p, s, _, _ = C.beam_select(np.zeros((1, 4, 2)), np.array([[0.0, -np.inf, -np.inf, -np.inf]]))
    assert t.tolist() == [[0, 1, 0, 1]] and p.tolist() == [[0, 0, 1, 1]]


def test_oracle_beam_select_orders_equal_ranks_by_beam_and_token():
    lowest = np.finfo(np.float32).min
    x = np.tile(np.array([0.0, 1.0, 2.0]), (1, 3, 1))
    t, p, _, _, _ = C.beam_select(x, np.full((1, 3), lowest))
    assert t.tolist() == [[0, 1, 2]] and p.tolist() == [[0, 0, 0]]
    t, p, _, _, _ = C.beam_select(x[..., :2], np.array([[lowest, lowest, -1.0]]))
    assert t.tolist() == [[1, 0, 0]] and p.tolist() == [[2, 2, 0]]
    t, p, _, _, _ = C.beam_select(x, np.array([[-5.0, -1.0, -2.0]]), eos=1, finished=np.ones((1, 3)), lengths=np.array([[5, 1, 1]]),
                                  penalty=1.0)
    assert t.tolist() == [[1, 1, 1]] and p.tolist() == [[0, 1, 2]]


def test_oracle_beam_reorder_by_hand():
    """Parents 1 1 0 1 of four beams with 10 tokens on pages of 4: beams 2 and 3 have no child."""
    table = np.array([[0, 1, 10, 90], [0, 2, 11, 91], [0, 3, 12, 92], [0, 4, 13, 93]], np.int32)
    x = np.arange(100, dtype=np.float32)[:, None, None] * np.ones((1, 1, 4), np.float32)
    t, (y,) = C.beam_reorder(np.array([[1, 1, 0, 1]]), [10] * 4, table, [x], 4)
    assert t.tolist() == [[0, 2, 11, 90], [0, 2, 12, 91], [0, 1, 10, 92], [0, 2, 13, 93]]
    assert y[12, 0].tolist() == [11, 11, 12, 12] and y[13, 0].tolist() == [11, 11, 13, 13]
    assert np.array_equal(np.delete(y, [12, 13], 0), np.delete(x, [12, 13], 0))


# ------------------------------------------------- the torch side, which refuses on the CPU

@pytest.fixture(scope="module")
def built():
    libbuild.build_all()
    return B.torch_module()


def test_the_torch_module_refuses_wrong_arguments(built):
    import torch
    mass, lens = torch.zeros(2, 1, 8), torch.zeros(2, dtype=torch.int32)
    k = torch.zeros(4, 1, 16, 128, dtype=torch.uint8)
    table = torch.zeros(2, 2, dtype=torch.int32)
    keep = torch.zeros(2, 1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="expected a CUDA device"):
        B.evict_select(mass, lens, budget=4)
    with pytest.raises(ValueError, match="expected a CUDA device"):
        B.kv_compact(keep, lens, table, k, k.clone())
    with pytest.raises(ValueError, match="expected a CUDA device"):
        B.beam_select(torch.zeros(1, 2, 9), torch.zeros(1, 2))
    with pytest.raises(ValueError, match="expected a CUDA device"):
        B.beam_reorder(torch.zeros(1, 2, dtype=torch.int32), lens, table, table.clone(), k, k.clone())
    with pytest.raises(ValueError, match="expected a CUDA device"):
        B.attn_mass(torch.zeros(2, 16, 128).bfloat16(), k, table, lens, torch.zeros(3, dtype=torch.int32), torch.zeros(2, 16), mass,
                    max_q_len=1)
    with pytest.raises(TypeError, match="expected a tensor"):
        B.evict_select(np.zeros((2, 1, 8), np.float32), lens, budget=4)
    with pytest.raises(TypeError):
        built.evict_select(mass, lens)


def test_torch_module_missing_fails_loudly(built, monkeypatch, tmp_path):
    """Without the compiled module the calls raise; there is no other path."""
    import torch
    monkeypatch.setattr(B, "_module", None)
    monkeypatch.setattr(libbuild, "torch_module_path", lambda: str(tmp_path / "pa_torch.so"))
    with pytest.raises(ImportError):
        B.evict_select(torch.zeros(2, 1, 8), torch.zeros(2, dtype=torch.int32), budget=4)


def test_the_torch_module_belongs_to_one_interpreter_and_one_set_of_flags(built, monkeypatch, tmp_path):
    """Another Python finds no module of its own rather than this one's, and changed flags rebuild both libraries."""
    import os
    import sysconfig
    mine = libbuild.torch_module_path()
    assert os.path.exists(mine) and libbuild.up_to_date(mine, libbuild._torch_module_inputs())
    assert os.path.abspath(libbuild.__file__) in libbuild._torch_module_inputs()
    assert os.path.abspath(libbuild.__file__) in libbuild._inputs()
    old = tmp_path / "old.so"
    old.write_bytes(b"")
    os.utime(old, (0, 0))
    assert not libbuild.up_to_date(str(old)) and not libbuild.up_to_date(str(old), [libbuild.__file__])
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda k: ".cpython-399-other.so" if k == "EXT_SUFFIX" else real(k))
    assert libbuild.torch_module_path() != mine and not os.path.exists(libbuild.torch_module_path())
