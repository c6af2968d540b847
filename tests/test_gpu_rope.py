"""pa_rope against its definition in 64 bits (needs a GPU).

Bounds.  A turned element is a c - b s in fp32: cosine and sine are CUDA's sincospif, within 2 units of their last place
(2^-22 of themselves) and 2^-25 from the angle's rounding to 24 bits; the scale, the two products and the
sum add a rounding of 2^-24 each, so the fp32 value is within 2^-21 (|a| + |b|) |scale| of the exact one.  An output
is that, rounded to its type: half a step, eps / 2 of its value."""
import math

import numpy as np
import pytest
import torch

from cache_util import dev
from oracle import prompt_ops as C
from paged_fp8_kv_04_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _f64(x):
    return x.double().cpu().numpy()


def _radians(freqs):
    return (freqs.cpu().numpy().astype(np.uint64).astype(np.longdouble) / np.longdouble(2) ** 64) * 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))


def _check(got, x, positions, freqs, half, inverse=False, scale=1.0, out_type=None):
    ref = C.rope(_f64(x), positions, _radians(freqs), half, inverse, scale)
    n = freqs.numel()
    a = np.abs(_f64(x))[..., :2 * n]
    both = a[..., :n] + a[..., n:] if half else a[..., 0::2] + a[..., 1::2]
    terms = np.concatenate([both, both], -1) if half else both.repeat(2, -1)
    tol = np.zeros_like(ref)
    tol[..., :2 * n] = 2.0 ** -21 * abs(scale) * terms
    tol[..., :2 * n] += torch.finfo(x.dtype).eps / 2 * (np.abs(ref[..., :2 * n]) + tol[..., :2 * n])
    err = np.abs(_f64(got) - ref)
    assert np.all(err <= tol), (float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(err > tol)[:3])


def _rows(g, T, heads, dtype):
    return torch.randn(T, heads, 128, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("rot", [128, 64, 96, 32, 16, 8, 2, 6, 34, 126])
def test_rope(rot, layout, dtype):
    g = torch.Generator(device="cuda").manual_seed(rot)
    freqs, _ = B.rope_frequencies(rot)
    for T, hq, hk in ((1, 16, 1), (7, 5, 3), (2055, 2, 1)):
        q, k = _rows(g, T, hq, dtype), _rows(g, T, hk, dtype)
        pos = torch.randint(0, 100000, (T,), generator=g, device="cuda", dtype=torch.int32)
        qo, ko = torch.full_like(q, math.nan), torch.full_like(k, math.nan)
        a, b = B.rope(q, k, pos, freqs, layout=layout, q_out=qo, k_out=ko)
        assert a is qo and b is ko
        _check(qo, q, pos.cpu().numpy(), freqs, layout == "half")
        _check(ko, k, pos.cpu().numpy(), freqs, layout == "half")
        assert torch.equal(qo[..., rot:], q[..., rot:])
        inplace = q.clone()
        a, b = B.rope(inplace, None, pos, freqs, layout=layout)
        assert a is inplace and b is None and torch.equal(inplace, qo)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rope_every_number_of_pairs(layout, dtype):
    """All accesses' widths: every rotation dimension, in place and not, at rows that are 16, 8, 4 and 2 bytes aligned."""
    g = torch.Generator(device="cuda").manual_seed(6)
    T, hq = 9, 3
    pos = torch.randint(-500, 70000, (T,), generator=g, device="cuda", dtype=torch.int32)
    for rot in range(2, 130, 2):
        freqs, _ = B.rope_frequencies(rot)
        for shift in (0, 4, 2, 1):
            buf = torch.randn(T, hq * 128 + 8, generator=g, device="cuda").to(dtype)
            q = buf[:, shift:shift + hq * 128].unflatten(1, (-1, 128))
            out, _ = B.rope(q, None, pos, freqs, layout=layout, q_out=torch.full((T, hq, 128), math.nan, dtype=dtype, device="cuda"))
            _check(out, q, pos.cpu().numpy(), freqs, layout == "half")
            B.rope(q, None, pos, freqs, layout=layout)
            assert torch.equal(q, out), (rot, shift)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
def test_rope_of_stretched_contexts(scaling):
    g = torch.Generator(device="cuda").manual_seed(1)
    freqs, scale = B.rope_frequencies(128, base=1e6, scaling=scaling, factor=32.0, original_len=8192)
    q, pos = _rows(g, 100, 3, torch.float32), torch.randint(0, 262144, (100,), generator=g, device="cuda", dtype=torch.int32)
    out, _ = B.rope(q, None, pos, freqs, scale=scale, q_out=torch.empty_like(q))
    _check(out, q, pos.cpu().numpy(), freqs, True, scale=np.float32(scale).item())


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rope_of_far_and_negative_positions(layout):
    g = torch.Generator(device="cuda").manual_seed(2)
    pos = np.array([0, 1, -1, 2**24 + 1, 2**31 - 1, -2**31, 123456789, -777777], np.int32)
    freqs, _ = B.rope_frequencies(128, base=500000.0)
    freqs[5], freqs[6], freqs[7] = 2**62, -2**63, -1      # a quarter of a turn, half of one, the smallest step back
    q = _rows(g, len(pos), 2, torch.float32)
    out, _ = B.rope(q, None, dev(pos), freqs, layout=layout, q_out=torch.empty_like(q))
    # the reference's angle from exact integers
    turns = np.array([[(int(p) * int(f)) % 2**64 for f in freqs.cpu()] for p in pos], dtype=np.uint64).astype(np.float64) / 2.0**64
    z = np.exp(2j * math.pi * turns)[:, None]
    x, n = _f64(q), 64
    one, two = (np.arange(n), np.arange(n) + n) if layout == "half" else (2 * np.arange(n), 2 * np.arange(n) + 1)
    w = (x[..., one] + 1j * x[..., two]) * z
    terms = np.abs(x[..., one]) + np.abs(x[..., two])
    for at, ref in ((one, w.real), (two, w.imag)):
        assert np.all(np.abs(_f64(out)[..., at] - ref) <= (2.0**-21 + 2.0**-24) * terms)
    assert torch.equal(out[0], q[0])


def test_rope_quarter_turns_are_exact():
    freqs = torch.tensor([2**62], dtype=torch.int64, device="cuda")
    q = torch.randn(8, 1, 128, device="cuda")
    out, _ = B.rope(q, None, torch.arange(8, dtype=torch.int32, device="cuda"), freqs, layout="pairs", q_out=torch.empty_like(q))
    a, b = q[..., 0], q[..., 1]
    for p, (x, y) in enumerate([(a, b), (-b, a), (-a, -b), (b, -a)] * 2):
        assert torch.equal(out[p, :, 0], x[p]) and torch.equal(out[p, :, 1], y[p])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rope_on_views_of_one_buffer(layout, dtype):
    """Queries and keys as the projection left them: turned in place, and out of it; rows that begin off a 16-byte
    boundary; the values between them, and elements behind the head's turned part, as they were."""
    g = torch.Generator(device="cuda").manual_seed(3)
    freqs, _ = B.rope_frequencies(64)
    T, hq, hk = 37, 4, 2
    for shift, gap in ((0, 0), (1, 0), (8, 3), (8, 16)):
        wide = (hq + 2 * hk) * 128
        buf = torch.randn(T, shift + wide + gap, generator=g, device="cuda").to(dtype)
        view = lambda b: [x.unflatten(1, (-1, 128)) for x in b[:, shift:shift + wide].split([hq * 128, hk * 128, hk * 128], 1)]  # noqa: E731
        q, k, _ = view(buf)
        pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32)
        qo, ko = B.rope(q, k, pos, freqs, layout=layout, q_out=torch.empty(T, hq, 128, dtype=dtype, device="cuda"),
                        k_out=torch.empty(T, hk, 128, dtype=dtype, device="cuda"))
        _check(qo, q, pos.cpu().numpy(), freqs, layout == "half")
        _check(ko, k, pos.cpu().numpy(), freqs, layout == "half")
        turned = buf.clone()
        tq, tk, tv = view(turned)
        B.rope(tq, tk, pos, freqs, layout=layout)
        assert torch.equal(tq, qo) and torch.equal(tk, ko)
        want = buf.clone()
        wq, wk, _ = view(want)
        wq.copy_(qo)
        wk.copy_(ko)
        assert torch.equal(turned, want)


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rope_inverse_is_the_gradient(layout):
    """y = R x is linear, so the gradient of g . y is R^T g: what inverse gives.  Against the formula in 64 bits, against the
    rotation's differences, and back to where it came from."""
    g = torch.Generator(device="cuda").manual_seed(4)
    freqs, scale = B.rope_frequencies(48, scaling="yarn", factor=4.0)
    T = 19
    x, gy, h = (_rows(g, T, 3, torch.float32) for _ in range(3))
    pos = torch.randint(0, 9000, (T,), generator=g, device="cuda", dtype=torch.int32)
    turn = lambda t, **kw: B.rope(t, None, pos, freqs, layout=layout, scale=scale, q_out=torch.empty_like(t), **kw)[0]  # noqa: E731
    gx = turn(gy, inverse=True)
    _check(gx, gy, pos.cpu().numpy(), freqs, layout == "half", inverse=True, scale=np.float32(scale).item())
    # <g, R (x + h) - R x> = <R^T g, h>: each turned element within 2^-21 (|a| + |b|) scale and 2^-24 of its value, the
    # inputs' sum within 2^-24 of itself; all of it weighed by g and added up
    up = x + h
    left = ((turn(up).double() - turn(x).double()) * gy.double()).sum()
    right = (gx.double() * h.double()).sum()
    size = (gy.abs().double().amax(-1) * (up.abs() + x.abs() + h.abs()).double().sum(-1)).sum() * 2 * scale
    assert abs(float(left - right)) <= 2.0**-20 * float(size)
    back = turn(turn(x), inverse=True)[..., :48] / scale**2
    assert float((back - x[..., :48]).abs().max()) <= 2.0**-19 * float(2 * x.abs().max())


def test_rope_large_batches_and_many_heads():
    g = torch.Generator(device="cuda").manual_seed(5)
    freqs, _ = B.rope_frequencies(128)
    for T, hq, hk in ((4099, 16, 1), (33, 64, 64), (3, 300, 7)):
        q, k = _rows(g, T, hq, torch.bfloat16), _rows(g, T, hk, torch.bfloat16)
        pos = torch.randint(0, 131072, (T,), generator=g, device="cuda", dtype=torch.int32)
        qo, ko = B.rope(q, k, pos, freqs, q_out=torch.empty_like(q), k_out=torch.empty_like(k))
        rows = np.r_[0, T // 2, T - 1]
        _check(qo[rows], q[rows], pos.cpu().numpy()[rows], freqs, True)
        _check(ko[rows], k[rows], pos.cpu().numpy()[rows], freqs, True)
        one, _ = B.rope(q[rows].contiguous(), None, pos[rows].contiguous(), freqs)
        assert torch.equal(one, qo[rows])


def test_rope_without_tokens_and_on_a_stream():
    freqs, _ = B.rope_frequencies(128)
    q = torch.empty(0, 4, 128, device="cuda", dtype=torch.bfloat16)
    assert B.rope(q, q[:, :1], torch.empty(0, dtype=torch.int32, device="cuda"), freqs)[0] is q
    side = torch.cuda.Stream()
    x, pos = torch.randn(50, 4, 128, device="cuda"), torch.arange(50, dtype=torch.int32, device="cuda")
    want, out = B.rope(x, None, pos, freqs, q_out=torch.empty_like(x))[0], torch.zeros_like(x)
    torch.cuda.synchronize()
    B.rope(x, None, pos, freqs, q_out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_rope_refuses_wrong_tensors():
    freqs, _ = B.rope_frequencies(128)
    q, k, pos = torch.zeros(4, 2, 128, device="cuda"), torch.zeros(4, 1, 128, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: B.rope(q.half(), None, pos, freqs), lambda: B.rope(q, k.bfloat16(), pos, freqs), lambda: B.rope(q, k, pos.long(), freqs),
                lambda: B.rope(q, k, pos, freqs.double())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: B.rope(q[0], k, pos, freqs), lambda: B.rope(q, k[:3], pos, freqs), lambda: B.rope(q, k, pos[:3], freqs),
                lambda: B.rope(q.transpose(0, 1), None, pos[:2], freqs), lambda: B.rope(q, None, pos, freqs, k_out=k),
                lambda: B.rope(q, None, pos, freqs.repeat(2)), lambda: B.rope(q.expand(4, 2, 128)[:, :, ::2], None, pos, freqs),
                lambda: B.rope(q, k, pos.cpu(), freqs), lambda: B.rope(k.expand(4, 2, 128), None, pos, freqs)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: B.rope(q, k, pos, freqs[:0]), lambda: B.rope(q, k, pos, freqs, scale=math.nan), lambda: B.rope(q, k, pos, freqs, k_out=q[:, 1:]),
                lambda: B.rope(q[..., :64].contiguous(), None, pos, freqs)):
        with pytest.raises(B.PaError):
            bad()
