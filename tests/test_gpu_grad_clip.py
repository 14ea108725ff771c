"""GPU parity of grad_clip against binary64: sizes, alignments, dtypes, many
tensors, values whose squares leave binary32, infinities and NaN, in place
and into other tensors."""
import math

import numpy as np
import pytest
import torch

from fp4_precision_numerics_b200 import mxfp4
from tests.routing_ref import HALF_F32, f64, half_step

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def rand(n, seed, std=1.0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * std).to(dtype)


def check(tensors, max_norm, outs=None):
    """Squares may be added in binary32 within runs of at most 16 (each sum a
    rounding) and the square root halves the relative error; the norm and the
    coefficient are rounded once each, the products once more."""
    before = [f64(t) for t in tensors]
    norm = math.sqrt(sum(float((b ** 2).sum()) for b in before))
    gl = mxfp4.GradList(tensors, out=outs)
    got = mxfp4.grad_clip(gl, max_norm)
    assert abs(float(got) - norm) <= 10 * HALF_F32 * norm
    coef = max_norm / norm if norm > max_norm else 1.0
    for b, t, o in zip(before, tensors, tensors if outs is None else outs):
        want = b * coef
        tol = (12 * HALF_F32 if coef != 1.0 else 0.0) + (half_step(t.dtype) if coef != 1.0 else 0.0)
        assert np.all(abs(f64(o) - want) <= tol * abs(want) + (2.0 ** -134 if coef != 1.0 else 0.0))
        if outs is not None:
            assert np.array_equal(f64(t), b)
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sizes", [[1], [7, 1, 3], [16384, 16385, 16383], [1 << 20, 5, 0, 12345], [0], [3000001]])
def test_grad_clip(sizes, dtype):
    for ratio in (0.5, 2.0):
        for into in (False, True):
            ts = [rand(n, i + 1, 0.01, dtype) for i, n in enumerate(sizes)]
            outs = [torch.full_like(t, 9.0) for t in ts] if into else None
            check(ts, ratio * 0.01 * math.sqrt(max(1, sum(sizes))), outs)


def test_many_tensors_mixed_dtypes_and_alignments():
    base32, base16 = rand(400000, 1), rand(400000, 2, dtype=BF16)
    ts, at = [], 0
    for i in range(301):
        n = (i * 37) % 611
        ts.append((base32 if i % 3 else base16)[at:at + n])    # odd starts: not 16-byte aligned
        at += n + i % 5
    check(ts, 3.0)
    o = [torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:] for t in ts]
    check(ts, 1.0, o)


def test_shapes_scalars_and_the_same_bits():
    t = [rand((33, 77), 1), rand((), 2), rand((2, 3, 5), 3, dtype=BF16)]
    a = mxfp4.grad_clip(mxfp4.GradList(t), float("inf"))
    for _ in range(3):
        assert torch.equal(a, mxfp4.grad_clip(t, float("inf")))
    assert abs(float(a) - math.sqrt(sum(float((f64(x) ** 2).sum()) for x in t))) <= 10 * HALF_F32 * float(a)


@pytest.mark.parametrize("std", [1e-30, 1e-22, 1e18, 1e25])
def test_squares_outside_binary32(std):
    t = [rand(100003, 5, std), rand(17, 6, std)]
    check(t, 0.5 * std)
    check([rand(1000, 5, 1e-25), rand(50000, 6, 1e10), rand(33, 7, 1e24)], 1.0)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(bad):
    for outs in (False, True):
        t = [rand(5000, 1), rand(40, 2, dtype=BF16)]
        t[0][4321] = bad
        before = [x.clone() for x in t]
        o = [torch.zeros_like(x) for x in t] if outs else None
        n = float(mxfp4.grad_clip(mxfp4.GradList(t, out=o), 1e-3))
        assert math.isnan(n) if math.isnan(bad) else n == math.inf
        for b, x in zip(before, o if outs else t):
            assert torch.equal(b.view(torch.int32 if b.dtype == F32 else torch.int16),
                               x.view(torch.int32 if b.dtype == F32 else torch.int16))


def test_zero_gradients():
    t = [torch.zeros(70000, device="cuda"), torch.zeros(3, device="cuda", dtype=BF16)]
    assert float(mxfp4.grad_clip(t, 1.0)) == 0.0
    assert float(t[0].abs().max()) == 0.0


def test_beyond_32_bit_offsets():
    n = (1 << 31) + 12345
    t = torch.zeros(n, dtype=BF16, device="cuda")
    t[-3:] = 3.0
    t[5] = 4.0
    norm = float(mxfp4.grad_clip([t], 1.0))
    want = math.sqrt(16 + 27)
    assert abs(norm - want) <= 10 * HALF_F32 * want
    c = 1.0 / want
    assert abs(float(t[-1]) - 3 * c) <= half_step(BF16) * 3 * c * 1.01 and abs(float(t[5]) - 4 * c) <= half_step(BF16) * 4 * c * 1.01
    assert float(t[6:-3].abs().max()) == 0.0


def test_graph_and_stream():
    t = [rand(100000, 1), rand(333, 2, dtype=BF16)]
    o = [torch.empty_like(x) for x in t]
    gl = mxfp4.GradList(t, out=o)
    want = mxfp4.grad_clip(gl, 2.0)
    keep = [x.clone() for x in o]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = mxfp4.grad_clip(gl, 2.0)
    for x in o + [got]:
        x.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(keep, o))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n = mxfp4.grad_clip(gl, 2.0, stream=s)
    s.synchronize()
    assert torch.equal(n, want)


def test_refusals():
    a, b = rand(100, 1), rand(100, 2)
    with pytest.raises(ValueError):
        mxfp4.GradList([a, a])                        # the same gradient twice
    with pytest.raises(ValueError):
        mxfp4.GradList([a[:60], a[50:]])              # overlapping views
    with pytest.raises(ValueError):
        mxfp4.GradList([a, b], out=[b, torch.empty_like(a)])      # an output over another gradient
    with pytest.raises(ValueError):
        mxfp4.GradList([a], out=[b[:50]])
    with pytest.raises(ValueError):
        mxfp4.GradList([a.view(10, 10).t()])
    with pytest.raises(ValueError):
        mxfp4.GradList([a, b.half()])
    mxfp4.GradList([a, b], out=[torch.empty_like(a), b])          # some in place, some not
    with pytest.raises(mxfp4.MXFP4Error):
        mxfp4.grad_clip([a], 0.0)
    with pytest.raises(mxfp4.MXFP4Error):
        mxfp4.grad_clip([a], float("nan"))
    gl = mxfp4.GradList([b])
    b.untyped_storage().resize_(0)
    with pytest.raises(ValueError):
        mxfp4.grad_clip(gl, 1.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [8, 16, 32, 33, 256, 5000, 300000])
def test_the_norm_is_off_by_one_rounding(n, dtype):
    """Squares are exact in binary64 and added there (n roundings of 2^-53), so
    that what is left is the norm's own rounding, half a step of binary32."""
    for seed in range(40 if n < 1000 else 4):
        for std in (1.0, 1e-3, 1e15):
            t = [rand(n, 100 * seed + n, std, dtype)]
            want = math.sqrt(float((f64(t[0]) ** 2).sum()))
            got = float(mxfp4.grad_clip(t, float("inf")))
            assert abs(got - want) <= HALF_F32 * want * (1 + 2.0 ** -20)


def test_a_norm_beyond_binary32_leaves_the_gradients():
    """Finite gradients whose norm reads as infinite are not scaled."""
    for n in (16, 1 << 20):
        for outs in (False, True):
            t = [torch.full((n,), 2e38, device="cuda"), rand(40, 2, dtype=BF16)]
            before = [x.clone() for x in t]
            o = [torch.zeros_like(x) for x in t] if outs else None
            assert float(mxfp4.grad_clip(mxfp4.GradList(t, out=o), 1.0)) == math.inf
            assert all(torch.equal(b, x) for b, x in zip(before, o if outs else t))


def test_a_list_whose_tensor_was_replaced_is_refused():
    """Not scaled in the place where its elements used to be."""
    for into in (False, True):
        a, b = rand(100, 1), rand(100, 2)
        outs = [torch.empty_like(a), torch.empty_like(b)] if into else None
        gl = mxfp4.GradList([a, b], out=outs)
        old = b.detach()
        before = old.clone()
        b.data = rand(100, 3)
        with pytest.raises(ValueError):
            mxfp4.grad_clip(gl, 0.1)
        b.set_(old)                      # the elements that the list was made for
        mxfp4.grad_clip(gl, 0.1)
        assert torch.equal(b, before) is into
        if into:
            outs[0].data = torch.empty_like(a)
            with pytest.raises(ValueError):
                mxfp4.grad_clip(gl, 0.1)
