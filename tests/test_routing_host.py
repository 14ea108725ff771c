"""CPU checks of the routing calls: host-side refusals of the C entry points
(fake pointers, nothing is dereferenced), the sizes they report, the checks of
the tensor helpers, and the plain forms the GPU tests compare with."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from fp4_precision_numerics_b200 import build, mxfp4, synth
from tests import routing_ref as ref

INV, SHAPE, ALIGN = -1, -2, -3


@pytest.fixture(scope="module")
def L():
    build.build()
    return mxfp4.lib()


def rp(score=0, top_k=2, groups=1, top_groups=1, best=1, renorm=1, scale=1.0):
    return mxfp4.RouteParams(score, top_k, groups, top_groups, best, renorm, scale)


def test_route_refusals(L):
    def call(logits=16, dtype=0, T=4, E=8, ld=8, bias=None, mask=None, p=None, ids=16, w=16):
        return L.mxfp4_route(logits, dtype, T, E, ld, bias, mask, ctypes.byref(p or rp()), ids, w, None)
    assert L.mxfp4_route(16, 0, 4, 8, 8, None, None, None, 16, 16, None) == INV
    assert call(dtype=5) == INV and call(p=rp(score=2)) == INV and call(E=0) == INV and call(ld=7) == INV
    assert call(T=-1) == INV and call(logits=None) == INV and call(ids=None) == INV and call(w=None) == INV
    assert call(E=1025, ld=1025) == SHAPE and call(T=1 << 31) == SHAPE
    assert call(p=rp(top_k=0)) == INV and call(p=rp(top_k=9)) == INV
    assert call(E=64, ld=64, p=rp(top_k=33)) == SHAPE
    assert call(p=rp(groups=3)) == INV and call(p=rp(groups=0)) == INV
    assert call(E=66, ld=66, p=rp(groups=33, top_groups=33)) == SHAPE
    assert call(p=rp(groups=4, top_groups=5)) == INV and call(p=rp(groups=4, top_groups=0)) == INV
    assert call(p=rp(best=3)) == INV and call(p=rp(best=0)) == INV
    assert call(p=rp(top_k=3, groups=4)) == INV            # one group of two experts for three slots
    assert call(p=rp(scale=float("nan"))) == INV and call(p=rp(scale=float("inf"))) == INV
    assert call(logits=17) == ALIGN and call(dtype=1, logits=18) == ALIGN
    assert call(ids=18) == ALIGN and call(w=18) == ALIGN and call(bias=18) == ALIGN
    assert call(T=0, logits=None, ids=None, w=None) == 0   # nothing to do


def test_route_bwd_refusals(L):
    def call(logits=16, dtype=1, T=4, E=8, ld=8, ids=16, dw=16, p=None, out=16, ldd=8):
        return L.mxfp4_route_bwd(logits, dtype, T, E, ld, ids, dw, ctypes.byref(p or rp()), out, ldd, None)
    assert call(ldd=7) == INV and call(ids=None) == INV and call(dw=None) == INV and call(out=None) == INV
    assert call(logits=None) == INV and call(p=rp(top_k=9)) == INV and call(E=1025, ld=1025, ldd=1025) == SHAPE
    assert call(out=18) == ALIGN and call(dw=18) == ALIGN and call(T=0, logits=None) == 0
    assert "route_bwd" in mxfp4.last_error()


def test_expert_plan_refusals(L):
    def call(ids=16, T=4, k=2, E=8, align=128, rows=1024, fill=0, c=16, o=16, r=16, s=16, ws=16, wb=1 << 20):
        return L.mxfp4_expert_plan(ids, T, k, E, align, rows, fill, c, o, r, s, ws, wb, None)
    assert call(T=-1) == INV and call(k=0) == INV and call(E=0) == INV and call(k=33) == SHAPE
    assert call(E=1025, rows=1 << 20) == SHAPE and call(T=1 << 30, k=4) == SHAPE
    assert call(align=0) == INV and call(align=96) == INV and call(align=1 << 17) == INV
    assert call(rows=1023) == INV and call(rows=1025, fill=1) == INV and call(rows=1 << 31) == SHAPE
    for name in ("ids", "c", "o", "r", "s"):
        assert call(**{name: None}) == INV, name
        assert call(**{name: 18}) == ALIGN, name
    big = dict(T=100000, k=4, rows=401920)
    assert L.mxfp4_expert_plan_workspace(100000, 4, 8) > 0
    assert L.mxfp4_expert_plan_workspace(1000, 4, 8) == 0
    assert call(ws=None, **big) == INV and call(wb=31, **big) == INV and call(ws=17, **big) == ALIGN


def test_expert_plan_rows_bound_every_split(L):
    rows = mxfp4.mxfp4_expert_plan_rows
    assert rows(0, 4, 32, 128) == 0 and rows(1, 1, 1, 1) == 1 and rows(16384, 4, 32, 128) == 69504
    assert rows(-1, 4, 32, 128) == 0 and rows(1 << 40, 4, 32, 128) == 0
    rng = np.random.default_rng(0)
    for _ in range(300):
        T, k, E = int(rng.integers(1, 60)), int(rng.integers(1, 5)), int(rng.integers(1, 40))
        align = int(2 ** rng.integers(0, 8))
        ids = rng.integers(0, E, (T, k))
        if rng.random() < 0.3:
            ids = np.arange(T * k).reshape(T, k) % E            # the split with the most padding
        used = ref.plan(ids, E, align, 1 << 16)["offsets"][-1]
        assert used <= rows(T, k, E, align) and rows(T, k, E, align) % align == 0


def test_rows_refusals(L):
    def disp(x=16, dtype=0, T=4, k=2, C=8, ldx=8, r=16, s=16, rows=128, out=16, ldo=8):
        return L.mxfp4_dispatch(x, dtype, T, k, C, ldx, r, s, rows, out, ldo, None)
    assert disp(dtype=3) == INV and disp(ldx=7) == INV and disp(ldo=7) == INV and disp(T=-1) == INV and disp(k=0) == INV
    assert disp(r=None) == INV and disp(r=18) == ALIGN
    assert disp(x=None) == INV and disp(s=None) == INV and disp(out=None) == INV
    assert disp(x=17) == ALIGN and disp(out=17) == ALIGN and disp(s=18) == ALIGN and disp(dtype=1, x=18) == ALIGN
    assert disp(k=33) == SHAPE and disp(rows=1 << 31) == SHAPE and disp(T=1 << 30) == SHAPE
    assert disp(rows=0) == 0 and disp(C=0) == 0

    def comb(y=16, yd=0, rows=128, C=8, ldy=8, r=16, w=16, T=4, k=2, out=16, od=0, ldo=8):
        return L.mxfp4_combine(y, yd, rows, C, ldy, r, w, T, k, out, od, ldo, None)
    assert comb(yd=2) == INV and comb(od=2) == INV and comb(ldy=7) == INV and comb(ldo=7) == INV
    assert comb(y=None) == INV and comb(r=None) == INV and comb(out=None) == INV and comb(k=33) == SHAPE
    assert comb(y=17) == ALIGN and comb(r=18) == ALIGN and comb(w=18) == ALIGN and comb(od=1, out=18) == ALIGN
    assert comb(T=0) == 0

    def bwd(d=16, dd=0, ldd=8, y=16, yd=0, rows=128, C=8, ldy=8, r=16, s=16, w=16, T=4, k=2, dy=16, lddy=8, dw=16):
        return L.mxfp4_combine_bwd(d, dd, ldd, y, yd, rows, C, ldy, r, s, w, T, k, dy, lddy, dw, None)
    for name in ("d", "y", "r", "s", "w", "dy", "dw"):
        assert bwd(**{name: None}) == INV, name
        assert bwd(**{name: 17}) == ALIGN, name
    assert bwd(ldd=7) == INV and bwd(ldy=7) == INV and bwd(lddy=7) == INV and bwd(dd=9) == INV and bwd(yd=9) == INV
    assert bwd(T=0, rows=0) == 0


def test_grad_clip_refusals(L):
    def call(ts=((16, 16, 4, 1),), max_norm=1.0, norm=16, ws=16, wb=1 << 20, count=None):
        arr = (mxfp4.GradTensor * max(1, len(ts)))(*[mxfp4.GradTensor(*t) for t in ts])
        return L.mxfp4_grad_clip(arr, len(ts) if count is None else count, max_norm, norm, ws, wb, None)
    assert call(count=-1) == INV and L.mxfp4_grad_clip(None, 1, 1.0, 16, 16, 1 << 20, None) == INV
    assert call(max_norm=0.0) == INV and call(max_norm=-1.0) == INV and call(max_norm=float("nan")) == INV
    assert call(norm=None) == INV
    big = ((16, 16, 1 << 22, 1),)
    assert call(ts=big, ws=None) == INV and call(ts=big, wb=8) == INV and call(ts=big * 97, wb=9472 * 2 - 1) == INV
    assert call(norm=18) == ALIGN and call(ws=20) == ALIGN
    assert call(ts=((16, 16, 4, 7),)) == INV and call(ts=((16, 16, -4, 1),)) == INV and call(ts=((None, 16, 4, 1),)) == INV
    assert call(ts=((16, 16, 4, 1), (32, None, 4, 1))) == INV
    assert call(ts=((18, 16, 4, 1),)) == ALIGN and call(ts=((16, 18, 4, 1),)) == ALIGN and call(ts=((16, 16, 1 << 41, 1),)) == SHAPE
    table = lambda *ts: (mxfp4.GradTensor * len(ts))(*[mxfp4.GradTensor(*t) for t in ts])
    need = mxfp4.mxfp4_grad_clip_workspace
    assert need(table((16, 16, 4, 1)), 1) == 0 and need(None, 0) == 0
    assert 0 < need(table(*big), 1) < need(table(*(big * 97)), 97)
    assert need(table(*(((16, 16, 4, 1),) * 97)), 97) > 0


def test_helpers_refuse_host_tensors_and_wrong_kinds():
    l = torch.zeros(4, 8)
    for call in (lambda: mxfp4.route(l, 2), lambda: mxfp4.route(None, 2),
                 lambda: mxfp4.route_bwd(l, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)),
                 lambda: mxfp4.expert_plan(torch.zeros(4, 2, dtype=torch.int32), 8), lambda: mxfp4.dispatch(l, {}),
                 lambda: mxfp4.combine(l, {}), lambda: mxfp4.combine_bwd(l, l, {}, l), lambda: mxfp4.grad_clip([l], 1.0),
                 lambda: mxfp4.grad_clip([], 1.0), lambda: mxfp4.GradList([l])):
        with pytest.raises(ValueError):
            call()


def test_plain_plan_equals_the_synthetic_layout():
    """The plain plan and the synthetic inputs' expert layout are the same
    thing where a token has each expert at most once."""
    r = synth.zipf_routing(500, 16, 4, seed=3)
    counts, offsets, tor = synth.expert_layout(r, 16)
    p = ref.plan(r, 16, 128, int(offsets[-1]))
    assert np.array_equal(p["counts"], counts) and np.array_equal(p["offsets"], offsets)
    assert np.array_equal(np.where(p["slot_of_row"] < 0, -1, p["slot_of_row"] // 4), tor)


def test_plain_route_gradient_against_differences():
    rng = np.random.default_rng(1)
    l, dw = rng.standard_normal((3, 9)), rng.standard_normal((3, 4))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, _ = ref.route(l, 4, score=score, renormalise=renorm)
            g, mag = ref.route_bwd(l, ids, dw, score, renorm, 1.5)
            for e in range(9):
                h = np.zeros_like(l)
                h[:, e] = 1e-6
                num = 0
                for sgn in (1, -1):
                    w = np.take_along_axis(ref.scores(l + sgn * h, score), ids, 1)
                    w = 1.5 * (w / w.sum(1, keepdims=True) if renorm else w)
                    num = num + sgn * (w * dw).sum(1)
                assert np.all(abs(num / 2e-6 - g[:, e]) < 1e-8)
            assert np.all(abs(g) <= mag * (1 + 1e-12) + 1e-15)


def test_the_module_imports_without_cuda_in_torch():
    """A torch built without CUDA has no current-stream handle to look up; only
    a call on tensors of a GPU needs one."""
    code = ("import torch; delattr(torch._C, '_cuda_getCurrentRawStream')\n"
            "from fp4_precision_numerics_b200 import mxfp4; print(mxfp4.mxfp4_mma_scale_bytes is not None)")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr


def test_a_number_is_not_a_stream(L):
    """A raw handle or a device index in place of a torch stream is refused by
    the entry points, before anything reaches the library."""
    p, q = mxfp4.QuantParams(), mxfp4.QuantOutputs()
    for call in (lambda s: mxfp4.mxfp4_check_device_status(s),
                 lambda s: mxfp4.mxfp4_quantize(16, 0, 1, 0, 32, 32, p, q, s),
                 lambda s: mxfp4.mxfp4_rht(16, 0, 0, 32, 32, 1, 16, 1, 16, 0, s),
                 lambda s: mxfp4.mxfp4_route(16, 0, 0, 8, 8, None, None, rp(), 16, 16, s),
                 lambda s: mxfp4.mxfp4_dispatch(16, 0, 0, 2, 8, 8, 16, 16, 0, 16, 8, s)):
        for stream in (0, 1, 7, True):
            with pytest.raises((AttributeError, TypeError)):
                call(stream)


def test_a_changed_scale_tensor_is_read_again():
    """Launch parameters are kept by value: a 0-dimensional tensor that was
    changed in place gives its new value."""
    t, k = torch.tensor(2.0), torch.tensor(4)
    p = mxfp4._route_params("softmax", k, 1, 1, 1, True, t)
    assert p.scale == 2.0 and p.top_k == 4
    t.fill_(5.0), k.fill_(3)
    p = mxfp4._route_params("softmax", k, 1, 1, 1, True, t)
    assert p.scale == 5.0 and p.top_k == 3
    a = np.array(1.5)
    assert mxfp4._route_params("sigmoid", 4, 1, 1, 1, False, a).scale == 1.5


def test_counts_beyond_an_int_are_refused():
    """Not cut to their low 32 bits, which may be a count that exists."""
    for kw in (dict(top_k=(1 << 32) + 4), dict(groups=(1 << 32) + 1), dict(top_groups=1 - (1 << 32)), dict(group_best=1 << 31)):
        args = {**dict(top_k=4, groups=1, top_groups=1, group_best=1), **kw}
        with pytest.raises(ValueError):
            mxfp4._route_params("softmax", args["top_k"], args["groups"], args["top_groups"], args["group_best"], True, 1.0)


def test_the_row_kernels_leave_a_bounded_wait_by_whole_warps():
    """A lane that gives up on a wait alone would leave the others of its warp
    to shuffles and barriers that name it.  The wait runs out on no test's
    machine, so the source is looked at: every bounded wait of the ring kernels
    is a vote of the warp."""
    here = os.path.dirname(os.path.abspath(mxfp4.__file__))
    with open(os.path.join(here, "csrc", "rows.cuh")) as f:
        text = " ".join(f.read().split())
    parts = text.split("mbar_wait_bounded(")
    assert len(parts) == 6      # dispatch's, combine's two, its gradient's two
    assert all(p.endswith("__all_sync(~0u, ") for p in parts[:-1])


def test_sizes_beyond_any_tensor_are_refused(L):
    """Products of sizes are bounded before they are formed: none wraps around
    to a size that looks small."""
    for T in (1 << 31, 1 << 61, 1 << 62, (1 << 63) - 1):
        for k in (1, 2, 4, 8):
            assert L.mxfp4_route(16, 0, T, 8, 8, None, None, ctypes.byref(rp(top_k=k)), 16, 16, None) == SHAPE
            assert L.mxfp4_route_bwd(16, 0, T, 8, 8, 16, 16, ctypes.byref(rp(top_k=k)), 16, 8, None) == SHAPE
    rows = mxfp4.mxfp4_expert_plan_rows
    big = (1 << 31) - 1
    assert rows(big, big, 1 << 62, 1 << 30) == 0               # beyond 64 bits
    assert rows(big, 1, 1 << 40, 2) == (big + big) // 2 * 2
    need = mxfp4.mxfp4_grad_clip_workspace
    for n in (1 << 40, 1 << 61, 1 << 62, (1 << 63) - 1):
        assert need((mxfp4.GradTensor * 1)(mxfp4.GradTensor(16, 16, n, 1)), 1) > 0
