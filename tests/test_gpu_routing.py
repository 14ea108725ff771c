"""GPU parity of the routing calls (route, route_bwd, expert_plan, dispatch,
combine, combine_bwd) against plain binary64 forms, at the sizes, masks and
layouts where they can go wrong.  Whole numbers are compared exactly; bounds
on the others count roundings (half a step of binary32 is 2^-24)."""
import numpy as np
import pytest
import torch

from fp4_precision_numerics_b200 import mxfp4
from tests import routing_ref as ref
from tests.routing_ref import HALF_F32, f64, half_step

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def rand(*shape, seed=0, std=1.0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


# ------------------------------------------------------------------ route
def check_route(logits, k, **kw):
    got = mxfp4.route(logits, k, **kw)
    rk = {n: (f64(v) if isinstance(v, torch.Tensor) else v) for n, v in kw.items() if n not in ("out", "stream")}
    ids, w = ref.route(f64(logits), k, **rk)
    assert np.array_equal(got["ids"].cpu().numpy(), ids)
    # exponents: the difference of logits is off by half a step of the largest one, the exponential by two steps;
    # then the sum of the scores, a division and the scale
    span = float(torch.nan_to_num(logits.float(), 0, 0, 0).abs().max()) if logits.numel() else 0.0
    tol = HALF_F32 * (2 * span + 4 + logits.shape[1] / 32 + 8 + 4)
    gw = f64(got["weights"])
    assert np.array_equal(np.isnan(gw), np.isnan(w))
    ok = ~np.isnan(w)
    assert np.all(abs(gw - w)[ok] <= tol * abs(w)[ok] + 1e-37)
    return got


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,E,k", [(1, 32, 4), (1, 1, 1), (5, 7, 7), (257, 33, 2), (64, 100, 8), (300, 256, 8),
                                   (33, 513, 6), (9, 1024, 32), (70, 32, 32), (4099, 64, 1)])
def test_route(T, E, k, dtype, score):
    l = rand(T, E, seed=T + E, std=1.5, dtype=dtype)
    check_route(l, k, score=score)
    check_route(l, k, score=score, renormalise=False, scale=2.5)
    b = rand(E, seed=9, std=0.2)
    check_route(l, k, score=score, bias=b)
    check_route(l, k, score=score, bias=torch.zeros_like(b), renormalise=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (64, 32, 3, 6), (39, 3, 2, 5), (128, 2, 1, 8), (32, 32, 4, 4),
                                            (1000, 20, 7, 9), (64, 8, 8, 4), (512, 16, 2, 8)])
def test_route_groups(E, groups, top, k, best, score):
    for dtype in (BF16, F32):
        l = rand(203, E, seed=E + groups, std=1.5, dtype=dtype)
        for bias in (None, rand(E, seed=4, std=0.1), torch.zeros(E, device="cuda")):
            check_route(l, k, score=score, groups=groups, top_groups=top, group_best=best, bias=bias, scale=1.5)


def test_route_ties_go_to_the_lowest_index():
    l = torch.zeros((3, 40), device="cuda")
    l[1, 7::9] = 1.0
    l[2, :] = -0.0
    l[2, 5] = 0.0     # one value with -0
    for kw in (dict(), dict(bias=torch.zeros(40, device="cuda")), dict(score="sigmoid", groups=4, top_groups=2, group_best=2)):
        check_route(l, 6, **kw)


def test_route_near_ties_are_decided_in_64_bits():
    """Scores plus bias that differ by less than a step of binary32: the
    choice is that of the binary64 scores."""
    rng = np.random.default_rng(0)
    l = torch.from_numpy(rng.standard_normal((512, 64)).astype(np.float32)).cuda()
    # a bias that brings the sigmoid scores of row 0's logits within ~1e-8 of one value; neighbouring rows repeat it
    l[:] = l[0]
    s = 1 / (1 + torch.exp(-l[0].double()))
    bias = (0.9 - s).float()
    for groups, best in ((1, 1), (4, 1), (8, 2)):
        check_route(l, 8, score="sigmoid", bias=bias, groups=groups, top_groups=max(1, groups // 2), group_best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_pairs_a_step_apart(score):
    """Two experts, or two whole groups, with the same logits whose biases
    differ by one step of binary32, the later one larger: binary32 scores often
    agree there, the choice is the later one's first."""
    for T, E, groups in ((1500, 96, 1), (1500, 96, 8), (700, 700, 4), (700, 64, 32)):
        l = rand(T, E, seed=T + E, std=1.5)
        bias = rand(E, seed=2, std=0.05)
        n = E // groups
        # one pair inside a group, high enough to be chosen often
        l[:, 1] = l[:, 1].abs() + 2
        l[:, 0] = l[:, 1]
        bias[0] = 0.1
        bias[1] = float(np.nextafter(np.float32(0.1), np.float32(1)))
        for best in (1, 2):
            check_route(l, 6, score=score, bias=bias, groups=groups, top_groups=max(1, groups * 3 // 4), group_best=best)
        if groups > 1:
            # two groups that differ by a step in every bias
            l2, b2 = l.clone(), bias.clone()
            l2[:, n:2 * n] = l2[:, 2 * n:3 * n]
            b2[n:2 * n] = bias[2 * n:3 * n]
            b2[2 * n:3 * n] = torch.from_numpy(np.nextafter(f64(bias[2 * n:3 * n]).astype(np.float32), np.float32(9))).cuda()
            for best in (1, 2):
                check_route(l2, min(4, n), score=score, bias=b2, groups=groups, top_groups=max(1, groups // 2), group_best=best)


def test_route_large_opposite_biases():
    """Biases far larger than the scores: sums of a group's two terms cancel."""
    l = rand(800, 64, seed=3, std=1.5)
    b = torch.zeros(64, device="cuda")
    b[::2], b[1::2] = 1000.0, -1000.0
    b += rand(64, seed=4, std=1e-4)
    for groups, best in ((1, 1), (8, 1), (8, 2), (32, 2), (32, 1)):
        for score in ("softmax", "sigmoid"):
            check_route(l, 4, score=score, bias=b, groups=groups, top_groups=max(1, groups // 2), group_best=best)


def test_route_excluded_experts():
    """A bias of -infinity keeps an expert out while others are left."""
    l = rand(300, 64, seed=5, std=1.5)
    b = rand(64, seed=6, std=0.1)
    b[::3] = -float("inf")
    for groups, best in ((1, 1), (8, 2), (4, 1)):
        got = check_route(l, 6, score="sigmoid", bias=b, groups=groups, top_groups=max(1, groups // 2), group_best=best)
        assert int((got["ids"] % 3 == 0).sum()) == 0
    b[:] = -float("inf")
    b[5] = 0.0
    check_route(l, 3, score="sigmoid", bias=b)


def test_route_masks_infinities_and_nan():
    inf, nan = float("inf"), float("nan")
    l = rand(12, 48, seed=1)
    l[0] = -inf
    l[1, 3:] = -inf                  # fewer finite logits than top_k
    l[2, 10] = nan
    l[3, 11] = inf
    l[4] = torch.finfo(torch.float32).min
    l[5] = nan
    l[6, 5] = -inf
    l[7] = nan
    mask = torch.ones(12, dtype=torch.bool, device="cuda")
    mask[7] = mask[9] = False        # NaN under a mask must not come through
    for score in ("softmax", "sigmoid"):
        for kw in (dict(), dict(renormalise=False), dict(groups=4, top_groups=2)):
            got = mxfp4.route(l, 5, score=score, mask=mask, **kw)
            ids, w = got["ids"].cpu().numpy(), f64(got["weights"])
            assert np.all(ids[[7, 9]] == -1) and np.all(w[[7, 9]] == 0)
            live = np.delete(np.arange(12), [7, 9])
            assert np.all((ids[live] >= 0) & (ids[live] < 48))
            assert all(len(set(r)) == 5 for r in ids[live].tolist())
            r_ids, r_w = ref.route(f64(l), 5, score=score, mask=f64(mask), **kw)
            finite = [0, 1, 4, 6, 8, 10, 11]
            assert np.array_equal(ids[finite], r_ids[finite])
            assert np.all(abs(w[finite] - r_w[finite]) <= 1e-5 * abs(r_w[finite]))
            if score == "softmax":
                assert np.all(np.isnan(w[[2, 3, 5]]))
                assert np.all(w[0] == 0)
            else:
                assert np.isfinite(w[2]).all() and ids[3, 0] == 11 and np.isfinite(w[3]).all()
                assert 10 not in ids[2]
    allm = mxfp4.route(l, 5, mask=torch.zeros(12, dtype=torch.uint8, device="cuda"))
    assert int(allm["ids"].max()) == -1 and float(allm["weights"].abs().max()) == 0


def test_route_strides_and_streams():
    big = rand(40, 100, seed=2, dtype=BF16)
    check_route(big[3:31, 5:70], 4)
    check_route(rand(40, 101, seed=2)[1::2, 1:66], 4, score="sigmoid", bias=rand(65, seed=3, std=0.1))
    s = torch.cuda.Stream()
    l = rand(1000, 32, seed=5)
    s.wait_stream(torch.cuda.current_stream())
    got = mxfp4.route(l, 4, stream=s)
    s.synchronize()
    assert np.array_equal(got["ids"].cpu().numpy(), ref.route(f64(l), 4)[0])
    assert mxfp4.route(l[:0], 4)["ids"].shape == (0, 4)


# ------------------------------------------------------------------ route_bwd
def check_route_bwd(l, ids, dw, **kw):
    got = mxfp4.route_bwd(l, ids, dw, **kw)
    g, mag = ref.route_bwd(f64(l), ids.cpu().numpy(), f64(dw), **kw)
    span = float(l.float().abs().max())
    tol = HALF_F32 * (4 * span + 8 + l.shape[1] / 32 + 8 + ids.shape[1] + 8)
    assert got.dtype == l.dtype
    assert np.all(abs(f64(got) - g) <= tol * mag + half_step(l.dtype) * (1 + tol) * abs(g) + 1e-37)
    return got


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 32, 4), (3, 1, 1), (65, 7, 3), (100, 128, 6), (33, 300, 8), (5, 1024, 32), (501, 33, 2)])
def test_route_bwd(T, E, k, renorm, score):
    for dtype in (BF16, F32):
        l = rand(T, E, seed=E, std=1.5, dtype=dtype)
        ids = mxfp4.route(l, k, score=score)["ids"]
        check_route_bwd(l, ids, rand(T, k, seed=2), score=score, renormalise=renorm, scale=1.5)


def test_route_bwd_dropped_and_repeated_slots():
    l = rand(6, 40, seed=3)
    ids = torch.tensor([[3, 3, 7], [-1, -1, -1], [39, -1, 0], [40, 5, 6], [1, 1, 1], [-5, 2, 1 << 30]], dtype=torch.int32,
                       device="cuda")
    dw = rand(6, 3, seed=4)
    dw[1] = float("nan")             # no slot of the row is live
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = check_route_bwd(l, ids, torch.where(dw.isnan(), 0.0, dw), score=score, renormalise=renorm)
            assert torch.equal(mxfp4.route_bwd(l, ids, dw, score=score, renormalise=renorm), got)
            assert float(got[1].abs().max()) == 0.0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_bwd_against_differences(renorm, score):
    """Central differences of the binary64 weights at a fixed choice."""
    l = rand(4, 12, seed=6)
    ids = mxfp4.route(l, 3, score=score)["ids"]
    dw = rand(4, 3, seed=7)
    got = f64(mxfp4.route_bwd(l, ids, dw, score=score, renormalise=renorm, scale=2.0))
    L, I, D, h = f64(l), ids.cpu().numpy(), f64(dw), 1e-5

    def weights(x):
        w = np.take_along_axis(ref.scores(x, score), I, axis=1)
        return 2.0 * (w / w.sum(1, keepdims=True) if renorm else w)
    for e in range(12):
        up, dn = L.copy(), L.copy()
        up[:, e] += h
        dn[:, e] -= h
        num = ((weights(up) - weights(dn)) / (2 * h) * D).sum(1)
        # differences: h^2 of the third derivative and 1e-16 / h of rounding; the kernel: a few steps of binary32
        assert np.all(abs(num - got[:, e]) <= 1e-8 + 64 * HALF_F32 * abs(D).sum(1) * 2)


def test_route_bwd_strides():
    l = rand(20, 70, seed=8, dtype=BF16)[:, 3:67]
    out = torch.full((20, 80), 7.0, device="cuda", dtype=BF16)
    ids = mxfp4.route(l, 4)["ids"]
    dw = rand(20, 4, seed=1)
    mxfp4.route_bwd(l, ids, dw, renormalise=False, out=out[:, 5:69])
    assert torch.equal(out[:, 5:69], mxfp4.route_bwd(l.contiguous(), ids, dw, renormalise=False))
    assert bool((out[:, :5] == 7).all()) and bool((out[:, 69:] == 7).all())


# ------------------------------------------------------------------ expert_plan
def check_plan(ids, E, align=128, rows=None, fill=False):
    got = mxfp4.expert_plan(ids, E, align=align, rows=rows, fill=fill)
    want = ref.plan(ids.cpu().numpy(), E, align, got["slot_of_row"].numel(), fill)
    for k in want:
        assert np.array_equal(got[k].cpu().numpy(), want[k]), k
    return got


@pytest.mark.parametrize("T,k,E,align", [(1, 1, 1, 1), (1, 4, 32, 128), (0, 4, 32, 128), (31, 3, 5, 128), (1024, 4, 32, 128),
                                         (1025, 4, 32, 64), (4097, 1, 1024, 128), (20011, 8, 256, 128), (3000, 2, 2, 1),
                                         (65536, 8, 256, 128), (140001, 4, 77, 256), (1366, 3, 9, 128), (16384, 4, 1024, 128),
                                         (65537, 1, 40, 32)])
def test_expert_plan(T, k, E, align):
    g = torch.Generator(device="cuda").manual_seed(T)
    u = torch.rand((T, k), generator=g, device="cuda")
    ids = (u * u * E).to(torch.int32).clamp_(max=E - 1)        # uneven, with repeats inside a token
    check_plan(ids, E, align)
    drop = torch.rand((T, k), generator=g, device="cuda") < 0.3
    check_plan(torch.where(drop, -1, ids).to(torch.int32), E, align)


def test_expert_plan_extremes():
    ids = torch.zeros((5000, 3), dtype=torch.int32, device="cuda")
    check_plan(ids + 6, 7)                                     # one expert takes all
    check_plan(ids - 1, 7)                                     # no slot has an expert
    check_plan(ids + 7, 7)                                     # ids behind the last expert
    check_plan(torch.full_like(ids, -(1 << 31)), 7)
    rows = mxfp4.mxfp4_expert_plan_rows(5000, 3, 7, 128)
    check_plan(ids, 7, rows=rows + 1280, fill=True)            # spare rows, the last segment takes them
    check_plan(ids + 6, 7, rows=rows + 77)
    assert mxfp4.expert_plan(ids, 7, fill=True)["offsets"][-1].item() == rows


def test_expert_plan_repeats_and_graph():
    """The same bits on every call, and two captured plans replayed together
    keep their own results."""
    g = torch.Generator(device="cuda").manual_seed(1)
    a = (torch.rand((30000, 4), generator=g, device="cuda") * 64).to(torch.int32)      # more than a cluster holds
    b = (torch.rand((30000, 4), generator=g, device="cuda") * 64).to(torch.int32)
    first = mxfp4.expert_plan(a, 64)
    for _ in range(3):
        again = mxfp4.expert_plan(a, 64)
        assert all(torch.equal(first[k], again[k]) for k in first)
    mxfp4.expert_plan(b, 64)
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for ids in (a, b):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(mxfp4.expert_plan(ids, 64))
        graphs.append(gr)
    for _ in range(5):
        for o in outs:
            for v in o.values():
                v.zero_()
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for ids, o in zip((a, b), outs):
            want = ref.plan(ids.cpu().numpy(), 64, 128, o["slot_of_row"].numel())
            assert all(np.array_equal(o[k].cpu().numpy(), want[k]) for k in want)


# ------------------------------------------------------------------ dispatch, combine
def make_plan(T, k, E, seed=0, drop=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    if drop:
        ids = torch.where(torch.rand((T, k), generator=g, device="cuda") < drop, -1, ids).to(torch.int32)
    return mxfp4.expert_plan(ids.contiguous(), E)


SHAPES = [(1, 1, 1, 1), (1, 4, 32, 2880), (48, 4, 32, 2880), (300, 2, 5, 1001), (1000, 4, 32, 64), (77, 8, 9, 5760),
          (130, 3, 4, 24), (5, 32, 40, 130), (2000, 1, 16, 8), (700, 5, 8, 1544), (601, 9, 16, 3080), (650, 4, 8, 4096),
          (90, 2, 4, 256), (90, 2, 4, 264)]


@pytest.mark.parametrize("T,k,E,C", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dispatch(T, k, E, C, dtype):
    for drop in (0.0, 0.4):
        plan = make_plan(T, k, E, drop=drop)
        x = rand(T, C, seed=T, dtype=dtype)
        got = mxfp4.dispatch(x, plan)
        slot = plan["slot_of_row"].long()
        want = torch.where((slot >= 0)[:, None], x[slot.clamp_min(0) // k], torch.zeros((), dtype=dtype, device="cuda"))
        assert torch.equal(got, want)


def test_no_tokens_leave_zero_rows():
    plan = mxfp4.expert_plan(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 8, rows=256)
    for C in (64, 33):
        for dtype in (BF16, F32):
            x = torch.empty((0, C), dtype=dtype, device="cuda")
            out = torch.full((256, C), 3.0, dtype=dtype, device="cuda")
            assert not bool(mxfp4.dispatch(x, plan, out=out).any())
            dy = torch.full((256, C), 3.0, dtype=dtype, device="cuda")
            w = torch.empty((0, 4), device="cuda")
            mxfp4.combine_bwd(x, out, plan, w, out={"dy": dy})
            assert not bool(dy.any())
            assert mxfp4.combine(out, plan, w).shape == (0, C)


def test_dispatch_layouts_and_nan_bits():
    plan = make_plan(60, 4, 8)
    for dtype, it in ((BF16, torch.int16), (F32, torch.int32)):
        x = rand(60, 300, seed=1, dtype=dtype)
        x[5, ::7] = float("nan")
        x[6] = float("-inf")
        for v in (x[:, 8:208], x[:, 1:200], x[:, 3:4]):
            out = torch.full((plan["slot_of_row"].numel(), 333), 3.0, dtype=dtype, device="cuda")
            for o0 in (0, 5, 8):
                o = out[:, o0:o0 + v.shape[1]]
                mxfp4.dispatch(v, plan, out=o)
                assert torch.equal(o.contiguous().view(it), mxfp4.dispatch(v.contiguous(), plan).view(it))
            assert bool((out[:, 300:] == 3).all())


@pytest.mark.parametrize("T,k,E,C", SHAPES)
@pytest.mark.parametrize("ydt", [BF16, F32])
@pytest.mark.parametrize("odt", [BF16, F32])
def test_combine(T, k, E, C, ydt, odt):
    for drop in (0.0, 0.4):
        plan = make_plan(T, k, E, seed=2, drop=drop)
        y = rand(plan["slot_of_row"].numel(), C, seed=3, dtype=ydt)
        y[plan["slot_of_row"] < 0] = float("nan")       # padding rows are never read into a sum
        w = rand(T, k, seed=4)
        w[plan["row_of_slot"] < 0] = float("nan")       # nor is the weight of a slot without a row
        for weights in (w, None):
            got = f64(mxfp4.combine(y, plan, weights, out_dtype=odt))
            want, mag = ref.combine(f64(y), plan["row_of_slot"].cpu().numpy(), None if weights is None else f64(w))
            assert np.all(abs(got - want) <= (k + 1) * HALF_F32 * mag + half_step(odt) * abs(want))


@pytest.mark.parametrize("T,k,E,C", SHAPES)
@pytest.mark.parametrize("ydt", [BF16, F32])
@pytest.mark.parametrize("ddt", [BF16, F32])
def test_combine_bwd(T, k, E, C, ydt, ddt):
    for drop in (0.0, 0.4):
        plan = make_plan(T, k, E, seed=5, drop=drop)
        rows = plan["slot_of_row"].numel()
        y, d = rand(rows, C, seed=6, dtype=ydt), rand(T, C, seed=7, dtype=ddt)
        y[plan["slot_of_row"] < 0] = float("nan")
        w = rand(T, k, seed=8)
        out = {"dy": torch.full((rows, C), float("nan"), dtype=ddt, device="cuda")}
        got = mxfp4.combine_bwd(d, y, plan, w, out=out)
        dy, dw, mag = ref.combine_bwd(f64(d), f64(y), plan["row_of_slot"].cpu().numpy(), f64(w))
        assert np.all(abs(f64(got["dy"]) - dy) <= (half_step(ddt) + HALF_F32) * abs(dy))
        assert np.all(abs(f64(got["d_weights"]) - dw) <= (C / 32 + 24) * HALF_F32 * mag)
        again = mxfp4.combine_bwd(d, y, plan, w)
        assert torch.equal(again["d_weights"], got["d_weights"]) and torch.equal(again["dy"], got["dy"])


def test_combine_gradients_against_differences():
    """<d_out, combine(y + h e, w)> by central differences, for y and w; and
    the gradient of dispatch, which is combine without weights."""
    T, k, C = 6, 3, 10
    plan = make_plan(T, k, 5, seed=9, drop=0.2)
    ros = plan["row_of_slot"].cpu().numpy()
    rows = plan["slot_of_row"].numel()
    y, w, d = rand(rows, C, seed=1), rand(T, k, seed=2), rand(T, C, seed=3)
    got = mxfp4.combine_bwd(d, y, plan, w)
    Y, W, D, h = f64(y), f64(w), f64(d), 0.5      # linear in each: differences of any width are exact
    loss = lambda a, b: (ref.combine(a, ros, b)[0] * D).sum()
    for t, j in ((0, 0), (2, 1), (5, 2), (3, 0)):
        up, dn = W.copy(), W.copy()
        up[t, j] += h
        dn[t, j] -= h
        assert abs((loss(Y, up) - loss(Y, dn)) / (2 * h) - f64(got["d_weights"])[t, j]) <= 1e-5
    for r in sorted(set(ros[ros >= 0].tolist()))[:6] + [rows - 1]:
        up, dn = Y.copy(), Y.copy()
        up[r, 4] += h
        dn[r, 4] -= h
        assert abs((loss(up, W) - loss(dn, W)) / (2 * h) - f64(got["dy"])[r, 4]) <= 1e-6
    g = rand(rows, C, seed=4)
    x = rand(T, C, seed=5)
    dx = f64(mxfp4.combine(g, plan))
    assert abs((f64(mxfp4.dispatch(x, plan)) * f64(g)).sum() - (f64(x) * dx).sum()) <= 1e-4


def test_combine_layouts():
    plan = make_plan(50, 4, 8, seed=3, drop=0.1)
    rows = plan["slot_of_row"].numel()
    w = rand(50, 4, seed=1)
    for dtype in (BF16, F32):
        y = rand(rows, 200, seed=2, dtype=dtype)
        d = rand(50, 210, seed=3, dtype=dtype)
        for c0, c1 in ((0, 64), (8, 72), (1, 65), (3, 10)):
            v, g = y[:, c0:c1], d[:, c0:c1]
            out = torch.full((50, 100), 2.0, dtype=dtype, device="cuda")
            mxfp4.combine(v, plan, w, out=out[:, :c1 - c0])
            assert torch.equal(out[:, :c1 - c0], mxfp4.combine(v.contiguous(), plan, w))
            assert bool((out[:, c1 - c0:] == 2).all())
            a, b = mxfp4.combine_bwd(g, v, plan, w), mxfp4.combine_bwd(g.contiguous(), v.contiguous(), plan, w)
            assert torch.equal(a["dy"], b["dy"])
            _, dw, mag = ref.combine_bwd(f64(g), f64(v), plan["row_of_slot"].cpu().numpy(), f64(w))
            for o in (a, b):
                assert np.all(abs(f64(o["d_weights"]) - dw) <= ((c1 - c0) / 32 + 24) * HALF_F32 * mag)


def test_offsets_beyond_32_bits():
    """Rows whose element offsets pass 2^31 and byte offsets pass 2^32."""
    T, k, C = 400000, 2, 2880
    g = torch.Generator(device="cuda").manual_seed(0)
    ids = (torch.rand((T, k), generator=g, device="cuda") * 4).to(torch.int32)
    plan = mxfp4.expert_plan(ids, 4)
    rows = plan["slot_of_row"].numel()
    assert rows * C > 1 << 31
    x = torch.empty((T, C), dtype=BF16, device="cuda").normal_(generator=g)
    xp = mxfp4.dispatch(x, plan)
    at = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    r = plan["row_of_slot"][at].long()
    assert int(r.max()) * C > 1 << 31
    for j in range(k):
        assert torch.equal(xp[r[:, j]], x[at])
    w = torch.rand((T, k), generator=g, device="cuda")
    y = mxfp4.combine(xp, plan, w, out_dtype=F32)
    want = x[at].double() * w[at].double().sum(1, keepdim=True)
    assert bool(((y[at].double() - want).abs() <= 4 * HALF_F32 * want.abs()).all())
    del y
    got = mxfp4.combine_bwd(x, xp, plan, w)
    for j in range(k):
        dy = x[at].float() * w[at, j, None]
        assert torch.equal(got["dy"][r[:, j]], dy.to(BF16))
    dw = (x[at].double() ** 2).sum(1, keepdim=True)
    assert bool(((got["d_weights"][at].double() - dw).abs() <= (C / 32 + 24) * HALF_F32 * dw).all())


# ------------------------------------------------------------------ together
def test_layer_forward_and_backward_together():
    """route -> expert_plan -> dispatch -> quantize_dual -> grouped GEMMs ->
    combine, then its backward to the tokens, the router and the weights, on
    one stream without reading the device (fill), eager and replayed from a
    graph.  Every step is held to the plain form of its own inputs."""
    T, E, k, H = 300, 8, 2, 256
    x = rand(T, H, seed=1, dtype=BF16)
    logits = rand(T, E, seed=2, std=1.5)
    W = rand(E, H, H, seed=3, std=0.05)
    d_out = rand(T, H, seed=4, dtype=BF16)
    wq = mxfp4.quantize(W, block="32x32", scales=False, scales_mma=True, transposed=True)

    def step():
        r = mxfp4.route(logits, k)
        p = mxfp4.expert_plan(r["ids"], E, fill=True)
        M = p["slot_of_row"].numel()
        xp = mxfp4.dispatch(x, p)
        xr, xc = mxfp4.quantize_dual(xp, col_rht_seed=1, scales=False, scales_mma=True)
        y = mxfp4.grouped_gemm(mxfp4.GEMM_FPROP, p["offsets"], xr["codes"], xr["scales_mma"], wq["codes"],
                               wq["scales_mma"], M, H, H)
        out = mxfp4.combine(y, p, r["weights"], out_dtype=BF16)
        g = mxfp4.combine_bwd(d_out, y, p, r["weights"])
        dr, dc = mxfp4.quantize_dual(g["dy"], col_rht_seed=1, scales=False, scales_mma=True)
        dxp = mxfp4.grouped_gemm(mxfp4.GEMM_DGRAD, p["offsets"], dr["codes"], dr["scales_mma"], wq["codes_t"],
                                 wq["scales_mma_t"], M, H, H)
        dW = mxfp4.grouped_gemm(mxfp4.GEMM_WGRAD, p["offsets"], dc["codes"], dc["scales_mma"], xc["codes"],
                                xc["scales_mma"], H, H, M)
        dx = mxfp4.combine(dxp, p, out_dtype=BF16)
        dl = mxfp4.route_bwd(logits, r["ids"], g["d_weights"])
        norm = mxfp4.grad_clip([dW, dl], 0.5)
        return dict(ids=r["ids"], weights=r["weights"], xp=xp, y=y, out=out, dy=g["dy"], dw=g["d_weights"], dxp=dxp, dx=dx,
                    dl=dl, dW=dW, norm=norm, offsets=p["offsets"], slot=p["slot_of_row"], ros=p["row_of_slot"])
    o = step()
    mxfp4.mxfp4_check_device_status()
    ids, w = ref.route(f64(logits), k)
    assert np.array_equal(o["ids"].cpu().numpy(), ids)
    M = o["slot"].numel()
    p = ref.plan(ids, E, 128, M, fill=True)
    assert np.array_equal(o["ros"].cpu().numpy(), p["row_of_slot"])
    assert torch.equal(o["xp"][o["ros"].long().reshape(-1)], x.repeat_interleave(k, 0))
    want, mag = ref.combine(f64(o["y"]), p["row_of_slot"], f64(o["weights"]))
    assert np.all(abs(f64(o["out"]) - want) <= (k + 1) * HALF_F32 * mag + half_step(BF16) * abs(want))
    want, mag = ref.combine(f64(o["dxp"]), p["row_of_slot"], None)
    assert np.all(abs(f64(o["dx"]) - want) <= (k + 1) * HALF_F32 * mag + half_step(BF16) * abs(want))
    # against the layer in 64 bits, where MXFP4 operands are off by up to a quarter of their value each
    full = np.zeros((T, H))
    for j in range(k):
        full += w[:, j, None] * np.einsum("th,toh->to", f64(x), f64(W)[ids[:, j]])
    cos = (full * f64(o["out"])).sum() / np.sqrt((full ** 2).sum() * (f64(o["out"]) ** 2).sum())
    assert cos > 0.95
    total = np.sqrt((f64(o["dW"]) ** 2).sum() + (f64(o["dl"]) ** 2).sum())
    assert abs(total - 0.5) <= 1e-5        # clipped: the plain norm is well above
    assert float(o["norm"]) > 0.5
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = step()
    for v in c.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for name in o:
        assert torch.equal(c[name], o[name]), name


def _chain(x, logits, k, E, W):
    r = mxfp4.route(logits, k)
    p = mxfp4.expert_plan(r["ids"], E)
    xp = mxfp4.dispatch(x, p)
    y = mxfp4.combine(xp, p, r["weights"], out_dtype=F32)
    g = mxfp4.combine_bwd(x, xp, p, r["weights"])
    dx = mxfp4.combine(g["dy"], p, out_dtype=F32)
    dl = mxfp4.route_bwd(logits, r["ids"], g["d_weights"])
    grads = [dx, dl, W.clone()]
    n = mxfp4.grad_clip(grads, 1.0)
    return [r["ids"], r["weights"], *p.values(), xp, y, g["dy"], g["d_weights"], *grads, n]


@pytest.mark.parametrize("T,E,k,C", [(40, 8, 2, 64), (700, 32, 4, 264), (30000, 32, 4, 40), (9000, 64, 8, 33)])
def test_calls_back_to_back_and_on_two_streams(T, E, k, C):
    """Every kernel may be put in place before the previous one has ended:
    chains of dependent calls, repeated without waiting on fresh and reused
    buffers, alone and on two streams at a time, give what each call gives
    when the device is idle before and after it."""
    sets = []
    for i in range(2):
        sets.append((rand(T, C, seed=i, dtype=BF16), rand(T, E, seed=10 + i, std=1.5), rand(1000 * (i + 1), seed=20 + i)))
    want = []
    for x, l, w in sets:
        torch.cuda.synchronize()
        # one call at a time
        r = mxfp4.route(l, k); torch.cuda.synchronize()
        p = mxfp4.expert_plan(r["ids"], E); torch.cuda.synchronize()
        xp = mxfp4.dispatch(x, p); torch.cuda.synchronize()
        y = mxfp4.combine(xp, p, r["weights"], out_dtype=F32); torch.cuda.synchronize()
        g = mxfp4.combine_bwd(x, xp, p, r["weights"]); torch.cuda.synchronize()
        dx = mxfp4.combine(g["dy"], p, out_dtype=F32); torch.cuda.synchronize()
        dl = mxfp4.route_bwd(l, r["ids"], g["d_weights"]); torch.cuda.synchronize()
        grads = [dx, dl, w.clone()]
        n = mxfp4.grad_clip(grads, 1.0); torch.cuda.synchronize()
        want.append([r["ids"], r["weights"], *p.values(), xp, y, g["dy"], g["d_weights"], *grads, n])
    for _ in range(3):
        got = [_chain(x, l, k, E, w) for x, l, w in sets for _ in range(2)]
        torch.cuda.synchronize()
        for i, o in enumerate(got):
            assert all(torch.equal(a, b) for a, b in zip(o, want[i // 2]))
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(4):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i] = _chain(sets[i][0], sets[i][1], k, E, sets[i][2])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


def test_captured_after_copies_fills_and_joins():
    """Capture with a copy, a fill and a join of two streams right before the
    calls, and with a copy right behind them."""
    T, E, k, C = 500, 16, 4, 128
    x, l, w = rand(T, C, seed=1, dtype=BF16), rand(T, E, seed=2, std=1.5), rand(100, seed=3)
    want = _chain(x, l, k, E, w)
    xs, ls = torch.zeros_like(x), torch.zeros_like(l)
    ws = torch.zeros_like(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            ls.copy_(l)
        xs.copy_(x)
        ws.zero_()
        ws.add_(w)
        main.wait_stream(side)
        out = _chain(xs, ls, k, E, ws)
        copies = [torch.empty_like(o) for o in out]
        for c, o in zip(copies, out):
            c.copy_(o)
    for _ in range(3):
        for c in copies:
            c.zero_()
        ls.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, want))


def test_named_streams_and_supplied_outputs():
    """Every call on a named stream, with its outputs supplied and with one of
    them missing, gives what it gives on the current stream."""
    T, E, k, C = 300, 16, 4, 136
    x, l = rand(T, C, seed=1, dtype=BF16), rand(T, E, seed=2, std=1.5)
    w = rand(50, seed=3)
    want = _chain(x, l, k, E, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = mxfp4.route(l, k, stream=s)
    rows = want[5].numel()
    p0 = {"slot_of_row": torch.empty(rows, dtype=torch.int32, device="cuda"), "note": "not a part"}
    torch.cuda.synchronize()
    p = mxfp4.expert_plan(r["ids"], E, out=p0, stream=s)
    assert p["slot_of_row"] is p0["slot_of_row"]
    xp = mxfp4.dispatch(x, p, stream=s)
    y = mxfp4.combine(xp, p, r["weights"], out_dtype=F32, stream=s)
    dw = torch.empty((T, k), device="cuda")
    torch.cuda.synchronize()
    g = mxfp4.combine_bwd(x, xp, p, r["weights"], out={"d_weights": dw}, stream=s)
    dx = mxfp4.combine(g["dy"], p, out_dtype=F32, stream=s)
    dl = mxfp4.route_bwd(l, r["ids"], g["d_weights"], stream=s)
    with torch.cuda.stream(s):
        grads = [dx, dl, w.clone()]
    n = mxfp4.grad_clip(grads, 1.0, stream=s)
    s.synchronize()
    got = [r["ids"], r["weights"], *(p[q] for q in ("counts", "offsets", "row_of_slot", "slot_of_row")), xp, y, g["dy"],
           g["d_weights"], *grads, n]
    assert g["d_weights"] is dw
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_helper_refusals():
    plan = make_plan(20, 2, 4)
    rows = plan["slot_of_row"].numel()
    x, y, w = rand(20, 16, dtype=BF16), rand(rows, 16), rand(20, 2)
    l = rand(20, 8)
    bad = [lambda: mxfp4.dispatch(x[:19], plan), lambda: mxfp4.dispatch(x.half(), plan), lambda: mxfp4.dispatch(x.t(), plan),
           lambda: mxfp4.dispatch(x, plan, out=torch.empty(rows, 16, device="cuda")),
           lambda: mxfp4.dispatch(x[:1].expand(20, 16), plan),
           lambda: mxfp4.dispatch(x, {**plan, "slot_of_row": plan["slot_of_row"].long()}),
           lambda: mxfp4.dispatch(x, {**plan, "row_of_slot": plan["row_of_slot"].cpu()}),
           lambda: mxfp4.combine(y[:-1], plan), lambda: mxfp4.combine(y, plan, w[:, :1]), lambda: mxfp4.combine(y, plan, w.half()),
           lambda: mxfp4.combine(y, plan, w, out=torch.empty(20, 15, device="cuda")),
           lambda: mxfp4.combine_bwd(x, y, plan, w.t().contiguous().t()), lambda: mxfp4.combine_bwd(x[:, :8], y, plan, w),
           lambda: mxfp4.combine_bwd(x, y, plan, w, out={"dy": torch.empty_like(y)}),
           lambda: mxfp4.route(l, 2, bias=rand(7)), lambda: mxfp4.route(l, 2, mask=torch.ones(19, dtype=torch.bool, device="cuda")),
           lambda: mxfp4.route(l, 2, mask=torch.ones(20, device="cuda")), lambda: mxfp4.route(l, 2, score="tanh"),
           lambda: mxfp4.route(l.double(), 2), lambda: mxfp4.route(l[0], 2), lambda: mxfp4.route(l, 2, bias=rand(8).cpu()),
           lambda: mxfp4.route_bwd(l, plan["row_of_slot"][:5], w[:5]), lambda: mxfp4.route_bwd(l, plan["row_of_slot"], w[:, :1]),
           lambda: mxfp4.route_bwd(l, plan["row_of_slot"], w, out=torch.empty(20, 8, dtype=BF16, device="cuda")),
           lambda: mxfp4.expert_plan(plan["row_of_slot"].long(), 4), lambda: mxfp4.expert_plan(plan["row_of_slot"].t(), 4),
           lambda: mxfp4.expert_plan(plan["row_of_slot"], 0),
           lambda: mxfp4.expert_plan(plan["row_of_slot"], 4, out={"counts": torch.empty(5, dtype=torch.int32, device="cuda")}),
           lambda: mxfp4.route(l, 2, stream=torch.cuda.Stream()) and mxfp4.route(l.cpu(), 2)]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            print("call", i, "was not refused")
    for call in (lambda: mxfp4.route(l, 9), lambda: mxfp4.route(l, 2, groups=3), lambda: mxfp4.route(l, 2, scale=float("inf")),
                 lambda: mxfp4.expert_plan(plan["row_of_slot"], 4, align=100),
                 lambda: mxfp4.expert_plan(plan["row_of_slot"], 4, rows=rows - 128)):
        with pytest.raises(mxfp4.MXFP4Error):
            call()
