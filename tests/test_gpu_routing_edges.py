"""GPU parity of the routing calls where values meet: experts behind a tie at
the cut, scores that vanish in binary32, and logits that are not finite where
binary32 scores make the choice."""
import itertools

import numpy as np
import pytest
import torch

from fp4_precision_numerics_b200 import mxfp4
from tests import routing_ref as ref
from tests.test_gpu_routing import check_route
from tests.routing_ref import HALF_F32, f64, half_step

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def ids_of(logits, k, **kw):
    got = mxfp4.route(logits, k, **kw)["ids"].cpu().numpy()
    rk = {n: (f64(v) if isinstance(v, torch.Tensor) else v) for n, v in kw.items()}
    return got, ref.route(f64(logits), k, **rk)[0]


def behind_a_tie(E, n, low, tied, best, top=(), seed=0):
    """Rows of E logits at `low`, the values of `top` on their first experts,
    and in each row three other experts with the logits tied, tied and best,
    in every order of index, and a fourth one with `tied` in every other row.
    The three lie in one lane's registers, in neighbouring lanes, or anywhere."""
    rng = np.random.default_rng(seed)
    l = np.full((n * 6, E), low, dtype=np.float32)
    l[:, :len(top)] = top
    t = 0
    for i in range(n):
        free = np.arange(len(top), E)
        if i % 3 == 0 and E >= 160:
            at = int(rng.integers(0, 32)) + 32 * np.arange(1, E // 32)     # a lane's
            at = at[at < E]
        elif i % 3 == 1:
            at = free[:6]
        else:
            at = free
        for order in itertools.permutations(range(3)):
            three = np.sort(rng.choice(at, 3, replace=False))[list(order)]
            l[t, three[0]] = l[t, three[1]] = tied
            l[t, three[2]] = best
            if t % 2:
                rest = np.setdiff1d(free, three)
                l[t, rng.choice(rest)] = tied
            t += 1
    return torch.from_numpy(l).cuda()


EXPERTS = [32, 64, 128, 250, 512, 1024]


@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_an_expert_behind_a_tie_at_the_cut_by_logits(E, score):
    """A binary32 logit one step above two equal ones, where the keys compared
    first leave out a logit's last bits."""
    for one in (1.0, -1.0, 1e-30):
        best = float(np.nextafter(np.float32(one), np.float32(9)))
        for top in ((), (5.0, 4.0)):
            l = behind_a_tie(E, 9, -3.0, one, best, top)
            for k in (1, 2, 3, 4):
                got, want = ids_of(l, k, score=score)
                assert np.array_equal(got, want), (one, top, k)
    g = 4 if E % 4 == 0 else 5
    l = behind_a_tie(E, 9, -3.0, 1.0, float(np.nextafter(np.float32(1), np.float32(2))))
    for k in (1, 2, 3):
        got, want = ids_of(l, k, score=score, groups=g, top_groups=2)
        assert np.array_equal(got, want), k


@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_an_expert_behind_a_tie_at_the_cut_by_scores(E, dtype):
    """Scores with a bias that are one value in binary32 and two in binary64:
    a saturated sigmoid, very negative logits, and a softmax's smallest terms."""
    def check(l, bias, **kw):
        for k in (1, 2, 3, 4):
            got, want = ids_of(l, k, bias=bias, **kw)
            assert np.array_equal(got, want), (k, kw)
    zero = torch.zeros(E, device="cuda")
    half = torch.full((E,), 0.5, device="cuda")
    groups = dict(groups=2, top_groups=1)
    for tied, best, low in ((17.0, 17.125, 1.0), (-19.0, -18.875, -30.0)):
        for top in ((), (25.0, 24.0)):
            l = behind_a_tie(E, 9, low, tied, best, top).to(dtype)
            for bias in (zero, half):
                check(l, bias, score="sigmoid")
                check(l, bias, score="sigmoid", group_best=2, **groups)
    l = behind_a_tie(E, 9, -40.0, -20.0, -19.875, (0.0, -0.5)).to(dtype)
    for bias in (zero, half):
        check(l, bias, score="softmax")
        check(l, bias, score="softmax", group_best=2, **groups)


def test_whole_rows_of_ties():
    """Every expert an exact tie, but for one in the last place."""
    for E in (33, 64, 256, 1000):
        l = torch.full((2, E), 1.0, device="cuda")
        l[1, E - 1] = float(np.nextafter(np.float32(1), np.float32(2)))
        for k in (1, 5, 32):
            for kw in (dict(), dict(score="sigmoid", bias=torch.zeros(E, device="cuda"))):
                got, want = ids_of(l, k, **kw)
                assert np.array_equal(got, want)


def low_logits(T, E, dtype, seed=0):
    """Rows of logits around -75 ... -650, and one row in eight below -720."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    at = -75.0 - 575.0 * torch.rand((T, 1), generator=g, device="cuda") ** 2
    l = at + 4.0 * torch.randn((T, E), generator=g, device="cuda")
    l[::8] -= 800.0
    return l.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_weights_and_gradients_of_very_negative_logits(dtype, renorm):
    """Scores below binary32's range still have weights when renormalised.
    Rounding: the difference from the largest logit is off by half a step of
    it (at most |x|), two exponentials by four half steps each, then three sums,
    two divisions and the scale; the gradient has two such scores and the
    dot product over the slots besides.  Below, half a step of the smallest
    binary32 numbers for each of at most 64 operations."""
    T, E, k = 200, 48, 5
    l = low_logits(T, E, dtype)
    l[1, 7], l[3, 7], l[5] = 3.0, -1.0, -85.0
    for bias in (None, torch.zeros(E, device="cuda")):
        got = mxfp4.route(l, k, score="sigmoid", renormalise=renorm, scale=2.0, bias=bias)
        ids, w = ref.route(f64(l), k, score="sigmoid", renormalise=renorm, scale=2.0)
        if bias is None:         # under a bias the scores of such rows are ties in binary64 too
            assert np.array_equal(got["ids"].cpu().numpy(), ids)
            tol = HALF_F32 * (2 * 700 + 8 + 3 + 2 + 1)
            assert np.all(abs(f64(got["weights"]) - w) <= tol * w + 64 * 2.0 ** -150)
        live = f64(l).max(1) > -700
        if renorm:
            assert np.all(abs(f64(got["weights"]).sum(1)[live] - 2.0) <= 16 * HALF_F32 * 2.0)
        assert not f64(got["weights"])[f64(l).max(1) < -710].any()
    ids = mxfp4.route(l, k, score="sigmoid")["ids"]
    dw = torch.randn((T, k), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    out = mxfp4.route_bwd(l, ids, dw, score="sigmoid", renormalise=renorm, scale=2.0)
    g, mag = ref.route_bwd(f64(l), ids.cpu().numpy(), f64(dw), "sigmoid", renorm, 2.0)
    tol = HALF_F32 * (4 * 700 + 2 * 16 + k + 8)
    assert np.all(abs(f64(out) - g) <= tol * mag + half_step(dtype) * (1 + tol) * abs(g) + 64 * 2.0 ** -150 +
                  (2.0 ** -134 if dtype == BF16 else 0.0))


@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_bias_is_for_the_choice_only(E, dtype):
    """The chosen experts' softmax weights are the same bits with and without
    a bias of zeros."""
    g = torch.Generator(device="cuda").manual_seed(E)
    for std in (0.0, 0.5, 1.5, 6.0):
        l = (torch.randn((300, E), generator=g, device="cuda") * std).to(dtype)
        l[:, 0] += 1.0
        for renorm in (True, False):
            a = mxfp4.route(l, 4, renormalise=renorm)
            b = mxfp4.route(l, 4, renormalise=renorm, bias=torch.zeros(E, device="cuda"))
            assert torch.equal(a["ids"], b["ids"])
            assert torch.equal(a["weights"], b["weights"]), (std, renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [48, 96, 256, 768])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinities_and_nan_where_scores_make_the_choice(score, E, dtype):
    """Logits, and then biases, that are not finite under a bias or with
    two-best groups, where binary32 scores are compared first."""
    inf, nan = float("inf"), float("nan")
    g = torch.Generator(device="cuda").manual_seed(E)
    l = torch.randn((24, E), generator=g, device="cuda") * 1.5
    l[0] = -inf
    l[1, 3:] = -inf                  # fewer finite logits than top_k
    l[2, 10] = nan
    l[3, 11] = inf
    l[4] = -1e4
    l[5] = nan
    l[6, 5] = -inf
    l[7, 1:] = nan                   # one score that counts
    l[8, ::2] = nan
    l[9] = inf
    l[10, ::3] = inf
    l[11, 2], l[11, 3], l[11, 4] = nan, inf, -inf
    l[12, E // 4:] = nan             # whole groups
    l[13, :E // 4] = -inf
    l[14, :E // 2] = nan
    l = l.to(dtype)
    mask = torch.rand(24, generator=g, device="cuda") < 0.8
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    odd = bias.clone()
    odd[1], odd[4], odd[E // 4 + 2], odd[E // 2:E // 2 + 3] = inf, nan, -inf, -inf
    for b in (bias, torch.zeros_like(bias), odd):
        for m in (None, mask):
            for renorm in (True, False):
                kw = dict(score=score, bias=b, mask=m, renormalise=renorm)
                check_route(l, 5, **kw)
                for best in (1, 2):
                    check_route(l, 5, groups=4, top_groups=2, group_best=best, **kw)
    check_route(l, 5, score=score, groups=4, top_groups=2, group_best=2)
    check_route(l, 5, score=score, groups=8, top_groups=1, group_best=2, renormalise=False)
