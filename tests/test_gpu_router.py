"""GPU parity of the expert router against a plain implementation in 64 bits on the CPU.

The choice has to be equal.  Tolerances of the weights: with u = 2^-24, exp is off by 2 u and its
argument's rounding by |l - m| u, sums of n terms by (n + 2) u at most, and the product and quotients
by u each; the gradients add the sum over the k chosen, whose terms' magnitudes are counted."""
import math

import pytest
import torch

import mixture_experts_ffn_permute_gb300 as moe
from mixture_experts_ffn_permute_gb300 import _build

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
NEG = -math.inf


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    moe.load()


def rank(values, live):
    """Ids of the live values, highest first, NaN last, ties to the lowest id."""
    ids = [i for i in range(len(values)) if live[i]]
    return sorted(ids, key=lambda i: (math.isnan(values[i]), 0 if math.isnan(values[i]) else -values[i], i))


def reference(p, logits, bias):
    """(ids [T][k], scores [T, E]) by the definition, token by token."""
    l64 = logits.double()
    s = torch.sigmoid(l64) if p.score else torch.softmax(l64, 1)
    ids = []
    for t in range(p.T):
        live = [x != NEG for x in l64[t].tolist()]
        key = (l64[t] if bias is None else s[t] + bias.double()).tolist()
        by = (s[t] if bias is None else s[t] + bias.double()).tolist()
        if not p.score and bool(s[t].isnan().any()):
            key = [math.nan] * p.E  # a softmax with a NaN is NaN everywhere
        per = p.E // p.groups
        score, some = [], []
        for g in range(p.groups):
            best = rank(by[g * per:(g + 1) * per], live[g * per:(g + 1) * per])[:p.group_top]
            score.append(sum(by[g * per + i] for i in best))
            some.append(bool(best))
        kept = set(rank(score, some)[:p.topk_groups])
        if p.topk_groups == p.groups:
            kept = set(range(p.groups))
        live = [live[e] and e // per in kept for e in range(p.E)]
        chosen = rank(key, live)[:p.k]
        ids.append(chosen + [-1] * (p.k - len(chosen)))
    return torch.tensor(ids, dtype=torch.int64).reshape(p.T, p.k), s


def weights_of(p, s, logits, ids):
    """Weights in 64 bits; small sigmoids relative to each other, as the ratio has them."""
    at, have = ids.clamp(min=0), ids >= 0
    w = torch.where(have, s.gather(1, at), torch.zeros((), dtype=torch.float64))
    if p.renormalize:
        w = torch.where(have, w / w.sum(1, keepdim=True), torch.zeros((), dtype=torch.float64))
    return w * p.scale


def run(p, logits, bias=None):
    idx = torch.full((p.T, p.k), -9, dtype=torch.int32, device=DEV)
    w = torch.full((p.T, p.k), math.nan, device=DEV)
    moe.router_forward(p, logits.to(DEV), idx, w, bias=None if bias is None else bias.to(DEV))
    torch.cuda.synchronize()
    return idx.cpu().long(), w.cpu()


def tolerance(p, logits):
    finite = torch.where(torch.isfinite(logits.double()), logits.double(), torch.zeros((), dtype=torch.float64))
    spread = float((finite.amax(1) - finite.amin(1)).amax()) if p.T else 0.0
    return (2 * (3 + spread) + p.E / 4 + 20) * 2.0 ** -24


def check(p, logits, bias=None):
    ids, s = reference(p, logits, bias)
    idx, w = run(p, logits, bias)
    assert torch.equal(idx, ids), (idx != ids).nonzero()[:4].tolist()
    want = weights_of(p, s, logits, ids)
    err = (w.double() - want).abs()
    assert (err <= tolerance(p, logits) * want.abs()).all(), float((err / want.abs()).nan_to_num().max())
    return ids, s


def draw(T, E, dtype=F32, seed=0, std=1.5):
    g = torch.Generator().manual_seed(seed + 1000 * E + T)
    return (torch.randn(T, E, generator=g) * std).to(dtype), torch.randn(E, generator=g) * 0.1


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (7, 3), (31, 5), (32, 32), (33, 1), (60, 4), (64, 8),
                                 (100, 10), (128, 8), (255, 8), (256, 31), (392, 7), (512, 8),
                                 (1000, 6), (1024, 32)])
def test_widths(E, k, score, dtype):
    logits, bias = draw(67, E, dtype)
    for renorm in (True, False):
        p = moe.RouterProblem.make(67, E, k, dtype, score, renormalize=renorm, scale=1.7)
        check(p, logits)
        check(p, logits, bias)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 1216, 1217, 3001])
def test_token_counts(T):
    logits, bias = draw(T, 64)
    check(moe.RouterProblem.make(T, 64, 6, score="sigmoid", groups=4, topk_groups=2, group_top=2),
          logits, bias)


@pytest.mark.parametrize("E,groups", [(256, 8), (128, 8), (64, 32), (64, 2), (60, 4), (60, 30), (24, 3),
                                      (400, 8), (512, 16), (96, 3), (1024, 32), (8, 4)])
def test_groups(E, groups):
    logits, bias = draw(101, E)
    for score in ("softmax", "sigmoid"):
        for top in (1, 2):
            for kept in sorted({1, (groups + 1) // 2, groups - 1, groups}):
                if kept < 1:
                    continue
                k = min(8, kept * (E // groups))
                p = moe.RouterProblem.make(101, E, k, score=score, groups=groups, topk_groups=kept,
                                           group_top=top)
                check(p, logits, bias)
                check(p, logits)


def test_equal_scores_go_to_the_lowest_id():
    T, E = 50, 256
    g = torch.Generator().manual_seed(3)
    few = torch.randint(0, 4, (T, E), generator=g).float()  # many equal logits
    bias = torch.randint(0, 3, (E,), generator=g).float() * 0.25
    for logits in (torch.zeros(T, E), few, -0.0 * few):
        for score in ("softmax", "sigmoid"):
            for b in (None, torch.zeros(E), bias):
                check(moe.RouterProblem.make(T, E, 8, score=score, groups=8, topk_groups=3, group_top=2),
                      logits, b)
                check(moe.RouterProblem.make(T, E, 9, score=score), logits, b)


def test_scores_that_fp32_cannot_tell():
    """Pairs whose scores differ by less than fp32 shows, in either order, and groups whose sums do."""
    T, E = 64, 128
    logits, bias = draw(T, E, std=1.0)
    g = torch.Generator().manual_seed(5)
    s = torch.sigmoid(logits.double())
    for t in range(T):  # experts 64.. copy the scores of 0.. through another bias, almost
        logits[t, 64:] = logits[t, :64]
    order = torch.randperm(64, generator=g)
    logits[:, 64:] = logits[:, :64][:, order]
    bias = torch.zeros(E)
    for score in ("softmax", "sigmoid"):
        for kept, top in ((2, 1), (1, 2), (1, 1)):
            p = moe.RouterProblem.make(T, E, 8, score=score, groups=2, topk_groups=kept, group_top=top)
            check(p, logits, bias)
    # scores next to each other: neighbouring floats as logits
    base = torch.linspace(-2, 2, T)[:, None].expand(T, E).contiguous()
    near = base.clone()
    steps = torch.randint(0, 6, (T, E), generator=g)
    for _ in range(6):
        near = torch.where(steps > 0, torch.nextafter(near, torch.full_like(near, 9.0)), near)
        steps -= 1
    tiny = torch.randint(0, 3, (E,), generator=g).float() * 2.0 ** -40
    for score in ("softmax", "sigmoid"):
        check(moe.RouterProblem.make(T, E, 8, score=score), near, tiny)
        check(moe.RouterProblem.make(T, E, 32, score=score), near, tiny)
        check(moe.RouterProblem.make(T, E, 8, score=score, groups=16, topk_groups=4, group_top=2), near, tiny)


@pytest.mark.parametrize("E", [64, 256, 512])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_groups_that_fp32_cannot_tell(E, dtype):
    """Groups that are copies of others but for steps of 2^-24 or of 2^-44, with and without a bias."""
    T, groups, half = 120, 8, E // 2
    logits, bias = draw(T, E, dtype, seed=21)
    g = torch.Generator().manual_seed(E)
    logits[:, half:] = logits[:, :half]
    if dtype == F32:
        up = torch.nextafter(logits[:, half:], torch.full((T, half), 9.0))
        logits[:, half:] = torch.where(torch.rand(T, half, generator=g) < 0.3, up, logits[:, half:])
    bias[half:] = bias[:half]
    tiny = torch.zeros(E)
    tiny[half:] = torch.randint(0, 3, (half,), generator=g).float() * 2.0 ** -44
    for score in ("softmax", "sigmoid"):
        for kept, top in ((1, 2), (3, 2), (5, 1)):
            for b in (None, bias, torch.zeros(E), tiny):
                check(moe.RouterProblem.make(T, E, 8, dtype, score, groups=groups, topk_groups=kept,
                                             group_top=top), logits, b)


@pytest.mark.parametrize("E", [200, 320, 512, 1000])
def test_neighbouring_scores_of_many_experts(E):
    """Logits a float or two apart, with biases that differ by less than fp32 shows, over all lanes."""
    T = 48
    g = torch.Generator().manual_seed(E)
    logits = torch.linspace(-2, 2, T)[:, None].expand(T, E).contiguous()
    steps = torch.randint(0, 4, (T, E), generator=g)
    for _ in range(4):
        logits = torch.where(steps > 0, torch.nextafter(logits, torch.full_like(logits, 9.0)), logits)
        steps -= 1
    far = torch.rand(T, E, generator=g) < 0.97
    logits = torch.where(far, logits - 3.0, logits)
    tiny = torch.randint(0, 3, (E,), generator=g).float() * 2.0 ** -41
    for score in ("softmax", "sigmoid"):
        for b in (tiny, torch.zeros(E), 0.5 + tiny):
            check(moe.RouterProblem.make(T, E, 8, score=score), logits, b)
            p = moe.RouterProblem.make(T, E, 8, score=score, groups=4, topk_groups=2, group_top=2)
            # Two pairs of neighbouring logits with the same sum have scores whose sums differ by
            # the curvature, some 2^-52: 64 bits do not tell such groups.  A score takes four
            # roundings of 2^-53 at most, its bias one, the sum of two one of 2^-52 (it is below
            # 4): 2^-49 for a group, 2^-48 for the difference of two.
            ids, s = reference(p, logits, b)
            sums = (s + b.double()).view(T, 4, E // 4).topk(2).values.sum(2).sort(1, descending=True).values
            told = (sums[:, 1] - sums[:, 2]) > 2.0 ** -48
            idx, _ = run(p, logits, b)
            assert torch.equal(idx[told], ids[told])
            assert told.sum() >= 16  # (22 of 48 at the fewest: E=1000 without a bias)


def test_biases_that_cancel_in_a_group():
    """Two best experts with biases of opposite sign and far above the scores: a sum as small as a score."""
    T, E = 300, 64
    logits, bias = draw(T, E, seed=31)
    bias = bias - 1000.0
    bias[0::8], bias[1::8] = 100.0, -100.0
    logits[:, 8:] = logits[:, :8].repeat(1, 7) + 1e-5 * torch.randn(T, 56, generator=torch.Generator().manual_seed(4))
    for score in ("softmax", "sigmoid"):
        for kept in (1, 4, 7):
            check(moe.RouterProblem.make(T, E, 5, score=score, groups=8, topk_groups=kept, group_top=2),
                  logits, bias)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("low", [NEG, torch.finfo(F32).min])
def test_experts_taken_out_by_their_bias(low, dtype):
    """-inf or the type's lowest value for some experts, for whole groups, for all but a few; +inf."""
    T, E = 40, 64
    logits, bias = draw(T, E, dtype, seed=41)
    some = bias.clone()
    some[torch.rand(E, generator=torch.Generator().manual_seed(6)) < 0.5] = low
    whole = some.clone()
    whole[8:32] = low
    few = torch.full((E,), low)
    few[50], few[51], few[9] = 0.0, math.inf, -0.25
    mixed = whole.clone()
    mixed[20], mixed[21] = NEG, torch.finfo(F32).min
    for b in (some, whole, few, mixed):
        for score in ("softmax", "sigmoid"):
            for kept, top, k in ((8, 1, 6), (2, 2, 12), (6, 2, 31), (5, 1, 32)):
                p = moe.RouterProblem.make(T, E, k, dtype, score, groups=8, topk_groups=kept, group_top=top)
                ids, _ = reference(p, logits, b)
                assert torch.equal(run(p, logits, b)[0], ids), (kept, top, k)


def test_experts_out_of_the_choice():
    T, E = 40, 64
    logits, bias = draw(T, E)
    g = torch.Generator().manual_seed(9)
    logits[torch.rand(T, E, generator=g) < 0.8] = NEG
    logits[0] = NEG          # none
    logits[1, 1:] = NEG      # one
    logits[2, :56] = NEG     # one group
    for dtype in (F32, BF):
        l = logits.to(dtype)
        for score in ("softmax", "sigmoid"):
            for b in (None, bias, -bias.abs() - 1):
                for kept, top, k in ((8, 1, 16), (2, 2, 12), (3, 1, 4)):
                    for renorm in (True, False):
                        p = moe.RouterProblem.make(T, E, k, dtype, score, groups=8, topk_groups=kept,
                                                   group_top=top, renormalize=renorm)
                        check(p, l, b)
    p = moe.RouterProblem.make(T, E, 8)
    idx, w = run(p, logits)
    assert (idx[0] == -1).all() and (w[0] == 0).all()
    assert (idx[1] == -1).all() and (w[1] == 0).all()  # (its expert 0 is out as well)
    one = torch.full((1, E), NEG)
    one[0, 41] = -3.0
    idx, w = run(moe.RouterProblem.make(1, E, 8), one)
    assert idx[0].tolist() == [41] + [-1] * 7 and w[0].tolist() == [1.0] + [0.0] * 7


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinities_and_nan(score):
    T, E, k = 8, 48, 5
    logits, bias = draw(T, E)
    logits[0, 7] = math.inf
    logits[1, 7] = math.nan
    logits[2, 7], logits[2, 9] = math.nan, NEG
    logits[3, :] = math.nan
    logits[4, :44] = NEG
    logits[4, 45] = math.nan
    for b in (None, bias):
        p = moe.RouterProblem.make(T, E, k, score=score)
        ids, s = reference(p, logits, b)
        idx, w = run(p, logits, b)
        assert torch.equal(idx, ids)
        for t in range(T):
            here = [float(s[t, e]) for e in ids[t].tolist() if e >= 0]
            nan = [math.isnan(x) for x in here]
            want = [any(nan)] * len(here)  # renormalised: by a sum that is NaN
            assert [math.isnan(x) for x in w[t].tolist()] == want + [False] * (k - len(here)), t
    bias[3] = math.nan
    bias[4], bias[5] = math.inf, NEG
    p = moe.RouterProblem.make(T, E, 48 // 2, score=score)
    idx, _ = run(p, logits, bias)
    assert torch.equal(idx, reference(p, logits, bias)[0])


def test_small_sigmoids_keep_their_ratio():
    logits = torch.tensor([[-200.0, -201.0, -90.0 - 200, -199.0], [-19.0, -21.0, -25.0, -40.0],
                           [-21.0, -22.0, -23.0, -120.0], [100.0, 50.0, -100.0, 0.0]])
    p = moe.RouterProblem.make(4, 4, 3, score="sigmoid")
    check(p, logits)
    q = moe.RouterProblem.make(4, 4, 3, score="sigmoid", renormalize=False)
    idx, w = run(q, logits)
    want = torch.sigmoid(logits.double()).gather(1, idx)
    # (what fp32 holds of them: to 2^-149)
    assert ((w.double() - want).abs() <= 220 * 2.0 ** -24 * want + 2.0 ** -148).all()


def test_strided_rows():
    big, bias = draw(33, 200)
    for lo, E, dtype in ((0, 64, F32), (1, 64, F32), (3, 100, BF), (8, 128, BF)):
        whole = big.to(dtype).to(DEV)
        view = whole[:, lo:lo + E]
        p = moe.RouterProblem.make(33, E, 5, dtype, "sigmoid", ld_logits=200)
        idx = torch.empty(33, 5, dtype=torch.int32, device=DEV)
        w = torch.empty(33, 5, device=DEV)
        moe.router_forward(p, view, idx, w, bias=bias[:E].to(DEV))
        ids, _ = reference(p, view.cpu(), bias[:E])
        assert torch.equal(idx.cpu().long(), ids)
        out = torch.full_like(whole, 7.0)
        moe.router_backward(p, view, idx, torch.ones_like(w), out[:, lo:lo + E])
        assert (out[:, :lo] == 7).all() and (out[:, lo + E:] == 7).all()
        assert (out[:, lo:lo + E] != 7).all()


# ------------------------------------------------------------------ backward
def exact_grad(p, logits, ids, dw):
    l = logits.double().requires_grad_()
    have = ids >= 0
    s = torch.sigmoid(l) if p.score else torch.softmax(l, 1)
    w = torch.where(have, s.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=torch.float64))
    if p.renormalize:
        w = w / torch.where(have.any(1, keepdim=True), w.sum(1, keepdim=True), torch.ones((), dtype=torch.float64))
    grad, = torch.autograd.grad((w * p.scale * torch.where(have, dw.double(), torch.zeros((), dtype=torch.float64))).sum(), l)
    return grad


def check_backward(p, dtype, ids, logits, seed=0):
    g = torch.Generator().manual_seed(seed)
    dw = torch.randn(p.T, p.k, generator=g)
    out = torch.full((p.T, p.E), math.nan, dtype=dtype, device=DEV)
    moe.router_backward(p, logits.to(DEV), ids.to(DEV, torch.int32), dw.to(DEV), out)
    want = exact_grad(p, logits, ids, dw)
    # the terms' magnitude: every dw_j of the token times a weight of the element's size
    s = torch.sigmoid(logits.double()) if p.score else torch.softmax(logits.double(), 1)
    have = ids >= 0
    w = torch.where(have, s.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=torch.float64))
    total = w.sum(1, keepdim=True) if p.renormalize else torch.ones(p.T, 1, dtype=torch.float64)
    total = torch.where(total > 0, total, torch.ones((), dtype=torch.float64))
    mag = p.scale * s / total * (dw.double().abs() * have).sum(1, keepdim=True)
    rounding = 2.0 ** -8 if dtype is BF else 2.0 ** -24
    tol = rounding * want.abs() + 3 * tolerance(p, logits) * mag
    err = (out.double().cpu() - want).abs()
    assert (err <= tol + 1e-300).all(), float((err - tol).max())
    return dw, out


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(1, 1), (7, 3), (33, 4), (60, 6), (128, 8), (256, 8), (500, 32),
                                 (1024, 10)])
def test_backward(E, k, score, dtype):
    logits, bias = draw(71, E, dtype)
    for renorm in (True, False):
        p = moe.RouterProblem.make(71, E, k, dtype, score, renormalize=renorm, scale=2.5)
        ids, _ = reference(p, logits, bias)
        check_backward(p, dtype, ids, logits)


def test_backward_of_masked_slots_and_experts():
    T, E, k = 30, 40, 4
    logits, _ = draw(T, E)
    logits[torch.rand(T, E, generator=torch.Generator().manual_seed(2)) < 0.5] = NEG
    logits[0] = NEG
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            p = moe.RouterProblem.make(T, E, k, score=score, renormalize=renorm)
            ids, _ = reference(p, logits, None)
            ids[5:9, 1] = -1
            ids[9] = -1
            safe = torch.where(torch.isfinite(logits), logits, torch.full_like(logits, -1e4))
            dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1))
            dev = torch.where(ids < 0, torch.full_like(dw, math.nan), dw).to(DEV)  # not used
            odd = ids.clone()
            odd[10:12][ids[10:12] < 0] = E + 3  # beyond the experts: masked
            out = torch.full((T, E), math.nan, device=DEV)
            moe.router_backward(p, logits.to(DEV), odd.to(DEV, torch.int32), dev, out)
            want = exact_grad(p, safe, ids, dw)
            got = out.double().cpu()
            assert (got[0] == 0).all() and (got[9] == 0).all()
            assert ((got - want).abs() <= 1e-5 * dw.abs().sum(1, keepdim=True)).all()


def test_backward_of_an_expert_in_several_slots():
    T, E, k = 20, 50, 5
    logits, _ = draw(T, E)
    for dtype in (F32, BF):
        l = logits.to(dtype)
        for score in ("softmax", "sigmoid"):
            for renorm in (True, False):
                p = moe.RouterProblem.make(T, E, k, dtype, score, renormalize=renorm)
                ids, _ = reference(p, l, None)
                ids[3, 4] = ids[3, 0]
                ids[7:9] = 49
                ids[9, :3] = ids[9, 3]
                check_backward(p, dtype, ids, l)


def test_gradient_against_differences():
    """Central differences of the forward's own weights, in the part of the logits where the choice
    stays: a step of 2^-6 is off by its square times the third derivative (below 1/8 of the largest
    weight), 2^-15, and the weights' rounding over the step 2^-23 / 2^-6."""
    T, E, k = 16, 24, 5
    logits, _ = draw(T, E, std=3.0)
    g = torch.Generator().manual_seed(1)
    dw = torch.randn(T, k, generator=g)
    direction = torch.randn(T, E, generator=g)
    direction /= direction.abs().amax()
    h = 2.0 ** -6
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            p = moe.RouterProblem.make(T, E, k, score=score, renormalize=renorm)
            ids, w0 = run(p, logits)
            i1, w1 = run(p, logits + h * direction)
            i2, w2 = run(p, logits - h * direction)
            same = (i1 == ids).all(1) & (i2 == ids).all(1)
            assert same.sum() >= T // 2
            out = torch.empty(T, E, device=DEV)
            moe.router_backward(p, logits.to(DEV), ids.to(DEV, torch.int32), dw.to(DEV), out)
            got = (out.cpu().double() * direction).sum(1)
            want = ((w1 - w2).double() * dw).sum(1) / (2 * h)
            err = (got - want).abs()[same]
            assert (err <= (2.0 ** -13 + 2.0 ** -16) * dw.abs().sum(1).double()[same]).all(), err


def test_graph_replay_and_streams():
    logits, bias = draw(300, 128)
    p = moe.RouterProblem.make(300, 128, 8, score="sigmoid", groups=8, topk_groups=3, group_top=2)
    buf, b = logits.to(DEV), bias.to(DEV)
    idx = torch.empty(300, 8, dtype=torch.int32, device=DEV)
    w, dl = torch.empty(300, 8, device=DEV), torch.empty(300, 128, device=DEV)
    dw = torch.ones(300, 8, device=DEV)
    moe.router_forward(p, buf, idx, w, bias=b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.router_forward(p, buf, idx, w, bias=b)
        moe.router_backward(p, buf, idx, dw, dl)
    other, _ = draw(300, 128, seed=4)
    buf.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    ids, _ = reference(p, other, bias)
    assert torch.equal(idx.cpu().long(), ids)
    first = (w.clone(), dl.clone())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.router_forward(p, buf, idx, w, bias=b, stream=s)
    moe.router_backward(p, buf, idx, dw, dl, stream=s)
    s.synchronize()
    assert torch.equal(w, first[0]) and torch.equal(dl, first[1])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E,groups", [(192, 8), (200, 4), (240, 6), (129, 3), (250, 10), (160, 4), (60, 4),
                                      (400, 8), (256, 8)])
def test_experts_out_of_the_choice_in_groups(E, groups, dtype):
    """Logits of -inf beside the best experts of groups, above all at the places 8 i + 7: they take
    nothing from their group's score."""
    T = 40
    logits, bias = draw(T, E, dtype, seed=61)
    g = torch.Generator().manual_seed(E)
    logits[torch.rand(T, E, generator=g) < 0.25] = NEG
    for t in range(T):
        for best in range(8 * (t % 5) + 7, E, 40):
            logits[t, best] = 3.0 + 0.125 * int(torch.randint(0, 16, (1,), generator=g))
            logits[t, best - 1 - t % 7] = NEG
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            for kept, top in ((1, 1), (groups // 2, 2), (groups - 1, 1)):
                check(moe.RouterProblem.make(T, E, 8, dtype, score, groups=groups, topk_groups=kept,
                                             group_top=top), logits, b)


@pytest.mark.parametrize("E", [33, 60, 256, 320, 512, 1000])
def test_runner_up_of_32_picks(E):
    """k = 32 with a bias: picks far apart but for the last one and the first left out, which differ by
    a step or two of fp32, by less than fp32 shows, or not at all."""
    T = 60
    g = torch.Generator().manual_seed(E)
    order = torch.stack([torch.randperm(E, generator=g) for _ in range(T)])
    place = torch.arange(E).clamp(max=60).float()
    values = 3.0 - 0.1 * place + 0.02 * torch.rand(T, E, generator=g)
    values[:, 32] = values[:, 31]
    for t in range(T):
        for _ in range(t % 3):
            values[t, 32] = torch.nextafter(values[t, 32], torch.tensor(9.0 if t % 2 else -9.0))
    logits = torch.empty(T, E).scatter_(1, order, values)
    tiny = torch.randint(0, 3, (E,), generator=g).float() * 2.0 ** -42
    for score in ("softmax", "sigmoid"):
        for b in (torch.zeros(E), tiny):
            check(moe.RouterProblem.make(T, E, 32, score=score), logits, b)
            if E % 4 == 0 and E > 60:
                check(moe.RouterProblem.make(T, E, 32, score=score, groups=4, topk_groups=3, group_top=2),
                      logits, b)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E", [37, 64, 100, 256, 320, 600, 1000])
def test_equal_experts_at_the_border_of_the_choice(E, dtype):
    """The last pick and the first expert left out are the same, and one behind them is higher by less
    than fp32 shows, or lower, or the same too; with and without groups, with picks above them."""
    T = 48
    g = torch.Generator().manual_seed(E)
    logits = torch.rand(T, E, generator=g) - 8.0
    next_up = float(torch.nextafter(torch.tensor(0.5), torch.tensor(9.0)))
    for t in range(T):
        ids = torch.randperm(E, generator=g)[:8].sort().values
        low, high = ((27.5, 81.5), (20.0, 20.125), (0.5, next_up), (0.5, 0.50390625))[t % 4]
        logits[t, ids] = low
        for i in ids[2 + t % 5:].tolist():
            logits[t, i] = (high, low, low - 0.125)[int(torch.randint(0, 3, (1,), generator=g))]
        if t % 4 > 1:
            logits[t, ids[torch.randperm(8, generator=g)[:2]]] = torch.tensor([3.0, 4.0])
    for score in ("sigmoid", "softmax"):
        l = logits if score == "sigmoid" else torch.where(logits > 0, logits * 2.0 ** -10, logits)
        for b in (torch.zeros(E), torch.full((E,), 0.25)):
            for k in (1, 2, 3, 5, 7, 31, 32):
                check(moe.RouterProblem.make(T, E, k, dtype, score), l.to(dtype), b)
            if E % 4 == 0:
                check(moe.RouterProblem.make(T, E, 2, dtype, score, groups=4, topk_groups=3), l.to(dtype), b)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E,groups", [(20, 4), (64, 8), (192, 8), (256, 8), (512, 8), (1000, 5)])
def test_an_infinite_bias_beside_the_lowest(E, groups, dtype):
    """A group's two best are an expert of +inf and one of the type's lowest value (their sum is +inf), of
    -inf (no number), or a few steps above the lowest."""
    T, per = 30, E // groups
    logits, bias = draw(T, E, dtype, seed=71)
    low = torch.finfo(F32).min
    for g, other in ((1, low), (2, NEG), (3, low * (1 - 2.0 ** -22))):
        lo = g * per
        logits[:, lo + 2:lo + per] = NEG
        logits[::3, lo + 1] = NEG  # (alone in its group)
        bias[lo], bias[lo + 1] = (math.inf, other) if g != 2 else (other, math.inf)
    for score in ("softmax", "sigmoid"):
        for kept, top in ((1, 2), (2, 2), (3, 2), (2, 1)):
            p = moe.RouterProblem.make(T, E, min(3, kept * per), dtype, score, groups=groups, topk_groups=kept,
                                       group_top=top)
            ids, _ = reference(p, logits, bias)
            assert torch.equal(run(p, logits, bias)[0], ids), (score, kept, top)
