"""GPU parity of the linear cross entropy (moe_linear_ce_*) against 64 bits.

Tolerances.  The operands are bf16, their products exact; a logit is the sum of
H of them, added sixteen at a time into an fp32 accumulator: within
ez = (H / 16 + 4) 2^-23 of its terms' magnitude.  lse moves by at most its
logits' error, plus the exponentials' and the sums' (2^-20 with room); the loss
takes one logit more.  The backward rounds d z to bf16 (2^-8 of it, and p times
its exponent's error) before the products with w and x, whose sums are fp32 and
whose results are rounded once (2^-8).  The bounds are worst cases, so the RMS
relative error is held to 5e-3 too, as for the layer's own gradients."""
import pytest
import torch

import mixture_experts_ffn_permute_gb300 as moe
from mixture_experts_ffn_permute_gb300 import _build

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    moe.load()


def inputs(T, H, V, seed=0, masked=0.2, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(BF).to(DEV)
    w = (torch.randn(V, H, generator=g) * spread / H ** 0.5).to(BF).to(DEV)
    labels = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    labels = torch.where(torch.rand(T, generator=g) < masked, -100, labels).to(torch.int32)
    d_loss = torch.rand(T, generator=g).to(DEV)
    return x, w, labels.to(DEV), d_loss


def forward(p, x, w, labels, ws, stream=None):
    nan = float("nan")
    loss, lse = (torch.full((p.T,), nan, device=DEV) for _ in range(2))
    moe.linear_ce_forward(p, x, w, labels, loss, lse, ws, stream=stream)
    return loss, lse


def backward(p, x, w, labels, lse, d_loss, ws, d_lse=None, stream=None):
    nan = float("nan")
    dx, dw = torch.full_like(x, nan), torch.full_like(w, nan)
    moe.linear_ce_backward(p, x, w, labels, lse, d_loss, dx, dw, ws, d_lse=d_lse, stream=stream)
    return dx, dw


def check(T, H, V, scale=1.0, seed=0, masked=0.2, use_d_lse=False, grads=True, spread=2.0):
    x, w, labels, d_loss = inputs(T, H, V, seed, masked, spread)
    d_lse = torch.randn(T, device=DEV) if use_d_lse else None
    p = moe.CEProblem.make(T, H, V, scale)
    ws = moe.alloc_linear_ce_workspace(p, backward=grads)
    loss, lse = forward(p, x, w, labels, ws)
    xd, wd = x.double(), w.double()
    z = scale * (xd @ wd.t())
    ez = (H / 16 + 4) * 2.0 ** -23 * abs(scale) * (xd.abs() @ wd.abs().t())
    want = torch.logsumexp(z, 1)
    tol = ez.max(1).values + 2.0 ** -20 * (1 + want.abs())
    assert ((lse.double() - want).abs() <= tol).all()
    valid = (labels >= 0) & (labels < V)
    at = torch.where(valid, labels, 0).long()[:, None]
    want_loss = torch.where(valid, want - z.gather(1, at)[:, 0], 0)
    tol = torch.where(valid, tol + ez.gather(1, at)[:, 0] + 2.0 ** -22 * z.gather(1, at)[:, 0].abs(), 0)
    assert ((loss.double() - want_loss).abs() <= tol).all()
    if grads:
        dx, dw = backward(p, x, w, labels, lse, d_loss, ws, d_lse)
        prob = torch.exp(z - want[:, None])
        dl = torch.where(valid, d_loss.double(), 0)
        a = dl + (d_lse.double() if use_d_lse else 0)
        g = a[:, None] * prob
        err = a.abs()[:, None] * prob * (2 * ez.max(1, keepdim=True).values + 2.0 ** -19 *
                                         (1 + want.abs()[:, None]))
        g.scatter_add_(1, at, -dl[:, None])
        err = scale * (err + 2.0 ** -8 * g.abs())
        g = scale * g
        for got, ref, mag, bound in (
                (dx, g @ wd, g.abs() @ wd.abs(), err.abs() @ wd.abs()),
                (dw, g.t() @ xd, g.abs().t() @ xd.abs(), err.abs().t() @ xd.abs())):
            tol = 1.1 * bound + 2.0 ** -8 * ref.abs() + (T + V) / 16 * 2.0 ** -23 * mag + 1e-30
            d = (got.double() - ref).abs()
            assert (d <= tol).all(), float((d / tol).max())
            norm = float(ref.norm())
            assert norm == 0 or float(d.norm()) <= 5e-3 * norm
    assert moe.get_device_status(ws) == moe.MOE_OK


# one token to several tiles of tokens; vocabularies of one row, round the 32-, 64- and 256-column
# units; widths round the 64-deep K step and the 256-column tile
@pytest.mark.parametrize("T", [1, 2, 31, 127, 128, 129, 255, 256, 257, 700])
def test_tokens(T):
    check(T, 136, 1000)


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 63, 64, 65, 255, 256, 257, 511, 513, 5000, 20011])
def test_vocabularies(V):
    check(40, 72, V)


@pytest.mark.parametrize("H", [8, 16, 56, 64, 72, 120, 128, 248, 256, 264, 512, 1000, 2056])
def test_widths(H):
    check(70, H, 300)


@pytest.mark.parametrize("T", [1, 33, 96, 127, 128, 129])
@pytest.mark.parametrize("H,V", [(64, 1), (64, 129), (128, 127), (64, 20011), (128, 60000),
                                 (1088, 5000), (2112, 20011)])
def test_tiles_of_one_cta(T, H, V):
    """Few tokens of whole 64-column planes take tiles of single CTAs; 129 take a pair's.  Several
    tiles per CTA, ragged last ones, and rows longer than one run of the accumulator."""
    check(T, H, V, use_d_lse=T % 2 == 0)


@pytest.mark.parametrize("T,V", [(300, 40000), (3, 60000), (2100, 20011)])
def test_several_waves_and_tile_widths(T, V):
    check(T, 256, V)


def test_several_pieces():
    """T V such that the backward takes the vocabulary in several pieces, the last one ragged."""
    check(8200, 64, 20011, seed=2)
    check(8200, 264, 9000, seed=3, use_d_lse=True)


@pytest.mark.parametrize("T,H,V", [(3, 64, 60000), (200, 1000, 50021), (300, 2056, 33000),
                                   (6000, 128, 700), (9000, 72, 300), (2500, 512, 2500)])
def test_products_split_along_k(T, H, V):
    """dx of few tokens sums over a large vocabulary, dW of a small vocabulary over many
    tokens: both cut into parts that are joined."""
    check(T, H, V, use_d_lse=T % 2 == 0)


def test_split_products_in_several_pieces():
    """dx split in every piece, the last piece shorter than the others (one stage of it)."""
    check(16500, 64, 4097, seed=4)
    check(16400, 64, 61441, seed=5)


@pytest.mark.parametrize("scale", [0.25, -1.5, 8.0])
def test_logit_scale_and_lse_gradient(scale):
    check(100, 128, 700, scale=scale, use_d_lse=True)


def test_large_logits():
    """Logits of some hundreds: the running maximum, not the exponential, carries them."""
    check(64, 256, 3000, spread=120.0, masked=0.0)


def test_all_masked():
    T, H, V = 90, 64, 500
    x, w, labels, d_loss = inputs(T, H, V)
    labels.fill_(-1)
    p = moe.CEProblem.make(T, H, V)
    ws = moe.alloc_linear_ce_workspace(p, backward=True)
    loss, lse = forward(p, x, w, labels, ws)
    assert not loss.any()
    dx, dw = backward(p, x, w, labels, lse, d_loss, ws)
    assert not dx.any() and not dw.any()


def test_labels_beyond_the_vocabulary():
    T, H, V = 50, 64, 100
    x, w, labels, d_loss = inputs(T, H, V, masked=0.0)
    labels[7] = V
    labels[20] = 1 << 30
    p = moe.CEProblem.make(T, H, V)
    ws = moe.alloc_linear_ce_workspace(p, backward=True)
    loss, lse = forward(p, x, w, labels, ws)
    assert moe.get_device_status(ws) == 7
    assert loss[7] == 0 and loss[20] == 0 and torch.isfinite(lse).all()
    dx, _ = backward(p, x, w, labels, lse, d_loss, ws)
    assert not dx[7].any() and not dx[20].any() and dx[8].any()


def test_no_tokens():
    p = moe.CEProblem.make(0, 64, 100)
    e, w = torch.empty(0, 64, dtype=BF, device=DEV), torch.ones(100, 64, dtype=BF, device=DEV)
    i, f = torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, device=DEV)
    ws = moe.alloc_linear_ce_workspace(p, backward=True)
    moe.linear_ce_forward(p, e, w, i, f, f, ws)
    moe.linear_ce_backward(p, e, w, i, f, f, e, w, ws)
    assert not w.any()


def test_not_finite():
    """A token of NaN touches its own loss and dx, and every row of dw; no other token's."""
    T, H, V = 300, 64, 900
    x, w, labels, d_loss = inputs(T, H, V, masked=0.0)
    p = moe.CEProblem.make(T, H, V)
    ws = moe.alloc_linear_ce_workspace(p, backward=True)
    clean, _ = forward(p, x, w, labels, ws)
    x[260, 3] = float("nan")
    loss, lse = forward(p, x, w, labels, ws)
    bad = torch.isnan(loss)
    assert bad[260] and bad.sum() == 1 and torch.equal(loss[~bad], clean[~bad])
    dx, dw = backward(p, x, w, labels, lse, d_loss, ws)
    assert torch.isnan(dx).any(1).sum() == 1 and torch.isnan(dw).all()


def test_against_differences():
    """Directional derivatives of sum(d_loss loss + d_lse lse) in x and w, in 64 bits."""
    T, H, V = 24, 64, 200
    x, w, labels, d_loss = inputs(T, H, V)
    d_lse = torch.randn(T, device=DEV)
    p = moe.CEProblem.make(T, H, V, 1.3)
    ws = moe.alloc_linear_ce_workspace(p, backward=True)
    _, lse = forward(p, x, w, labels, ws)
    dx, dw = backward(p, x, w, labels, lse, d_loss, ws, d_lse)
    valid, at = labels >= 0, labels.clamp(min=0).long()[:, None]

    def value(xd, wd):
        z = 1.3 * (xd @ wd.t())
        l = torch.logsumexp(z, 1)
        per = torch.where(valid, l - z.gather(1, at)[:, 0], 0)
        return float((d_loss.double() * per + d_lse.double() * l).sum())

    h = 1e-4
    for t, grad, at_x in ((x, dx, True), (w, dw, False)):
        v = torch.randn(t.shape, dtype=torch.float64, device=DEV)
        args = [((x.double() + s * h * v, w.double()) if at_x else
                 (x.double(), w.double() + s * h * v)) for s in (1, -1)]
        num = (value(*args[0]) - value(*args[1])) / (2 * h)
        # the gradient's bf16 roundings, two of 2^-8 an element with random signs
        tol = 4 * 2.0 ** -8 * float((grad.double() * v).norm()) + 1e-4
        assert abs(num - float((grad.double() * v).sum())) <= tol


def test_reproducible_and_on_another_stream():
    x, w, labels, d_loss = inputs(600, 264, 30011)
    p = moe.CEProblem.make(600, 264, 30011)

    def once(stream=None):
        ws = moe.alloc_linear_ce_workspace(p, backward=True)
        nan = float("nan")
        loss, lse = (torch.full((600,), nan, device=DEV) for _ in range(2))
        dx, dw = torch.full_like(x, nan), torch.full_like(w, nan)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        moe.linear_ce_forward(p, x, w, labels, loss, lse, ws, stream=stream)
        moe.linear_ce_backward(p, x, w, labels, lse, d_loss, dx, dw, ws, stream=stream)
        torch.cuda.synchronize()
        return loss, lse, dx, dw

    a, b, c = once(), once(), once(torch.cuda.Stream())
    assert all(torch.equal(i, j) and torch.equal(i, k) for i, j, k in zip(a, b, c))


def test_binding_refuses_wrong_tensors():
    x, w, labels, _ = inputs(8, 64, 100)
    p = moe.CEProblem.make(8, 64, 100)
    ws = moe.alloc_linear_ce_workspace(p)
    f = torch.empty(8, device=DEV)
    for a in ((x.float(), w, labels, f, f), (x, w[:99], labels, f, f), (x, w, labels.long(), f, f),
              (x, w, labels, f[:7], f), (x, w, labels, f, f.cpu()), (x[:, ::2], w, labels, f, f)):
        with pytest.raises(ValueError):
            moe.linear_ce_forward(p, *a, ws)
    with pytest.raises(moe.MoEError):
        moe.linear_ce_forward(p, x, w, labels, f, f, ws[:256])


def logits_of(x, w):
    return x.double() @ w.double().t()


@pytest.mark.parametrize("T,H", [(4, 64), (4, 72), (200, 64), (300, 1088)])
@pytest.mark.parametrize("V", [1, 2, 33, 65, 129, 257, 700, 40001])
def test_lse_of_logits_that_are_not_finite(T, H, V):
    """NaN in a token (masked or not), NaN in the vocabulary's last row alone, infinite logits of
    either sign, and nothing but -inf: lse as the formula has it in 64 bits, and no other token
    touched.  V - 1 is the first column of a tile, of a warp's half or of a chunk of 32."""
    x, w, labels, _ = inputs(T, H, V, masked=0.0)
    labels[1], labels[2] = -1, 0
    p = moe.CEProblem.make(T, H, V)
    ws = moe.alloc_linear_ce_workspace(p)
    clean_loss, clean = forward(p, x, w, labels, ws)

    bad = x.clone()
    bad[1, 3], bad[2, 5] = float("nan"), float("nan")
    loss, lse = forward(p, bad, w, labels, ws)
    assert torch.isnan(lse).nonzero()[:, 0].tolist() == [1, 2]
    assert loss[1] == 0 and torch.isnan(loss[2])
    keep = ~torch.isnan(lse)
    assert torch.equal(lse[keep], clean[keep]) and torch.equal(loss[keep], clean_loss[keep])

    bad = w.clone()
    bad[V - 1, 7] = float("nan")
    loss, lse = forward(p, x, bad, labels, ws)
    assert torch.isnan(lse).all() and torch.isnan(loss[labels >= 0]).all() and loss[1] == 0

    for value in (float("inf"), float("-inf")):
        bad = w.clone()
        bad[V // 2, 0] = value  # +inf or -inf by the sign of x's first column
        _, lse = forward(p, x, bad, labels, ws)
        want = torch.logsumexp(logits_of(x, bad), 1)
        assert (x[:, 0] != 0).all() and torch.equal(torch.isinf(want), torch.isinf(lse))
        inf = torch.isinf(want)
        assert torch.equal(want[inf], lse[inf].double()) and not torch.isnan(lse).any()
        assert ((lse.double() - want)[~inf].abs() <= 1e-4 * (1 + want[~inf].abs())).all()

    bad = w.clone()
    bad[:, 0] = float("-inf")
    positive = x.clone()
    positive[:, 0] = 1.0
    _, lse = forward(p, positive, bad, labels, ws)
    assert torch.equal(lse, torch.full_like(lse, float("-inf")))


def test_backward_records_labels_beyond_the_vocabulary():
    T, H, V = 300, 64, 100
    x, w, labels, d_loss = inputs(T, H, V, masked=0.3)
    p = moe.CEProblem.make(T, H, V)
    ws = moe.alloc_linear_ce_workspace(p, backward=True)
    _, lse = forward(p, x, w, labels, ws)
    backward(p, x, w, labels, lse, d_loss, ws)
    assert moe.get_device_status(ws) == moe.MOE_OK
    labels[T - 1] = V
    backward(p, x, w, labels, lse, d_loss, ws)
    assert moe.get_device_status(ws) == 7
