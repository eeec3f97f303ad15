"""GPU parity of the block norms (moe_block_norm_forward / _backward) against
the formulas in 64 bits on the CPU, their gradients against differences, and
their refusals.

Tolerances.  One output is its exact value plus the fp32 error of its row sum
(relative 2^-22 with room: sums of squares have no cancellation, rsqrt is
within 2 ulp, a handful of products) and one rounding to its type (2^-9 for
bf16).  A gradient is a difference of terms, so its bound is relative to the
magnitude of its terms, which the reference computes beside the value; a
column sum over T rows adds the sum's own rounding, T 2^-24 at most in any
order.  All bounds double these to leave room for the order of operations.
"""
import itertools

import pytest
import torch

import mixture_experts_ffn_permute_gb300 as moe
from mixture_experts_ffn_permute_gb300 import _build

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    moe.load()


def rounding(dtype):
    return 2.0 ** -8 if dtype is BF else 2.0 ** -23


def close(got, want, mag, dtype, sums=1):
    """|got - want| <= 2 (type rounding of want + fp32 error of the terms)."""
    got = got.double().cpu()
    tol = rounding(dtype) * want.abs() + 2.0 ** -20 * mag + sums * 2.0 ** -23 * mag
    tol = tol + 1e-30
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol).max()))


def inputs(T, H, tb, tr, tw, gate, seed=0, ld=0):
    g = torch.Generator().manual_seed(seed)

    def rows(dtype, std):
        t = torch.randn(T, ld or H, generator=g) * std
        return t.to(dtype)[:, :H]

    s = {"branch": rows(tb, 0.7), "residual": rows(tr, 2.0), "d_normed": rows(tb, 1.0),
         "d_residual_out": rows(tr, 1.0),
         "w_post": (torch.randn(H, generator=g) * 0.2 + 1).to(tw),
         "w_pre": (torch.randn(H, generator=g) * 0.2 + 1).to(tw)}
    shape = {"none": None, "channel": (H,), "token": (T,), "element": (T, H)}[gate]
    s["gate"] = None if shape is None else (torch.randn(*shape, generator=g)).to(tw)
    return s


def spread(gate, kind):
    return 1.0 if gate is None else gate.double()[:, None] if kind == "token" else gate.double()


def ref_forward(s, kind, off, rs, bs, post=True):
    y, r = s["branch"].double(), s["residual"].double()
    if post:
        y = y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS) * (s["w_post"].double() + off)
    b = bs * spread(s["gate"], kind) * y
    out = rs * r + b
    n = out / torch.sqrt((out * out).mean(1, keepdim=True) + EPS) * (s["w_pre"].double() + off)
    mag = (rs * r).abs() + b.abs()
    rms = torch.sqrt((out * out).mean(1, keepdim=True) + EPS)
    n_mag = n.abs() + mag / rms * (s["w_pre"].double() + off).abs()
    return out, mag, n, n_mag


def ref_backward(s, kind, off, rs, bs, post=True, pre=True, later=True):
    """Values and magnitudes of the terms of every gradient."""
    y, r = s["branch"].double(), s["residual"].double()
    H = r.shape[1]
    dr = s["d_residual_out"].double() if later else torch.zeros_like(r)
    g, gm = dr.clone(), dr.abs()
    o = {}
    if pre:
        dn, w = s["d_normed"].double(), s["w_pre"].double() + off
        rstd = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + EPS)
        u, a = r * rstd, dn * w
        g = g + rstd * (a - u * (a * u).mean(1, keepdim=True))
        gm = gm + rstd * (a.abs() + u.abs() * (a * u).abs().mean(1, keepdim=True))
        o["w_pre"] = ((dn * u).sum(0), (dn * u).abs().sum(0))
    o["residual"] = (rs * g, abs(rs) * gm)
    if post:
        ystd = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)
        w = s["w_post"].double() + off
    else:
        ystd, w = torch.ones(y.shape[0], 1, dtype=torch.float64), torch.ones(H, dtype=torch.float64)
    v, gate = y * ystd, spread(s["gate"], kind)
    absg = gate.abs() if torch.is_tensor(gate) else 1.0
    B, Bm = bs * g, abs(bs) * gm
    c, cm = B * gate * w, Bm * absg * w.abs()
    if post:
        o["branch"] = (ystd * (c - v * (c * v).mean(1, keepdim=True)),
                       ystd * (cm + v.abs() * (cm * v.abs()).mean(1, keepdim=True)))
        o["w_post"] = ((B * gate * v).sum(0), (Bm * absg * v.abs()).sum(0))
    else:
        o["branch"] = (c, cm)
    d, dm = B * v * w, Bm * (v * w).abs()
    if kind == "channel":
        o["gate"] = (d.sum(0), dm.sum(0))
    elif kind == "token":
        o["gate"] = (d.sum(1), dm.sum(1))
    elif kind == "element":
        o["gate"] = (d, dm)
    return o


def dev(t, ld=0):
    """On the GPU with the row stride kept."""
    if t is None:
        return None
    if t.dim() == 2 and ld:
        full = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device=DEV)
        full[:, :t.shape[1]] = t.to(DEV)
        return full[:, :t.shape[1]]
    return t.to(DEV)


def like(t, ld=0):
    """An output filled with NaN, of t's shape, and its padding (or None)."""
    if t.dim() == 2 and ld:
        full = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device=DEV)
        return full[:, :t.shape[1]], full[:, t.shape[1]:]
    return torch.full(t.shape, float("nan"), dtype=t.dtype, device=DEV), None


def problem(T, H, tb, tr, tw, kind, off, rs, bs, ld=0):
    return moe.NormProblem.make(T, H, branch_dtype=tb, residual_dtype=tr, weight_dtype=tw,
                                gate=kind, eps=EPS, weight_offset=off, residual_scale=rs,
                                branch_scale=bs, ld_branch=ld, ld_residual=ld,
                                ld_residual_out=ld, ld_normed=ld)


def check(T, H, tb, tr, tw, kind, off=0.0, rs=0.9, bs=0.5, ld=0, post=True, pre=True, later=True,
          seed=0):
    s = inputs(T, H, tb, tr, tw, kind, seed, ld)
    if not post:
        s["w_post"] = None
    p = problem(T, H, tb, tr, tw, kind, off, rs, bs, ld)
    d = {k: dev(v, ld) if k not in ("w_post", "w_pre", "gate") else dev(v) for k, v in s.items()}
    # forward
    out, pad = like(s["residual"], ld)
    nrm, npad = like(s["branch"], ld) if pre else (None, None)
    moe.block_norm_forward(p, d["residual"], branch=d["branch"], w_post=d["w_post"],
                           gate=d["gate"], w_pre=d["w_pre"] if pre else None, residual_out=out,
                           normed=nrm)
    want, mag, n, n_mag = ref_forward(s, kind, off, rs, bs, post)
    close(out, want, mag, tr)
    if pre:
        close(nrm, n, n_mag, tb)
    for q in (pad, npad):
        assert q is None or torch.isnan(q).all()
    # backward of the same inputs, `residual` standing for the stored residual_out
    o = {k: like(s[k], ld if k in ("branch", "residual") else 0)
         for k in ("branch", "residual", "w_post", "w_pre", "gate") if s[k] is not None}
    if not pre:
        o.pop("w_pre")
    ws = moe.alloc_block_norm_workspace(p)
    moe.block_norm_backward(p, d["residual"], o["residual"][0], ws, branch=d["branch"],
                            w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"] if pre else None,
                            d_normed=d["d_normed"] if pre else None,
                            d_residual_out=d["d_residual_out"] if later else None,
                            d_branch=o["branch"][0],
                            **{"d_" + k: o[k][0] for k in ("w_post", "gate", "w_pre") if k in o})
    ref = ref_backward(s, kind, off, rs, bs, post, pre, later)
    assert set(ref) == set(o)
    for k, (want, mag) in ref.items():
        dtype = {"branch": tb, "residual": tr}.get(k, tw)
        close(o[k][0], want, mag, dtype,
              sums=T if want.shape == (H,) else H if want.dim() == 1 else 1)
        assert o[k][1] is None or torch.isnan(o[k][1]).all(), k
    assert moe.get_device_status(ws) == moe.MOE_OK


# every width class: a warp's row (1, 2, 4 steps), a block's (1 and 2 steps, up to 1024 threads),
# each with rows that take 16-byte accesses and rows that do not
@pytest.mark.parametrize("H", [1, 7, 8, 255, 256, 257, 264, 511, 520, 1001, 1024, 1025, 2048, 4095,
                               4096, 4104, 7168, 8191, 8192, 8200, 16383, 16384])
def test_widths(H):
    check(37, H, BF, BF, F32, "channel")


@pytest.mark.parametrize("tb,tr,tw,kind", list(itertools.product(
    (BF, F32), (BF, F32), (BF, F32), ("none", "channel", "token", "element"))))
def test_types_and_gates(tb, tr, tw, kind):
    for H in (200, 1003, 2304):
        check(19, H, tb, tr, tw, kind, off=1.0, seed=H)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 151, 153, 607, 609, 2500])
def test_row_counts(T):
    check(T, 128, BF, F32, F32, "token")
    check(T, 1288, F32, BF, BF, "channel")


# enough rows that they are streamed through shared memory, in every depth of the ring
@pytest.mark.parametrize("H", [264, 1032, 2048, 4096, 7168, 8192])
@pytest.mark.parametrize("tb,tr", list(itertools.product((BF, F32), repeat=2)))
def test_streamed_rows(tb, tr, H):
    for kind, T in (("channel", 611), ("element", 1000)):
        check(T, H, tb, tr, F32, kind, off=0.5, seed=T)
    check(700, H, tb, tr, BF, "token", ld=H + 8)


# rows that do not start on 16 bytes: dense ones are streamed as octets of the whole tensor
@pytest.mark.parametrize("H", [257, 566, 1025, 1254, 2047, 5897, 8191])
@pytest.mark.parametrize("tb,tr", list(itertools.product((BF, F32), repeat=2)))
def test_streamed_narrow_rows(tb, tr, H):
    check(613, H, tb, tr, F32, "channel", off=0.5)
    check(1, H, tb, tr, BF, "element")
    check(620, H, tb, tr, BF, "token", ld=H + 5)


@pytest.mark.parametrize("shift,H", [(0, 1031), (0, 1026), (8, 1029), (1, 1032), (2, 1031),
                                     (3, 1032), (5, 1032), (7, 1032)])
def test_rows_of_a_shifted_tensor(shift, H):
    """The tensors start `shift` elements behind a 32-byte boundary and end where the last eight
    elements' place is not whole; what lies round them is NaN and stays."""
    T = 701
    s = inputs(T, H, BF, F32, F32, "channel")
    p = problem(T, H, BF, F32, F32, "channel", 0.0, 0.9, 0.5)
    whole = {}

    def put(name, t):
        whole[name] = torch.full((T * H + 16,), float("nan"), dtype=t.dtype, device=DEV)
        view = whole[name][shift:shift + T * H].view(T, H)
        return view.copy_(t)

    d = {k: put(k, v) if v.dim() == 2 else v.to(DEV) for k, v in s.items()}
    o = {k: put("o" + k, torch.zeros_like(s[k])) for k in ("branch", "residual")}
    out, n = put("out", torch.zeros_like(s["residual"])), put("n", torch.zeros_like(s["branch"]))
    kw = dict(branch=d["branch"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"])
    moe.block_norm_forward(p, d["residual"], residual_out=out, normed=n, **kw)
    want, mag, nw, n_mag = ref_forward(s, "channel", 0.0, 0.9, 0.5)
    close(out, want, mag, F32)
    close(n, nw, n_mag, BF)
    w = {k: torch.empty_like(d[k]) for k in ("w_post", "gate", "w_pre")}
    moe.block_norm_backward(p, d["residual"], o["residual"], moe.alloc_block_norm_workspace(p),
                            d_normed=d["d_normed"], d_residual_out=d["d_residual_out"],
                            d_branch=o["branch"], **kw, **{"d_" + k: v for k, v in w.items()})
    for k, (want, mag) in ref_backward(s, "channel", 0.0, 0.9, 0.5).items():
        got = o[k] if k in o else w[k]
        close(got, want, mag, got.dtype, sums=T if want.dim() == 1 else 1)
    for name, t in whole.items():
        assert torch.isnan(t[:shift]).all() and torch.isnan(t[shift + T * H:]).all(), name


@pytest.mark.parametrize("kind", ["none", "token", "element"])
@pytest.mark.parametrize("post,pre,later", [(False, True, True), (True, False, True),
                                            (True, True, False), (False, False, True)])
def test_streamed_rows_with_parts_left_out(kind, post, pre, later):
    check(1300, 1288, BF, F32, F32, kind, post=post, pre=pre, later=later)
    check(1300, 1288, BF, BF, F32, kind, post=post, pre=pre, later=later)
    check(650, 1291, BF, F32, F32, kind, post=post, pre=pre, later=later)


@pytest.mark.parametrize("kind", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("post,pre,later", [(False, True, True), (True, False, True),
                                            (True, True, False), (False, False, True),
                                            (False, True, False)])
def test_parts_left_out(kind, post, pre, later):
    for H in (96, 1500):
        check(23, H, BF, F32, F32, kind, post=post, pre=pre, later=later)


@pytest.mark.parametrize("H,ld", [(256, 264), (200, 201), (2048, 2056), (2048, 2049), (5000, 6001)])
def test_row_strides(H, ld):
    check(29, H, BF, BF, BF, "element", ld=ld)
    check(29, H, F32, F32, F32, "none", ld=ld)


@pytest.mark.parametrize("H", [64, 333, 2048])
@pytest.mark.parametrize("T", [11, 900])
def test_norm_alone(T, H):
    s = inputs(T, H, BF, F32, F32, "none")
    p = problem(T, H, BF, F32, F32, "none", 0.0, 0.3, 0.4)
    d = {k: dev(v) for k, v in s.items()}
    n = like(s["branch"])[0]
    moe.block_norm_forward(p, d["residual"], w_pre=d["w_pre"], normed=n)
    r, w = s["residual"].double(), s["w_pre"].double()
    want = r / torch.sqrt((r * r).mean(1, keepdim=True) + EPS) * w
    close(n, want, want.abs(), BF)
    dr, dw = like(s["residual"])[0], like(s["w_pre"])[0]
    ws = moe.alloc_block_norm_workspace(p)
    moe.block_norm_backward(p, d["residual"], dr, ws, w_pre=d["w_pre"], d_normed=d["d_normed"],
                            d_residual_out=d["d_residual_out"], d_w_pre=dw)
    ref = ref_backward(s, "none", 0.0, 1.0, 0.4)  # the scales do not apply
    close(dr, *ref["residual"], F32)
    close(dw, *ref["w_pre"], F32, sums=T)


def test_in_place():
    s = inputs(300, 1536, BF, BF, BF, "channel")
    p = problem(300, 1536, BF, BF, BF, "channel", 0.0, 0.9, 0.5)
    d = {k: dev(v) for k, v in s.items()}
    out, n1, n2 = (torch.empty_like(d["branch"]) for _ in range(3))
    kw = dict(branch=d["branch"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"])
    moe.block_norm_forward(p, d["residual"], residual_out=out, normed=n1, **kw)
    r = d["residual"].clone()
    moe.block_norm_forward(p, r, residual_out=r, normed=n2, **kw)
    assert torch.equal(r, out) and torch.equal(n1, n2)
    ws = moe.alloc_block_norm_workspace(p)

    def back(dro, dres):
        o = {k: torch.empty_like(d[k]) for k in ("branch", "w_post", "gate", "w_pre")}
        moe.block_norm_backward(p, out, dres, ws, d_normed=d["d_normed"], d_residual_out=dro,
                                **kw, **{"d_" + k: v for k, v in o.items()})
        return dres, o

    a, oa = back(d["d_residual_out"], torch.empty_like(out))
    same = d["d_residual_out"].clone()
    b, ob = back(same, same)
    assert torch.equal(a, b) and all(torch.equal(oa[k], ob[k]) for k in oa)


def test_zero_rows_and_values():
    """No rows: the weights' gradients are zero; a row of zeros keeps finite values."""
    p = problem(0, 96, BF, BF, F32, "channel", 0.0, 1.0, 1.0)
    e, w = torch.empty(0, 96, dtype=BF, device=DEV), torch.ones(96, device=DEV)
    moe.block_norm_forward(p, e, branch=e, w_post=w, gate=w, w_pre=w, residual_out=e, normed=e)
    o = [torch.full((96,), float("nan"), device=DEV) for _ in range(3)]
    moe.block_norm_backward(p, e, e, moe.alloc_block_norm_workspace(p), branch=e, w_post=w, gate=w,
                            w_pre=w, d_normed=e, d_residual_out=e, d_branch=e, d_w_post=o[0],
                            d_gate=o[1], d_w_pre=o[2])
    assert all(torch.equal(t, torch.zeros_like(t)) for t in o)
    p = problem(3, 96, BF, F32, F32, "none", 0.0, 1.0, 1.0)
    z, zf = torch.zeros(3, 96, dtype=BF, device=DEV), torch.zeros(3, 96, device=DEV)
    out, n = torch.empty_like(zf), torch.empty_like(z)
    moe.block_norm_forward(p, zf, branch=z, w_post=w, w_pre=w, residual_out=out, normed=n)
    assert not out.any() and not n.any()


def test_infinite_gate_stays_in_its_columns():
    """A width that leaves a thread's vector partly outside the row: the columns outside do not
    turn an infinite gate into NaN sums, and a NaN row does not touch the others."""
    for H in (1003, 1000, 264):
        s = inputs(9, H, BF, F32, F32, "element")
        s["branch"][4, 5] = float("nan")
        p = problem(9, H, BF, F32, F32, "element", 0.0, 0.9, 0.5)
        d = {k: dev(v) for k, v in s.items()}
        out, n = torch.empty_like(d["residual"]), torch.empty_like(d["branch"])
        moe.block_norm_forward(p, d["residual"], branch=d["branch"], w_post=d["w_post"],
                               gate=d["gate"], w_pre=d["w_pre"], residual_out=out, normed=n)
        bad = torch.isnan(n.float()).all(1).cpu()
        assert bad.tolist() == [t == 4 for t in range(9)]
        assert not torch.isnan(n.float()).any(1).cpu()[[t for t in range(9) if t != 4]].any()


def test_against_differences():
    """Directional derivatives of <dn, normed> + <dr, residual_out> in every input, fp32."""
    T, H = 5, 40
    for kind in ("channel", "token", "element"):
        s = inputs(T, H, F32, F32, F32, kind, seed=3)
        p = problem(T, H, F32, F32, F32, kind, 0.0, 0.9, 0.5)
        names = ("residual", "branch", "w_post", "w_pre", "gate")

        def value(q):
            out, _, n, _ = ref_forward(q, kind, 0.0, 0.9, 0.5)
            return float((s["d_normed"].double() * n).sum() +
                         (s["d_residual_out"].double() * out).sum())

        d = {k: dev(v) for k, v in s.items()}
        out, nrm = torch.empty_like(d["residual"]), torch.empty_like(d["branch"])
        kw = dict(branch=d["branch"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"])
        moe.block_norm_forward(p, d["residual"], residual_out=out, normed=nrm, **kw)
        o = {k: torch.empty_like(d[k]) for k in names}
        moe.block_norm_backward(p, out, o["residual"], moe.alloc_block_norm_workspace(p),
                                d_normed=d["d_normed"], d_residual_out=d["d_residual_out"],
                                **kw, **{"d_" + k: o[k] for k in names[1:]})
        g = torch.Generator().manual_seed(9)
        for k in names:
            v = torch.randn(s[k].shape, generator=g, dtype=torch.float64)
            h = 1e-5
            up = value({**s, k: s[k].double() + h * v})
            down = value({**s, k: s[k].double() - h * v})
            num, got = (up - down) / (2 * h), float((o[k].double().cpu() * v).sum())
            # fp32 gradients of a few hundred terms of order one
            assert abs(num - got) <= 1e-4 * max(1.0, abs(num)), (kind, k, num, got)


def test_reproducible_and_on_another_stream():
    s = inputs(1500, 1288, BF, F32, F32, "channel")
    p = problem(1500, 1288, BF, F32, F32, "channel", 0.0, 0.9, 0.5)
    d = {k: dev(v) for k, v in s.items()}
    kw = dict(branch=d["branch"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"],
              d_normed=d["d_normed"], d_residual_out=d["d_residual_out"])

    def once(stream=None):
        o = {k: torch.empty_like(d[k]) for k in ("residual", "branch", "w_post", "gate", "w_pre")}
        ws = moe.alloc_block_norm_workspace(p)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        moe.block_norm_backward(p, d["residual"], o["residual"], ws, stream=stream, **kw,
                                **{"d_" + k: o[k] for k in o if k != "residual"})
        torch.cuda.synchronize()
        return o

    a, b, c = once(), once(), once(torch.cuda.Stream())
    assert all(torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]) for k in a)


def test_binding_refuses_wrong_tensors():
    p = problem(4, 64, BF, BF, F32, "none", 0.0, 1.0, 1.0)
    r = torch.zeros(4, 64, dtype=BF, device=DEV)
    w = torch.ones(64, device=DEV)
    n = torch.empty_like(r)
    for bad in (dict(w_pre=w.to(BF)), dict(w_pre=w[:32]), dict(w_pre=w.cpu()),
                dict(normed=n.float()), dict(normed=torch.empty(64, 4, dtype=BF, device=DEV).t())):
        with pytest.raises(ValueError):
            moe.block_norm_forward(p, r, **{**dict(w_pre=w, normed=n), **bad})
    with pytest.raises(moe.MoEError):
        moe.block_norm_forward(p, r)  # nothing to compute


@pytest.mark.parametrize("kind", ["channel", "token", "element"])
@pytest.mark.parametrize("H,ld", [(200, 0), (203, 0), (1000, 0), (1003, 0), (2304, 0), (2301, 0),
                                  (2301, 2307)])
@pytest.mark.parametrize("T", [9, 700])
def test_infinite_gates(T, H, ld, kind):
    """An infinite gate value, and a NaN in another row: the forward has infinities and NaN where
    the formula in 64 bits has them, and the backward is finite where it is (sums of infinities of
    both signs are NaN in one order of the factors and infinite in another)."""
    s = inputs(T, H, BF, F32, F32, kind, seed=5, ld=ld)
    at = {"channel": H - 2, "token": 6, "element": (6, H - 2)}[kind]
    s["gate"][at] = float("inf")
    s["branch"][4, 5] = float("nan")
    p = problem(T, H, BF, F32, F32, kind, 0.0, 0.9, 0.5, ld)
    d = {k: dev(v, ld) if k not in ("w_post", "w_pre", "gate") else dev(v) for k, v in s.items()}
    kw = dict(branch=d["branch"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"])
    out, n = like(s["residual"], ld)[0], like(s["branch"], ld)[0]
    moe.block_norm_forward(p, d["residual"], residual_out=out, normed=n, **kw)
    want, mag, nw, n_mag = ref_forward(s, kind, 0.0, 0.9, 0.5)
    for got, ref, m, dtype in ((out, want, mag, F32), (n, nw, n_mag, BF)):
        g = got.double().cpu()
        assert torch.equal(torch.isnan(g), torch.isnan(ref))
        inf = torch.isinf(ref)
        assert torch.equal(torch.isinf(g), inf) and torch.equal(g[inf], ref[inf])
        fine = torch.isfinite(ref)
        m = torch.where(torch.isfinite(m), m, ref.abs())  # a finite value's terms may be infinite
        close(got.cpu()[fine], ref[fine], m[fine], dtype)
    o = {k: like(s[k], ld if k in ("branch", "residual") else 0)[0]
         for k in ("branch", "residual", "w_post", "w_pre", "gate")}
    moe.block_norm_backward(p, d["residual"], o["residual"], moe.alloc_block_norm_workspace(p),
                            d_normed=d["d_normed"], d_residual_out=d["d_residual_out"],
                            d_branch=o["branch"], **kw,
                            **{"d_" + k: o[k] for k in ("w_post", "gate", "w_pre")})
    for k, (ref, m) in ref_backward(s, kind, 0.0, 0.9, 0.5).items():
        fine = torch.isfinite(ref)
        assert torch.equal(torch.isfinite(o[k]).cpu(), fine), k
        dtype = BF if k == "branch" else F32
        close(o[k].cpu()[fine], ref[fine], m[fine], dtype,
              sums=T if ref.shape == (H,) else H if ref.dim() == 1 else 1)
