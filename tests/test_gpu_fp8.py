"""GPU parity of the quantisation to E4M3 and of the product of the codes against 64 bits.

Quantisation: a scale is one quotient in fp32 (2^-24 of it; SwiGLU's values are off by their fast
exponential, (|g| + 4) 2^-23).  A code is that of the quotient v / scale in fp32: its distance from
the exact quotient is at most half a step and 2^-22 of it, with room; bit by bit it is looked at by
the tests of the borders between codes.

Product: one rounding of the result; every block's sum is taken by the tensor core in four steps of
32 products (each rounded or cut in the accumulator: 36 2^-23 of the terms' magnitude at most) and
scaled and added in fp32 (2^-24 of the magnitude a block, and the factor's rounding)."""
import math

import pytest
import torch

import mixture_experts_ffn_permute_gb300 as moe
from mixture_experts_ffn_permute_gb300 import _build

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    moe.load()


def blocks(n):
    return -(-n // 128)


def per_value(scales, rows, cols):
    """Scales of 128 x 128 blocks (or, rows None, of 1 x 128) as one for every value."""
    s = scales.repeat_interleave(128, -1)[..., :cols]
    return s if rows is None else s.repeat_interleave(128, -2)[..., :rows, :]


def step_of(q):
    """Half the distance between neighbouring codes about a value of at most 448."""
    e = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e - 4)


def check_codes(v, codes, scales, spread, slack):
    """v in 64 bits, scales spread to its shape."""
    s = spread(scales.double())
    q = v / s
    got = codes.to(F32).double()
    tol = step_of(q) * (1 + 1e-12) + slack * q.abs()
    err = (got - q).abs()
    assert (err <= tol).all(), float((err / tol).max())


def rows_case(T, H, dtype, swiglu=False, interleave=0, clamp=0.0, ld=0, seed=0, src=None):
    width = 2 * H if swiglu else H
    g = torch.Generator().manual_seed(seed + T + H)
    if src is None:
        src = torch.randn(T, width, generator=g) * torch.exp(torch.randn(T, 1, generator=g))
        src = src.to(dtype)
    dev = torch.zeros(T, ld or width, dtype=dtype, device=DEV)
    dev[:, :width] = src.to(DEV)
    p = moe.QuantProblem.make(T, H, dtype, swiglu, interleave, clamp, ld)
    codes = torch.full((T, H), 255, dtype=torch.uint8, device=DEV).view(E4M3)
    scales = torch.full((T, blocks(H)), math.nan, device=DEV)
    moe.fp8_quantize_rows(p, dev[:, :width], codes, scales)
    torch.cuda.synchronize()
    return src, codes.cpu(), scales.cpu()


def swiglu_of(src, H, interleave, clamp):
    x = src.double()
    I = interleave or H
    pairs = x.reshape(x.shape[0], H // I, 2, I)
    g, u = pairs[:, :, 0].reshape(-1, H), pairs[:, :, 1].reshape(-1, H)
    if clamp > 0:
        g, u = g.clamp(max=clamp), u.clamp(-clamp, clamp)
    return g / (1 + torch.exp(-g)) * u, g


def check_rows(T, H, dtype, **kw):
    src, codes, scales = rows_case(T, H, dtype, **kw)
    if kw.get("swiglu"):
        v, g = swiglu_of(src, H, kw.get("interleave", 0), kw.get("clamp", 0.0))
        off = float((g.abs().amax() + 6) * 2.0 ** -23) if T else 0.0
    else:
        v, off = src.double(), 0.0
    pad = torch.nn.functional.pad(v, (0, -H % 128)).reshape(T, -1, 128).abs().amax(2)
    want = torch.where(pad > 0, pad / 448, torch.ones_like(pad))
    assert ((scales.double() - want).abs() <= (2.0 ** -23 + off) * want).all()
    check_codes(v, codes, scales, lambda s: per_value(s, None, H), 2.0 ** -22 + off)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [16, 48, 112, 128, 144, 256, 1040, 2048, 7168])
@pytest.mark.parametrize("T", [1, 3, 65])
def test_rows(T, H, dtype):
    check_rows(T, H, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,interleave", [(16, 0), (128, 0), (208, 0), (208, 16), (768, 32), (768, 64),
                                          (768, 128), (768, 256), (1024, 1024)])
def test_swiglu_rows(H, interleave, dtype):
    for clamp in (0.0, 1.5):
        check_rows(37, H, dtype, swiglu=True, interleave=interleave, clamp=clamp)


def test_rows_many():
    check_rows(5000, 640, BF)
    check_rows(2500, 256, BF, swiglu=True)


def test_rows_with_strides():
    for dtype, ld in ((BF, 280), (BF, 272), (F32, 264), (F32, 1024)):  # (off the 32 bytes, on them)
        check_rows(9, 256, dtype, ld=ld)
        check_rows(9, 112, dtype, swiglu=True, ld=ld)
    # rows that begin 16 bytes behind a multiple of 32
    whole = torch.randn(6, 272).to(BF)
    dev = whole.to(DEV)
    p = moe.QuantProblem.make(6, 256, BF, ld_src=272)
    codes = torch.empty(6, 256, dtype=E4M3, device=DEV)
    scales = torch.empty(6, 2, device=DEV)
    moe.fp8_quantize_rows(p, dev[:, 8:264], codes, scales)
    check_codes(whole[:, 8:264].double(), codes.cpu(), scales.cpu(), lambda s: per_value(s, None, 256),
                2.0 ** -22)


def test_rows_of_zeros_and_small_values():
    H = 256
    src = torch.zeros(6, H)
    src[1, 5] = -0.0
    src[2, :128] = 1e-44      # subnormal: scale 2^-126
    src[3, 130] = 3e38
    src[4, 1] = -448.0
    src[5, :] = torch.linspace(-1e-36, 1e-36, H)
    _, codes, scales = rows_case(6, H, F32, src=src)
    assert (scales[:2] == 1).all() and (codes[:2].to(F32) == 0).all()
    assert scales[2, 0] == 2.0 ** -126 and scales[2, 1] == 1
    assert scales[4, 0] == 1 and codes[4, 1].to(F32) == -448
    assert codes[3, 130].to(F32) == 448
    check_codes(src.double(), codes, scales, lambda s: per_value(s, None, H), 2.0 ** -22)


def test_rows_with_infinities_and_nan():
    src = torch.randn(4, 256)
    src[0, 3] = math.nan
    src[1, 200] = math.inf
    src[2, 7] = -math.inf
    for dtype in (BF, F32):
        s, codes, scales = rows_case(4, 256, dtype, src=src.to(dtype))
        c = codes.to(F32)
        assert math.isnan(scales[0, 0]) and c[0, :128].isnan().all() and not c[0, 128:].isnan().any()
        assert scales[1, 1] == math.inf and scales[2, 0] == math.inf
        assert c[1, 200].isnan() and c[2, 7].isnan()
        assert (c[1, 128:200] == 0).all() and (c[2, 8:128] == 0).all()
        assert not c[3].isnan().any() and scales[3].isfinite().all()
    pre = torch.randn(3, 512)
    pre[0, 3] = -200.0   # silu of it is -0
    pre[1, 300] = math.nan
    pre[2, 9] = math.inf
    _, codes, scales = rows_case(3, 256, F32, swiglu=True, src=pre)
    c = codes.to(F32)
    assert c[0, 3] == 0 and not c[0].isnan().any()
    assert c[1, :128].isnan().all() and not c[1, 128:].isnan().any()
    assert scales[2, 0] == math.inf and c[2, 9].isnan()


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (2, 128, 128), (1, 130, 272), (3, 400, 144), (2, 256, 1024),
                                   (1, 16, 2048), (5, 208, 400)])
def test_weights(E, N, K, dtype):
    g = torch.Generator().manual_seed(N + K)
    src = (torch.randn(E, N, K, generator=g) * torch.exp(torch.randn(E, N, 1, generator=g))).to(dtype)
    src[0, :, :16] = 0
    p = moe.QuantWeightsProblem.make(E, N, K, dtype)
    for transposed in (False, True) if N % 16 == 0 else (False,):
        codes = torch.full((E, N, K), 255, dtype=torch.uint8, device=DEV).view(E4M3)
        scales = torch.full((E, blocks(N), blocks(K)), math.nan, device=DEV)
        t = (torch.full((E, K, N), 255, dtype=torch.uint8, device=DEV).view(E4M3),
             torch.full((E, blocks(K), blocks(N)), math.nan, device=DEV)) if transposed else (None, None)
        moe.fp8_quantize_weights(p, src.to(DEV), codes, scales, codes_t=t[0], scales_t=t[1])
        pad = torch.nn.functional.pad(src.double().abs(), (0, -K % 128, 0, -N % 128))
        pad = pad.reshape(E, blocks(N), 128, blocks(K), 128).amax((2, 4))
        want = torch.where(pad > 0, pad / 448, torch.ones_like(pad))
        assert ((scales.cpu().double() - want).abs() <= 2.0 ** -23 * want).all()
        check_codes(src.double(), codes.cpu(), scales.cpu(), lambda s: per_value(s, N, K), 2.0 ** -22)
        if transposed:
            assert torch.equal(t[0].view(torch.uint8), codes.view(torch.uint8).transpose(1, 2))
            assert torch.equal(t[1], scales.transpose(1, 2))


def test_weights_with_infinities_and_nan():
    src = torch.randn(1, 256, 256)
    src[0, 3, 5], src[0, 200, 9] = math.nan, math.inf
    p = moe.QuantWeightsProblem.make(1, 256, 256, F32)
    codes, scales = torch.empty(1, 256, 256, dtype=E4M3, device=DEV), torch.empty(1, 2, 2, device=DEV)
    moe.fp8_quantize_weights(p, src.to(DEV), codes, scales)
    c = codes.to(F32).cpu()[0]
    assert c[:128, :128].isnan().all() and math.isnan(scales[0, 0, 0])
    assert scales[0, 1, 0] == math.inf and c[200, 9].isnan() and (c[201:, :128] == 0).all()
    assert not c[:, 128:].isnan().any() and scales[0, :, 1].isfinite().all()


def codes_by_quotient(src, scale):
    """What the definition gives of one scale a row: E4M3 of the quotient in fp32."""
    return (src.float() / scale[:, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)


def blocks_of_ties(dtype):
    """Rows of one block each, [n, 128]: every mantissa of bf16 over every other, at twelve sizes;
    and (fp32) values a few steps from every border between two codes, of scales of every size."""
    c, top = torch.arange(127), 2 * (1 + torch.arange(128) / 128)
    rows = []
    for j in range(12):
        v = (1 + ((c + 11 * j) % 128) / 128) * 2.0 ** -j * (1 - 2 * (c % 2))
        rows.append(torch.cat([top[:, None], v.expand(128, -1)], 1))
    rows = torch.cat(rows)
    if dtype is BF:
        return rows
    g = torch.Generator().manual_seed(12)
    n = 4000
    size = torch.exp2(torch.randint(-148, 126, (n,), generator=g).double())
    size[: n // 2] = 1.0
    top = ((1 + torch.rand(n, generator=g, dtype=torch.float64)) * size).float()
    scale = (top / torch.full_like(top, 448.0)).clamp(min=2.0 ** -126)
    odd = torch.cat([torch.arange(17, 32, 2) * 2.0 ** e for e in range(-10, 4)]
                    + [torch.arange(1, 16, 2) * 2.0 ** -10])  # the borders
    v = odd[torch.randint(0, len(odd), (n, 127), generator=g)].double() * scale[:, None].double()
    bits = v.float().view(torch.int32) + torch.randint(-3, 4, (n, 127), generator=g, dtype=torch.int32)
    v = torch.minimum(bits.clamp(min=0).view(F32), top[:, None])
    v = v * (1 - 2 * torch.randint(0, 2, (n, 127), generator=g))
    return torch.cat([rows, torch.cat([top[:, None], v], 1)])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_codes_are_those_of_the_quotient(dtype):
    """scale = max |v| / 448 and code = E4M3(v / scale), both quotients in fp32, bit by bit: ties go to
    the even code.  (Block maximum 1.078125, v = 0.80859375: 336 in fp32, code 320; times a rounded
    reciprocal 336.00003, code 352.)"""
    src = blocks_of_ties(dtype).to(dtype)
    src[5, 9] = -0.0
    n = src.shape[0]
    want_s = (src.float().abs().amax(1) / torch.full((n,), 448.0)).clamp(min=2.0 ** -126)
    want = codes_by_quotient(src, want_s)
    _, codes, scales = rows_case(n, 128, dtype, src=src)
    assert torch.equal(scales[:, 0], want_s)
    assert torch.equal(codes.view(torch.uint8), want), int((codes.view(torch.uint8) != want).sum())
    # the same as blocks of weights, [1, 128] each
    p = moe.QuantWeightsProblem.make(n, 1, 128, dtype)
    codes, scales = torch.empty(n, 1, 128, dtype=E4M3, device=DEV), torch.empty(n, 1, 1, device=DEV)
    moe.fp8_quantize_weights(p, src.view(n, 1, 128).to(DEV), codes, scales)
    assert torch.equal(scales.view(-1).cpu(), want_s)
    assert torch.equal(codes.view(torch.uint8).cpu().view(n, 128), want)


# ------------------------------------------------------------------ product
def operands(M, N, K, E, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed + M + N + K)
    code = lambda *s: (torch.randn(*s, generator=g) * 128).clamp(-448, 448).to(E4M3)  # noqa: E731
    size = lambda *s: torch.exp(torch.randn(*s, generator=g)) / 128 * std  # noqa: E731
    return code(M, K), size(M, blocks(K)), code(E, N, K), size(E, blocks(N), blocks(K))


def cut(M, E, seed=0, tail=0):
    """Offsets of E experts in [0, M - tail], empty ones among them."""
    g = torch.Generator().manual_seed(seed + M + 7 * E)
    at = torch.randint(0, M - tail + 1, (E + 1,), generator=g).sort().values
    at[0], at[E] = 0, M - tail
    return at.to(torch.int32)


def check_product(M, N, K, E=1, dtype=F32, offsets=None, seed=0, ops=None):
    x, xs, w, ws = ops or operands(M, N, K, E, seed)
    p = moe.FP8Problem.make(M, N, K, E, dtype)
    work = moe.alloc_fp8_matmul_workspace(p)
    out = torch.full((M, N), math.nan, dtype=dtype, device=DEV)
    moe.fp8_matmul(p, x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), out, work,
                   expert_offsets=None if offsets is None else offsets.to(DEV))
    torch.cuda.synchronize()
    assert moe.get_device_status(work) == moe.MOE_OK
    got = out.double().cpu()
    ends = [0, M] if offsets is None else offsets.tolist()
    a = (x.to(F32).to(DEV).double() * per_value(xs.to(DEV).double(), None, K))
    for e in range(E):
        r = slice(ends[e], ends[e + 1])
        b = w[e].to(F32).to(DEV).double() * per_value(ws[e].to(DEV).double(), N, K)
        want, mag = (a[r] @ b.t()).cpu(), (a[r].abs() @ b.abs().t()).cpu()
        tol = (2.0 ** -8 if dtype is BF else 2.0 ** -24) * want.abs() + (75 + blocks(K)) * 2.0 ** -24 * mag
        err = (got[r] - want).abs()
        assert (err <= tol).all(), (e, float((err / tol).max()))
    inside = torch.zeros(M, dtype=torch.bool)
    inside[ends[0]:ends[-1]] = True
    assert out.cpu()[~inside].isnan().all()  # left as they were
    return out, p


@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 64, 100, 128, 129, 255, 300, 513])
def test_product_rows(M):
    check_product(M, 256, 384)
    check_product(M, 200, 272, dtype=BF)


@pytest.mark.parametrize("N", [1, 7, 16, 100, 127, 128, 129, 144, 255, 256, 300, 640])
def test_product_columns(N):
    for M in (5, 140):
        check_product(M, N, 256, dtype=BF)
        check_product(M, N, 256)


@pytest.mark.parametrize("K", [16, 112, 128, 144, 256, 272, 384, 640, 1040, 4096, 16384])
def test_product_lengths(K):
    for M in (3, 150):
        check_product(M, 144, K)
        check_product(M, 144, K, dtype=BF)


@pytest.mark.parametrize("M,N,K,E", [(1, 1000, 4096, 1), (1, 128, 2048, 1), (33, 130, 2064, 1), (64, 512, 4112, 1),
                                     (100, 300, 8192, 1), (128, 17, 16384, 1), (65, 1024, 2048, 1),
                                     (5, 512, 4096, 4), (40, 130, 6144, 3), (3, 512, 4096, 60)])
def test_product_of_few_rows_and_long_sums(M, N, K, E):
    """Few tiles: several CTAs share one along K."""
    offsets = None if E == 1 else cut(M, E, tail=min(2, M - 1))
    for dtype in (F32, BF):
        first, p = check_product(M, N, K, E, dtype, offsets)
        again, _ = check_product(M, N, K, E, dtype, offsets)
        assert torch.equal(first.nan_to_num(0.0), again.nan_to_num(0.0))


@pytest.mark.parametrize("M,E", [(1, 3), (8, 128), (40, 7), (256, 128), (300, 4), (777, 5), (1000, 64),
                                 (2000, 3), (600, 1024)])
def test_product_of_experts(M, E):
    for tail in (0, min(M, 13)):
        check_product(M, 144 if E > 64 else 272, 256, E, offsets=cut(M, E, tail=tail))
    check_product(M, 128, 144, E, BF, cut(M, E, seed=3))


def test_product_of_one_crowded_expert():
    for M, E, at in ((700, 6, 3), (40, 6, 0), (40, 200, 199)):
        offsets = torch.zeros(E + 1, dtype=torch.int32)
        offsets[at + 1:] = M
        check_product(M, 272, 400, E, offsets=offsets)


def test_product_without_rows():
    p = moe.FP8Problem.make(64, 64, 64, 2)
    x, xs, w, ws = (t.to(DEV) for t in operands(64, 64, 64, 2))
    out = torch.full((64, 64), 3.0, dtype=BF, device=DEV)
    work = moe.alloc_fp8_matmul_workspace(p)
    moe.fp8_matmul(p, x, xs, w, ws, out, work, expert_offsets=torch.zeros(3, dtype=torch.int32, device=DEV))
    assert (out == 3).all() and moe.get_device_status(work) == moe.MOE_OK


@pytest.mark.parametrize("offsets", [[0, 40, 30], [0, 10, 65], [-1, 10, 20], [5, 3, 64]])
def test_bad_offsets_are_recorded_and_nothing_is_written(offsets):
    for M in (64, 600):
        offs = [M + 1 if o == 65 else o for o in offsets]
        p = moe.FP8Problem.make(M, 64, 64, 2)
        x, xs, w, ws = (t.to(DEV) for t in operands(M, 64, 64, 2))
        out = torch.full((M, 64), 3.0, dtype=BF, device=DEV)
        work = moe.alloc_fp8_matmul_workspace(p)
        moe.fp8_matmul(p, x, xs, w, ws, out, work,
                       expert_offsets=torch.tensor(offs, dtype=torch.int32, device=DEV))
        assert (out == 3).all() and moe.get_device_status(work) == 7
        moe.clear_device_status(work)
        assert moe.get_device_status(work) == moe.MOE_OK


def test_offsets_that_do_not_start_at_zero():
    check_product(300, 144, 256, 2, offsets=torch.tensor([17, 140, 290], dtype=torch.int32))
    check_product(30, 144, 256, 2, offsets=torch.tensor([3, 14, 28], dtype=torch.int32))


def test_product_with_nan_and_infinities():
    M, N, K = 140, 144, 384
    for rows in (M, 9):
        x, xs, w, ws = operands(rows, N, K, 1)
        x.view(torch.uint8)[2, 5] = 0x7F       # NaN code
        w.view(torch.uint8)[0, 7, 300] = 0x7F
        xs[4, 1] = math.inf
        xs[5, 2] = math.nan
        xs[6, 0] = 0.0
        ws[0, 1, 1] = math.inf
        p = moe.FP8Problem.make(rows, N, K, 1, F32)
        out = torch.zeros(rows, N, device=DEV)
        moe.fp8_matmul(p, x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), out,
                       moe.alloc_fp8_matmul_workspace(p))
        got = out.cpu()
        assert got[2].isnan().all() and got[5].isnan().all() and got[:, 7].isnan().all()
        assert not got[4, :128].isfinite().any() and not got[:, 128:].isfinite().any()
        rest = got[:, :128].clone()
        rest[[2, 4, 5]] = 0
        rest[:, 7] = 0
        assert rest.isfinite().all()


def test_product_takes_codes_as_bytes_and_repeats_bitwise():
    x, xs, w, ws = operands(300, 144, 384, 3)
    offs = cut(300, 3)
    out, p = check_product(300, 144, 384, 3, BF, offs, ops=(x, xs, w, ws))
    again = torch.full_like(out, math.nan)
    work = moe.alloc_fp8_matmul_workspace(p)
    moe.fp8_matmul(p, x.view(torch.uint8).to(DEV), xs.to(DEV), w.view(torch.uint8).to(DEV), ws.to(DEV), again,
                   work, expert_offsets=offs.to(DEV))
    assert torch.equal(out[offs[0]:offs[-1]], again[offs[0]:offs[-1]])


def test_unaligned_outputs():
    """Out 16 bytes behind a multiple of 32, and scales at any element."""
    for dtype, M in ((BF, 140), (F32, 140), (BF, 6), (F32, 6)):
        x, xs, w, ws = (t.to(DEV) for t in operands(M, 144, 256, 1))
        p = moe.FP8Problem.make(M, 144, 256, 1, dtype)
        want = torch.empty(M, 144, dtype=dtype, device=DEV)
        work = moe.alloc_fp8_matmul_workspace(p)
        moe.fp8_matmul(p, x, xs, w, ws, want, work)
        shift = 16 // want.element_size()
        flat = torch.full((M * 144 + 2 * shift,), 5.0, dtype=dtype, device=DEV)
        off = flat[shift:shift + M * 144].view(M, 144)
        odd = torch.empty(xs.numel() + 1, device=DEV)[1:].view_as(xs)
        odd.copy_(xs)
        moe.fp8_matmul(p, x, odd, w, ws, off, work)
        assert torch.equal(off, want) and (flat[:shift] == 5).all() and (flat[-shift:] == 5).all()


def test_gradient_of_the_rows_by_the_transposed_weights():
    """d_x = d_out W by the transposed codes, against autograd of the product in 64 bits: d_out's
    quantisation is off by half a step of each value, 2^-4 of it, or 2^-10 of its block's largest."""
    M, N, K = 150, 272, 400
    g = torch.Generator().manual_seed(0)
    wf = torch.randn(1, N, K, generator=g) / math.sqrt(K)
    d_out = torch.randn(M, N, generator=g).to(BF)
    q = moe.QuantWeightsProblem.make(1, N, K, F32)
    w, ws = torch.empty(1, N, K, dtype=E4M3, device=DEV), torch.empty(1, blocks(N), blocks(K), device=DEV)
    wt, wts = torch.empty(1, K, N, dtype=E4M3, device=DEV), torch.empty(1, blocks(K), blocks(N), device=DEV)
    moe.fp8_quantize_weights(q, wf.to(DEV), w, ws, codes_t=wt, scales_t=wts)
    dq, ds = torch.empty(M, N, dtype=E4M3, device=DEV), torch.empty(M, blocks(N), device=DEV)
    moe.fp8_quantize_rows(moe.QuantProblem.make(M, N), d_out.to(DEV), dq, ds)
    p = moe.FP8Problem.make(M, K, N, 1, F32)
    dx = torch.empty(M, K, device=DEV)
    moe.fp8_matmul(p, dq, ds, wt, wts, dx, moe.alloc_fp8_matmul_workspace(p))
    weight = (w[0].to(F32).double() * per_value(ws[0].double(), N, K)).cpu()
    x = torch.zeros(M, K, dtype=torch.float64, requires_grad=True)
    want, = torch.autograd.grad(x @ weight.t(), x, d_out.double())
    d = d_out.double()
    amax = torch.nn.functional.pad(d.abs(), (0, -N % 128)).reshape(M, -1, 128).amax(2)
    off = torch.maximum(2.0 ** -4 * d.abs(), 2.0 ** -10 / 448 * per_value(amax, None, N))
    mag = d.abs() @ weight.abs()
    tol = off @ weight.abs() + (75 + blocks(N)) * 2.0 ** -24 * mag + 2.0 ** -20 * mag
    assert ((dx.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("M,N,K,E", [(300, 272, 400, 5), (64, 512, 256, 40), (700, 144, 128, 3)])
def test_gradient_of_the_rows_of_experts(M, N, K, E):
    """d_x of rows grouped by expert, empty experts and rows of none among them: the product with the
    transposed codes of the weights, which are the codes themselves turned around."""
    g = torch.Generator().manual_seed(M)
    wf = (torch.randn(E, N, K, generator=g) / math.sqrt(K)).to(BF)
    d_out = torch.randn(M, N, generator=g).to(BF)
    w, ws = torch.empty(E, N, K, dtype=E4M3, device=DEV), torch.empty(E, blocks(N), blocks(K), device=DEV)
    wt, wts = torch.empty(E, K, N, dtype=E4M3, device=DEV), torch.empty(E, blocks(K), blocks(N), device=DEV)
    moe.fp8_quantize_weights(moe.QuantWeightsProblem.make(E, N, K), wf.to(DEV), w, ws, codes_t=wt, scales_t=wts)
    dq, ds = torch.empty(M, N, dtype=E4M3, device=DEV), torch.empty(M, blocks(N), device=DEV)
    moe.fp8_quantize_rows(moe.QuantProblem.make(M, N), d_out.to(DEV), dq, ds)
    back = (w.view(torch.uint8).transpose(1, 2).contiguous().view(E4M3), ws.transpose(1, 2).contiguous())
    assert torch.equal(wt.view(torch.uint8), back[0].view(torch.uint8)) and torch.equal(wts, back[1])
    for dtype in (BF, F32):
        check_product(M, K, N, E, dtype, cut(M, E, tail=7), ops=[t.cpu() for t in (dq, ds, wt, wts)])


def test_graph_replay_and_streams():
    M, N, K, E = 200, 272, 384, 4
    x, xs, w, ws = (t.to(DEV) for t in operands(M, N, K, E))
    offs = cut(M, E).to(DEV)
    p = moe.FP8Problem.make(M, N, K, E)
    work = moe.alloc_fp8_matmul_workspace(p)
    out = torch.zeros(M, N, dtype=BF, device=DEV)
    moe.fp8_matmul(p, x, xs, w, ws, out, work, expert_offsets=offs)
    want = out.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.fp8_matmul(p, x, xs, w, ws, out, work, expert_offsets=offs)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    x2 = x.flip(0).contiguous()
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = torch.zeros_like(out)
    moe.fp8_matmul(p, x, xs, w, ws, other, work, expert_offsets=offs, stream=s)
    s.synchronize()
    assert torch.equal(out, other)


# ------------------------------------------------------------------ the run of them
def test_layer_of_the_operators():
    """FP8Experts behind router_forward against the layer in 64 bits on the weights that the codes
    stand for.  x and h are quantised (half a step, 2^-4 of a value at most, in either product), the
    two products' outputs and the result are rounded to bf16."""
    for T, H, F, E, k, interleave in ((1, 256, 256, 8, 2, 0), (200, 256, 384, 8, 3, 0), (70, 512, 128, 40, 4, 32)):
        g = torch.Generator().manual_seed(T)
        x = torch.randn(T, H, generator=g).to(BF)
        w1 = (torch.randn(E, 2 * F, H, generator=g) / math.sqrt(H)).to(BF)
        w2 = (torch.randn(E, H, F, generator=g) / math.sqrt(F)).to(BF)
        logits, bias = torch.randn(T, E, generator=g), torch.randn(E, generator=g) * 0.1
        p = moe.RouterProblem.make(T, E, k, score="sigmoid", groups=4, topk_groups=2, group_top=2)
        idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
        w = torch.empty(T, k, device=DEV)
        moe.router_forward(p, logits.to(DEV), idx, w, bias=bias.to(DEV))
        if T > 1:
            idx[3, 1] = -1  # a masked route
        layer = moe.FP8Experts(w1.to(DEV), w2.to(DEV), k, interleave)
        out = layer(x.to(DEV), idx, w)
        assert moe.get_device_status(layer.ws) == moe.get_device_status(layer.ws_matmul) == moe.MOE_OK
        a = layer.w1.to(F32).double().cpu() * per_value(layer.s1.double().cpu(), 2 * F, H)
        b = layer.w2.to(F32).double().cpu() * per_value(layer.s2.double().cpu(), H, F)
        want = torch.zeros(T, H, dtype=torch.float64)
        for t in range(T):
            for j in range(k):
                e = int(idx[t, j])
                if e >= 0:
                    h, _ = swiglu_of((a[e] @ x[t].double())[None], F, interleave, 0.0)
                    want[t] += float(w[t, j]) * (b[e] @ h[0])
        err = (out.double().cpu() - want).norm() / want.norm()
        # two quantisations of independent roundings, each of 2^-4 / sqrt(3) of a value at most
        # (uniform in half a step), through sums of random signs
        assert err <= 2 * 2.0 ** -4 / math.sqrt(3), float(err)
