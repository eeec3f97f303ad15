"""GPU parity of the embedding and its gradient against 64 bits on the CPU.

Tolerances: the forward is one fp32 product and one rounding.  A gradient row
adds its n tokens in fp32 (n 2^-24 of the terms' magnitude at most, in any
order), multiplies by the scale and rounds once."""
import itertools

import pytest
import torch

import mixture_experts_ffn_permute_gb300 as moe
from mixture_experts_ffn_permute_gb300 import _build

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    moe.load()


def rounding(dtype):
    return 2.0 ** -8 if dtype is BF else 2.0 ** -22


def check_forward(ids, V, H, tt, to, scale=1.7):
    T = ids.numel()
    g = torch.Generator().manual_seed(T + H)
    table = torch.randn(V, H, generator=g).to(tt)
    out = torch.full((T, H), float("nan"), dtype=to, device=DEV)
    p = moe.EmbedProblem.make(T, V, H, tt, to, scale)
    moe.embedding_forward(p, ids.to(DEV), table.to(DEV), out)
    ok = (ids >= 0) & (ids < V)
    want = table.double()[torch.where(ok, ids, 0).long()] * scale * ok[:, None]
    assert ((out.double().cpu() - want).abs() <= rounding(to) * want.abs()).all()


def check_backward(ids, V, H, tt=F32, to=F32, scale=0.7, seed=0):
    T = ids.numel()
    g = torch.Generator().manual_seed(seed)
    d_out = torch.randn(T, H, generator=g).to(to)
    d_table = torch.full((V, H), float("nan"), dtype=tt, device=DEV)
    p = moe.EmbedProblem.make(T, V, H, tt, to, scale)
    ws = moe.alloc_embedding_workspace(p)
    moe.embedding_backward(p, ids.to(DEV), d_out.to(DEV), d_table, ws)
    ok = (ids >= 0) & (ids < V)
    at = ids[ok].long()
    want = torch.zeros(V, H, dtype=torch.float64).index_add_(0, at, d_out.double()[ok]) * scale
    mag = torch.zeros(V, H, dtype=torch.float64).index_add_(0, at, d_out.double()[ok].abs()) * scale
    n = torch.bincount(at, minlength=V).double()[:, None]
    tol = rounding(tt) * want.abs() + (n + 2) * 2.0 ** -24 * mag
    err = (d_table.double().cpu() - want).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())
    return p, ws, d_table


def ids_of(T, V, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "uniform":
        return torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    if kind == "one":
        return torch.full((T,), V // 2, dtype=torch.int32)
    if kind == "masked":
        return torch.full((T,), -1, dtype=torch.int32)
    if kind == "few":  # long runs of a few ids, single ones between
        return (torch.randint(0, 3, (T,), generator=g) ** 5 * (V - 1) // 32).to(torch.int32)
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    ids = torch.where(torch.rand(T, generator=g) < 0.4, V // 3, ids)  # frequent, rare, masked
    return torch.where(torch.rand(T, generator=g) < 0.2, -7, ids).to(torch.int32)


@pytest.mark.parametrize("H", [1, 5, 8, 64, 511, 512, 520, 1000, 1001, 2048])
def test_forward_widths(H):
    check_forward(ids_of(77, 50, "mixed"), 50, H, BF, F32)
    check_forward(ids_of(3, 1, "uniform"), 1, H, F32, BF)


@pytest.mark.parametrize("tt,to", list(itertools.product((BF, F32), repeat=2)))
def test_types(tt, to):
    check_forward(ids_of(200, 1000, "mixed"), 1000, 264, tt, to)
    for H in (264, 77):
        check_backward(ids_of(700, 90, "mixed"), 90, H, tt, to)


@pytest.mark.parametrize("kind", ["uniform", "one", "masked", "few", "mixed"])
@pytest.mark.parametrize("T", [1, 2, 31, 63, 64, 65, 128, 129, 1000, 5000])
def test_backward_ids(kind, T):
    check_backward(ids_of(T, 200, kind, T), 200, 40)


@pytest.mark.parametrize("V", [1, 2, 31, 33, 152 * 32, 152 * 32 + 1, 50021, 152 * 1024, 200003])
def test_backward_vocabularies(V):
    check_backward(ids_of(900, V, "mixed"), V, 24)


@pytest.mark.parametrize("H", [1, 7, 8, 511, 512, 513, 1001, 2056])
def test_backward_widths(H):
    check_backward(ids_of(400, 37, "mixed"), 37, H, BF, BF)


@pytest.mark.parametrize("H", [40, 248, 256, 264, 513, 1024, 1025, 2047, 2048, 2049, 2056, 4104])
def test_groups_and_column_blocks(H):
    """Every group size (32 to 256 threads) and several column blocks, with long, short and
    empty runs of ids."""
    for V, T, kind in ((1000, 300, "uniform"), (37, 600, "mixed"), (600, 900, "few")):
        check_backward(ids_of(T, V, kind, H), V, H, BF, F32)
        check_backward(ids_of(T, V, kind, H), V, H, F32, BF)


def test_unaligned_rows():
    """A table and gradients that start off a 16-byte boundary."""
    for shift in (1, 3):
        ids = ids_of(500, 90, "mixed")
        d = torch.randn(500 * 64 + shift, device=DEV).to(BF)[shift:].view(500, 64)
        full = torch.full((90 * 64 + 16,), float("nan"), dtype=BF, device=DEV)
        t = full[shift:shift + 90 * 64].view(90, 64)
        p = moe.EmbedProblem.make(500, 90, 64, BF, BF)
        moe.embedding_backward(p, ids.to(DEV), d, t, moe.alloc_embedding_workspace(p))
        ok = ids >= 0
        want = torch.zeros(90, 64, dtype=torch.float64).index_add_(
            0, ids[ok].long(), d.double().cpu()[ok])
        err = (t.double().cpu() - want).abs()
        assert (err <= 2.0 ** -8 * want.abs() + 1e-3).all()
        assert torch.isnan(full[:shift]).all() and torch.isnan(full[shift + 90 * 64:]).all()
        out = torch.empty(500 * 64 + shift, dtype=BF, device=DEV)[shift:].view(500, 64)
        moe.embedding_forward(p, ids.to(DEV), t, out)
        assert torch.equal(out[ok.to(DEV)], t[ids[ok].long().to(DEV)])


def test_runs_round_the_piece_boundaries():
    """Runs of 64, 65 and more tokens that start at, before and after multiples of 64."""
    for lead in (0, 1, 63, 64, 65):
        for n in (1, 63, 64, 65, 66, 127, 128, 129, 200):
            runs = [(0, lead), (1, n), (2, 65), (3, 64), (4, 300), (5, 1)]
            ids = torch.cat([torch.full((c,), v, dtype=torch.int32) for v, c in runs])
            ids = ids[torch.randperm(ids.numel(), generator=torch.Generator().manual_seed(n))]
            check_backward(ids, 7, 16)


def test_no_tokens():
    p = moe.EmbedProblem.make(0, 9, 16, BF, BF)
    ids = torch.empty(0, dtype=torch.int32, device=DEV)
    e, t = torch.empty(0, 16, dtype=BF, device=DEV), torch.ones(9, 16, dtype=BF, device=DEV)
    moe.embedding_forward(p, ids, t, e)
    moe.embedding_backward(p, ids, e, t, moe.alloc_embedding_workspace(p))
    assert not t.any()


def test_ids_beyond_the_vocabulary():
    """Treated as masked and recorded in the status word."""
    ids = torch.tensor([3, 50, 2, 1 << 30, -1, 49], dtype=torch.int32)
    check_forward(ids, 50, 40, F32, F32)
    p, ws, _ = check_backward(ids, 50, 40)
    assert moe.get_device_status(ws) == 7
    moe.clear_device_status(ws)
    t, o = torch.zeros(50, 40, device=DEV), torch.zeros(6, 40, device=DEV)
    moe.embedding_forward(p, ids.to(DEV), t, o, ws=ws)
    assert moe.get_device_status(ws) == 7
    _, ws, _ = check_backward(ids.clamp(max=49), 50, 40)
    assert moe.get_device_status(ws) == moe.MOE_OK


def test_values_that_are_not_finite_stay_in_their_rows():
    ids = torch.tensor([1, 2, 1, 4, -1], dtype=torch.int32, device=DEV)
    d = torch.ones(5, 24, device=DEV)
    d[1, 3], d[4] = float("nan"), float("inf")  # a token of id 2; a masked token
    t = torch.empty(6, 24, device=DEV)
    p = moe.EmbedProblem.make(5, 6, 24, F32, F32)
    moe.embedding_backward(p, ids, d, t, moe.alloc_embedding_workspace(p))
    bad = torch.isnan(t) | torch.isinf(t)
    assert bad.sum() == 1 and bad[2, 3]


def test_large_offsets():
    """Rows beyond 2^31 elements of the table."""
    V, H = 70000, 32768
    table = torch.zeros(V, H, dtype=BF, device=DEV)
    table[V - 1] = 3.0
    ids = torch.tensor([V - 1, 0, V - 1], dtype=torch.int32, device=DEV)
    out = torch.empty(3, H, dtype=BF, device=DEV)
    p = moe.EmbedProblem.make(3, V, H, BF, BF)
    moe.embedding_forward(p, ids, table, out)
    assert (out[0] == 3).all() and (out[2] == 3).all() and not out[1].any()
    moe.embedding_backward(p, ids, out, table, moe.alloc_embedding_workspace(p))
    assert (table[V - 1] == 6).all() and not table[: V - 1].any()


def test_against_differences():
    """<G, out> is linear in the table: its gradient is its difference."""
    ids = ids_of(60, 20, "mixed")
    g = torch.Generator().manual_seed(5)
    table, G = torch.randn(20, 33, generator=g), torch.randn(60, 33, generator=g)
    p = moe.EmbedProblem.make(60, 20, 33, F32, F32, 0.5)
    d = torch.empty(20, 33, device=DEV)
    moe.embedding_backward(p, ids.to(DEV), G.to(DEV), d, moe.alloc_embedding_workspace(p))
    v = torch.randn(20, 33, generator=g)

    def value(t):
        out = torch.empty(60, 33, device=DEV)
        moe.embedding_forward(p, ids.to(DEV), t.to(DEV), out)
        return float((out.double().cpu() * G.double()).sum())

    num = (value(table + v) - value(table - v)) / 2
    assert abs(num - float((d.double().cpu() * v.double()).sum())) <= 1e-4 * abs(num) + 1e-4


def test_reproducible_and_on_another_stream():
    ids = ids_of(5000, 300, "mixed").to(DEV)
    d = torch.randn(5000, 264, device=DEV)
    p = moe.EmbedProblem.make(5000, 300, 264, F32, F32)

    def once(stream=None):
        t, ws = torch.empty(300, 264, device=DEV), moe.alloc_embedding_workspace(p)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        moe.embedding_backward(p, ids, d, t, ws, stream=stream)
        torch.cuda.synchronize()
        return t

    a = once()
    assert torch.equal(a, once()) and torch.equal(a, once(torch.cuda.Stream()))


def test_binding_refuses_wrong_tensors():
    p = moe.EmbedProblem.make(4, 10, 16)
    ids = torch.zeros(4, dtype=torch.int32, device=DEV)
    t, o = torch.zeros(10, 16, dtype=BF, device=DEV), torch.zeros(4, 16, dtype=BF, device=DEV)
    for a in ((ids.long(), t, o), (ids[:3], t, o), (ids, t.float(), o), (ids, t[:9], o),
              (ids, t, o.cpu()), (ids, t, torch.zeros(16, 4, dtype=BF, device=DEV).t())):
        with pytest.raises(ValueError):
            moe.embedding_forward(p, *a)


def pieces_of(p):
    """The pieces of the sorted list, from what the workspace holds past the lists."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    lists = 256 + 2 * up(4 * p.T) + up(4 * (p.V + 1))
    part = moe.alloc_embedding_workspace(p).numel() - lists
    return next(n for n in (8, 16, 32) if up(8 * -(-p.T // n) * p.H) == part)


# pieces of 16 and of 32 tokens, which sizes of training take: rows of wide accesses and of single
# elements, and every number of tokens in flight
@pytest.mark.parametrize("T,piece", [(4500, 16), (10000, 32), (10015, 32)])
@pytest.mark.parametrize("H", [4104, 4101])
@pytest.mark.parametrize("tt,to", [(BF, BF), (F32, F32), (F32, BF)])
def test_longer_pieces(T, piece, H, tt, to):
    V = 701
    p = moe.EmbedProblem.make(T, V, H, tt, to, 0.7)
    assert pieces_of(p) == piece
    g = torch.Generator(device=DEV).manual_seed(T + H)
    d_out = torch.randn(T, H, generator=g, device=DEV).to(to)
    # runs that end at, one before and one behind the pieces' ends; single tokens; one long run
    edges = [n for q in range(1, 12) for n in (q * piece - 1, q * piece, q * piece + 1)]
    runs, at = [], 0
    for e in edges:
        runs.append(e - at)
        at = e
    runs += [1] * 200 + [3000] + [5, 11] * 20
    bounded = torch.repeat_interleave(torch.arange(len(runs)), torch.tensor(runs))
    bounded = torch.cat([bounded, torch.full((T - bounded.numel(),), 400)])
    bounded = bounded[torch.randperm(T, generator=torch.Generator().manual_seed(T))]
    for ids in (bounded.to(torch.int32), ids_of(T, V, "mixed"), ids_of(T, V, "one"),
                ids_of(T, V, "few"), ids_of(T, V, "uniform")):
        d_table = torch.full((V, H), float("nan"), dtype=tt, device=DEV)
        moe.embedding_backward(p, ids.to(DEV), d_out, d_table, moe.alloc_embedding_workspace(p))
        at = ids.to(DEV).long()
        ok = at >= 0
        d = d_out.double()[ok] * 0.7
        want, mag = (torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, at[ok], t)
                     for t in (d, d.abs()))
        n = torch.bincount(at[ok], minlength=V).double()[:, None]
        tol = rounding(tt) * want.abs() + (n + 2) * 2.0 ** -24 * mag
        err = (d_table.double() - want).abs()
        assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())
