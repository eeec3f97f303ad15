"""The router, the quantisation and the product of the codes beyond 2^31 elements; what they
allocate; workspaces and streams used at once.

Large tensors are filled on the GPU with a few known rows (or with one value), so that the expected
values are those of the rows alone."""
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


def test_router_rows_beyond_31_bits():
    """The last rows of logits of 2.3 billion elements (a stride of 1100), against them alone."""
    T, E, ld, n = 2_100_000, 100, 1100, 9
    big = torch.zeros(T, ld, dtype=BF, device=DEV)
    tail = torch.randn(n, E, generator=torch.Generator(device=DEV).manual_seed(0), device=DEV).to(BF)
    big[-n:, :E] = tail
    bias = torch.rand(E, device=DEV)

    def run(rows, l, stride):
        p = moe.RouterProblem.make(rows, E, 6, BF, "sigmoid", ld_logits=stride)
        idx = torch.empty(rows, 6, dtype=torch.int32, device=DEV)
        w, dl = torch.empty(rows, 6, device=DEV), torch.zeros(rows, stride or E, dtype=BF, device=DEV)[:, :E]
        moe.router_forward(p, l, idx, w, bias=bias)
        moe.router_backward(p, l, idx, torch.ones_like(w) * torch.arange(6, device=DEV), dl)
        return idx[-n:], w[-n:], dl[-n:]

    for a, b in zip(run(n, tail, 0), run(T, big[:, :E], ld)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("swiglu", [False, True])
def test_quantised_rows_beyond_32_bits(swiglu):
    T, H, n = (300_000, 8192, 5) if swiglu else (600_000, 8192, 5)
    width = 2 * H if swiglu else H
    tail = torch.randn(n, width, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(BF)
    big = torch.zeros(T, width, dtype=BF, device=DEV)
    big[-n:] = tail

    def run(rows, src):
        codes = torch.empty(rows, H, dtype=E4M3, device=DEV)
        scales = torch.empty(rows, H // 128, device=DEV)
        moe.fp8_quantize_rows(moe.QuantProblem.make(rows, H, swiglu=swiglu), src, codes, scales)
        return codes.view(torch.uint8), scales

    (c0, s0), (c1, s1) = run(n, tail), run(T, big)
    assert torch.equal(c0, c1[-n:]) and torch.equal(s0, s1[-n:])
    assert not c1[T // 2:T // 2 + 100].any() and (s1[T // 2:T // 2 + 100] == 1).all()


def test_weights_and_product_beyond_32_bits():
    """The last of 270 experts of 4096 x 4096 (4.5 billion codes), quantised there and multiplied."""
    E, N, K, M = 270, 4096, 4096, 300
    g = torch.Generator(device=DEV).manual_seed(2)
    last = (torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K)).to(BF)
    src = torch.zeros(E, N, K, dtype=BF, device=DEV)
    src[-1] = last

    def quantise(w):
        e = w.shape[0]
        out = [torch.empty(e, N, K, dtype=E4M3, device=DEV), torch.empty(e, N // 128, K // 128, device=DEV),
               torch.empty(e, K, N, dtype=E4M3, device=DEV), torch.empty(e, K // 128, N // 128, device=DEV)]
        moe.fp8_quantize_weights(moe.QuantWeightsProblem.make(e, N, K), w, *out[:2], codes_t=out[2],
                                 scales_t=out[3])
        return out

    one, all_ = quantise(last[None]), quantise(src)
    for a, b in zip(one, all_):
        assert torch.equal(a[0].view(torch.uint8), b[-1].view(torch.uint8))
    del src
    x = torch.randn(M, K, generator=g, device=DEV).to(BF)
    xq, xs = torch.empty(M, K, dtype=E4M3, device=DEV), torch.empty(M, K // 128, device=DEV)
    moe.fp8_quantize_rows(moe.QuantProblem.make(M, K), x, xq, xs)
    for rows in (M, 70, 5):
        offs = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        offs[-1] = rows
        got = []
        for e, w, s, o in ((1, one[0], one[1], None), (E, all_[0], all_[1], offs)):
            p = moe.FP8Problem.make(rows, N, K, e, F32)
            out = torch.empty(rows, N, device=DEV)
            moe.fp8_matmul(p, xq[:rows], xs[:rows], w, s, out, moe.alloc_fp8_matmul_workspace(p),
                           expert_offsets=o)
            got.append(out)
        # another tiling or split of the sums: 32 blocks' order in fp32
        assert (got[0] - got[1]).abs().max() <= 64 * 2.0 ** -24 * got[0].abs().max() * 32
    del all_


@pytest.mark.parametrize("N", [65536, 65535])
def test_product_rows_beyond_32_bits(N):
    M, K, n = 70_000, 128, 300
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.zeros(M, K, dtype=torch.uint8, device=DEV)
    x[-n:] = (torch.randn(n, K, generator=g, device=DEV) * 100).clamp(-448, 448).to(E4M3).view(torch.uint8)
    w = (torch.randn(1, N, K, generator=g, device=DEV) * 100).clamp(-448, 448).to(E4M3)
    xs, ws = torch.ones(M, 1, device=DEV), torch.full((1, 512, 1), 1.0 / 1024, device=DEV)
    out = torch.full((M, N), 3.0, dtype=BF, device=DEV)
    p = moe.FP8Problem.make(M, N, K)
    moe.fp8_matmul(p, x, xs, w, ws, out, moe.alloc_fp8_matmul_workspace(p))
    want = x[-n:].view(E4M3).double() @ w[0].double().t() / 1024
    mag = x[-n:].view(E4M3).double().abs() @ w[0].double().abs().t() / 1024
    assert ((out[-n:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 80 * 2.0 ** -24 * mag).all()
    assert not out[M // 2:M // 2 + 50].any()


def test_nothing_is_allocated():
    T, E, H = 500, 64, 512
    logits, bias = torch.randn(T, E, device=DEV), torch.randn(E, device=DEV)
    p = moe.RouterProblem.make(T, E, 4, score="sigmoid", groups=4, topk_groups=2, group_top=2)
    idx, w = torch.empty(T, 4, dtype=torch.int32, device=DEV), torch.empty(T, 4, device=DEV)
    dl = torch.empty_like(logits)
    src = torch.randn(E, H, H, device=DEV).to(BF)
    qw = moe.QuantWeightsProblem.make(E, H, H)
    cw, sw = torch.empty(E, H, H, dtype=E4M3, device=DEV), torch.empty(E, 4, 4, device=DEV)
    x = torch.randn(T, H, device=DEV).to(BF)
    qx = moe.QuantProblem.make(T, H)
    cx, sx = torch.empty(T, H, dtype=E4M3, device=DEV), torch.empty(T, 4, device=DEV)
    problems = [moe.FP8Problem.make(T, H, H, e) for e in (1, E)]
    offs = torch.arange(E + 1, dtype=torch.int32, device=DEV) * (T // E)
    work = moe.alloc_fp8_matmul_workspace(problems[0])
    out = torch.empty(T, H, dtype=BF, device=DEV)

    def run():
        moe.router_forward(p, logits, idx, w, bias=bias)
        moe.router_backward(p, logits, idx, w, dl)
        moe.fp8_quantize_weights(qw, src, cw, sw)
        moe.fp8_quantize_rows(qx, x, cx, sx)
        moe.fp8_matmul(problems[0], cx, sx, cw[:1], sw[:1], out, work)
        moe.fp8_matmul(problems[1], cx, sx, cw, sw, out, work, expert_offsets=offs)

    run()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(5):
        run()
    torch.cuda.synchronize()
    assert before == (torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"])
    assert moe.get_device_status(work) == moe.MOE_OK


def test_calls_at_once_on_two_streams_and_in_two_graphs_of_one_workspace():
    """Products on two streams and of two captured graphs share a workspace: it holds a status only."""
    M, N, K = 300, 512, 1024
    g = torch.Generator(device=DEV).manual_seed(5)
    code = lambda *s: (torch.randn(*s, generator=g, device=DEV) * 100).clamp(-448, 448).to(E4M3)  # noqa: E731
    w, ws = code(1, N, K), torch.rand(1, 4, 8, generator=g, device=DEV)
    xs = torch.rand(M, 8, generator=g, device=DEV)
    a, b = code(M, K), code(M, K)
    p = moe.FP8Problem.make(M, N, K)
    work = moe.alloc_fp8_matmul_workspace(p)
    want = [torch.empty(M, N, dtype=BF, device=DEV) for _ in range(2)]
    for x, o in zip((a, b), want):
        moe.fp8_matmul(p, x, xs, w, ws, o, work)
    torch.cuda.synchronize()
    got = [torch.zeros(M, N, dtype=BF, device=DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for x, o, s in zip((a, b), got, streams):
            moe.fp8_matmul(p, x, xs, w, ws, o, work, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graphs = []
    for x, o in zip((a, b), got):
        o.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.fp8_matmul(p, x, xs, w, ws, o, work)
        graphs.append(graph)
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_layer_changes_its_token_count_and_masks():
    """FP8Experts with other counts of tokens between, padded tokens masked throughout."""
    E, H, F, k = 8, 256, 256, 2
    g = torch.Generator(device=DEV).manual_seed(6)
    layer = moe.FP8Experts(torch.randn(E, 2 * F, H, generator=g, device=DEV) / 16,
                           torch.randn(E, H, F, generator=g, device=DEV) / 16, k)
    x = torch.randn(64, H, generator=g, device=DEV).to(BF)
    logits = torch.randn(64, E, generator=g, device=DEV)
    logits[40:] = -math.inf  # padding
    p = moe.RouterProblem.make(64, E, k)
    idx, w = torch.empty(64, k, dtype=torch.int32, device=DEV), torch.empty(64, k, device=DEV)
    moe.router_forward(p, logits, idx, w)
    assert (idx[40:] == -1).all() and (w[40:] == 0).all()
    whole = layer(x, idx, w)
    assert not whole[40:].any() and whole[:40].any()
    part = layer(x[:40], idx[:40].contiguous(), w[:40].contiguous())
    # the same codes and the same rows per expert: the same sums
    assert torch.equal(part, whole[:40])
    again = layer(x, idx, w)
    assert torch.equal(again, whole)
    assert layer(x[:0], idx[:0], w[:0]).shape == (0, H)
    assert moe.get_device_status(layer.ws) == moe.MOE_OK


def test_layer_in_a_graph_while_its_token_count_changes():
    """A captured call of FP8Experts replays into its own buffers after eager calls of other counts
    took new ones; memory freed meanwhile belongs to others and stays as they wrote it."""
    E, H, F, k, T = 8, 256, 256, 2, 96
    g = torch.Generator(device=DEV).manual_seed(7)
    layer = moe.FP8Experts(torch.randn(E, 2 * F, H, generator=g, device=DEV) / 16,
                           torch.randn(E, H, F, generator=g, device=DEV) / 16, k)
    x = torch.randn(T, H, generator=g, device=DEV).to(BF)
    p = moe.RouterProblem.make(T, E, k, score="sigmoid")
    idx, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    moe.router_forward(p, torch.randn(T, E, generator=g, device=DEV), idx, w)
    want = layer(x, idx, w)  # (and the plan, outside the graph)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, idx, w, out=out)
    others = []
    for n in (8, 96, 40):
        part = layer(x[:n], idx[:n].contiguous(), w[:n].contiguous())
        others.append((n, part))
        others += [(None, torch.full((n * H,), 5, dtype=torch.uint8, device=DEV)) for _ in range(40)]
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for n, t in others:
        assert torch.equal(t, want[:n]) if n else (t == 5).all()
    assert moe.get_device_status(layer.ws) == moe.get_device_status(layer.ws_matmul) == moe.MOE_OK


def test_layer_on_two_streams_while_its_token_count_changes():
    """Buffers made on one stream and used on another are not given away under the other's work."""
    E, H, F, k = 8, 512, 512, 2
    g = torch.Generator(device=DEV).manual_seed(8)
    layer = moe.FP8Experts(torch.randn(E, 2 * F, H, generator=g, device=DEV) / 22,
                           torch.randn(E, H, F, generator=g, device=DEV) / 22, k)
    x = torch.randn(2048, H, generator=g, device=DEV).to(BF)
    idx = torch.randint(0, E, (2048, k), generator=g, device=DEV, dtype=torch.int32)
    w = torch.rand(2048, k, generator=g, device=DEV)
    want = layer(x, idx, w)
    small = layer(x[:64], idx[:64].contiguous(), w[:64].contiguous())
    outs = []
    s = torch.cuda.Stream()
    layer(x, idx, w)
    for _ in range(5):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(layer(x, idx, w))
        filler = [torch.full((2048 * k, 2 * F), 1.0, dtype=BF, device=DEV) for _ in range(4)]
        layer._plan(64, x.device)
        del filler
        torch.cuda.current_stream().wait_stream(s)
        outs.append(layer(x[:64], idx[:64].contiguous(), w[:64].contiguous()))
        layer._plan(2048, x.device)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want if o.shape[0] == 2048 else small)


def test_layer_captured_without_a_call_before():
    """Two graphs of a layer whose first calls they are; an eager call before the first replay."""
    E, H, F, k, T = 8, 256, 256, 2, 50
    g = torch.Generator(device=DEV).manual_seed(9)
    w1, w2 = torch.randn(E, 2 * F, H, generator=g, device=DEV) / 16, torch.randn(E, H, F, generator=g, device=DEV) / 16
    x = torch.randn(T, H, generator=g, device=DEV).to(BF)
    idx = torch.stack([torch.randperm(E, generator=g, device=DEV)[:k] for _ in range(T)]).to(torch.int32)
    w = torch.rand(T, k, generator=g, device=DEV)
    want = moe.FP8Experts(w1, w2, k)(x, idx, w)
    layer = moe.FP8Experts(w1, w2, k)
    outs, graphs, status = [torch.zeros_like(want) for _ in range(2)], [], []
    torch.cuda.synchronize()
    for o in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer(x, idx, w, out=o)
        graphs.append(graph)
        status.append((layer.ws, layer.ws_matmul))
    assert torch.equal(layer(x, idx, w), want)
    status.append((layer.ws, layer.ws_matmul))
    for graph in reversed(graphs):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    for a, b in status:
        assert moe.get_device_status(a) == moe.get_device_status(b) == moe.MOE_OK
