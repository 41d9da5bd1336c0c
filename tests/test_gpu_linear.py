"""The dense product with its fused epilogue against a 64-bit reference: formats,
sizes on both sides of every choice of kernel, strides, in-place residual, capture."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_31_b200 as moe
import ops_ref as ref
import synth

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
FORMATS = [("bf16", "bf16"), ("int8", "bf16"), ("int4", "bf16"), ("int4b128", "bf16"), ("f32", "f32"), ("f32", "bf16"),
           ("bf16", "f32"), ("int8", "f32"), ("int4", "f32"), ("int4b128", "f32")]


@pytest.fixture(autouse=True)
def _clear_flags():
    moe.moe_device_flags(clear=True)
    yield
    assert moe.moe_device_flags(clear=True) == 0


class Product:
    def __init__(self, K, N, wfmt="bf16", xfmt="bf16", yfmt=None, act="none", gated=False, bias=False, seed=3):
        self.K, self.N, self.wfmt, self.act = K, N, wfmt, act
        self.x_dtype, self.y_dtype = DT[xfmt], DT[yfmt or xfmt]
        W, s, self.W = ref.weights(N, K, wfmt, seed)
        Wu, su, self.Wu = ref.weights(N, K, wfmt, seed + 1) if gated else (None, None, None)
        mk = lambda n: torch.from_numpy(synth.normal_f32((N,), n, 4, 0.0, 1.0)) if bias else None
        b, bu = mk(seed + 2), mk(seed + 3) if gated else None
        self.b, self.bu = (None if t is None else t.double() for t in (b, bu))
        self.dev = moe.Linear(K=K, N=N, wfmt=wfmt, xfmt=xfmt, yfmt=yfmt, act=act, W=W, s=s, b=b, W_up=Wu, s_up=su, b_up=bu)

    def x(self, M, seed=7):
        return torch.from_numpy(synth.normal_f32((M, self.K), seed, 9, 0.0, 1.0)).to(self.x_dtype)

    def residual(self, M, seed=8):
        return torch.from_numpy(synth.normal_f32((M, self.N), seed, 9, 0.0, 1.0)).to(self.y_dtype)

    def compare(self, x, y, residual=None, what=""):
        # int4 weights are widened exactly for up to 40 tokens and for fp32 outputs; else each is rounded
        # to bf16 once, which is off by half a step of bf16 at most, or kept in two parts (moe_linear)
        exact = x.shape[0] <= 40 or self.y_dtype == torch.float32
        want, bound = ref.linear(x, self.W, self.b, None if self.Wu is None else (self.Wu, self.bu), self.act, residual,
                                 self.y_dtype, self.wfmt, 0 if exact else (1 if self.Wu is None else 2))
        ref.check(y, want, bound, what)

    def run(self, M, residual=False):
        x = self.x(M)
        r = self.residual(M) if residual else None
        y = self.dev(x.cuda(), residual=None if r is None else r.cuda())
        torch.cuda.synchronize()
        self.compare(x, y, r, "M=%d" % M)
        return x, y


@pytest.mark.parametrize("wfmt,xfmt", FORMATS)
@pytest.mark.parametrize("M", [1, 7, 16, 17, 24, 25, 32, 33, 40, 41, 48, 49, 64, 65, 200])
def test_formats(wfmt, xfmt, M):
    Product(384, 200, wfmt, xfmt, bias=True, act="silu").run(M, residual=M % 2 == 0)


@pytest.mark.parametrize("wfmt,xfmt", FORMATS)
@pytest.mark.parametrize("M", [1, 16, 33, 130])
def test_gated(wfmt, xfmt, M):
    Product(256, 136, wfmt, xfmt, act="gelu_tanh", gated=True, bias=M != 16).run(M, residual=M == 33)


@pytest.mark.parametrize("wfmt", ["bf16", "int8", "int4", "int4b128", "f32"])
@pytest.mark.parametrize("yfmt", ["f32", "bf16"])
@pytest.mark.parametrize("M", [3, 20, 90])
def test_output_formats(wfmt, yfmt, M):
    Product(256, 77, wfmt, "f32" if wfmt == "f32" else "bf16", yfmt=yfmt, bias=True).run(M, residual=True)


@pytest.mark.parametrize("M", [1, 2, 15, 17, 63, 127, 128, 129, 255, 257, 300])
@pytest.mark.parametrize("N", [1, 63, 129, 513])
def test_ragged_sizes(M, N):
    Product(192, N, "bf16", bias=True, seed=M + N).run(M, residual=True)


@pytest.mark.parametrize("wfmt,xfmt,K", [("bf16", "bf16", 8), ("bf16", "bf16", 40), ("bf16", "bf16", 1000), ("int8", "bf16", 16),
                                         ("int8", "bf16", 336), ("int4", "bf16", 32), ("int4", "bf16", 96),
                                         ("int4", "bf16", 1056), ("int4b128", "bf16", 128), ("int4b128", "bf16", 640),
                                         ("f32", "f32", 4), ("f32", "f32", 300), ("f32", "bf16", 8), ("int8", "f32", 16)])
@pytest.mark.parametrize("M", [1, 20, 150])
def test_short_and_ragged_reductions(wfmt, xfmt, K, M):
    Product(K, 70, wfmt, xfmt, bias=True, gated=K % 3 == 0, act="silu").run(M, residual=True)


@pytest.mark.parametrize("wfmt", ["bf16", "int8", "int4", "int4b128"])
@pytest.mark.parametrize("M", [1, 2, 8, 13, 24, 32, 40, 48, 64, 90])
def test_many_columns(wfmt, M):
    """Columns enough for units of two row tiles."""
    Product(384, 9533, wfmt, bias=True).run(M)


@pytest.mark.parametrize("wfmt", ["bf16", "int8", "int4", "int4b128"])
@pytest.mark.parametrize("M", [1, 2, 8, 48, 100, 500])
@pytest.mark.parametrize("yfmt", ["bf16", "f32"])
def test_long_reductions(wfmt, M, yfmt):
    """Sums long enough to be split over several CTAs."""
    Product(9216, 96, wfmt, yfmt=yfmt).run(M, residual=True)


@pytest.mark.parametrize("wfmt,xfmt,gated", [("bf16", "bf16", False), ("bf16", "bf16", True), ("f32", "f32", False),
                                             ("f32", "f32", True), ("int8", "f32", False), ("int4", "f32", False),
                                             ("f32", "bf16", False)])
def test_fp32_outputs_drained_in_segments(wfmt, xfmt, gated):
    """Enough tiles that the reduction is not split, and columns for several segments."""
    Product(1664, 2000, wfmt, xfmt, yfmt="f32", gated=gated, act="silu", bias=True).run(2500)


@pytest.mark.parametrize("wfmt", ["bf16", "int8", "int4"])
def test_many_tiles(wfmt):
    Product(512, 1537, wfmt, act="silu", gated=True).run(1111)


@pytest.mark.parametrize("wfmt,xfmt", [("bf16", "bf16"), ("int8", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("M", [2, 50, 140])
def test_strided_rows_and_untouched_neighbours(wfmt, xfmt, M):
    p = Product(128, 101, wfmt, xfmt, bias=True)
    pad = 24
    xs = torch.full((M + 2, p.K + pad), float("nan"), dtype=p.x_dtype, device="cuda")
    rs = torch.full((M + 2, p.N + 7), float("nan"), dtype=p.y_dtype, device="cuda")
    ys = torch.full((M + 2, p.N + 3), 5.0, dtype=p.y_dtype, device="cuda")
    x, r = p.x(M), p.residual(M)
    xs[:M, : p.K], rs[:M, : p.N] = x.cuda(), r.cuda()
    p.dev(xs[:M, : p.K], residual=rs[:M, : p.N], y=ys[:M, : p.N])
    torch.cuda.synchronize()
    p.compare(x, ys[:M, : p.N], r)
    assert bool((ys[M:] == 5).all()) and bool((ys[:, p.N:] == 5).all())


@pytest.mark.parametrize("M", [1, 30, 150])
def test_in_place_residual(M):
    p = Product(256, 160, "int8", act="silu", bias=True)
    x, r = p.x(M).cuda(), p.residual(M).cuda()
    y = p.dev(x, residual=r.clone())
    p.dev(x, residual=r, y=r)
    assert torch.equal(y, r)


@pytest.mark.parametrize("wfmt", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("M", [0, 1, 4, 14, 40, 200])
def test_infinity_and_nan_stay_in_their_row(M, wfmt):
    p = Product(256, 96, wfmt)
    x = p.x(M + 2)
    x[M:] = 1  # the same number of rows, so the same kernel
    clean = p.dev(x.cuda())
    x[M, 3], x[M + 1, 9] = float("nan"), float("inf")
    y = p.dev(x.cuda())
    assert torch.equal(y[:M].view(torch.int16), clean[:M].view(torch.int16))
    assert bool(y[M].isnan().all()) and not bool(y[M + 1].isfinite().any())


@pytest.mark.parametrize("wfmt", ["int8", "int4", "int4b128"])
@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e6, 1e18])
def test_tokens_of_any_magnitude(wfmt, scale):
    """Digits are relative to the token's largest value: its magnitude does not matter."""
    p = Product(512, 80, wfmt, yfmt="f32")
    x = (p.x(2).float() * torch.tensor([scale, 0.0])[:, None]).to(torch.bfloat16)
    p.compare(x, p.dev(x.cuda()))


@pytest.mark.parametrize("wfmt,xfmt", [("bf16", "bf16"), ("int8", "bf16"), ("int4", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("M", [2, 6, 18, 300])
def test_outliers_in_a_row(wfmt, xfmt, M):
    """A few columns thousands of times the others, as hidden states have them."""
    p = Product(640, 75, wfmt, xfmt, bias=True)
    x = p.x(M).float()
    x[:, 7] *= 4000
    x[0, 200] = -30000.0
    x = x.to(p.x_dtype)
    p.compare(x, p.dev(x.cuda()))


@pytest.mark.parametrize("wfmt,xfmt", [("bf16", "bf16"), ("int8", "bf16"), ("int4", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("M", [2, 4, 60, 300])
def test_same_call_same_bits_on_a_dirty_workspace(wfmt, xfmt, M):
    p = Product(1024, 272, wfmt, xfmt)
    x = p.x(M).cuda()
    y = p.dev(x).clone()
    for fill in (0, 255):
        for ws in p.dev._ws.values():
            ws.fill_(fill)
        assert torch.equal(p.dev(x), y)


@pytest.mark.parametrize("M", [3, 50, 200])
def test_captured_and_replayed_with_new_inputs(M):
    p = Product(512, 300, "int4", bias=True, act="gelu_tanh")
    x = p.x(M).cuda()
    y = p.dev(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.dev(x, y=y)
    for seed in (31, 32):
        new = p.x(M, seed)
        x.copy_(new)
        y.zero_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        p.compare(new, y)


@pytest.mark.parametrize("wfmt,xfmt,M", [("int8", "bf16", 4), ("int4", "bf16", 60), ("f32", "f32", 100)])
def test_graphs_keep_workspaces_of_their_own(wfmt, xfmt, M):
    """Two captured calls replayed at once, after the eager workspace was replaced by a larger one."""
    p = Product(1024, 320, wfmt, xfmt)
    xs = [p.x(M, 60 + n).cuda() for n in range(2)]
    want = [p.dev(x).clone() for x in xs]
    ys, graphs = [torch.empty_like(w) for w in want], []
    for x, y in zip(xs, ys):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            p.dev(x, y=y)
    p.dev(p.x(M + 200).cuda())
    other = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(16)]
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for y, w in zip(ys, want))
    assert all(bool((t == 255).all()) for t in other)


@pytest.mark.parametrize("M", [2, 48, 160])
def test_several_streams_at_once(M):
    p = Product(2048, 320, "int8")
    xs = [p.x(M, 50 + n).cuda() for n in range(4)]
    want = [p.dev(x).clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(p.dev(x))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[n % 4]) for n, y in enumerate(got))


def _sampled(p_dev, x, W, rows, cols, y):
    """Checks y at sampled rows and columns against 64-bit dot products of the device tensors."""
    xr, Wr = x[rows].double().cpu(), W[cols].double().cpu()
    want = xr @ Wr.T
    bound = ref.sum_error(W.shape[1], xr.abs() @ Wr.abs().T) + ref.HALF[y.dtype] * want.abs()
    ref.check(y[rows][:, cols], want, bound * (1 + ref.HALF[y.dtype]))


@pytest.mark.parametrize("M", [5, 70])
def test_weight_offsets_beyond_32_bits(M):
    """bf16 weights of 2^31 + elements; the last rows are the ones far out."""
    K, N = 8192, (1 << 18) + 37
    W = torch.empty((N, K), dtype=torch.bfloat16, device="cuda").normal_(0, 0.02)
    lin = moe.Linear(K=K, N=N, wfmt="bf16", xfmt="bf16", W=W)
    x = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    y = lin(x)
    torch.cuda.synchronize()
    _sampled(lin, x, W, torch.tensor([0, M - 1]), torch.tensor([0, 77, N // 2, N - 38, N - 1]), y)


@pytest.mark.parametrize("N", [40, 300])
def test_row_offsets_beyond_32_bits(N):
    """Rows of x and y so far apart that the last ones lie beyond 2^31 elements."""
    K, ld = 64, 1 << 23
    for M, wfmt in ((260, "bf16"), (260, "int8")):
        p = Product(K, N, wfmt)
        base = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")
        x = p.x(M)
        base[:, :K] = x.cuda()
        y = base[:, 4096 : 4096 + N]
        p.dev(base[:, :K], y=y)
        torch.cuda.synchronize()
        p.compare(x, y)
        del base, y


def test_wrapper_refusals():
    p = Product(64, 10)
    x = p.x(4).cuda()
    for bad in (x.float(), x[:, :32], x.cpu(), p.x(64).cuda()[:64].T, torch.empty(4, 68, dtype=torch.bfloat16, device="cuda")[:, :64],
                torch.empty(4, 72, dtype=torch.bfloat16, device="cuda")[:, 4:68]):
        with pytest.raises(moe.MoeError):
            p.dev(bad)
    with pytest.raises(moe.MoeError):
        p.dev(x, residual=x)
    assert p.dev(x[:0]).shape == (0, 10)
